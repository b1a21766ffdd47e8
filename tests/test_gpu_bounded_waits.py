"""Both kinds of bounded wait (by global time, by a number of tries that the hardware suspends for about 4 us each) give
up when their limit is over: not long before, and not much later."""
import pytest
import torch

import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _build, _native

pytestmark = pytest.mark.gpu


def test_each_wait_takes_its_limit():
    _build.build()
    sd.sdnq_selftest_wait_timeout(1000)
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_TIMEOUT
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    sd.sdnq_selftest_wait_timeout(20_000_000)      # 20 ms, then 5001 tries
    end.record()
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_TIMEOUT
    assert 30.0 < begin.elapsed_time(end) < 120.0   # the second takes between half and five times its limit
    assert sd.sdnq_device_status() == 0
