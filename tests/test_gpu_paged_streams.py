"""The paged cache's calls on several streams, without a synchronisation between them: every result bit for bit that
of the same call made alone."""
import numpy as np
import pytest
import torch

import oracle
import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _build
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    oracle.build()
    torch.cuda.init()
    yield
    assert sd.sdnq_device_status() == 0


def setup(D, lens, new, seed):
    cache = ref.Cache(2, 16, D, ref.pages_of(lens, 16), seed)
    cu = ref.offsets(new)
    return (cache.gpu(), torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(cu).cuda(),
            [ref.queries(int(cu[-1]), 8, D, seed + i).cuda() for i in range(6)])


@pytest.mark.parametrize("D,lens,new", [(128, [30000, 9000, 700], [1, 1, 1]), (64, [9000, 4000], [600, 500]),
                                        (128, [6000, 3000, 90], [400, 1, 33])])
def test_a_call_on_another_stream_right_behind_one_on_the_current(D, lens, new):
    """Workspaces and outputs made by the calls: the second call's may not be the first one's, which is still running
    when it starts."""
    gpu, gl, gc, qs = setup(D, lens, new, 61)
    call = lambda q, **kw: sd.sdnq_attention_paged(q, *gpu, gl, cu_q=gc, max_q=max(new), **kw)    # noqa: E731
    slots = torch.from_numpy(np.random.default_rng(3).permutation(gpu[0].shape[0] * 16)).cuda()
    want, rows = [call(q) for q in qs], sd.sdnq_kv_read(slots, *gpu[:2])
    side = torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        got = [call(qs[0]), call(qs[1], stream=side), call(qs[2]), call(qs[3], stream=side.cuda_stream)]
        a, b = sd.sdnq_kv_read(slots, *gpu[:2]), sd.sdnq_kv_read(slots, *gpu[:2], stream=side)
        got += [call(qs[4], stream=side), call(qs[5])]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        assert all(torch.equal(x, y) for r in (a, b) for x, y in zip(r, rows))
