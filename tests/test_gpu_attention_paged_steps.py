"""Attention over the paged cache where one step of keys differs from the next: scales, missing pages, and ranges that
begin and end inside a step. Against the plain 64-bit implementation, with the bound derived there."""
import numpy as np
import pytest
import torch

import oracle
import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _build, _native
from tests import paged_reference as ref
from tests.test_gpu_attention_paged import call, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    oracle.build()
    torch.cuda.init()
    yield
    assert sd.sdnq_device_status() == 0


@pytest.mark.parametrize("D,page,share,new", [(128, 16, 4, [300, 5, 77]), (64, 32, 4, [300, 5, 77]),
                                              (128, 64, 1, [600, 40, 129]), (64, 256, 9, [100, 1, 50])])
def test_every_step_uses_its_own_scales_and_pages(D, page, share, new):
    """Value scales that grow and shrink by powers of two from one 64 keys to the next, pages missing in a pattern with
    a period of its own: a step that used its neighbour's would be off by whole factors."""
    lens = [1500, 700, 900]
    cache = ref.Cache(1, page, D, ref.pages_of(lens, page), 71)
    for b, L in enumerate(lens):
        for n in range(-(-L // page)):
            at = n * page + np.arange(page)
            cache.scales[cache.table[b, n], 0, 1] *= 2.0 ** ((at // 64 * 5) % 11 - 5)
            cache.scales[cache.table[b, n], 0, 0] *= 2.0 ** -(at // 64 % 3)
    for b in range(3):
        gone = np.arange(1, cache.table.shape[1], max(2, 7 * 16 // page))
        cache.table[b, gone[gone < -(-lens[b] // page) - 1]] = -1
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), share, D, 72)
    out = call(q, cache.gpu(), lens, cu, max(new))
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_INDEX
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, 256, D ** -0.5)
    check(out, o, size, max(lens))


@pytest.mark.parametrize("D,page", [(128, 16), (128, 64), (128, 256), (64, 32)])
@pytest.mark.parametrize("window,sinks,new", [(300, 4, [1, 1, 1]), (100, 0, [3, 1, 2]), (70, 20, [1, 1, 1]),
                                              (300, 4, [200, 40, 3]), (65, 0, [50, 140, 257]), (1, 1, [1, 90, 2])])
def test_pages_that_no_row_sees_may_be_gone(D, page, window, sinks, new):
    """A sliding window's owner gives back the pages between the sinks and the window; their entries name nothing."""
    lens = [1500, 700, 601]
    cache = ref.Cache(2, page, D, ref.pages_of(lens, page), 81)
    table = cache.table.copy()
    for b, L in enumerate(lens):
        for n in range(table.shape[1]):
            j = n * page + np.arange(page)
            if not (((j > L - new[b] - window) & (j < L)) | (j < min(sinks, L))).any():
                table[b, n] = (-1, -2 ** 31, cache.P, 2 ** 31 - 1)[n % 4]
    assert (table != cache.table).any()
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 4, D, 82)
    gpu = cache.gpu()
    out = call(q, (*gpu[:2], torch.from_numpy(table).cuda()), lens, cu, max(new), window=window, sinks=sinks)
    assert sd.sdnq_device_status() == 0
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, 256, D ** -0.5, window, sinks)
    check(out, o, size, max(lens))


@pytest.mark.parametrize("new", [[1], [60]])
def test_a_missing_page_that_a_row_sees_is_still_reported(new):
    lens, window, sinks = [900], 200, 20
    cache = ref.Cache(1, 16, 128, ref.pages_of(lens, 16), 83)
    q = ref.queries(sum(new), 4, 128, 84)
    for gone in (0, 1, (900 - new[0] - window + 1) // 16, 899 // 16):
        table = cache.table.copy()
        table[0, gone] = -1
        gpu = cache.gpu()
        out = call(q, (*gpu[:2], torch.from_numpy(table).cuda()), lens, ref.offsets(new), max(new), window=window,
                   sinks=sinks)
        assert sd.sdnq_device_status() == _native.SDNQ_ERR_INDEX, gone
        o, size = ref.attention(q, cache.codes, cache.scales, table, lens, ref.offsets(new), 256, 128 ** -0.5, window,
                                sinks)
        check(out, o, size, 900)


@pytest.mark.parametrize("new", [None, [1, 40, 2]])
def test_sequences_without_pages(new):
    """A table without columns: no key to see, rows of zeros."""
    cache = ref.Cache(2, 16, 128, [1], 91)
    c, s, _ = cache.gpu()
    cu = ref.offsets(new or [1, 1, 1])
    q = ref.queries(int(cu[-1]), 4, 128, 92)
    out = call(q, (c, s, torch.empty((3, 0), dtype=torch.int32, device="cuda")), [0, 0, 0], new and cu, max(new or [1]))
    assert sd.sdnq_device_status() == 0 and not out.any()


def test_sequences_behind_a_blocks_last_piece_cost_nothing():
    """A chunk in front of 40000 sequences without new tokens takes what it takes behind them: the blocks that have its
    last pieces do not look at those sequences one by one."""
    E, times = 40000, []
    cache = ref.Cache(1, 16, 128, ref.pages_of([600], 16), 95)
    c, s, t = cache.gpu()
    q = ref.queries(300, 4, 128, 96).cuda()
    for at in (0, E):
        new, lens = np.zeros(E + 1, np.int64), np.zeros(E + 1, np.int32)
        new[at], lens[at] = 300, 600
        args = (q, c, s, t.expand(E + 1, -1).contiguous(), torch.from_numpy(lens).cuda())
        cu = torch.from_numpy(ref.offsets(new)).cuda()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        for e in (begin, end):      # the second call is the timed one
            begin.record()
            out = sd.sdnq_attention_paged(*args, cu_q=cu)
            e.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end))
        o, size = ref.attention(q[-1:].cpu(), cache.codes, cache.scales, cache.table, [600], [0, 1], 256, 128 ** -0.5)
        check(out[-1:], o, size, 600)
    assert times[0] < 3 * times[1], times


def excess(out, o):
    """How far each row's elements are from o beyond half a bf16 step, in the 2-norm: what the row's error before its
    last rounding is at least."""
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(o), 2.0 ** -126))) - 7)
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - o)
    return np.linalg.norm(np.maximum(err - 0.5 * step, 0.0), axis=-1)


@pytest.mark.parametrize("lens,new,share,Hkv,D,page,window,sinks", [
    ([1, 2, 3, 5, 9, 17, 33, 40], None, 4, 2, 128, 16, 0, 0), ([1, 4, 30], None, 8, 1, 64, 32, 0, 0),
    ([4, 3, 20], [4, 3, 2], 4, 2, 128, 64, 0, 0), ([7, 300], [2, 4], 6, 1, 64, 16, 90, 4),
    ([9000], None, 3, 1, 128, 64, 0, 0), ([1500, 3], None, 20, 1, 128, 16, 200, 1)])
def test_few_rows_keep_11_bits_of_the_weights(lens, new, share, Hkv, D, page, window, sinks):
    """Up to 32 query rows a kv head: before its last rounding a row is off by half an f16 step of each weight (2^-11)
    and the fp32 sums over the keys, logits up to 64 a few roundings off, the exponential's 2^-22 and the butterfly."""
    cache = ref.Cache(Hkv, page, D, ref.pages_of(lens, page), 97)
    cu = ref.offsets(new or [1] * len(lens))
    q = ref.queries(int(cu[-1]), share * Hkv, D, 98)
    out = call(q, cache.gpu(), lens, None if new is None else cu, max(new or [1]), window=window, sinks=sinks)
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, 256, D ** -0.5, window, sinks)
    rel = 2.0 ** -11 + 2 * max(lens) * 2.0 ** -24 + 4 * 64 * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -20
    assert np.all(excess(out, o) <= rel * size)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 1, 2], [120, 70, 1]])
@pytest.mark.parametrize("power", [-100, -60, 0, 60, 110])
def test_value_scales_of_any_size(D, new, power):
    """Value scales around 2^power, some of them zero, some rows of zeros, and a hidden key's 2^120: what a row sees
    sets the range that its weights are held in."""
    lens, window = [700, 260, 150], 100
    cache = ref.Cache(1, 16, D, ref.pages_of(lens, 16), 99)
    cache.scales[:, :, 1] = np.minimum(cache.scales[:, :, 1].astype(np.float64) * 2.0 ** power, 2.0 ** 112)
    cu = ref.offsets(new)
    for b, L in enumerate(lens):
        for j in range(0, L, 7):
            cache.scales[cache.table[b, j // 16], :, 1, j % 16] = 0.0
            cache.codes[cache.table[b, j // 16], :, 1, j % 16] = 0
        for j in range(max(0, L - new[b] - window + 1)):
            cache.scales[cache.table[b, j // 16], :, 1, j % 16] = 2.0 ** 120
    q = ref.queries(int(cu[-1]), 4, D, 100)
    out = call(q, cache.gpu(), lens, cu, max(new), window=window)
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, 256, D ** -0.5, window)
    check(out, o, size, 700)
