"""Rows that are not finite, in the paged cache and the attention over it: they stay NaN, they reach only what sees
them, and rows without keys stay zeros."""
import numpy as np
import pytest
import torch

import oracle
import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _build
from tests import paged_reference as ref
from tests.test_gpu_attention_paged import call, check

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    oracle.build()
    torch.cuda.init()
    yield
    assert sd.sdnq_device_status() == 0


@pytest.mark.parametrize("D,group", [(64, 8), (64, 64), (128, 8), (128, 32), (128, 128)])
def test_rows_that_are_not_finite_are_stored_as_such(D, group):
    T, Hkv = 40, 3
    k, v = ref.queries(T, Hkv, D, 1), ref.queries(T, Hkv, D, 2)
    want = [k.clone(), v.clone()]
    rng = np.random.default_rng(3)
    bad = np.zeros((2, T, Hkv), bool)
    kinds = [(NAN,), (INF,), (-INF,), (INF, -INF), (NAN, INF), (3e38,) * 8]   # (the last: sums past the range)
    for n, x in enumerate((k, v)):
        for t in range(0, T, 3):
            h, at = int(rng.integers(Hkv)), int(rng.integers(D // 8)) * 8
            x[t, h, at:at + len(kinds[t // 3 % 6])] = torch.tensor(kinds[t // 3 % 6], dtype=torch.bfloat16)
            bad[n, t, h] = True
            want[n][t, h] = 0.0
    codes, scales = sd.kv_cache(4, Hkv, 16, D)
    slots = torch.from_numpy(rng.permutation(64)[:T])
    sd.sdnq_kv_write(k.cuda(), v.cuda(), slots.cuda(), codes, scales, group)
    back = sd.sdnq_kv_read(slots.cuda(), codes, scales, group)
    ids, off = slots.numpy() // 16, slots.numpy() % 16
    for n in range(2):
        c, s = ref.quantize_rows(want[n], group)
        got = scales.cpu().numpy()[ids, :, n, off]
        assert np.array_equal(codes.cpu().numpy()[ids, :, n, off], c)
        assert np.array_equal(np.isnan(got), bad[n])
        assert np.array_equal(got[~bad[n]].view(np.uint32), s[~bad[n]].view(np.uint32))
        x = back[n].float().cpu().numpy()
        assert np.isnan(x[bad[n]]).all() and np.isfinite(x[~bad[n]]).all()


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,new", [(0, [1, 1]), (90, [1, 3]), (0, [120, 70]), (90, [150, 129])])
def test_a_stored_row_reaches_the_rows_that_see_it(which, D, window, new):
    """One key or one value whose scale is NaN, near the window's edge of the first new rows."""
    lens = [700, 333]
    cache = ref.Cache(1, 16, D, ref.pages_of(lens, 16), 5)
    j = [L - n - max(window - 2, 50) for L, n in zip(lens, new)]
    clean = cache.scales.copy()
    for b in range(2):
        cache.codes[cache.table[b, j[b] // 16], 0, which, j[b] % 16] = 0
        cache.scales[cache.table[b, j[b] // 16], 0, which, j[b] % 16] = np.nan
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 4, D, 6)
    out = call(q, cache.gpu(), lens, cu, max(new), window=window).float().cpu()
    o, size = ref.attention(q, cache.codes, clean, cache.table, lens, cu, 256, D ** -0.5, window)
    see = np.zeros(int(cu[-1]), bool)
    for b, n in enumerate(new):
        for i in range(n):
            see[cu[b] + i] = ref.visible(lens[b] - n + i, lens[b], window, 0)[j[b]]
    assert see.any() and (window == 0 or max(new) == 1 or not see.all())
    assert np.isnan(out[torch.from_numpy(see)].numpy()).all()
    check(out[torch.from_numpy(~see)], o[~see], size[~see], 700) if not see.all() else None


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [4, 3, 1, 2], [150, 20, 5, 40]])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_query_row_stays_to_itself_and_needs_a_key(D, new, bad):
    """Rows that are not finite among others: NaN where they see a key, zeros where they see none (a length of 0, and
    rows before the first key)."""
    lens = [400, 200, 0, 15]
    cache = ref.Cache(2, 16, D, ref.pages_of(lens, 16), 7)
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 6, D, 8)
    rng = np.random.default_rng(9)
    hit = rng.random((int(cu[-1]), 6)) < 0.3
    hit[cu[2]:cu[2] + 1, :3] = True
    hit[cu[3]] = True
    clean = q.clone()
    q[torch.from_numpy(hit)] = q[torch.from_numpy(hit)].index_fill(1, torch.tensor([5]), bad)
    out = call(q, cache.gpu(), lens, cu, max(new)).float().cpu()
    o, size = ref.attention(clean, cache.codes, cache.scales, cache.table, lens, cu, 256, D ** -0.5)
    sees = size > 0
    assert np.isnan(out[torch.from_numpy(hit & sees)].numpy()).all()
    assert not out[torch.from_numpy(~sees)].any() and (hit & ~sees).any()
    rest = torch.from_numpy(~hit)
    check(out[rest], o[~hit], size[~hit], 400)


def test_a_bad_row_of_a_long_context_that_several_blocks_share():
    lens = [20000]
    cache = ref.Cache(1, 64, 128, ref.pages_of(lens, 64), 11)
    cache.scales[cache.table[0, 100], 0, 0, 7] = np.nan
    q = ref.queries(300, 4, 128, 12)
    gpu = cache.gpu()
    assert bool(call(q[-1:], gpu, lens, None, 1).isnan().all())
    assert bool(call(q, gpu, lens, [0, 300], 300).isnan().all())
    cache.scales[cache.table[0, 100], 0, 0, 7] = 1.0
    gpu = cache.gpu()
    q[7, 2, 0] = NAN
    out = call(q, gpu, lens, [0, 300], 300).isnan()
    assert bool(out[7, 2].all()) and int(out.any(-1).sum()) == 1
