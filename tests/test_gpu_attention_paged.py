"""Attention over the paged cache against the plain 64-bit implementation (paged_reference), row by row in the
2-norm with the bound derived there; masks, empty rows, strides, pages and indexes where it can go wrong."""
import math

import numpy as np
import pytest
import torch

import oracle
import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _build, _native
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    oracle.build()
    torch.cuda.init()
    yield
    assert sd.sdnq_device_status() == 0


def call(q, gpu, lens, cu, max_q, **kw):
    c, s, t = gpu
    return sd.sdnq_attention_paged(q.cuda() if not q.is_cuda else q, c, s, t,
                                   torch.tensor(np.asarray(lens), dtype=torch.int32, device="cuda"),
                                   cu_q=None if cu is None else torch.from_numpy(np.asarray(cu, np.int32)).cuda(),
                                   max_q=max_q, **kw)


def check(out, o, size, keys):
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    err = np.linalg.norm(got - o, axis=-1)
    lim = ref.bound(o, size, keys)
    assert np.all(err <= lim), (float((err / lim).max()), np.argwhere(err > lim)[:5].tolist())


# lengths, new tokens of each sequence (None: one each, without offsets), query heads per kv head, kv heads, D, page,
# window, sinks, group
CASES = [
    ([1], None, 1, 1, 128, 16, 0, 0, 256),
    ([1, 2, 15, 16, 17], None, 4, 2, 128, 16, 0, 0, 256),
    ([63, 64, 65, 127, 128, 129, 300], None, 4, 2, 128, 16, 0, 0, 256),
    ([200, 1, 77], None, 16, 1, 128, 32, 0, 0, 64),
    ([200, 1, 77], None, 17, 1, 128, 32, 0, 0, 256),          # more rows than one small tile
    ([513, 40], None, 3, 2, 128, 64, 0, 0, 8),
    ([1000], None, 8, 1, 128, 128, 0, 0, 16),
    ([700, 255], None, 6, 2, 128, 256, 0, 0, 32),
    ([100, 1, 33], None, 4, 2, 64, 16, 0, 0, 256),
    ([300, 257], None, 5, 1, 64, 64, 0, 0, 32),
    ([300, 129], None, 1, 3, 64, 256, 0, 0, 8),
    ([400, 90, 5], None, 4, 2, 128, 16, 50, 0, 256),
    ([400, 90, 5], None, 4, 2, 128, 16, 50, 4, 256),
    ([700, 300], None, 2, 1, 64, 32, 64, 130, 256),           # more sinks than a tile
    ([500], None, 4, 1, 128, 16, 1, 0, 256),                  # a window of one key: itself
    ([500], None, 4, 1, 128, 16, 1 << 40, 3, 256),            # a window longer than anything
    ([40, 20, 9], [4, 4, 4], 4, 2, 128, 16, 0, 0, 256),       # drafted tokens
    ([140, 70], [3, 2], 5, 1, 64, 16, 37, 2, 256),
    ([30], [30], 1, 1, 128, 16, 0, 0, 256),                   # a whole prompt
    ([130], [130], 2, 1, 128, 32, 0, 0, 256),
    ([300, 129, 1], [300, 1, 1], 4, 1, 128, 16, 0, 0, 256),   # a prompt and single tokens
    ([300, 500, 64, 20], [45, 130, 0, 20], 4, 2, 128, 64, 0, 0, 256),
    ([257, 400], [129, 200], 3, 1, 128, 128, 0, 0, 64),
    ([600], [260], 1, 2, 128, 256, 100, 5, 256),
    ([600, 333], [128, 40], 7, 1, 128, 16, 64, 0, 256),
    ([300, 200], [100, 90], 4, 1, 64, 16, 0, 0, 256),
    ([420], [200], 2, 2, 64, 128, 129, 1, 16),
    ([280], [70], 4, 1, 64, 256, 0, 0, 256),
    ([900, 30], [17, 30], 8, 1, 128, 16, 0, 0, 128),
    ([777], [1], 20, 1, 128, 64, 300, 70, 256),
    ([300, 77], None, 40, 1, 64, 32, 0, 0, 256),              # single tokens with more rows than the small tiles take
    ([500], None, 300, 1, 128, 16, 100, 3, 8),
]


@pytest.mark.parametrize("lens,new,share,Hkv,D,page,window,sinks,group", CASES)
def test_attention(lens, new, share, Hkv, D, page, window, sinks, group):
    seed = sum(lens) + share + D + page
    cache = ref.Cache(Hkv, page, D, ref.pages_of(lens, page), seed, group=group)
    cu = ref.offsets(new or [1] * len(lens))
    q = ref.queries(int(cu[-1]), share * Hkv, D, seed)
    out = call(q, cache.gpu(), lens, None if new is None else cu, max(new or [1]), window=window, sinks=sinks,
               group=group)
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, group, 1 / math.sqrt(D),
                            min(window, 1 << 30), sinks)
    check(out, o, size, max(lens))
    assert sd.sdnq_device_status() == 0


@pytest.mark.parametrize("new,max_q", [([1, 1, 1], 1), ([1, 1, 1], 64), ([5, 40, 2], 1), ([5, 40, 2], 40),
                                       ([5, 40, 2], 5000)])
def test_max_q_changes_no_more_than_roundings(new, max_q):
    lens = [150, 300, 64]
    cache = ref.Cache(2, 16, 128, ref.pages_of(lens, 16), 5)
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 8, 128, 6)
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, 256, 128 ** -0.5)
    check(call(q, cache.gpu(), lens, cu, max_q), o, size, 300)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 4, 1], [150, 70, 1]])
def test_only_visible_keys_count(D, new):
    """Equal logits (q = 0), visible values of one kind and huge ones everywhere else: the mean over visible keys,
    in which every key shows. The largest visible weight sits on the ends of the visible ranges."""
    lens, page, window, sinks = [400, 333, 130], 16, 90, 3
    cache = ref.Cache(1, page, D, ref.pages_of(lens, page), 3)
    cu = ref.offsets(new)
    q = torch.zeros(int(cu[-1]), 4, D, dtype=torch.bfloat16)
    for win, snk in ((0, 0), (window, 0), (window, sinks)):
        scales = cache.scales.copy()
        for b, L in enumerate(lens):   # slots behind the end of each sequence: huge
            last = cache.table[b, (L - 1) // page]
            scales[last, :, :, (L - 1) % page + 1:] = 1e30
            if win and snk < L - win - new[b]:   # keys between the sinks and the first row's window
                for j in range(snk, L - new[b] - win + 1):
                    scales[cache.table[b, j // page], :, 1, j % page] = 1e30
                j = L - new[b] - win + 1         # the first row's first key
                scales[cache.table[b, j // page], :, 1, j % page] *= 50
            j = L - new[b]                       # the first row's last key
            scales[cache.table[b, j // page], :, 1, j % page] *= 50
        gpu = (torch.from_numpy(cache.codes).cuda(), torch.from_numpy(scales).cuda(),
               torch.from_numpy(cache.table).cuda())
        out = call(q, gpu, lens, cu, max(new), window=win, sinks=snk)
        o, size = ref.attention(q, cache.codes, scales, cache.table, lens, cu, 256, D ** -0.5, win, snk)
        check(out, o, size, max(lens))


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [2, 3, 1, 4], [140, 20, 150, 1]])
def test_rows_without_keys_are_zero(new):
    """A length of zero, and more new tokens than the length (the first ones sit before key 0)."""
    lens = [0, 1, 100, 0]
    cache = ref.Cache(2, 16, 128, [0, 1, 3, 0], 4, width=3)   # 48 keys at most: the length counts as 48
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 6, 128, 5)
    out = call(q, cache.gpu(), lens, cu, max(new))
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_INDEX
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, [0, 1, 48, 0], cu, 256, 128 ** -0.5)
    check(out, o, size, 100)
    got = out.float().cpu().numpy()
    assert not got[size == 0].any() and (size == 0).any()
    out = call(q, cache.gpu(), [0, 1, 48, -3], cu, max(new), window=1)
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_INDEX
    assert not out[cu[3]:].any()


@pytest.mark.parametrize("D,page", [(128, 16), (128, 128), (64, 32)])
@pytest.mark.parametrize("new", [[1, 1], [130, 33]])
def test_memory_that_was_never_written_has_no_effect(D, page, new):
    """Infinite and NaN scales and any codes in every slot behind the sequences, and in visible pages outside the
    window."""
    lens = [page * 3 + 5, page * 2 + 40]
    blank = ref.Cache(2, page, D, ref.pages_of(lens, page), 8, fill=False)
    full = ref.Cache(2, page, D, ref.pages_of(lens, page), 8)
    window = 20
    for b, L in enumerate(lens):
        for j in range(max(0, L - new[b] - window + 1), L):
            at = (blank.table[b, j // page], slice(None), slice(None), j % page)
            blank.codes[at], blank.scales[at] = full.codes[at], full.scales[at]
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 4, D, 9)
    out = call(q, blank.gpu(), lens, cu, max(new), window=window)
    o, size = ref.attention(q, blank.codes, blank.scales, blank.table, lens, cu, 256, D ** -0.5, window)
    check(out, o, size, max(lens))


@pytest.mark.parametrize("new", [[1, 1, 1], [60, 1, 33]])
def test_rows_behind_the_last_sequence_and_strides(new):
    lens = [100, 50, 33]
    cache = ref.Cache(2, 16, 128, ref.pages_of(lens, 16), 2, width=11)
    cu = ref.offsets(new)
    T, n = int(cu[-1]) + 5, int(cu[-1])
    q = ref.queries(T, 6, 128, 3)
    wide = torch.zeros(T, 10 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    gq = wide[:, 8:8 + 768].unflatten(1, (6, 128))
    gq.copy_(q)
    hold = torch.full((T, 800), 3.0, dtype=torch.bfloat16, device="cuda")
    out = hold[:, 16:784].unflatten(1, (6, 128))
    c, s, t = cache.gpu()
    far = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    far[:, 4:15] = t
    r = sd.sdnq_attention_paged(gq, c, s, far[:, 4:15], torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                cu_q=torch.from_numpy(cu).cuda(), max_q=max(new), out=out)
    assert r is out
    o, size = ref.attention(q[:n], cache.codes, cache.scales, cache.table, lens, cu, 256, 128 ** -0.5)
    check(out[:n], o, size, 100)
    assert bool((out[n:] == 3.0).all()) and bool((hold[:, :16] == 3.0).all()) and bool((hold[:, 784:] == 3.0).all())


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("new", [[1, 1], [40, 150]])
def test_pages_outside_the_pool_hide_their_keys(new, page):
    lens = [page * 4 + 3, page * 3]
    cache = ref.Cache(2, page, 128, ref.pages_of(lens, page), 6)
    cache.table[0, 1] = cache.P
    cache.table[0, 4] = -1
    cache.table[1, 0] = 2 ** 31 - 1
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 4, 128, 7)
    out = call(q, cache.gpu(), lens, cu, max(new))
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_INDEX
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, 256, 128 ** -0.5)
    check(out, o, size, max(lens))


@pytest.mark.parametrize("max_q", [1, 50])
def test_row_offsets_that_make_no_sense_leave_their_sequence_out(max_q):
    lens = [60, 70, 80, 90]
    cache = ref.Cache(1, 16, 128, ref.pages_of(lens, 16), 6)
    q = ref.queries(30, 4, 128, 7)
    cu = np.array([0, 10, 5, 20, 31], np.int32)    # the second decreases, the last ends past the rows
    hold = torch.full((30, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    out = call(q, cache.gpu(), lens, cu, max_q, out=hold)
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_INDEX
    o, size = ref.attention(q[:10], cache.codes, cache.scales, cache.table[:1], lens[:1], [0, 10], 256, 128 ** -0.5)
    check(out[:5], o[:5], size[:5], 90)            # rows 5..9 belong to two sequences
    o, size = ref.attention(q[5:20], cache.codes, cache.scales, cache.table[2:3], lens[2:3], [0, 15], 256, 128 ** -0.5)
    check(out[10:20], o[5:], size[5:], 90)
    assert bool((out[20:] == 9.0).all())


def test_zero_scale_and_zero_rows():
    lens = [70, 130]
    cache = ref.Cache(1, 16, 64, ref.pages_of(lens, 16), 6)
    cache.codes[cache.table[0, 1], :, 0, 3] = 0
    cache.scales[cache.table[0, 1], :, 0, 3] = 0.0
    q = ref.queries(2, 4, 64, 7)
    q[0, 1] = 0.0
    for scale in (0.0, 1e-30, 0.125):
        out = call(q, cache.gpu(), lens, None, 1, scale=scale)
        o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, [0, 1, 2], 256, scale)
        check(out, o, size, 130)


@pytest.mark.parametrize("new", [[1, 1], [100, 140]])
def test_wide_logits(new):
    """Logits of several hundred in base 2: the running maximum moves again and again."""
    lens = [700, 333]
    cache = ref.Cache(1, 16, 128, ref.pages_of(lens, 16), 16, k_amp=6.0)
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 4, 128, 7, amp=6.0)
    out = call(q, cache.gpu(), lens, cu, max(new))
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, 256, 128 ** -0.5)
    got = out.float().cpu().numpy().astype(np.float64)
    err = np.linalg.norm(got - o, axis=-1)
    assert np.all(err <= ref.bound(o, size, 700, logit=1500.0))


@pytest.mark.parametrize("new,page", [([1] * 5, 16), ([3, 1, 4, 2, 1], 64), ([700, 1, 90, 333, 256], 32)])
def test_long_contexts_sampled_rows(new, page):
    """Contexts that are split over many blocks and joined: sampled rows, and the same bits twice."""
    lens = [9000, 1, 12345, 3500, 6000]
    cache = ref.Cache(1, page, 128, ref.pages_of(lens, page), 11)
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 4, 128, 12)
    out = call(q, cache.gpu(), lens, cu, max(new))
    again = call(q, cache.gpu(), lens, cu, max(new))
    assert torch.equal(out, again)
    rng = np.random.default_rng(1)
    for b, n in enumerate(new):
        for i in {0, n - 1, int(rng.integers(0, n))}:
            t = int(cu[b]) + i
            L = lens[b] - n + i + 1     # row i alone sees as the last of a context of L
            if L < 1:
                continue
            o, size = ref.attention(q[t:t + 1], cache.codes, cache.scales, cache.table[b:b + 1], [L], [0, 1], 256,
                                    128 ** -0.5)
            check(out[t:t + 1], o, size, 12345)


def test_many_sequences():
    """More sequences than blocks, most of them short, of every kind together."""
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 60, 1500)
    new = np.minimum(rng.integers(0, 4, 1500), np.maximum(lens, 1))
    cache = ref.Cache(1, 16, 64, ref.pages_of(lens, 16), 11)
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 2, 64, 12)
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, lens, cu, 256, 0.125)
    for max_q in (3, 100):
        check(call(q, cache.gpu(), lens, cu, max_q), o, size, 60)


def test_other_stream_and_given_workspace():
    lens, new = [3000, 500], [1, 90]
    cache = ref.Cache(2, 16, 128, ref.pages_of(lens, 16), 21)
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), 8, 128, 22)
    gpu = cache.gpu()
    want = call(q, gpu, lens, cu, 90)
    gq, gl, gc = q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(cu).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [sd.sdnq_attention_paged(gq, *gpu, gl, cu_q=gc, max_q=90, stream=side) for _ in range(3)]
    got.append(sd.sdnq_attention_paged(gq, *gpu, gl, cu_q=gc, max_q=90, stream=side.cuda_stream))
    ws = torch.full((sd.attention_paged_workspace(8, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    got.append(sd.sdnq_attention_paged(gq, *gpu, gl, cu_q=gc, max_q=90, ws=ws))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_captured_steps_share_a_workspace():
    """Two captured graphs with one workspace, replayed in turn with changed lengths and inputs."""
    lens = [2000, 37, 650]
    cache = ref.Cache(2, 16, 128, ref.pages_of([2100, 60, 700], 16), 31)
    gpu = cache.gpu()
    gl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(sd.attention_paged_workspace(8, 2, 128), dtype=torch.uint8, device="cuda")
    q1, q2 = ref.queries(3, 8, 128, 1).cuda(), ref.queries(270, 8, 128, 2).cuda()
    cu2 = torch.tensor([0, 200, 210, 270], dtype=torch.int32, device="cuda")
    o1, o2 = torch.empty_like(q1), torch.empty_like(q2)
    run1 = lambda: sd.sdnq_attention_paged(q1, *gpu, gl, ws=ws, out=o1)                            # noqa: E731
    run2 = lambda: sd.sdnq_attention_paged(q2, *gpu, gl, cu_q=cu2, max_q=200, ws=ws, out=o2)       # noqa: E731
    run1(), run2()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        run1()
    with torch.cuda.graph(g2):
        run2()
    for step in range(3):
        gl.copy_(torch.tensor([2000 + 30 * step, 37 + step, 650 - 100 * step], dtype=torch.int32))
        q1.copy_(ref.queries(3, 8, 128, 10 + step))
        g1.replay(), g2.replay()
        a, b = o1.clone(), o2.clone()
        run1(), run2()
        assert torch.equal(a, o1) and torch.equal(b, o2)


@pytest.mark.parametrize("D,page,window,sinks", [(128, 16, 0, 0), (64, 64, 70, 4)])
def test_a_prompt_and_its_next_tokens(D, page, window, sinks):
    """The set as a server uses it: a prompt stored in two chunks, each attending as it comes, then tokens one by one,
    two sequences sharing the batch. Each step against the 64-bit form over what the oracle stores."""
    Hkv, share, total = 2, 3, [190, 260]
    P = sum(ref.pages_of(total, page)) + 1
    codes, scales = sd.kv_cache(P, Hkv, page, D)
    ids = np.random.default_rng(1).permutation(P)
    width = max(ref.pages_of(total, page))
    table = np.full((2, width), -1, np.int32)
    table[0, :ref.pages_of(total, page)[0]] = ids[:ref.pages_of(total, page)[0]]
    table[1, :ref.pages_of(total, page)[1]] = ids[ref.pages_of(total, page)[0]:-1]
    held_c, held_s = codes.cpu().numpy(), scales.cpu().numpy()
    gt = torch.from_numpy(table).cuda()
    lens = [0, 0]
    for step, new in enumerate([[100, 33], [80, 200], [1, 1], [1, 1], [4, 0], [1, 3]]):
        qkv = ref.queries(sum(new), (share + 2) * Hkv, D, 50 + step)
        g = qkv.cuda()
        q, k, v = g[:, :share * Hkv], g[:, share * Hkv:-Hkv], g[:, -Hkv:]
        pos = [(b, lens[b] + i) for b in range(2) for i in range(new[b])]
        slots = np.array([table[b, p // page] * page + p % page for b, p in pos], np.int64)
        lens = [lens[0] + new[0], lens[1] + new[1]]
        sd.sdnq_kv_write(k, v, torch.from_numpy(slots).cuda(), codes, scales)
        out = call(q, (codes, scales, gt), lens, ref.offsets(new), max(new), window=window, sinks=sinks)
        for which, x in ((0, qkv[:, share * Hkv:-Hkv]), (1, qkv[:, -Hkv:])):
            c, s = ref.quantize_rows(x, 256)
            held_c[slots // page, :, which, slots % page] = c
            held_s[slots // page, :, which, slots % page] = s
        o, size = ref.attention(qkv[:, :share * Hkv], held_c, held_s, table, lens, ref.offsets(new), 256, D ** -0.5,
                                window, sinks)
        check(out, o, size, 300)
    assert np.array_equal(codes.cpu().numpy(), held_c)


def test_more_query_rows_than_a_grid_dimension():
    """65536 and more rows of one head, a context of one page each."""
    B = 66000
    cache = ref.Cache(1, 16, 64, [1] * 40, 3)
    table = torch.from_numpy(cache.table[np.arange(B) % 40]).cuda()
    c, s, _ = cache.gpu()
    q = ref.queries(40, 1, 64, 3)
    lens = torch.from_numpy((np.arange(B) % 40 % 16 + 1).astype(np.int32)).cuda()
    big = q[torch.arange(B) % 40].cuda()
    out = sd.sdnq_attention_paged(big, c, s, table, lens)
    o, size = ref.attention(q, cache.codes, cache.scales, cache.table, [i % 16 + 1 for i in range(40)],
                            np.arange(41), 256, 0.125)
    check(out[:40], o, size, 16)
    assert torch.equal(out, out[:40][torch.arange(B, device="cuda") % 40])


@pytest.mark.parametrize("share,D,window,sinks", [(1, 128, 70, 0), (1, 64, 40, 130), (3, 128, 10, 3), (1, 128, 0, 0)])
def test_short_chunks_of_many_lengths(share, D, window, sinks):
    """Chunks whose key ranges are a few steps long, tiles with and without a second half, several to a block, with
    single tokens and empty sequences in between."""
    rng = np.random.default_rng(share + D)
    B, Hkv, page = 150, 2, 16
    new = rng.choice([0, 1, 2, 33, 40, 65, 127, 128, 129, 200, 256, 257, 300], B)
    lens = new + rng.choice([0, 1, 15, 64, 90], B)
    cache = ref.Cache(Hkv, page, D, ref.pages_of(lens, page), 41, group=64)
    cu = ref.offsets(new)
    q = ref.queries(int(cu[-1]), share * Hkv, D, 42)
    out = call(q, cache.gpu(), lens, cu, int(new.max()), window=window, sinks=sinks, group=64)
    assert sd.sdnq_device_status() == 0
    for b in rng.permutation(B)[:25]:
        n, L, t = int(new[b]), int(lens[b]), int(cu[b])
        for i in sorted({0, n // 2, 127, 128, n - 1} & set(range(n))):
            at = L - n + i      # row i sees what the last row of a context of at + 1 keys sees
            o, size = ref.attention(q[t + i:t + i + 1], cache.codes, cache.scales, cache.table[b:b + 1], [at + 1], [0, 1],
                                    64, D ** -0.5, window, sinks)
            check(out[t + i:t + i + 1], o, size, 400)
    assert torch.equal(out, call(q, cache.gpu(), lens, cu, int(new.max()), window=window, sinks=sinks, group=64))


def test_two_calls_at_once_on_two_streams():
    """Calls that overlap on the GPU, each with its own workspace, in both forms."""
    lens, new = [3000, 700, 90], [400, 1, 33]
    cache = ref.Cache(2, 16, 128, ref.pages_of(lens, 16), 51)
    gpu = cache.gpu()
    gl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    gc = torch.from_numpy(ref.offsets(new)).cuda()
    q1, q2 = ref.queries(434, 8, 128, 1).cuda(), ref.queries(3, 8, 128, 2).cuda()
    want1 = sd.sdnq_attention_paged(q1, *gpu, gl, cu_q=gc, max_q=400)
    want2 = sd.sdnq_attention_paged(q2, *gpu, gl)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append((sd.sdnq_attention_paged(q1, *gpu, gl, cu_q=gc, max_q=400, stream=a), want1))
        got.append((sd.sdnq_attention_paged(q2, *gpu, gl, stream=b), want2))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)
