"""The paged rotated-int8 cache on the GPU: codes and scales bit for bit against the oracle's row quantizer, rows
read back against 64 bits, and every slot that is not named left as it was."""
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


def rows(T, H, D, seed):
    """Rows with outlier channels, one all-zero row, one of the smallest numbers, one of large ones."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=gen)
    x[..., 3] *= 25.0
    x = x.to(torch.bfloat16)
    x[0, 0] = 0.0
    if T > 2:
        x[1, 0] = (x[1, 0].float() * 2.0 ** -126).to(torch.bfloat16)
        x[2, 0] = (x[2, 0].float() * 2.0 ** 100).to(torch.bfloat16)
    return x


def write_case(T, Hkv, D, page, group, seed, strided):
    rng = np.random.default_rng(seed)
    P = -(-T // page) + 2
    slots = rng.permutation(P * page)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1 - int(rng.integers(0, 1 << 40))
    codes = rng.integers(-128, 128, (P, Hkv, 2, page, D), dtype=np.int8)
    scales = rng.standard_normal((P, Hkv, 2, page)).astype(np.float32)
    k, v = rows(T, Hkv, D, seed), rows(T, Hkv, D, seed + 1)
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    if strided:   # parts of a fused projection's rows, at an odd multiple of 16 bytes
        wide = torch.zeros(T, 3 * Hkv * D + 8, dtype=torch.bfloat16, device="cuda")
        gk, gv = (wide[:, a:a + Hkv * D].unflatten(1, (Hkv, D)) for a in (Hkv * D + 8, 2 * Hkv * D + 8))
        gk.copy_(k), gv.copy_(v)
    else:
        gk, gv = k.cuda(), v.cuda()
    return codes, scales, slots, k, v, c, s, gk, gv


@pytest.mark.parametrize("T,Hkv,D,page,group,strided", [
    (1, 1, 128, 16, 256, False), (1, 8, 64, 16, 256, False), (7, 3, 128, 16, 128, True), (33, 2, 64, 32, 64, True),
    (130, 5, 128, 64, 64, False), (300, 1, 64, 128, 32, True), (65, 8, 128, 256, 16, True), (40, 4, 64, 16, 8, False),
    (9, 2, 128, 32, 8, False), (50, 3, 64, 16, 16, False), (21, 1, 128, 16, 32, True),
])
def test_write_and_read(T, Hkv, D, page, group, strided):
    codes, scales, slots, k, v, c, s, gk, gv = write_case(T, Hkv, D, page, group, T + D + group, strided)
    sd.sdnq_kv_write(gk, gv, torch.from_numpy(slots).cuda(), c, s, group)
    for which, x in ((0, k), (1, v)):
        qc, qs = ref.quantize_rows(x, group)
        for t in np.flatnonzero(slots >= 0):
            codes[slots[t] // page, :, which, slots[t] % page] = qc[t]
            scales[slots[t] // page, :, which, slots[t] % page] = qs[t]
    assert np.array_equal(c.cpu().numpy(), codes)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    # read back: repeats, an order of its own, negative slots; x = code sums (exact) * fp32(s c), rounded once
    rng = np.random.default_rng(5)
    want = np.concatenate([slots, rng.integers(0, codes.shape[0] * page, 11), [-5]]).astype(np.int64)
    gk2, gv2 = sd.sdnq_kv_read(torch.from_numpy(want).cuda(), c, s, group)
    for which, got in ((0, gk2), (1, gv2)):
        at = np.maximum(want, 0)
        held = codes[at // page, :, which, at % page].astype(np.float64)
        held = ref.unrotate(held, group) * scales[at // page, :, which, at % page].astype(np.float64)[..., None]
        held[want < 0] = 0.0
        err = np.abs(got.float().cpu().numpy().astype(np.float64) - held)
        # half a bf16 step, three fp32 roundings; 2^-134 is half the smallest bf16
        assert np.all(err <= (2.0 ** -8 + 2.0 ** -21) * np.abs(held) + 2.0 ** -133), float(err.max())


def test_read_into_strided_outputs():
    codes, scales, slots, k, v, c, s, gk, gv = write_case(50, 2, 128, 16, 256, 3, False)
    sl = torch.from_numpy(np.maximum(slots, 0)).cuda()
    a, b = sd.sdnq_kv_read(sl, c, s)
    wide = torch.full((50, 2 * 256 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    ka, va = wide[:, 8:264].unflatten(1, (2, 128)), wide[:, 264:520].unflatten(1, (2, 128))
    r = sd.sdnq_kv_read(sl, c, s, k=ka, v=va)
    assert r[0] is ka and torch.equal(ka.nan_to_num(), a.nan_to_num()) and torch.equal(va.nan_to_num(), b.nan_to_num())
    assert bool((wide[:, :8] == 7.0).all()) and bool((wide[:, 520:] == 7.0).all())


def test_slots_past_the_pool_are_left_out_and_reported():
    """The kernel compares every slot with the pool's size before it forms an address."""
    codes, scales, slots, k, v, c, s, gk, gv = write_case(20, 2, 64, 16, 256, 9, False)
    slots = np.arange(20, dtype=np.int64)
    slots[4], slots[11], slots[17] = codes.shape[0] * 16, 1 << 40, (1 << 62)
    sl = torch.from_numpy(slots).cuda()
    sd.sdnq_kv_write(gk, gv, sl, c, s)
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_INDEX
    assert sd.sdnq_device_status() == 0
    for which, x in ((0, k), (1, v)):
        qc, qs = ref.quantize_rows(x, 256)
        for t in set(range(20)) - {4, 11, 17}:
            codes[t // 16, :, which, t % 16] = qc[t]
            scales[t // 16, :, which, t % 16] = qs[t]
    assert np.array_equal(c.cpu().numpy(), codes)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    a, b = sd.sdnq_kv_read(sl, c, s)
    assert sd.sdnq_device_status() == _native.SDNQ_ERR_INDEX
    assert not a[[4, 11, 17]].any() and not b[[4, 11, 17]].any() and bool(a[5].any())


def test_empty_calls():
    c, s = sd.kv_cache(2, 3, 16, 64)
    none = torch.empty(0, 3, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    sd.sdnq_kv_write(none, none, slots, c, s)
    a, b = sd.sdnq_kv_read(slots, c, s)
    assert a.shape == b.shape == (0, 3, 64) and not c.any() and not s.any()


def test_offsets_past_32_bits():
    """A pool of 2^32 bytes and more of codes: the first and the last pages."""
    P, Hkv, page, D = 262150, 1, 64, 128
    c = torch.empty((P, Hkv, 2, page, D), dtype=torch.int8, device="cuda")
    s = torch.empty((P, Hkv, 2, page), dtype=torch.float32, device="cuda")
    assert c.numel() > 1 << 32
    T = 70
    k, v = rows(T, Hkv, D, 1), rows(T, Hkv, D, 2)
    slots = torch.cat([torch.arange(35), P * page - 35 + torch.arange(35)]).cuda()
    sd.sdnq_kv_write(k.cuda(), v.cuda(), slots, c, s)
    for which, x in ((0, k), (1, v)):
        qc, qs = ref.quantize_rows(x, 256)
        assert np.array_equal(c[slots // page, :, which, slots % page].cpu().numpy(), qc)
        assert np.array_equal(s[slots // page, :, which, slots % page].cpu().numpy(), qs)
    # and attention over them: one sequence of 70 tokens in the first page and the last two
    table = torch.tensor([[0, P - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    c[0, 0, :, 35:] = 0
    s[0, 0, :, 35:] = 0.0
    c[P - 1, 0, :, :29] = 0
    s[P - 1, 0, :, :29] = 0.0
    q = ref.queries(1, 4, D, 3)
    small_c = torch.stack([c[0], c[P - 1]]).cpu().numpy()
    small_s = torch.stack([s[0], s[P - 1]]).cpu().numpy()
    out = sd.sdnq_attention_paged(q.cuda(), c, s, table, lens)
    o, size = ref.attention(q, small_c, small_s, np.array([[0, 1]], np.int32), [100], [0, 1], 256, D ** -0.5)
    err = np.linalg.norm(out.float().cpu().numpy() - o, axis=-1)
    assert np.all(err <= ref.bound(o, size, 100))
