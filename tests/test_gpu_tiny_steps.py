"""Rows whose quantization step is small but not subnormal. The kernels replace the quotient z / s by a product with the
reciprocal and a correction (Markstein), whose residual z - q s has to be exact: it needs bits down to
ulp(q) ulp(s), which lie below the smallest fp32 number once s is under 2^-102 (codes of 1/2 and more of the int8 grid)
or 2^-93 (2^-10 and more of the e4m3 grid). Each row here has one element on the border between two codes, or next to
it, where an inexact residual gives the other code. Bit for bit against the oracle, which divides."""
import numpy as np
import pytest
import torch

import oracle
import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _build, _native, synthetic

pytestmark = pytest.mark.gpu

# (largest rotated magnitude, another one) of a row, in units of the smallest bf16 number, 2^-133: pairs where the
# corrected quotient without an exact residual falls on the wrong side, found by evaluating its fp32 steps in 64 bits
INT8 = [(16470, 8235), (260161, 44043), (260415, 44086), (1040390, 176129), (4161560, 704516), (4161621, 49153),
        (16646168, 720897), (66584664, 786433), (266338400, 3145729), (1065353344, 12582913),
        (4261413376, 50331652), (17045653504, 201326608), (17045657600, 201326656)]
FP8 = [(14680078, 1114113), (14680862, 1638489), (58720312, 2228226), (234881248, 1114113), (939524992, 2228226),
       (3758099968, 1114113), (15032399872, 2228226), (60129599488, 3276803), (60132622336, 917551)]


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    oracle.build()
    torch.cuda.init()
    yield
    assert sd.sdnq_device_status() == 0


def pieces(n):
    """Up to 8 bf16 numbers, in units, whose sum is n."""
    out = []
    while n:
        shift = max(0, n.bit_length() - 8)
        out.append(n >> shift << shift)
        n -= out[-1]
    assert len(out) <= 8
    return out + [0] * (8 - len(out))


def rows(pairs, K, group):
    """[len(pairs), K] bf16: the first group's sum is the row's largest rotated magnitude, the second group's the
    element on the border; every other rotated element of a group is a difference of its pieces."""
    x = np.zeros((len(pairs), K))
    for i, (a, z) in enumerate(pairs):
        x[i, :8] = pieces(a)
        x[i, group:group + 8] = pieces(z)
    return torch.from_numpy(x * 2.0 ** -133).to(torch.bfloat16)


def same(codes, scales, want):
    assert np.array_equal(codes, want[0])
    assert np.array_equal(scales.view(np.uint32), want[1].view(np.uint32))


def test_rows_are_what_they_say():
    x = rows(INT8, 64, 8).double() * 2.0 ** 133
    assert [(int(r[:8].sum()), int(r[8:16].sum())) for r in x] == INT8


@pytest.mark.parametrize("K,group", [(64, 8), (1024, 8), (2048, 128), (4096, 256), (8192, 16)])
def test_linear_path(K, group):
    x = rows(INT8, K, group)
    c, s = sd.sdnq_rotquant_act(x.cuda(), group)
    same(c.cpu().numpy(), s.cpu().numpy(), oracle.rotate_quantize(synthetic.bits(x), group))


@pytest.mark.parametrize("K,group", [(64, 8), (1024, 8), (2048, 128), (4096, 256), (8192, 16)])
def test_fp8(K, group):
    x = rows(FP8, K, group)
    c, s = sd.sdnq_rotquant_fp8(x.cuda(), group)
    same(c.cpu().numpy(), s.cpu().numpy(), oracle.rotate_quantize_fp8(synthetic.bits(x), group))


@pytest.mark.parametrize("group", [8, 16, 64])
def test_attention_preparation(group):
    x = rows(INT8, 128, group)
    q = x.reshape(1, -1, 1, 128).cuda()
    ws = _native.sdnq_attention_prep(q, q, group, smooth_k=False)
    off = _native.attention_workspace(1, len(INT8), len(INT8), 1, 128)[1]
    c = ws[off[0]:off[0] + x.numel()].view(torch.int8).reshape(x.shape)
    s = ws[off[2]:off[2] + 4 * len(INT8)].view(torch.float32)
    same(c.cpu().numpy(), s.cpu().numpy(), oracle.rotate_quantize(synthetic.bits(x), group))


@pytest.mark.parametrize("D,group", [(64, 8), (128, 8), (128, 64)])
def test_stored_rows(D, group):
    x = rows(INT8, D, group)
    n = len(INT8)
    k = torch.cat([x, rows([(a, z) for a, z in INT8[::-1]], D, group)]).reshape(n, 2, D)
    codes, scales = sd.kv_cache(1, 2, 16, D)
    slots = torch.arange(n, device="cuda")
    sd.sdnq_kv_write(k.cuda(), (-k).cuda(), slots, codes, scales, group)
    for which, r in ((0, k), (1, -k)):
        want = oracle.rotate_quantize(synthetic.bits(r.reshape(-1, D)), group)
        same(codes[0, :, which, :n].transpose(0, 1).reshape(-1, D).cpu().numpy(),
             scales[0, :, which, :n].t().reshape(-1).cpu().numpy(), want)
