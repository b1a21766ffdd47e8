"""Plain 64-bit implementation of the paged rotated-int8 cache and of the attention over it, in numpy, and the
builders of the inputs that its tests share. Row codes and scales come from the oracle's row quantizer (the fp32
definition, bit for bit); everything after them is 64-bit."""
import math

import numpy as np
import torch

import oracle
from hadamard_rotated_int8_b200 import synthetic


def quantize_rows(x: torch.Tensor, group: int):
    """[..., D] bf16 -> (int8 codes [..., D], fp32 scales [...]) by the oracle."""
    D = x.shape[-1]
    flat = np.ascontiguousarray(synthetic.bits(x.contiguous().reshape(-1, D)))
    if flat.shape[0] == 0:
        return np.zeros(x.shape, np.int8), np.zeros(x.shape[:-1], np.float32)
    c, s = oracle.rotate_quantize(flat, min(group, D))
    return c.reshape(x.shape), s.reshape(x.shape[:-1])


def unrotate(z: np.ndarray, group: int) -> np.ndarray:
    """z [..., D] float64 times the normalised block-diagonal Sylvester matrix of groups of min(group, D)."""
    D = z.shape[-1]
    g = min(group, D)
    i = np.arange(g)
    ones = np.array([[bin(a & b).count("1") for b in i] for a in i])
    H = np.where(ones % 2 == 0, 1.0, -1.0)   # signs only: sums of whole numbers stay exact
    return (z.reshape(z.shape[:-1] + (D // g, g)) @ H).reshape(z.shape) / math.sqrt(g)


def visible(pos: int, n: int, window: int, sinks: int) -> np.ndarray:
    j = np.arange(n)
    see = j <= pos
    if window > 0:
        see &= (j > pos - window) | (j < sinks)
    return see


def attention(q: torch.Tensor, codes, scales, table, lens, cu, group, scale, window=0, sinks=0):
    """o [T, H, D] float64, and per row the sum over visible keys of probability times |v| (2-norm of the row):
    the size that roundings of the probabilities scale with. codes, scales, table: numpy."""
    T, H, D = q.shape
    P, Hkv, _, page, _ = codes.shape
    share = H // Hkv
    qc, qs = quantize_rows(q, group)
    o = np.zeros((T, H, D))
    size = np.zeros((T, H))
    for b in range(len(lens)):
        L, n = int(lens[b]), int(cu[b + 1] - cu[b])
        ids = table[b, :-(-L // page)].astype(np.int64) if L > 0 else np.zeros(0, np.int64)
        good = np.repeat((ids >= 0) & (ids < P), page)[:L]
        ids = np.clip(ids, 0, P - 1)
        for h in range(H):
            kv = h // share
            with np.errstate(all="ignore"):
                kc = codes[ids, kv, 0].reshape(-1, D)[:L].astype(np.int64)
                vc = codes[ids, kv, 1].reshape(-1, D)[:L].astype(np.float64)
                ks = scales[ids, kv, 0].reshape(-1)[:L].astype(np.float64)
                vs = scales[ids, kv, 1].reshape(-1)[:L].astype(np.float64)
                for i in range(n):
                    t = int(cu[b]) + i
                    see = visible(L - n + i, L, window, sinks) & good
                    if not see.any():
                        continue
                    x = (kc[see] @ qc[t, h].astype(np.int64)) * (float(qs[t, h]) * ks[see]) * scale
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    held = vc[see] * vs[see][:, None]
                    o[t, h] = unrotate(w @ held, group)
                    size[t, h] = w @ np.linalg.norm(held, axis=1)
    return o, size


def bound(o, size, keys: int, logit: float = 64.0):
    """Row-norm bound on |out - o|: the rotation keeps norms, so roundings of the probabilities (half a bf16 step,
    2^-8 relative each) move a row by at most 2^-8 of `size`; the fp32 sums over `keys` keys add 2 keys 2^-24; logits
    of up to `logit` in base e a few fp32 roundings off and the exponential's 2^-22 move a probability by
    (4 logit 2^-24 + 2^-21); the butterfly adds log2(D) + 2 fp32 roundings (2^-20); o is rounded once, half a bf16
    step of each element."""
    rel = 2.0 ** -8 + 2 * keys * 2.0 ** -24 + 4 * logit * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -20
    return rel * size * (1 + 2.0 ** -7) + 2.0 ** -8 * np.linalg.norm(o, axis=-1) + 1e-30


class Cache:
    """A pool on the CPU (numpy) and on the GPU (torch) with the same bytes, and page tables over it."""

    def __init__(self, Hkv, page, D, need, seed, spare=2, group=256, width=None, k_amp=1.0, fill=True):
        """need: pages of each sequence; ids are a random permutation. Entries past a sequence's pages are -7."""
        rng = np.random.default_rng(seed)
        P = int(sum(need)) + spare
        self.Hkv, self.page, self.D, self.group, self.P = Hkv, page, D, group, P
        ids = rng.permutation(P)
        self.table = np.full((len(need), width or max([1] + list(need))), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        if fill:
            rows = torch.from_numpy(rng.standard_normal((P * Hkv * 2 * page, D)).astype(np.float32))
            rows *= torch.from_numpy(np.exp(0.5 * rng.standard_normal((rows.shape[0], 1))).astype(np.float32)) * k_amp
            c, s = quantize_rows(rows.to(torch.bfloat16), group)
            self.codes, self.scales = c.reshape(P, Hkv, 2, page, D), s.reshape(P, Hkv, 2, page)
        else:  # what memory that was never written may hold
            self.codes = rng.integers(-128, 128, (P, Hkv, 2, page, D), dtype=np.int8)
            self.scales = np.where(rng.random((P, Hkv, 2, page)) < 0.5, np.nan, np.inf).astype(np.float32)

    def gpu(self):
        return (torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scales).cuda(),
                torch.from_numpy(self.table).cuda())


def pages_of(lens, page):
    return [-(-int(n) // page) for n in lens]


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def queries(T, H, D, seed, amp=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, D, generator=gen) * amp).to(torch.bfloat16)
