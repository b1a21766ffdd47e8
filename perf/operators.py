"""The paged, rotated int8 key/value cache and the attention over it: cases, their plain forms in elementary
torch operations, and the framework's calls.

A case's "op" is one of

* ``store``      keys and values of new tokens written into pages of the cache and read back from it, as the
                 bfloat16 rows that the 8-bit codes stand for
* ``fetch``      a stored prefix read back from its pages
* ``attention``  new tokens of a batch of sequences (one, a few or a chunk each) attending to their pages
"""
import math
import random

import torch

own = False

GROUP = 256


# ------------------------------------------------------------------------------------------- cases

def _store(name, tokens, kv_heads, dim, page, fused):
    return {"name": name, "op": "store", "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page,
            "fused": fused}


def _fetch(name, tokens, kv_heads, dim, page):
    return {"name": name, "op": "fetch", "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page}


def _attention(name, batch, len_min, len_max, new_min, new_max, heads, kv_heads, dim, page, window=0, sinks=0):
    return {"name": name, "op": "attention", "batch": batch, "len_min": len_min, "len_max": len_max,
            "new_min": new_min, "new_max": new_max, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "window": window, "sinks": sinks}


def listed():
    return [
        # one new token of one sequence: the smallest write, where latency is all
        _store("store_1_token", 1, 8, 128, 16, True),
        # the step of a batch whose heads are small
        _store("store_96_tokens_d64", 96, 4, 64, 32, True),
        # a long prompt's keys and values, taken out of a fused projection's rows
        _store("store_16400_tokens", 16400, 8, 128, 64, True),
        # a short prefix taken out of the cache
        _fetch("fetch_333_tokens", 333, 8, 128, 16),
        # a long shared prefix taken out of the cache, to be kept elsewhere
        _fetch("fetch_100k_tokens", 100003, 8, 128, 64),
        # a chat's next token: one sequence, a few hundred tokens
        _attention("decode_1x300", 1, 300, 300, 1, 1, 32, 8, 128, 16),
        # one sequence with a long document before it
        _attention("decode_1x131071", 1, 131071, 131071, 1, 1, 32, 8, 128, 64),
        # a server's batch, contexts of every length, grouped heads
        _attention("decode_64x8k_ragged", 64, 1, 8192, 1, 1, 32, 8, 128, 16),
        # a batch that streams without end: a window and the first tokens stay, six queries to a head
        _attention("decode_96x8k_window", 96, 3000, 8192, 1, 1, 48, 8, 128, 32, 2048, 4),
        # drafted tokens verified together, small heads
        _attention("verify_16x4k_d64", 16, 700, 4099, 2, 4, 32, 8, 64, 16),
        # a chunk of a long prompt over what was stored before it
        _attention("chunk_2048_of_16384", 1, 16384, 16384, 2048, 2048, 32, 8, 128, 64),
        # a mixed batch: single tokens and chunks of odd sizes, no grouping, a window and sinks
        _attention("mixed_8_chunks_window", 8, 1600, 5003, 1, 1500, 24, 24, 128, 128, 1000, 5),
    ]


def _spread(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["store", "fetch", "attention", "attention", "attention"])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 8, 24])
    if op == "store":
        return {"op": op, "tokens": _spread(rng, 1, 16400 * 8 // max(kv, 8)), "kv_heads": kv, "dim": dim,
                "page": page, "fused": rng.random() < 0.5}
    if op == "fetch":
        return {"op": op, "tokens": _spread(rng, 17, 100003 * 8 // max(kv, 8)), "kv_heads": kv, "dim": dim,
                "page": page}
    share = rng.choice([1, 2, 3, 4, 5, 6, 8]) if kv < 24 else 1
    window = rng.choice([0, 0, 0, _spread(rng, 128, 4096)])
    sinks = rng.choice([0, 1, 4, 70]) if window else 0
    if rng.random() < 0.6:  # one or a few tokens each
        batch = _spread(rng, 1, 128)
        most = min(131071, 250000 * 8 // max(kv, 8) // batch)
        high = _spread(rng, 64, max(65, most))
        new = rng.choice([1, 1, 1, 2, 4, 7])
    else:  # chunks
        batch = rng.choice([1, 1, 2, 3, 5, 8])
        new = _spread(rng, 17, 2048 // batch)
        high = new + _spread(rng, 1, 12000 // batch)
    low = max(new, rng.choice([high, 1 + high // 2, 1]))
    return {"op": op, "batch": batch, "len_min": low, "len_max": max(low, high),
            "new_min": rng.choice([new, 1]), "new_max": new, "heads": kv * share, "kv_heads": kv, "dim": dim,
            "page": page, "window": window, "sinks": sinks}


def _lengths(case):
    """Every sequence's context length and number of new tokens: the case's own, whatever the seed."""
    r = random.Random("%(batch)d %(len_min)d %(len_max)d %(new_min)d %(new_max)d" % case)
    lens = [r.randint(case["len_min"], case["len_max"]) for _ in range(case["batch"])]
    lens[-1] = case["len_max"]
    new = [min(n, r.randint(case["new_min"], case["new_max"])) for n in lens]
    new[-1] = min(lens[-1], case["new_max"])
    return lens, new


# ------------------------------------------------------------------------------------------- inputs

def _codes(gen, rows, dim):
    """Codes of rotated rows: nearly normal, the largest of a row at the grid's end."""
    c = torch.randn((rows, dim), generator=gen, device="cuda").mul_(40.0).round_().clamp_(-126, 126).to(torch.int8)
    c[:, 0] = torch.where(c[:, 0] < 0, -127, 127).to(torch.int8)
    at = torch.randint(0, dim, (rows, 1), generator=gen, device="cuda")
    first, there = c[:, :1].clone(), c.gather(1, at)
    c[:, :1] = there
    return c.scatter_(1, at, first)


def _pool(gen, pages, kv, page, dim):
    codes = torch.empty((pages, kv, 2, page, dim), dtype=torch.int8, device="cuda")
    flat = codes.view(-1, dim)
    for at in range(0, flat.shape[0], 1 << 21):
        n = min(1 << 21, flat.shape[0] - at)
        flat[at:at + n] = _codes(gen, n, dim)
    scales = torch.randn((pages, kv, 2, page), generator=gen, device="cuda").mul_(0.15).exp_().mul_(0.025)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] in ("store", "fetch"):
        n = case["tokens"]
        pages = -(-n // page) + 3
        slots = (torch.randperm(pages, generator=gen, device="cuda")[:, None] * page
                 + torch.arange(page, device="cuda")).reshape(-1)[3:n + 3].contiguous()
        codes, scales = _pool(gen, pages, kv, page, dim)
        state = {"case": dict(case), "slots": slots, "codes": codes, "scales": scales}
        if case["op"] == "store":
            # keys have a few channels that are far larger than the others; a fused projection gives the rows of
            # queries, keys and values side by side (four query heads to each here)
            wide = (6 if case["fused"] else 2) * kv
            rows = torch.randn((n, wide, dim), generator=gen, device="cuda")
            big = torch.randint(0, dim, (4,), generator=gen, device="cuda")
            rows[:, -2 * kv:-kv, big] *= 12.0
            rows = rows.to(torch.bfloat16)
            state["k"], state["v"] = rows[:, -2 * kv:-kv], rows[:, -kv:]
        return state
    lens, new = _lengths(case)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    codes, scales = _pool(gen, pages, kv, page, dim)
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["batch"], max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = (torch.randn((cu[-1], case["heads"], dim), generator=gen, device="cuda") * 2.0).to(torch.bfloat16)
    return {"case": dict(case), "codes": codes, "scales": scales, "table": table, "q": q, "max_new": max(new),
            "pages": max(need), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
            "one_each": all(n == 1 for n in new)}


# ------------------------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](state)
    return _PLAIN[case["op"]](state)


def _own_store(s):
    import hadamard_rotated_int8_b200 as sd
    sd.sdnq_kv_write(s["k"], s["v"], s["slots"], s["codes"], s["scales"], GROUP)
    return sd.sdnq_kv_read(s["slots"], s["codes"], s["scales"], GROUP)


def _own_fetch(s):
    import hadamard_rotated_int8_b200 as sd
    return sd.sdnq_kv_read(s["slots"], s["codes"], s["scales"], GROUP)


def _own_attention(s):
    import hadamard_rotated_int8_b200 as sd
    return sd.sdnq_attention_paged(s["q"], s["codes"], s["scales"], s["table"], s["lens"],
                                   cu_q=None if s["one_each"] else s["cu"], max_q=s["max_new"], group=GROUP,
                                   window=s["case"]["window"], sinks=s["case"]["sinks"])


_OWN = {"store": _own_store, "fetch": _own_fetch, "attention": _own_attention}


# ---- plain forms

def _stage(z, h):
    """One stage of the butterfly over the last dimension: (a, b) -> (a + b, a - b) at distance h."""
    p = z.unflatten(-1, (-1, 2, h))
    a, b = p[..., 0, :], p[..., 1, :]
    return torch.stack((a + b, a - b), dim=-2).flatten(-3)


def _butterfly(z):
    z = _stage(_stage(_stage(_stage(_stage(_stage(z, 1), 2), 4), 8), 16), 32)
    return _stage(z, 64) if z.shape[-1] == 128 else z


def _factor(dim):
    return float(torch.tensor(1.0 / math.sqrt(min(GROUP, dim)), dtype=torch.float32))


def _quantize(x):
    """Rows of x rotated, as whole numbers in 32-bit floats, and their scales."""
    z = _butterfly(x.float())
    step = z.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=x.device)
    codes = torch.where(step > 0, torch.round(z / step).clamp(-127.0, 127.0), 0.0)
    return codes, (step * _factor(x.shape[-1])).squeeze(-1)


def _values(codes, scales):
    return (_butterfly(codes.float()) * (scales * _factor(codes.shape[-1]))[..., None]).to(torch.bfloat16)


def _plain_store(s):
    page = s["case"]["page"]
    ids, off = s["slots"] // page, s["slots"] % page
    for_k, k_scale = _quantize(s["k"])
    for_v, v_scale = _quantize(s["v"])
    s["codes"][ids, :, 0, off] = for_k.to(torch.int8)
    s["codes"][ids, :, 1, off] = for_v.to(torch.int8)
    s["scales"][ids, :, 0, off] = k_scale
    s["scales"][ids, :, 1, off] = v_scale
    return _plain_fetch(s)


def _plain_fetch(s):
    page = s["case"]["page"]
    ids, off = s["slots"] // page, s["slots"] % page
    return (_values(s["codes"][ids, :, 0, off], s["scales"][ids, :, 0, off]),
            _values(s["codes"][ids, :, 1, off], s["scales"][ids, :, 1, off]))


def _plain_attention(s):
    case, q, lens, cu = s["case"], s["q"], s["lens"].long(), s["cu"].long()
    kv, dim, window, sinks = case["kv_heads"], case["dim"], case["window"], case["sinks"]
    share = case["heads"] // kv
    batch, new = case["batch"], s["max_new"]
    ids = s["table"][:, :s["pages"]].long().clamp(min=0)
    held = s["codes"][ids].permute(0, 2, 3, 1, 4, 5).flatten(3, 4).float()        # [B, kv, 2, L, D]
    scale = s["scales"][ids].permute(0, 2, 3, 1, 4).flatten(3, 4)                 # [B, kv, 2, L]
    count = cu[1:] - cu[:-1]
    i = torch.arange(new, device=q.device)
    have = i < count[:, None]                                                     # [B, new]
    rows = torch.where(have, cu[:-1, None] + i, 0)
    qc, qs = _quantize(q)
    qc = qc[rows].view(batch, new, kv, share, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    qs = qs[rows].view(batch, new, kv, share).permute(0, 2, 1, 3).flatten(2, 3)
    # products of whole numbers, exact in 32 bits
    logits = qc @ held[:, :, 0].transpose(-1, -2)
    logits = logits * (qs[..., None] * scale[:, :, 0, None, :]) * (1.0 / math.sqrt(dim))
    at = (lens - count)[:, None] + i                                              # [B, new]
    j = torch.arange(logits.shape[-1], device=q.device)
    sees = j <= at[..., None]
    if window > 0:
        sees = sees & ((j > at[..., None] - window) | (j < sinks))
    sees = sees.repeat_interleave(share, dim=1)[:, None]
    logits = logits.masked_fill(~sees, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = p @ (held[:, :, 1] * torch.where(j < lens[:, None], 1.0, 0.0)[:, None, :, None] * scale[:, :, 1, :, None])
    o = _butterfly(torch.where(total > 0, o / total, 0.0)) * _factor(dim)
    o = o.view(batch, kv, new, share, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, new, H, D]
    t = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return o[b, t - cu[b]].to(torch.bfloat16)


_PLAIN = {"store": _plain_store, "fetch": _plain_fetch, "attention": _plain_attention}


# ------------------------------------------------------------------------------------------- work

def work(case):
    kv, dim = case["kv_heads"], case["dim"]
    if case["op"] != "attention":
        rows = 2 * case["tokens"] * kv
        levels = int(math.log2(dim))
        held, plain = rows * (dim + 4), rows * 2 * dim + 8 * case["tokens"]
        if case["op"] == "store":  # the rows once, the codes written and read back, the rows written
            return {"bytes": 2 * plain + 2 * held, "flops": rows * dim * (2 * levels + 3)}
        return {"bytes": plain + held, "flops": rows * dim * (levels + 1)}
    lens, new = _lengths(case)
    window, sinks = case["window"], case["sinks"]
    pairs = keys = 0
    for n, m in zip(lens, new):
        first = n - m
        if window <= 0:
            keys += n
            pairs += m * first + m * (m + 1) // 2
        else:
            low = max(0, first - window + 1)
            keys += n - low + min(sinks, low)
            for p in range(first, n):
                low = max(0, p - window + 1)
                pairs += p + 1 - low + min(sinks, low)
    return {"bytes": keys * kv * 2 * (dim + 4) + 4 * sum(new) * case["heads"] * dim,
            "flops": 4 * dim * pairs * case["heads"]}


# ------------------------------------------------------------------------------------------- 64 bits

def _sylvester(dim):
    """The rotation's matrix from its definition, H[i][j] = (-1)^(number of ones in i & j), divided by sqrt(dim)."""
    i = torch.arange(dim)
    both = i[:, None] & i
    ones = sum((both >> b) & 1 for b in range(8))
    return ((1 - 2 * (ones % 2)).double() / math.sqrt(dim)).cuda()


def _round64(x):
    """Rows rotated in 64 bits and put on their grid of 127 steps to each side."""
    z = x.double() @ _sylvester(x.shape[-1])
    step = z.abs().amax(-1, keepdim=True) / 127.0
    return torch.where(step > 0, torch.round(z / step), 0.0) * step


def exact(case, seed):
    s = prepare(case, seed)
    rotation = _sylvester(case["dim"])
    page = case["page"]
    if case["op"] == "store":
        return tuple(_round64(s[x]) @ rotation for x in ("k", "v"))
    if case["op"] == "fetch":
        held, scale = s["codes"].transpose(1, 3).flatten(0, 1), s["scales"].transpose(1, 3).flatten(0, 1)
        rows = held[s["slots"]].double() * scale[s["slots"]].double()[..., None]  # [T, 2, kv, D]
        return rows[:, 0] @ rotation, rows[:, 1] @ rotation
    lens, new = _lengths(case)
    share = case["heads"] // case["kv_heads"]
    parts, first = [], 0
    for b, (n, m) in enumerate(zip(lens, new)):
        ids = s["table"][b, :-(-n // page)].long()
        q = _round64(s["q"][first:first + m])                                    # [m, H, D]
        first += m
        at = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None]
        hidden = j > at
        if case["window"] > 0:
            hidden = hidden | ((j <= at - case["window"]) & (j >= case["sinks"]))
        o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        for h in range(case["kv_heads"]):
            held = s["codes"][ids, h].transpose(0, 1).flatten(1, 2)[:, :n].double()
            held *= s["scales"][ids, h].transpose(0, 1).flatten(1, 2)[:, :n, None].double()
            for g in range(h * share, (h + 1) * share):
                w = (q[:, g] @ held[0].T / math.sqrt(case["dim"])).masked_fill_(hidden, -math.inf)
                o[:, g] = torch.softmax(w, dim=-1) @ held[1] @ rotation
        parts.append(o)
    return torch.cat(parts)
