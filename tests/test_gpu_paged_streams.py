"""The paged cache's calls on several streams, without a synchronisation between them: every result bit for bit that
of the same call made alone."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _build
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def test_every_call_at_once_from_host_threads():
    r = subprocess.run([sys.executable, "-m", "tests.paged_concurrency_case"], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "CONCURRENCY ok 10" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.parametrize("D,page", [(128, 16), (64, 128)])
def test_back_to_back_on_one_stream(D, page):
    """Rounds of store, chunk, single tokens and read-back with no synchronisation between, the same slots, workspace and
    cache written over in each round. The kernels start while the one before drains; one that read the cache or the
    workspace before that was complete would see another round's."""
    Hkv, H, lens, rounds = 2, 8, [900, 300], 5
    codes, scales = sd.kv_cache(1 + sum(ref.pages_of(lens, page)), Hkv, page, D)
    ids = torch.randperm(codes.shape[0], generator=torch.Generator().manual_seed(4)).to(torch.int32)
    table = torch.full((2, max(ref.pages_of(lens, page))), -1, dtype=torch.int32)
    first = ref.pages_of(lens, page)[0]
    table[0, :first], table[1, :ref.pages_of(lens, page)[1]] = ids[:first], ids[first:-1]
    slots = torch.cat([table[b, torch.arange(n) // page].long() * page + torch.arange(n) % page
                       for b, n in enumerate(lens)]).cuda()
    table, gl = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    new = [200, 40]
    cu = torch.from_numpy(ref.offsets(new)).cuda()
    ks, vs, qs, ones = ([ref.queries(n, h, D, 10 * r + i).cuda() for r in range(rounds)]
                        for i, (n, h) in enumerate([(sum(lens), Hkv), (sum(lens), Hkv), (240, H), (2, H)]))
    ws = torch.empty(sd.attention_paged_workspace(H, Hkv, D), dtype=torch.uint8, device="cuda")

    def round_(r, wait):
        sd.sdnq_kv_write(ks[r], vs[r], slots, codes, scales)
        wait()
        a = sd.sdnq_attention_paged(qs[r], codes, scales, table, gl, cu_q=cu, max_q=200, ws=ws)
        wait()
        b = sd.sdnq_attention_paged(ones[r], codes, scales, table, gl, ws=ws, window=100, sinks=2)
        wait()
        c = sd.sdnq_kv_read(slots, codes, scales)
        wait()
        return a, b, *c

    alone = [round_(r, torch.cuda.synchronize) for r in range(rounds)]
    together = [round_(r, lambda: None) for r in range(rounds)]
    torch.cuda.synchronize()
    for r, (x, y) in enumerate(zip(alone, together)):
        assert all(torch.equal(g, w) for g, w in zip(x, y)), r


def test_a_captured_fork_with_memory_of_its_own():
    """Two branches of one graph, on the capturing stream and on another that joined the capture, whose calls make
    their workspaces and outputs themselves; replayed with other inputs and lengths."""
    gpu, gl, gc, qs = setup(128, [3000, 900, 64], [150, 1, 40], 101)
    ones = [ref.queries(3, 8, 128, 110 + i).cuda() for i in range(3)]
    q, one = qs[0].clone(), ones[0].clone()
    chunk = lambda **kw: sd.sdnq_attention_paged(q, *gpu, gl, cu_q=gc, max_q=150, **kw)           # noqa: E731
    single = lambda **kw: sd.sdnq_attention_paged(one, *gpu, gl, window=500, sinks=3, **kw)       # noqa: E731
    chunk(), single()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        a, b = chunk(), [single(stream=side) for _ in range(2)]
        c = single()
        here.wait_stream(side)
    for i in range(3):
        q.copy_(qs[i])
        one.copy_(ones[i])
        gl.copy_(torch.tensor([3000 - 700 * i, 900 + 5 * i, 64]))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (a, *b, c)]
        want = [chunk(), single(), single(), single()]
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i
