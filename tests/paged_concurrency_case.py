"""The paged cache's calls at once, beside linear layers and the dense attention: one host thread per call, each on its
own CUDA stream, started together in a fresh process, so that the library's once-per-device set-up happens while other
calls run. Each thread repeats its call a few times; every result is compared bit for bit with the same call made alone
afterwards. Run as ``python -m tests.paged_concurrency_case``; prints ``CONCURRENCY ok <n>`` on success."""
import sys
import threading

import torch

import hadamard_rotated_int8_b200 as sd

REPEATS = 4


def main():
    torch.cuda.set_device(0)
    gen = torch.Generator().manual_seed(91)

    def rows(T, H, D):
        return torch.randn(T, H, D, generator=gen).to(torch.bfloat16).cuda()

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    jobs = {}
    for D, page in ((128, 16), (64, 64)):
        pages = 2048 // page
        codes = torch.randint(-127, 128, (pages, 2, 2, page, D), dtype=torch.int8, generator=gen).cuda()
        scales = (0.02 + 0.01 * torch.rand(pages, 2, 2, page, generator=gen)).cuda()
        table = torch.randperm(pages, generator=gen).to(torch.int32).cuda().view(2, -1)
        slots = torch.randperm(2048, generator=gen)[:700].cuda()
        lens = i32(1000, 700)
        one, few, many = rows(2, 8, D), rows(7, 8, D), rows(500, 8, D)
        cu_few, cu_many = i32(0, 3, 7), i32(0, 499, 500)
        k, v = rows(700, 2, D), rows(700, 2, D)

        def stored(codes=codes, scales=scales, slots=slots, k=k, v=v):
            c, s = torch.zeros_like(codes), torch.zeros_like(scales)
            sd.sdnq_kv_write(k, v, slots, c, s)
            return [c, s, *sd.sdnq_kv_read(slots, c, s)]

        args = (codes, scales, table, lens)
        jobs[f"store_{D}"] = stored
        jobs[f"one_{D}"] = lambda q=one, a=args: [sd.sdnq_attention_paged(q, *a)]
        jobs[f"few_{D}"] = lambda q=few, a=args, cu=cu_few: [sd.sdnq_attention_paged(q, *a, cu_q=cu, max_q=4)]
        jobs[f"many_{D}"] = lambda q=many, a=args, cu=cu_many: [sd.sdnq_attention_paged(q, *a, cu_q=cu, window=300,
                                                                                       sinks=5)]
    x = torch.randn(640, 1024, generator=gen).to(torch.bfloat16).cuda()
    W = torch.randn(768, 1024, generator=gen).to(torch.bfloat16).cuda()
    qkv = [torch.randn(1, 700, 4, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(3)]
    qW, sW = sd.sdnq_rotate_quant_weight(W)
    jobs["linear"] = lambda: [sd.linear(x, qW, sW)]
    jobs["attention"] = lambda: [sd.sdnq_attention_int8qk(*qkv)]
    torch.cuda.synchronize()
    results, errors, start = {}, [], threading.Barrier(len(jobs))

    def worker(name, fn):
        try:
            stream = torch.cuda.Stream()
            start.wait(timeout=60)
            with torch.cuda.stream(stream):
                results[name] = [fn() for _ in range(REPEATS)]
            stream.synchronize()
        except Exception as e:  # reported below
            errors.append(f"{name}: {e!r}")

    threads = [threading.Thread(target=worker, args=j) for j in jobs.items()]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    torch.cuda.synchronize()
    if errors or any(t.is_alive() for t in threads):
        print("CONCURRENCY errors", errors, file=sys.stderr)
        return 1
    bad = []
    for name, fn in jobs.items():
        alone = fn()
        torch.cuda.synchronize()
        bad += [name for r in results[name] for a, b in zip(alone, r) if not torch.equal(a, b)]
    status = sd.sdnq_device_status()
    if bad or status != 0:
        print("CONCURRENCY mismatch", bad, "device status", status, file=sys.stderr)
        return 1
    print(f"CONCURRENCY ok {len(jobs)}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
