"""Concurrent callers: host threads, each with its own CUDA stream and its own layouts (and so
its own workspace), run the whole path at once on different workloads, several times over.
Every result must equal, byte for byte, the same calls made one after another on one stream:
the library keeps no state between calls other than per-device launch settings looked up under
a lock (the no-allocation layout, whose shared array is documented as not to be used by
overlapping calls, is left out)."""
import threading

import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import dev, dev_bf16

pytestmark = pytest.mark.gpu

# (workload, tokens, hidden size): the fused call's staged dispatch (qwen3, dsv3), top-2 routing
# over 8 experts (mixtral), and the two-kernel layout beyond one cluster (the large microbatch's
# routing at 40,000 tokens, 320,000 ids; a short hidden size keeps the host-side inputs small)
CASES = [("qwen3", 1500, None), ("dsv3", 600, None), ("mixtral", 3000, None), ("dsv3_large", 40000, 256)]
REPEATS = 3


def host_inputs(cfg) -> tuple:
    return W.make_inputs(cfg), W.make_expert_out(cfg)


def run_path(ep, cfg, host, stream, start=None) -> dict:
    T, H, E, K, S, P = cfg.T, cfg.H, cfg.E, cfg.K, cfg.S, cfg.P
    C = cfg.rerun_C if cfg.rerun_C else cfg.capacity
    inp, y_h = host
    with torch.cuda.stream(stream):
        ids, probs, x, y = dev(inp["topk_ids"]), dev(inp["probs"]), dev_bf16(inp["x"]), dev_bf16(y_h)
        if start is not None:
            start.wait()          # every thread launches its work at the same time
        res = {}
        for rep in range(REPEATS):
            L = ep.Layout(T, K, E, P, bool(S))
            _, nv = ep.dispatch_layout_nvfp4(ids, x, E, P, C, bool(S), out_layout=L, stream=stream)
            L2 = ep.dispatch_layout(ids, E, P, C, bool(S), stream=stream)
            bf = ep.dispatch_bf16(x, L2, stream=stream)
            f8 = ep.dispatch_fp8(x, L2, stream=stream)
            out = ep.combine(y, probs, L, stream=stream)
            gy, gp = ep.combine_bwd(x, y, probs, L2, stream=stream)
            gx = ep.dispatch_bwd(y, L2, stream=stream)
            stream.synchronize()
            got = {"row_of": L.row_of, "row_offsets": L.row_offsets, "expert_ids": L2.expert_ids,
                   "src_info": L2.src_info, "fp4": nv[0], "sc": nv[1], "inv": nv[2], "bf16": bf,
                   "fp8": f8[0], "fp8_scales": f8[1], "out": out, "gy": gy, "gp": gp, "gx": gx}
            got = {k: v.contiguous().view(torch.uint8).cpu().numpy() for k, v in got.items()}
            if rep == 0:
                res = got
            else:
                for k in res:
                    assert np.array_equal(res[k], got[k]), f"{cfg.name}: {k} changed between repeats"
    return res


def test_concurrent_streams_match_serial():
    import combine_topk_ids_histogram_gb300 as ep
    cfgs = [W.scaled(W.CONFIGS[n], T=T, H=H) for n, T, H in CASES]
    hosts = [host_inputs(c) for c in cfgs]
    serial = [run_path(ep, c, h, torch.cuda.current_stream()) for c, h in zip(cfgs, hosts)]

    results, errors = [None] * len(cfgs), []
    start = threading.Barrier(len(cfgs), timeout=300)

    def worker(i):
        try:
            results[i] = run_path(ep, cfgs[i], hosts[i], torch.cuda.Stream(), start)
        except Exception as e:   # reported below, from the main thread
            errors.append(f"{cfgs[i].name}: {e!r}")

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(cfgs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=600)
    assert not errors, "\n".join(errors)
    for cfg, want, got in zip(cfgs, serial, results):
        assert got is not None, f"{cfg.name}: no result"
        for k in want:
            assert np.array_equal(want[k], got[k]), f"{cfg.name}: {k} differs from the serial run"


def test_threads_that_share_a_layout_and_a_stream():
    """The expert products are two launches through a workspace: host threads that call them at once, on one stream and
    one layout but for their own x, must not meet in it."""
    import combine_topk_ids_histogram_gb300 as ep
    T, K, E, H, N, n_threads, calls = 64, 4, 64, 512, 2600, 4, 40        # several items per CTA: they are drawn
    g = torch.Generator().manual_seed(5)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int().cuda()
    L = ep.dispatch_layout(ids, E)
    w = (torch.randint(0, 256, (E, N, H // 2), generator=g, dtype=torch.uint8).cuda(),
         torch.randint(0, 0x7F, (E, N, H // 16), generator=g, dtype=torch.uint8).cuda(),
         torch.rand(E, N, generator=g).cuda())
    xs = [torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(n_threads)]
    want = [ep.expert_matvec(x, *w, L) for x in xs]
    outs = [[torch.full_like(want[0], float("nan")) for _ in range(calls)] for _ in xs]
    errors, start = [], threading.Barrier(n_threads, timeout=300)

    def worker(i):
        try:
            start.wait()
            for out in outs[i]:
                ep.expert_matvec(xs[i], *w, L, out=out)
        except Exception as e:   # reported below, from the main thread
            errors.append(repr(e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=worker, args=(i,)) for i in range(n_threads)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=600)
    torch.cuda.synchronize()
    assert not errors, errors
    for i in range(n_threads):
        assert all(torch.equal(o, want[i]) for o in outs[i]), f"thread {i}"


def test_operators_on_concurrent_streams_match_serial():
    """The norm, the router and the expert products, each thread on its own stream with its own inputs."""
    import combine_topk_ids_histogram_gb300 as ep

    def run(seed, stream):
        T, H, E, K, N = 300 + 777 * seed, 512, 32, 4, 192
        g = torch.Generator().manual_seed(seed)
        with torch.cuda.stream(stream):
            x, gy = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(2))
            wn, bn = torch.randn(H, generator=g).bfloat16().cuda(), torch.randn(H, generator=g).bfloat16().cuda()
            logits, gp = torch.randn(T, E, generator=g).cuda(), torch.randn(T, K, generator=g).cuda()
            codes = torch.randint(0, 256, (E, N, H // 2), generator=g, dtype=torch.uint8).cuda()
            scales = torch.randint(0, 0x7F, (E, N, H // 16), generator=g, dtype=torch.uint8).cuda()
            rs = torch.rand(E, N, generator=g).cuda()
            res = []
            for _ in range(5):
                y, mean, rstd = ep.layer_norm(x, wn, bn)
                dx, dw, db = ep.layer_norm_bwd(gy, x, wn, mean, rstd, bias=True)
                ids, p = ep.router_topk(logits, K)
                dl = ep.router_topk_bwd(gp, logits, ids)
                L = ep.dispatch_layout(ids, E)
                o = ep.expert_matvec(y, codes, scales, rs, L, swiglu=True)
                res.append([y, mean, rstd, dx, dw, db, ids, p, dl, o])
            stream.synchronize()
            return [[t.contiguous().view(torch.uint8).cpu() for t in r] for r in res]

    seeds = range(4)
    serial = [run(s, torch.cuda.current_stream()) for s in seeds]
    got, errors = [None] * len(serial), []

    def worker(s):
        try:
            got[s] = run(s, torch.cuda.Stream())
        except Exception as e:   # reported below, from the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(s,)) for s in seeds]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=600)
    assert not errors, errors
    for a, b in zip(serial, got):
        assert all(torch.equal(u, v) for r in b for u, v in zip(a[0], r))


def test_expert_products_keep_no_memory():
    """A call's workspace is the call's own: nothing of it stays with the layout."""
    import combine_topk_ids_histogram_gb300 as ep
    T, E, H, N = 2048, 8, 1024, 32
    ids = torch.arange(2 * T, dtype=torch.int32, device="cuda").view(T, 2) % E
    L = ep.dispatch_layout(ids, E)
    x = torch.randn(T, H, device="cuda").bfloat16()
    w = (torch.zeros(E, N, H // 2, dtype=torch.uint8, device="cuda"), torch.zeros(E, N, H // 16, dtype=torch.uint8, device="cuda"),
         torch.ones(E, N, device="cuda"))
    out = torch.empty(L.R_max, N, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        ep.expert_matvec(x, *w, L, out=out)
    assert torch.cuda.memory_allocated() == before
