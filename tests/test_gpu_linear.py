"""The grouped 16-bit products and their gradients against the 64-bit definition."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def normal(seed, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def guarded(rows, cols, dtype):
    """A buffer of rows x cols in front of guard values."""
    buf = torch.full((rows * cols + 4096,), 7.0, dtype=dtype, device="cuda")
    return buf, buf[:rows * cols].view(rows, cols)


def check_forward(ep, L, x, w, swiglu):
    G, N, K = w.shape
    n_out = N // 2 if swiglu else N
    buf, out = guarded(L.R_max, n_out, w.dtype)
    gbuf, gu = guarded(L.R_max, N, w.dtype)
    if swiglu:
        ep.expert_linear(x, w, L, swiglu=True, save=True, out=(out, gu))
        assert torch.equal(ep.expert_linear(x, w, L, swiglu=True)[:L.row_offsets[-1]], out[:L.row_offsets[-1]])
    else:
        ep.expert_linear(x, w, L, out=out)
    assert ep.read_status(L) == 0
    for g, rows in enumerate(ref.extents(L)):
        y, err = ref.linear(x[rows], w[g])
        if swiglu:
            ref.assert_within(gu[rows], y, ref.rounded(y, err, w.dtype), f"gate and up of group {g}")
            y, err = ref.glu(y, err)
        ref.assert_within(out[rows], y, ref.rounded(y, err, w.dtype), f"group {g}")
    R = int(L.row_offsets[-1])
    assert (buf[R * n_out:] == 7).all() and (gbuf[R * N if swiglu else 0:] == 7).all(), "rows behind the last one were written"
    return out


def check_backward(ep, L, grad, x, w, gate_up, wide, before=None):
    G, N, K = w.shape
    cols = K if gate_up is None else 2 * K
    buf, gx = guarded(L.R_max, cols, w.dtype)
    wt = torch.float32 if wide else w.dtype
    wbuf = torch.full((G * N * K + 4096,), 7.0, dtype=wt, device="cuda")
    gw = wbuf[:G * N * K].view(G, N, K)
    if before is not None:
        gw.copy_(before)
    ep.expert_linear_bwd(grad, x, w, L, gate_up=gate_up, accumulate=before is not None, out=(gx, gw))
    assert ep.read_status(L) == 0
    for g, rows in enumerate(ref.extents(L)):
        d, err = ref.linear(grad[rows], w[g].t())
        if gate_up is not None:
            d, err = ref.grad_gate(d, err, gate_up[rows])
        ref.assert_within(gx[rows], d, ref.rounded(d, err, w.dtype), f"grad_x of group {g}")
        dw, err = ref.grad_w(grad[rows], x[rows])
        if before is not None:
            dw = dw + before[g].double()
            err = err + 2.0 ** -23 * (dw.abs() + before[g].abs().double()) * (1 + (rows.stop - rows.start) / 2048)
        ref.assert_within(gw[g], dw, ref.rounded(dw, err, wt), f"grad_w of group {g}")
    R = int(L.row_offsets[-1])
    assert (buf[R * cols:] == 7).all() and (wbuf[G * N * K:] == 7).all(), "something behind the outputs was written"
    return gx, gw


# Rows per group around the steps of 16, 32, 64, 128 and 256 rows; empty groups at both ends and between; one row in all.
COUNTS = {"one": [0, 1, 0], "few": [1, 2, 0, 3, 15, 16, 17], "edges": [31, 32, 33, 63, 64, 65, 0, 127], "tiles": [128, 129, 255, 256, 257, 0],
          "long": [1, 700, 0, 0, 513], "many": [i % 5 for i in range(200)]}
# (K, N): the smallest, one block and a bit, more than a tile, odd multiples of 16
SIZES = [(16, 32), (64, 64), (80, 160), (272, 544), (128, 256), (2048, 96), (48, 1056)]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N", SIZES)
def test_forward(counts, K, N):
    import combine_topk_ids_histogram_gb300 as ep
    dtype = F16 if (K + N) % 32 else BF16
    L = ref.layout_of(ep, COUNTS[counts])
    x, w = normal(K, L.R_max, K, dtype=dtype), normal(N, L.G, N, K, dtype=dtype, scale=K ** -0.5)
    check_forward(ep, L, x, w, False)
    check_forward(ep, L, x, w, True)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N", SIZES)
def test_backward(counts, K, N):
    import combine_topk_ids_histogram_gb300 as ep
    dtype = BF16 if (K + N) % 32 else F16
    L = ref.layout_of(ep, COUNTS[counts], seed=1)
    x, w, g = normal(K, L.R_max, K, dtype=dtype), normal(N, L.G, N, K, dtype=dtype, scale=N ** -0.5), normal(K + N, L.R_max, N, dtype=dtype)
    check_backward(ep, L, g, x, w, None, False)
    check_backward(ep, L, g, x, w, normal(3, L.R_max, 2 * K, dtype=dtype, scale=2.0), True)


@pytest.mark.parametrize("T,E,K,S,pad,capacity", [(100, 8, 2, 1, 1, None), (77, 5, 3, 1, 128, None), (300, 16, 4, 0, 16, 2000), (0, 4, 2, 0, 1, None),
                                                  (0, 3, 1, 1, 8, None), (40, 4, 1, 0, 1, 64)])
def test_layouts(T, E, K, S, pad, capacity):
    """Shared experts, padded groups, capacities, unused slots, no token at all."""
    import combine_topk_ids_histogram_gb300 as ep
    g = torch.Generator().manual_seed(T)
    ids = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :K].int()
    ids[torch.rand(T, K, generator=g) < 0.1] = -1
    L = ep.dispatch_layout_routed(E, topk_ids=ids.cuda(), fused_shared=bool(S), pad_multiple=pad, num_permuted_tokens=capacity)[0]
    H, N = 144, 96
    tokens = normal(1, T, H)
    x = ep.dispatch_bf16(tokens, L) if T else torch.empty(L.R_max, H, dtype=BF16, device="cuda")
    grad = normal(2, L.R_max, N)
    pads = (L.src_info[:, 0] < 0).nonzero()[:, 0] if T else []
    if T:
        pads = pads[pads < L.row_offsets[-1]]
        grad[pads] = 0
        assert (x[pads] == 0).all()
    w = normal(3, L.G, N, H, scale=H ** -0.5)
    out = check_forward(ep, L, x, w, False)
    check_forward(ep, L, x, w, True)
    if len(pads):
        assert (out[pads] == 0).all()
    check_backward(ep, L, grad, x, w, None, True)
    check_backward(ep, L, grad, x, w, None, True, before=normal(5, L.G, N, H, dtype=torch.float32))


def test_long_sums():
    """Weight gradients over more rows than the tensor cores add at a time, and their 16-bit form."""
    import combine_topk_ids_histogram_gb300 as ep
    L = ref.layout_of(ep, [2047, 2048, 2049, 4100, 1])
    x, w, g = normal(1, L.R_max, 80), normal(2, 5, 64, 80), normal(3, L.R_max, 64)
    check_backward(ep, L, g, x, w, None, False)
    check_backward(ep, L, g, x, w, None, True)
    check_backward(ep, L, g, x, w, None, True, before=normal(4, 5, 64, 80, dtype=torch.float32))
    # all of one sign, where a truncating adder loses most
    gx, gw = ep.expert_linear_bwd(g.abs(), x.abs(), w, L, grad_w_dtype=torch.float32)
    for i, rows in enumerate(ref.extents(L)):
        dw, err = ref.grad_w(g[rows].abs(), x[rows].abs())
        ref.assert_within(gw[i], dw, ref.rounded(dw, err, torch.float32), f"group {i}")


def test_strided_rows():
    import combine_topk_ids_histogram_gb300 as ep
    L = ref.layout_of(ep, [5, 0, 200, 17])
    wide, gwide = normal(1, L.R_max, 400), normal(2, L.R_max, 320)
    x, g = wide[:, 80:80 + 144], gwide[:, 8:8 + 96]
    w = normal(3, 4, 96, 144)
    check_forward(ep, L, x, w, False)
    check_forward(ep, L, x, w, True)
    check_backward(ep, L, g, x, w, None, True)
    with pytest.raises(ep.EPError):                      # rows that do not begin on 16 bytes
        ep.expert_linear(wide[:, 1:145], w, L)
    with pytest.raises(ep.EPError):
        ep.expert_linear(normal(1, L.R_max, 151)[:, :144], w, L)
    with pytest.raises(ValueError):
        ep.expert_linear(normal(1, 144, L.R_max).t(), w, L)


def test_rows_do_not_mix():
    """A row that holds NaN or infinities changes its own results and its group's weight gradient, nothing else; rows
    behind the last group's are not read into anything."""
    import combine_topk_ids_histogram_gb300 as ep
    counts, K, N = [3, 20, 0, 70, 9], 96, 64
    ids = torch.repeat_interleave(torch.arange(5), torch.tensor(counts)).int().view(-1, 1).cuda()
    L = ep.dispatch_layout_routed(5, topk_ids=ids, num_permuted_tokens=160)[0]
    x, w, g = normal(1, 160, K), normal(2, 5, N, K), normal(3, 160, N)
    clean = ep.expert_linear(x, w, L), *ep.expert_linear_bwd(g, x, w, L)
    x2, g2 = x.clone(), g.clone()
    x2[102:], g2[102:] = float("nan"), float("inf")
    for a, b in zip(clean, (ep.expert_linear(x2, w, L), *ep.expert_linear_bwd(g2, x2, w, L))):
        n = 102 if a.dim() == 2 else None
        assert torch.equal(a[:n], b[:n])
    x2[22], g2[22] = float("nan"), float("-inf")         # the last row of group 1
    y, (gx, gw) = ep.expert_linear(x2, w, L), ep.expert_linear_bwd(g2, x2, w, L)
    other = [i for i in range(102) if i != 22]
    assert torch.equal(y[other], clean[0][other]) and torch.equal(gx[other], clean[1][other])
    assert y[22].isnan().all() and not gx[22].isfinite().any()
    for i in (0, 2, 3, 4):
        assert torch.equal(gw[i], clean[2][i])
    assert gw[1].isnan().all()
    # an infinite weight reaches its output column only
    w2 = w.clone()
    w2[3, 10, 5] = float("inf")
    y = ep.expert_linear(x, w2, L)
    keep = [n for n in range(N) if n != 10]
    assert torch.equal(y[:102, keep], clean[0][:102, keep]) and not y[23:93, 10].isfinite().any()


def test_extreme_gates():
    """Gates whose exponential overflows or vanishes."""
    import combine_topk_ids_histogram_gb300 as ep
    L = ref.layout_of(ep, [40])
    x = torch.zeros(40, 16, dtype=BF16, device="cuda")
    x[:, 0] = torch.tensor([-1e4, -200, -90, -88, -87, -20, -1e-3, -0.0, 0.0, 1e-3, 20, 87, 88, 90, 200, 1e4] + [1.0] * 24).bfloat16()
    x[:, 1] = 1
    w = torch.zeros(1, 32, 16, dtype=BF16, device="cuda")
    w[0, :16, 0], w[0, 16:, 1] = 1, 3
    check_forward(ep, L, x, w, True)
    gu = torch.cat([x[:, :1].expand(40, 16), torch.full((40, 16), 3.0, device="cuda")], 1).bfloat16().contiguous()
    check_backward(ep, L, normal(1, 40, 48), x, normal(2, 1, 48, 16), gu, True)


def test_refusals(monkeypatch):
    """What the binding checks before the library sees it."""
    import combine_topk_ids_histogram_gb300 as ep
    L = ref.layout_of(ep, [30, 50])
    x, w, g, a, b = normal(1, 80, 64), normal(2, 2, 96, 64), normal(3, 80, 96), normal(4, 2, 8, 64), normal(5, 2, 64, 8)
    wrong = [lambda: ep.expert_linear(x[:79], w, L), lambda: ep.expert_linear(x[:, :48], w, L), lambda: ep.expert_linear(x, w[:1], L),
             lambda: ep.expert_linear(x, w[0], L), lambda: ep.expert_linear(x, w, L, save=True), lambda: ep.expert_linear(x, w, L, out=x),
             lambda: ep.expert_linear(x.cpu(), w, L), lambda: ep.expert_linear_bwd(g[:, :80], x, w, L),
             lambda: ep.expert_linear_bwd(g, None, w, L), lambda: ep.expert_linear_bwd(g, x, w, L, accumulate=True),
             lambda: ep.expert_linear_bwd(g, x, w, L, gate_up=x), lambda: ep.expert_linear_bwd(g, x, w, L, gate_up=x, need=(False, True)),
             lambda: ep.lora_add(x, x[:70], a, b, L, by_token=False),
             lambda: ep.lora_add(x, x, a, b[:1], L, by_token=False), lambda: ep.lora_add(x, x, a, a, L, by_token=False)]
    for i, f in enumerate(wrong):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ep.expert_linear(x.half(), w, L), lambda: ep.expert_linear(x.float(), w.float(), L),
              lambda: ep.expert_linear_bwd(g, x, w, L, grad_w_dtype=F16), lambda: ep.lora_add(x, x.half(), a, b, L, by_token=False)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ep.EPError):
        ep.expert_linear_bwd(g, x, w, L, need=(False, False))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for f in (lambda: ep.expert_linear(x, w, L, stream=s), lambda: ep.expert_linear_bwd(g, x, w, L, stream=s),
              lambda: ep.lora_add(x, x, a, b, L, by_token=False, stream=s)):
        s = torch.cuda.Stream(device=0)
        with pytest.raises(ValueError, match="current device"):
            f()


def test_one_of_the_gradients():
    import combine_topk_ids_histogram_gb300 as ep
    L = ref.layout_of(ep, [30, 50])
    x, w, g = normal(1, 80, 64), normal(2, 2, 96, 64), normal(3, 80, 96)
    gx, gw = ep.expert_linear_bwd(g, x, w, L)
    only, none = ep.expert_linear_bwd(g, None, w, L, need=(True, False))
    assert none is None and torch.equal(only, gx)
    none, only = ep.expert_linear_bwd(g, x, w, L, need=(False, True))
    assert none is None and torch.equal(only, gw)


def test_gradients_against_differences():
    """The gradient of sum(c * out) in a direction, against the difference of two forward passes in 64 bits."""
    import combine_topk_ids_histogram_gb300 as ep
    L = ref.layout_of(ep, [6, 0, 11])
    K, F, N = 32, 48, 64
    x, w13, w2, c = normal(1, 17, K), normal(2, 3, 2 * F, K, scale=K ** -0.5), normal(3, 3, N, F, scale=F ** -0.5), normal(4, 17, N)

    def loss(x, w13, w2):
        total = 0.0
        for g, rows in enumerate(ref.extents(L)):
            gate, up = (x[rows] @ w13[g].t()).chunk(2, 1)
            total += (c[rows].double() * ((gate * torch.sigmoid(gate) * up) @ w2[g].t())).sum().item()
        return total

    act, gu = ep.expert_linear(x, w13, L, swiglu=True, save=True)
    ggu, gw2 = ep.expert_linear_bwd(c, act, w2, L, gate_up=gu, grad_w_dtype=torch.float32)
    gx, gw13 = ep.expert_linear_bwd(ggu, x, w13, L, grad_w_dtype=torch.float32)
    at = [v.double() for v in (x, w13, w2)]
    for i, grad in enumerate((gx, gw13, gw2)):
        d = normal(9 + i, *grad.shape, dtype=torch.float64)
        h = 1e-6
        up, down = [[v + s * h * d if j == i else v for j, v in enumerate(at)] for s in (1, -1)]
        want, terms_ = (loss(*up) - loss(*down)) / (2 * h), grad.double() * d
        # four roundings to bf16 on the way (act, gate and up, their gradient, grad_x), each of its term at most
        assert abs(terms_.sum().item() - want) <= 4 * 2.0 ** -8 * terms_.abs().sum().item()


def test_status_means_nothing_is_written():
    import combine_topk_ids_histogram_gb300 as ep
    ids = torch.zeros(20, 1, dtype=torch.int32, device="cuda")
    L = ep.dispatch_layout(ids, 2, capacity=10)
    assert ep.read_status(L) == ep.STATUS_OVERFLOW
    x, w = normal(1, 20, 64), normal(2, 2, 64, 64)
    out, gu, gx, gw = (torch.full(s, 7.0, dtype=BF16, device="cuda") for s in ((20, 32), (20, 64), (20, 64), (2, 64, 64)))
    ep.expert_linear(x, w, L, swiglu=True, save=True, out=(out, gu))
    ep.expert_linear(x, w, L, out=gx)
    ep.expert_linear_bwd(x, x, w, L, out=(gx, gw))
    for t in (out, gu, gx, gw):
        assert (t == 7).all()


def test_graph_streams_and_repeats():
    """The same bits again: in a CUDA graph replayed on other data, on another stream, from two threads at once."""
    import combine_topk_ids_histogram_gb300 as ep
    E, T, K, H, F = 8, 200, 2, 256, 96
    w13, w2 = normal(1, E, 2 * F, H, scale=H ** -0.5), normal(2, E, H, F, scale=F ** -0.5)

    def step(ids, x, c, stream=None):
        L = ep.dispatch_layout(ids, E, stream=stream)
        rows = ep.dispatch_bf16(x, L, stream=stream)
        act, gu = ep.expert_linear(rows, w13, L, swiglu=True, save=True, stream=stream)
        y = ep.expert_linear(act, w2, L, stream=stream)
        ggu, gw2 = ep.expert_linear_bwd(c, act, w2, L, gate_up=gu, stream=stream)
        gx, gw13 = ep.expert_linear_bwd(ggu, rows, w13, L, grad_w_dtype=torch.float32, stream=stream)
        return y, gw2, gx, gw13

    def data(seed):
        g = torch.Generator().manual_seed(seed)
        ids = torch.argsort(torch.rand(T, E, generator=g) ** (1 + seed), dim=1)[:, :K].int().cuda()
        return ids, normal(seed + 10, T, H), normal(seed + 20, T * K, H)

    ids, x, c = data(0)
    step(ids, x, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(ids, x, c)
    sets = [data(s) for s in (1, 2, 3)]
    eager = [[v.clone() for v in step(*d)] for d in sets]
    for d, want in zip(sets, eager):
        for dst, src in zip((ids, x, c), d):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
    torch.cuda.synchronize()
    got, start = [None] * 3, threading.Barrier(3, timeout=60)

    def worker(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            start.wait()
            for _ in range(5):
                got[i] = step(*sets[i], stream=s)
        s.synchronize()

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(3)]
    [t.start() for t in threads]
    [t.join(timeout=120) for t in threads]
    for g, want in zip(got, eager):
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    """More than 2^32 output elements, and rows whose last lie behind them."""
    import combine_topk_ids_histogram_gb300 as ep
    R, N, K = 66_000, 65_536, 16
    L = ref.layout_of(ep, [R - 300, 300])
    x, w = normal(1, R, K), normal(2, 2, N, K)
    out = ep.expert_linear(x, w, L)
    for rows in (slice(0, 64), slice(32_700, 32_800), slice(R - 364, R - 236), slice(R - 64, R)):
        g = torch.tensor([0 if i < R - 300 else 1 for i in range(R)][rows])
        y = torch.stack([x[rows][i].double() @ w[g[i]].double().t() for i in range(len(g))])
        err = torch.stack([ref.terms(K) * (x[rows][i].double().abs() @ w[g[i]].double().abs().t()) for i in range(len(g))])
        ref.assert_within(out[rows], y, ref.rounded(y, err, BF16), str(rows))
    gu = torch.randn(R, 2 * K, device="cuda").bfloat16()
    gx, _ = ep.expert_linear_bwd(out, None, w, L, gate_up=gu, need=(True, False))
    for rows in (slice(0, 40), slice(R - 310, R - 290)):
        parts = [ref.grad_gate(*ref.linear(out[i:i + 1], w[0 if i < R - 300 else 1].t()), gu[i:i + 1]) for i in range(R)[rows]]
        d, err = (torch.cat(v) for v in zip(*parts))
        ref.assert_within(gx[rows], d, ref.rounded(d, err, BF16), str(rows))


def test_offsets_outside_the_buffers():
    """A layout whose extents a caller has overwritten: nothing behind the buffers' rows is written or taken into a sum, and the
    bounds-checked build reports it."""
    import combine_topk_ids_histogram_gb300 as ep
    L = ref.layout_of(ep, [10, 20, 30])
    L.row_offsets.copy_(torch.tensor([-7, 10, 30, 1 << 30], dtype=torch.int32))
    x, w, g = normal(1, 60, 64), normal(2, 3, 96, 64), normal(3, 60, 96)
    buf, out = guarded(60, 96, BF16)
    ep.expert_linear(x, w, L, out=out)
    got = [out.clone(), None, None]
    L.status.zero_()
    got[1:] = ep.expert_linear_bwd(g, x, w, L)
    torch.cuda.synchronize()
    assert (buf[60 * 96:] == 7).all()
    assert (L.status[0].item() & ep.STATUS_BOUNDS != 0) == bool(ep.CHECKED)
    L = ref.layout_of(ep, [10, 20, 30])
    want = [ep.expert_linear(x, w, L), *ep.expert_linear_bwd(g, x, w, L)]
    if not ep.CHECKED:                                   # (there the second kernel of a call may see the first one's report)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_on_the_bounds_checked_build():
    if os.environ.get("EP_GB300_CHECKED", "0") == "1":
        pytest.skip("this process runs on it already")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu and not slow", "tests/test_gpu_linear.py", "tests/test_gpu_lora.py",
                        "-k", "not bounds_checked"], cwd=root, env=dict(os.environ, EP_GB300_CHECKED="1"), capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
