"""Low-rank adapters beside a shared projection against the 64-bit definition."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def normal(seed, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def make(T, G, r, H, N, dtype, seed, none=0.2):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, G, (T, 1), generator=g, dtype=torch.int32)
    ids[torch.rand(T, 1, generator=g) < none] = -1
    a, b = normal(seed + 1, G, r, H, dtype=dtype, scale=H ** -0.5), normal(seed + 2, G, N, r, dtype=dtype, scale=r ** -0.5)
    scale = (0.5 + torch.rand(G, generator=g)).cuda()
    return ids.cuda(), normal(seed + 3, T, N, dtype=dtype), normal(seed + 4, T, H, dtype=dtype), a, b, scale


def expected(y, x, a, b, scale, rows_of):
    """out and its bound; rows_of[g]: the rows of adapter g."""
    want, err = y.double(), torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    for g, rows in enumerate(rows_of):
        if len(rows):
            d, e = ref.lora(x[rows], a[g], b[g], 1.0 if scale is None else scale[g].double(), y.dtype)
            want[rows] += d
            err[rows] = e + 2.0 ** -23 * (d.abs() + e)
    return want, ref.rounded(want, err, y.dtype)


def check(ep, ids, y, x, a, b, scale, in_place=False):
    L = ep.dispatch_layout(ids, a.shape[0])
    rows_of = [(ids[:, 0] == g).nonzero()[:, 0] for g in range(a.shape[0])]
    want, tol = expected(y, x, a, b, scale, rows_of)
    before = y.clone()
    out = ep.lora_add(y, x, a, b, L, scale=scale, out=y if in_place else None)
    assert ep.read_status(L) == 0
    ref.assert_within(out, want, tol, "out")
    none = ids[:, 0] < 0
    assert torch.equal(out[none], before[none])
    return out


# (T, adapters, r, H, N): one token; every tile of rows; each width of the rank; odd sizes; one adapter for all
CASES = [(1, 1, 8, 16, 16), (1, 32, 16, 2048, 2048), (7, 3, 24, 80, 48), (16, 1, 32, 256, 272), (33, 2, 40, 272, 96), (64, 48, 32, 1024, 512),
         (65, 1, 64, 144, 1040), (100, 5, 72, 528, 304), (300, 4, 128, 512, 160), (500, 7, 64, 384, 208), (130, 1000, 16, 64, 32),
         (2000, 3, 16, 96, 64), (40, 2, 104, 32768, 16), (24, 8, 8, 7168, 4096),
         # enough of everything for tiles of 128 rows: each width of the rank, odd sizes, one adapter, ragged ends
         (3000, 3, 72, 7168, 1456), (20000, 7, 24, 1040, 1520), (9000, 2, 128, 1136, 720), (70000, 5, 8, 512, 608), (8200, 1, 16, 4096, 4112),
         (14000, 9, 64, 48, 2064), (12000, 2, 40, 3200, 32)]


@pytest.mark.parametrize("T,G,r,H,N", CASES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_by_token(T, G, r, H, N, dtype):
    import combine_topk_ids_histogram_gb300 as ep
    data = make(T, G, r, H, N, dtype, T + r, none=0.0 if T == 1 else 0.2)
    out = check(ep, *data)
    ids, y, x, a, b, scale = data
    assert torch.equal(out, check(ep, ids, y.clone(), x, a, b, scale, in_place=True))
    check(ep, ids, y, x, a, b, None)


@pytest.mark.parametrize("T,G,r,H,N", CASES)
def test_in_row_order(T, G, r, H, N):
    """Adapters of experts: any layout, padded groups and a shared expert among them; rows behind the last stay as they are."""
    import combine_topk_ids_histogram_gb300 as ep
    K = min(G, 2)
    g = torch.Generator().manual_seed(T)
    ids = torch.argsort(torch.rand(T, G, generator=g), dim=1)[:, :K].int()
    ids[torch.rand(T, K, generator=g) < 0.2] = -1
    L = ep.dispatch_layout_routed(G, topk_ids=ids.cuda(), fused_shared=G < 1000, pad_multiple=1 + T % 3)[0]
    dtype = F16 if T % 2 else BF16
    a, b = normal(1, L.G, r, H, dtype=dtype, scale=H ** -0.5), normal(2, L.G, N, r, dtype=dtype, scale=r ** -0.5)
    y, x = normal(3, L.R_max, N, dtype=dtype), normal(4, L.R_max, H, dtype=dtype)
    buf = torch.full(((L.R_max + 2) * N,), 7.0, dtype=dtype, device="cuda")
    out = buf[:L.R_max * N].view(L.R_max, N)
    ep.lora_add(y, x, a, b, L, by_token=False, out=out)
    assert ep.read_status(L) == 0
    off = L.row_offsets.tolist()
    want, tol = expected(y, x, a, b, None, [torch.arange(p, q, device="cuda") for p, q in zip(off, off[1:])])
    ref.assert_within(out[:off[-1]], want[:off[-1]], tol[:off[-1]], "out")
    assert (buf[off[-1] * N:] == 7).all()


def test_nobody_has_an_adapter():
    import combine_topk_ids_histogram_gb300 as ep
    ids, y, x, a, b, scale = make(50, 3, 16, 64, 48, BF16, 0, none=2.0)
    assert torch.equal(check(ep, ids, y, x, a, b, scale), y)
    assert torch.equal(check(ep, ids, y.clone(), x, a, b, scale, in_place=True), y)
    L = ep.dispatch_layout(ids[:0].contiguous(), 3)
    assert ep.lora_add(y[:0], x[:0], a, b, L).shape == (0, 48)


def test_strides():
    """Slices of wider matrices: y and out of a fused projection, x of its input."""
    import combine_topk_ids_histogram_gb300 as ep
    ids, _, _, a, b, scale = make(90, 4, 16, 144, 96, BF16, 1)
    ywide, xwide = normal(1, 90, 304), normal(2, 90, 200)
    y, x = ywide[:, 104:200], xwide[:, 8:152]
    want = check(ep, ids, y.contiguous(), x.contiguous(), a, b, scale)
    guard = ywide.clone()
    assert torch.equal(check(ep, ids, y, x, a, b, scale, in_place=True), want)
    assert torch.equal(ywide[:, :104], guard[:, :104]) and torch.equal(ywide[:, 200:], guard[:, 200:])
    L = ep.dispatch_layout(ids, 4)
    owide = torch.full((90, 160), 7.0, dtype=BF16, device="cuda")
    ep.lora_add(guard[:, 104:200], x, a, b, L, scale=scale, out=owide[:, 16:112])
    assert torch.equal(owide[:, 16:112], want) and (owide[:, :16] == 7).all() and (owide[:, 112:] == 7).all()
    with pytest.raises(ep.EPError):
        ep.lora_add(ywide[:, 100:196], x, a, b, L)


def test_rows_do_not_mix():
    import combine_topk_ids_histogram_gb300 as ep
    ids, y, x, a, b, scale = make(70, 4, 24, 96, 64, BF16, 5, none=0.1)
    clean = check(ep, ids, y, x, a, b, scale)
    x2, y2 = x.clone(), y.clone()
    at = [3, 20, 69]
    ids[at, 0] = torch.tensor([0, -1, 2], dtype=torch.int32, device="cuda")
    base = ep.lora_add(y, x, a, b, ep.dispatch_layout(ids, 4), scale=scale)
    x2[at] = float("nan")
    y2[3] = float("inf")
    out = ep.lora_add(y2, x2, a, b, ep.dispatch_layout(ids, 4), scale=scale)
    others = [t for t in range(70) if t not in at]
    assert torch.equal(out[others], base[others]) and torch.equal(out[20], y2[20])
    assert out[3].isnan().all() and out[69].isnan().all() and clean.isfinite().all()
    # an adapter that nobody uses may hold anything
    a2, b2 = a.clone(), b.clone()
    a2[1], b2[1] = float("nan"), float("inf")
    ids2 = torch.where(ids == 1, -1, ids)
    out = ep.lora_add(y, x, a2, b2, ep.dispatch_layout(ids2, 4), scale=scale)
    assert out.isfinite().all()


@pytest.mark.parametrize("T,N", [(40, 96), (18000, 144)])                # tiles of 16 rows, and of 128
@pytest.mark.parametrize("size", [1e-6, 1.0, 3000.0])
def test_size_of_the_low_rank_values(size, T, N):
    """A x from below fp16's normal numbers to above its largest, brought back by B."""
    import combine_topk_ids_histogram_gb300 as ep
    ids, y, x, a, b, scale = make(T, 3, 16, 4096, N, F16, 2)
    ids[:] = ids.abs() % 3
    x = (x.abs() * 10 * min(size, 1.0)).half()
    a = (a.abs() * max(size, 1.0)).half()
    b = (b / 64 / max(size, 1.0)).half()
    check(ep, ids, y, x, a, b, scale)


@pytest.mark.parametrize("T,G,r,H,N", [(50, 4, 24, 80, 48), (9000, 2, 72, 2560, 496)])
def test_padded_layouts_by_token(T, G, r, H, N):
    """Padding rows have no token and change nothing."""
    import combine_topk_ids_histogram_gb300 as ep
    ids, y, x, a, b, scale = make(T, G, r, H, N, BF16, 6)
    want, tol = expected(y, x, a, b, scale, [(ids[:, 0] == g).nonzero()[:, 0] for g in range(G)])
    for pad, capacity in ((16, None), (128, T + 300 * G)):
        L = ep.dispatch_layout_routed(G, topk_ids=ids, pad_multiple=pad, num_permuted_tokens=capacity)[0]
        ref.assert_within(ep.lora_add(y, x, a, b, L, scale=scale), want, tol, f"padded to {pad}")


def test_tiles_of_128_rows():
    """What the tests above ask of few rows: strides, in place, rows with NaN, a status, a CUDA graph on other ids."""
    import combine_topk_ids_histogram_gb300 as ep
    T, G, r, H, N = 9000, 3, 40, 3200, 1136
    ids, _, _, a, b, scale = make(T, G, r, H, N, BF16, 1)
    ywide, xwide = normal(1, T, N + 64), normal(2, T, H + 16)
    y, x = ywide[:, 24:24 + N], xwide[:, 8:8 + H]
    want = check(ep, ids, y.contiguous(), x.contiguous(), a, b, scale)
    guard = ywide.clone()
    assert torch.equal(check(ep, ids, y, x, a, b, scale, in_place=True), want)
    assert torch.equal(ywide[:, :24], guard[:, :24]) and torch.equal(ywide[:, 24 + N:], guard[:, 24 + N:])
    y = guard[:, 24:24 + N]
    x2 = x.clone()
    at = [0, 77, 4000, T - 1]
    x2[at] = float("nan")
    out = ep.lora_add(y, x2, a, b, ep.dispatch_layout(ids, G), scale=scale)
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[at] = False
    assert torch.equal(out[others], want[others])
    for t in at:
        assert out[t].isnan().all() or ids[t, 0] < 0
    L = ep.dispatch_layout(ids.clamp(min=0), G, capacity=10)
    kept = torch.full_like(want, 7.0)
    ep.lora_add(y, x, a, b, L, out=kept)
    assert ep.read_status(L) == ep.STATUS_OVERFLOW and (kept == 7).all()
    graph, ids_s = torch.cuda.CUDAGraph(), ids.clone()
    with torch.cuda.graph(graph):
        held = ep.lora_add(y, x, a, b, ep.dispatch_layout(ids_s, G), scale=scale)
    for new in (ids, ids.flip(0), torch.full_like(ids, 2), torch.full_like(ids, -1)):
        ids_s.copy_(new)
        graph.replay()
        assert torch.equal(held, ep.lora_add(y, x, a, b, ep.dispatch_layout(ids_s, G), scale=scale))


def test_status_graph_and_streams():
    import combine_topk_ids_histogram_gb300 as ep
    ids, y, x, a, b, scale = make(60, 4, 16, 256, 128, BF16, 3)
    L = ep.dispatch_layout(torch.zeros_like(ids), 4, capacity=5)
    out = torch.full_like(y, 7.0)
    ep.lora_add(y, x, a, b, L, out=out)
    assert ep.read_status(L) == ep.STATUS_OVERFLOW and (out == 7).all()
    want = check(ep, ids, y, x, a, b, scale)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    xs, ids_s = x.clone(), ids.clone()
    with torch.cuda.graph(graph):
        held = ep.lora_add(y, xs, a, b, ep.dispatch_layout(ids_s, 4), scale=scale)
    for seed in (7, 8):
        xs.copy_(normal(seed, 60, 256))
        ids_s.copy_(ids.flip(0) if seed == 8 else ids)
        graph.replay()
        assert torch.equal(held, ep.lora_add(y, xs, a, b, ep.dispatch_layout(ids_s, 4), scale=scale))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L = ep.dispatch_layout(ids, 4, stream=s)
        out = ep.lora_add(y, x, a, b, L, scale=scale, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_decode_step_with_adapters():
    """The example's block with an adapter per request, in and out of a CUDA graph."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import combine_topk_ids_histogram_gb300 as ep
    import moe_block as M
    T, H, F, E, K = 20, 256, 96, 8, 2
    p = M.make_weights(H, F, E)
    q13, q2 = M.quantise(p["w13"]), M.quantise(p["w2"])
    ids, x, _, a, b, scale = make(T, 3, 16, H, H, BF16, 4)
    without = M.decode_step(x, p, q13, q2, K)
    out = M.decode_step(x, p, q13, q2, K, (ids, a, b, scale))
    h, _, _ = ep.layer_norm(x, p["norm"], rms=True)
    want, tol = expected(without, h, a, b, scale, [(ids[:, 0] == g).nonzero()[:, 0] for g in range(3)])
    ref.assert_within(out, want, tol, "out")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = M.decode_step(x, p, q13, q2, K, (ids, a, b, scale))
    graph.replay()
    assert torch.equal(held, out)
