"""The 4-bit expert products on layout rows against the 64-bit definition."""
import numpy as np
import pytest
import torch

import operator_ref as ref

pytestmark = pytest.mark.gpu


def weights(G, N, H, seed, signed_scales=False):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (G, N, H // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(0, 0x7F, (G, N, H // 16), generator=g, dtype=torch.uint8)
    if signed_scales:
        scales |= torch.randint(0, 2, scales.shape, generator=g, dtype=torch.uint8) << 7
    row_scale = (torch.rand(G, N, generator=g) + 0.5) / 300
    return codes.cuda(), scales.cuda(), row_scale.cuda()


def routing(T, K, E, seed, unused=0.0, only=None):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    if only is not None:
        ids[:] = only
    ids[rng.random((T, K)) < unused] = -1
    return torch.from_numpy(ids).cuda()


def check(ep, L, w, by_token, swiglu, seed, zero=()):
    codes, scales, row_scale = w
    G, N, half = codes.shape
    H = 2 * half
    rows = L.T if by_token else L.R_max
    x = torch.randn(max(rows, 1), H, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)[:rows].cuda()
    for r in zero:
        x[r] = 0
    n_out = N // 2 if swiglu else N
    buf = torch.full(((L.R_max + 2) * n_out + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:L.R_max * n_out].view(L.R_max, n_out)
    nws = ep.expert_matvec_workspace_bytes(L, H) if L.T else 16
    ws = torch.full((nws + 256,), 0xFF, dtype=torch.uint8, device="cuda")        # NaN where nothing is written
    got = ep.expert_matvec(x, codes, scales, row_scale, L, by_token=by_token, swiglu=swiglu, out=out, workspace=ws[:nws])
    assert (ws[nws:] == 0xFF).all()
    assert ep.read_status(L) == 0
    off = L.row_offsets.cpu().numpy()
    src = L.src_info.cpu().numpy()
    xs = x.double().cpu().numpy()
    for g in range(G):
        a, b = off[g], off[g + 1]
        if a == b:
            continue
        wm = ref.weights(codes[g].cpu().numpy(), scales[g].cpu().numpy(), row_scale[g].cpu().numpy())
        if by_token:
            tok = src[a:b, 0]
            xr = np.where(tok[:, None] >= 0, xs[np.maximum(tok, 0)], 0.0)
        else:
            xr = xs[a:b]
        want, tol = ref.experts(xr, wm, swiglu)
        ref.assert_within(got[a:b], want, tol, f"group {g}")
    R = int(off[G])
    assert (buf[R * n_out:] == 7).all(), "rows past the last one were written"
    return got


# (T, K, E, S, H, N): one token, every row count around the tiles, widths of each alignment, odd output rows
CASES = [(1, 1, 1, 0, 16, 1), (1, 8, 16, 0, 2048, 96), (1, 2, 8, 1, 64, 34), (2, 2, 4, 0, 48, 5), (3, 2, 8, 0, 32, 17),
         (7, 1, 1, 0, 80, 33), (8, 1, 1, 1, 128, 64), (9, 1, 1, 0, 144, 40), (16, 2, 4, 0, 256, 130), (17, 1, 1, 0, 272, 31),
         (31, 4, 8, 1, 320, 66), (33, 2, 2, 0, 512, 20), (65, 3, 4, 0, 1040, 24), (130, 8, 8, 0, 96, 48), (40, 8, 64, 1, 384, 36),
         (4, 2, 1000, 0, 64, 16), (5, 3, 6, 0, 7168, 18), (1500, 2, 3, 1, 128, 40), (12, 2, 8, 0, 14336, 22), (2, 2, 4, 0, 32768, 8),
         (1, 4, 6, 1, 1040, 70), (1, 8, 8, 0, 2080, 300), (1, 3, 5, 1, 32768, 20), (1, 2, 3, 0, 7168, 600), (1, 1, 2, 0, 272, 1001)]


@pytest.mark.parametrize("T,K,E,S,H,N", CASES)
@pytest.mark.parametrize("by_token", [True, False])
def test_products(T, K, E, S, H, N, by_token):
    import combine_topk_ids_histogram_gb300 as ep
    L = ep.dispatch_layout(routing(T, K, E, T + H), E, fused_shared=bool(S))
    check(ep, L, weights(E + S, N, H, N), by_token, False, H)


@pytest.mark.parametrize("T,K,E,S,H,N", [c for c in CASES if c[5] % 2 == 0])
def test_gated_products(T, K, E, S, H, N):
    import combine_topk_ids_histogram_gb300 as ep
    L = ep.dispatch_layout(routing(T, K, E, T + H), E, fused_shared=bool(S))
    check(ep, L, weights(E + S, N, H, N + 1), True, True, H + 1)


# more items than the resident CTAs begin with, so that each takes several: in passes of 8 rows and of 16, with one step of
# k per item (items in turn) and with more (drawn), on weight rows of each alignment
MANY = [(64, 4, 64, 0, 512, 2600), (128, 2, 8, 0, 512, 8200), (64, 4, 64, 0, 48, 2600), (128, 2, 8, 1, 256, 8200),
        (64, 4, 64, 0, 528, 2600), (64, 4, 64, 1, 544, 2600), (100, 2, 8, 0, 784, 6000), (64, 4, 64, 0, 2048, 1400)]


@pytest.mark.parametrize("T,K,E,S,H,N", MANY)
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_items(T, K, E, S, H, N, swiglu):
    import combine_topk_ids_histogram_gb300 as ep
    L = ep.dispatch_layout(routing(T, K, E, T + H), E, fused_shared=bool(S))
    w = weights(E + S, N, H, N)
    first = check(ep, L, w, True, swiglu, H).clone()
    assert torch.equal(check(ep, L, w, True, swiglu, H), first), "two runs differ"


@pytest.mark.parametrize("swiglu", [False, True])
def test_unused_slots_and_empty_groups(swiglu):
    import combine_topk_ids_histogram_gb300 as ep
    for unused in (0.3, 0.97, 1.0):
        ids = routing(24, 4, 32, 3, unused)
        L = ep.dispatch_layout(ids, 32)
        check(ep, L, weights(32, 48, 160, 2), True, swiglu, 4)
        check(ep, L, weights(32, 48, 160, 2), False, swiglu, 4)


@pytest.mark.parametrize("H", [16, 48, 80, 272, 304, 1040])
def test_a_nan_scale_stays_in_its_weight_row(H):
    """Rows whose scales begin at any byte: the block after a row's last one is the next row's."""
    import combine_topk_ids_histogram_gb300 as ep
    N = 37
    codes, scales, row_scale = weights(2, N, H, 9)
    scales[0, 5, 0] = scales[1, 20, -1] = scales[1, N - 1, -1] = 0x7F
    codes |= 0x11                                                       # no zero weight
    L = ep.dispatch_layout(routing(4, 2, 2, 1), 2)
    x = torch.randn(4, H, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    got = ep.expert_matvec(x, codes, scales, row_scale, L)
    bad = torch.isnan(got)
    want = torch.zeros_like(bad)
    want[:4, 5] = want[4:, 20] = want[4:, N - 1] = True
    assert torch.equal(bad, want)


def test_all_rows_in_one_expert_and_negative_scales():
    import combine_topk_ids_histogram_gb300 as ep
    L = ep.dispatch_layout(routing(100, 2, 5, 1, only=3), 5)
    check(ep, L, weights(5, 34, 192, 6, signed_scales=True), True, False, 1)
    check(ep, L, weights(5, 34, 192, 6, signed_scales=True), False, True, 1)


def test_padded_layout():
    """Padding rows are the product of a zero row."""
    import combine_topk_ids_histogram_gb300 as ep
    ids = routing(19, 2, 6, 5, 0.1)
    for S in (False, True):
        L, _, _ = ep.dispatch_layout_routed(6, topk_ids=ids, pad_multiple=8, fused_shared=S)
        w = weights(6 + S, 40, 208, 3)
        got = check(ep, L, w, True, False, 2)
        off, src = L.row_offsets.cpu().numpy(), L.src_info.cpu().numpy()
        pad = [r for r in range(off[-1]) if src[r, 0] < 0]
        assert pad and (got[pad] == 0).all()
        check(ep, L, w, False, False, 2, zero=pad)


def test_weights_of_the_dispatch_quantiser():
    """dispatch_nvfp4 of a weight matrix (N tokens, one expert) gives the format this call takes."""
    import combine_topk_ids_histogram_gb300 as ep
    E, N, H, T = 3, 64, 512, 9
    dense = torch.randn(E * N, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda() / 16
    Lw = ep.dispatch_layout(torch.zeros(E * N, 1, dtype=torch.int32, device="cuda"), 1)
    codes, scales, inv, _ = ep.dispatch_nvfp4(dense, Lw)
    w = codes.view(E, N, H // 2), scales.view(E, N, H // 16), inv.float().view(E, N)
    L = ep.dispatch_layout(routing(T, 2, E, 4), E)
    got = check(ep, L, w, True, False, 8)
    # and the products are near those of the unquantised weights: 4-bit rounding is within 1/4 of the spacing
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    off, src = L.row_offsets.cpu(), L.src_info.cpu()
    for g in range(E):
        a, b = int(off[g]), int(off[g + 1])
        full = x[src[a:b, 0].long()].float() @ dense.view(E, N, H)[g].float().t()
        rel = (got[a:b].float() - full).norm() / full.norm()
        assert rel < 0.2


def test_special_values():
    """Zero weights times finite values are 0; an infinity or NaN in a row shows in that row alone."""
    import combine_topk_ids_histogram_gb300 as ep
    E, N, H, T = 2, 40, 256, 6
    L = ep.dispatch_layout(torch.tensor([[0], [0], [0], [1], [1], [1]], dtype=torch.int32, device="cuda"), E)
    codes, scales, row_scale = weights(E, N, H, 1)
    scales.clamp_(min=0x30)
    codes &= 0x77
    codes |= 0x22                                                       # no zero weight
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    clean = ep.expert_matvec(x, codes, scales, row_scale, L)
    x[1, 100], x[4, 255] = float("nan"), float("inf")
    got = ep.expert_matvec(x, codes, scales, row_scale, L)
    rows = [0, 2, 3, 5]
    assert torch.equal(got[rows], clean[rows])
    assert torch.isnan(got[1]).all() and (got[4] == float("inf")).all()
    zero = ep.expert_matvec(x[[0, 0, 2, 3, 3, 5]].contiguous(), torch.zeros_like(codes), scales, row_scale, L)
    assert (zero == 0).all()
    big = torch.full((T, H), 3e38, dtype=torch.bfloat16, device="cuda")
    assert (ep.expert_matvec(big, codes, scales, row_scale, L) == float("inf")).all()


# one token, few rows per expert, many
TOKENS = [(1, 2, 4), (6, 1, 2), (40, 1, 2)]


@pytest.mark.parametrize("T,K,E", TOKENS)
@pytest.mark.parametrize("x_exp,row_scale", [(110, 2.0 ** -40), (-112, 1.37 * 2.0 ** -20), (120, -1.2 * 2.0 ** -100), (-60, 1.1 * 2.0 ** 100)])
def test_large_and_small_values_times_their_scales(T, K, E, x_exp, row_scale):
    """Sums that leave fp32's range before the row's scale brings them back."""
    import combine_topk_ids_histogram_gb300 as ep
    N, H = 70, 512
    codes, scales, _ = weights(E, N, H, 3)
    rs = torch.full((E, N), row_scale, device="cuda")
    x = (torch.randn(T, H, generator=torch.Generator().manual_seed(8)).clamp(-2, 2) * 2.0 ** x_exp).to(torch.bfloat16).cuda()
    L = ep.dispatch_layout(routing(T, K, E, 5), E)
    got = ep.expert_matvec(x, codes, scales, rs, L)
    off, src = L.row_offsets.cpu().numpy(), L.src_info.cpu().numpy()
    for g in range(E):
        a, b = off[g], off[g + 1]
        wm = ref.weights(codes[g].cpu().numpy(), scales[g].cpu().numpy(), rs[g].cpu().numpy())
        want, tol = ref.experts(x.double().cpu().numpy()[src[a:b, 0]], wm, False)
        ref.assert_within(got[a:b], want, tol, f"group {g}")


@pytest.mark.parametrize("T,K,E,N", [(1, 2, 4, 64), (6, 1, 2, 64), (16, 2, 8, 4096), (64, 2, 8, 4096)])
def test_long_sums_keep_their_last_bits(T, K, E, N):
    """1 - 1 and thousands of terms far below them.  The products are added on the tensor cores over at most 2048 k, 128 steps
    that are each off by at most 2^-22 of what they add, and those sums in fp32: within (128 + 8 + 16) * 2^-22 * sum|w x|
    whatever the width.  (All of these terms together are more than that.)"""
    import combine_topk_ids_histogram_gb300 as ep
    H, small = 14336, 0.8984375 * 2.0 ** -27
    codes = torch.full((E, N, H // 2), 0x22, dtype=torch.uint8, device="cuda")
    scales = torch.full((E, N, H // 16), 0x38, dtype=torch.uint8, device="cuda")
    rs = torch.ones(E, N, device="cuda")
    x = torch.full((T, H), small, device="cuda")
    x[:, 0], x[:, -1] = 1.0, -1.0
    L = ep.dispatch_layout(routing(T, K, E, 5), E)
    got = ep.expert_matvec(x.bfloat16(), codes, scales, rs, L)
    want = (H - 2) * small
    tol = 152 * 2.0 ** -22 * (2 + want) + 2.0 ** -8 * want
    assert tol < want
    err = (got.double() - want).abs().max().item()
    assert err <= tol, (err, tol, want)


def test_status_repeat_and_streams():
    import combine_topk_ids_histogram_gb300 as ep
    ids = routing(20, 4, 16, 5)
    w = weights(16, 80, 640, 3)
    x = torch.randn(20, 640, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    L = ep.dispatch_layout(ids, 16)
    a = ep.expert_matvec(x, *w, L)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = ep.expert_matvec(x, *w, L)
    s.synchronize()
    assert torch.equal(a, b)
    # a layout in error writes nothing
    over = ep.dispatch_layout(ids, 16, n_parts=2, capacity=3)
    out = torch.full((over.R_max, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_matvec(x, *w, over, out=out)
    assert ep.read_status(over) == ep.STATUS_OVERFLOW and (out == 7).all()


def test_calls_on_layouts_without_rows_stay_in_order():
    """A call on a layout without rows, between calls that share its workspace and draw their items: nothing of it may
    run beside the next one, whose counter of drawn items lies in that workspace."""
    import combine_topk_ids_histogram_gb300 as ep
    T, E, H, N = 64, 64, 512, 2600                                     # several items per CTA
    ids = routing(T, 4, E, 7)
    full, none = ep.dispatch_layout(ids, E), ep.dispatch_layout(torch.full_like(ids, -1), E)
    w = weights(E, N, H, 4)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    ws = torch.empty(ep.expert_matvec_workspace_bytes(full, H), dtype=torch.uint8, device="cuda")
    want = ep.expert_matvec(x, *w, full, workspace=ws).clone()
    outs = [torch.full_like(want, float("nan")) for _ in range(20)]
    empty = torch.full((none.R_max, N), 7.0, dtype=torch.bfloat16, device="cuda")
    for out in outs:
        ep.expert_matvec(x, *w, none, out=empty, workspace=ws)
        ep.expert_matvec(x, *w, full, out=out, workspace=ws)
    torch.cuda.synchronize()
    R = int(full.row_offsets[-1])
    assert all(torch.equal(o[:R], want[:R]) for o in outs) and (empty == 7).all()


def test_rows_outside_the_layout_are_not_used():
    """A src_info entry that names no token is a zero row, and row_offsets past R_max are cut there; the bounds-checked
    build reports such an entry and writes nothing."""
    import combine_topk_ids_histogram_gb300 as ep
    L = ep.dispatch_layout(routing(6, 2, 4, 5), 4)
    w = weights(4, 24, 96, 3)
    x = torch.randn(6, 96, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    good = ep.expert_matvec(x, *w, L)
    L.src_info[3, 0], L.src_info[5, 0] = 6, -9
    buf = torch.full((L.R_max + 4, 24), 7.0, dtype=torch.bfloat16, device="cuda")
    L.row_offsets[4] = L.R_max + 3
    ep.expert_matvec(x, *w, L, out=buf)
    torch.cuda.synchronize()
    if ep.CHECKED:
        assert ep.read_status(L) == ep.STATUS_BOUNDS and (buf == 7).all()
        return
    keep = [r for r in range(L.R_max) if r not in (3, 5)]
    assert torch.equal(buf[keep], good[keep])
    assert (buf[L.R_max:] == 7).all() and (buf[[3, 5]] == 0).all()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("H,N", [(2048, 96), (784, 40), (96, 300)])
def test_one_token_without_expert_ids_and_padded(H, N, swiglu):
    """A layout's expert_ids may be absent: the general kernels give the same products within the bound; so do a padded
    layout and one whose slots are partly unused."""
    import combine_topk_ids_histogram_gb300 as ep
    ids = routing(1, 4, 8, 3)
    w = weights(8, N, H, 5)
    L = ep.dispatch_layout(ids, 8)
    check(ep, L, w, True, swiglu, 2)
    kept, L.c.expert_ids = L.c.expert_ids, None
    check(ep, L, w, True, swiglu, 2)
    L.c.expert_ids = kept
    ids[0, 1] = -1
    check(ep, ep.dispatch_layout(ids, 8), w, True, swiglu, 2)
    check(ep, ep.dispatch_layout(torch.full_like(ids, -1), 8), w, True, swiglu, 2)
    for pad in (2, 16):
        check(ep, ep.dispatch_layout_routed(8, topk_ids=ids[:, :1].contiguous(), pad_multiple=pad)[0], w, True, swiglu, 2)


def test_no_tokens_and_refusals():
    import combine_topk_ids_histogram_gb300 as ep
    L = ep.dispatch_layout(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    codes, scales, row_scale = weights(4, 24, 96, 3)
    ep.expert_matvec(torch.empty(0, 96, dtype=torch.bfloat16, device="cuda"), codes, scales, row_scale, L)
    L = ep.dispatch_layout(routing(6, 2, 4, 5), 4)
    x = torch.zeros(6, 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        ep.expert_matvec(x, codes[:3], scales, row_scale, L)
    with pytest.raises(ValueError):
        ep.expert_matvec(x, codes, scales[:, :, :5], row_scale, L)
    with pytest.raises(ValueError):
        ep.expert_matvec(x, codes, scales, row_scale[:, :20].contiguous(), L)
    with pytest.raises(TypeError):
        ep.expert_matvec(x, codes.int(), scales, row_scale, L)
    with pytest.raises(ValueError):
        ep.expert_matvec(x.cpu(), codes, scales, row_scale, L)
    with pytest.raises(TypeError):
        ep.expert_matvec(x.float(), codes, scales, row_scale, L)
    with pytest.raises(ValueError):
        ep.expert_matvec(x[:5], codes, scales, row_scale, L)
    with pytest.raises(ValueError):
        ep.expert_matvec(x, codes, scales, row_scale, L, by_token=False)      # needs R_max rows
    odd = codes[:, :23].contiguous(), scales[:, :23].contiguous(), row_scale[:, :23].contiguous()
    with pytest.raises(ep.EPError):
        ep.expert_matvec(x, *odd, L, swiglu=True)                             # gate and up rows: an even number
    with pytest.raises(ValueError):
        ep.expert_matvec(x, codes, scales, row_scale, L, out=torch.empty(3, 24, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ep.EPError):
        ep.expert_matvec(x, codes, scales, row_scale, L, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
