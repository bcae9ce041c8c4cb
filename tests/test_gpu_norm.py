"""Layer norm and RMS norm, forward and backward, against the 64-bit definition: every type, widths that no
vector divides, strided rows, rows that are constant or hold infinities, one token and none."""
import os
import re

import numpy as np
import pytest
import torch

import operator_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32), (torch.float32, torch.float32)]
# (T, H): one element, odd widths, each register layout's edges, the widest rows, ragged row counts
SIZES = [(1, 1), (3, 2), (5, 8), (7, 33), (2, 255), (9, 256), (400, 256), (33, 264), (700, 511), (600, 512), (310, 520),
         (1, 2048), (320, 2048), (37, 2056), (5, 4096), (3, 4097), (311, 1111), (6, 7168), (610, 7168), (2, 8192),
         (3, 8200), (330, 8200), (2, 16384), (2, 32767), (3, 32768),
         (457, 256), (801, 264), (830, 1111), (810, 7168), (820, 8192), (805, 8200), (4000, 40), (2500, 520)]


def make(T, H, dt, wdt, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g) * (1 + torch.arange(T)[:, None] % 5) + 0.5
    w = 1 + 0.2 * torch.randn(H, generator=g)
    b = 0.3 * torch.randn(H, generator=g) if bias else None
    gy = torch.randn(T, H, generator=g)
    to = lambda t, d: t.to(d).cuda()
    return to(x, dt), to(w, wdt), None if b is None else to(b, wdt), to(gy, dt)


def check_forward(ep, x, w, b, eps, rms, out=None):
    y, mean, rstd = ep.layer_norm(x, w, b, eps=eps, rms=rms, out=out)
    ry, rmean, rrstd = ref.norm(x, w, b, eps, rms)
    ty, tmean, trstd = ref.norm_tol(x, w, b, eps, rms, x.dtype)
    ref.assert_within(y, ry, ty, "y")
    ref.assert_within(rstd, rrstd, trstd, "rstd")
    if rms:
        assert mean is None
    else:
        ref.assert_within(mean, rmean, tmean, "mean")
    return y, mean, rstd


def check_backward(ep, gy, x, w, mean, rstd, rms, bias=True):
    dx, dw, db = ep.layer_norm_bwd(gy, x, w, mean, rstd, rms=rms, bias=bias)
    rx, rw, rb = ref.norm_bwd(gy, x, w, mean, rstd, rms)
    tx, tw, tb = ref.norm_bwd_tol(gy, x, w, mean, rstd, rms, x.dtype)
    assert dw.dtype == torch.float32
    ref.assert_within(dx, rx, tx, "dx")
    ref.assert_within(dw, rw, tw, "dw")
    if bias:
        ref.assert_within(db, rb, tb, "db")
    else:
        assert db is None


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("rms", [False, True])
def test_sizes_bf16(T, H, rms):
    import combine_topk_ids_histogram_gb300 as ep
    x, w, b, gy = make(T, H, torch.bfloat16, torch.bfloat16, T * 7 + H, bias=not rms)
    _, mean, rstd = check_forward(ep, x, w, b, 1e-5, rms)
    check_backward(ep, gy, x, w, mean, rstd, rms, bias=not rms)


@pytest.mark.parametrize("dt,wdt", TYPES[1:])
@pytest.mark.parametrize("T,H", [(1, 7), (35, 100), (340, 132), (320, 2048), (61, 2049), (5, 4100), (320, 7168), (2, 8196),
                                 (2, 32768), (457, 132), (820, 132), (815, 2048), (803, 2049), (810, 7168), (801, 8196)])
def test_types(dt, wdt, T, H):
    import combine_topk_ids_histogram_gb300 as ep
    x, w, b, gy = make(T, H, dt, wdt, T + 3 * H)
    _, mean, rstd = check_forward(ep, x, w, b, 1e-6, False)
    check_backward(ep, gy, x, w, mean, rstd, False)
    _, mean, rstd = check_forward(ep, x, w, b, 1e-6, True)            # RMS with a bias
    check_backward(ep, gy, x, w, mean, rstd, True)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,extra", [(0, 8), (0, 3), (1, 7), (8, 24), (5, 0)])
@pytest.mark.parametrize("T,H", [(45, 256), (450, 256), (330, 1030), (310, 4099), (2, 9000), (820, 256), (830, 1030),
                                 (810, 4099), (802, 8185)])
def test_strided_and_unaligned_rows(dt, offset, extra, T, H):
    """Rows inside a wider matrix, on and off 16-byte boundaries."""
    import combine_topk_ids_histogram_gb300 as ep
    x, w, b, gy = make(T, H, dt, dt, offset + extra)
    wide = torch.full((T, offset + H + extra), float("nan"), dtype=dt, device="cuda")
    wide[:, offset:offset + H] = x
    gwide = torch.full((T, 2 * H + 1), float("nan"), dtype=dt, device="cuda")
    gwide[:, H:2 * H] = gy
    xs, gs = wide[:, offset:offset + H], gwide[:, H:2 * H]
    _, mean, rstd = check_forward(ep, xs, w, b, 1e-5, False)
    check_backward(ep, gs, xs, w, mean, rstd, False)


@pytest.mark.parametrize("T,H", [(1, 3), (7, 5), (310, 9), (500, 1111), (777, 2047), (40, 8191), (831, 9), (1003, 1111), (823, 2047),
                                 (809, 8191)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_dense_matrices_off_boundaries(dt, T, H):
    """Dense matrices of odd width that all begin at the same distance from a 16-byte boundary."""
    import combine_topk_ids_histogram_gb300 as ep
    x, w, b, gy = make(T, H, dt, dt, T + H)
    for off in (0, 1, 3):
        bufs = [torch.full((off + T * H + 16,), float("nan"), dtype=dt, device="cuda") for _ in range(3)]
        xs, gs, ys = (v[off:off + T * H].view(T, H) for v in bufs)
        xs.copy_(x)
        gs.copy_(gy)
        f32 = dict(device="cuda")
        out = ys, torch.empty(T, **f32), torch.empty(T, **f32)
        _, mean, rstd = check_forward(ep, xs, w, b, 1e-5, False, out=out)
        check_backward(ep, gs, xs, w, mean, rstd, False)
        assert torch.isnan(bufs[2][:off]).all() and torch.isnan(bufs[2][off + T * H:]).all()
        dx = ep.layer_norm_bwd(gs, xs, w, mean, rstd, bias=True, out=(ys, torch.empty(H, **f32), torch.empty(H, **f32)))[0]
        ref.assert_within(dx, ref.norm_bwd(gs, xs, w, mean, rstd, False)[0],
                          ref.norm_bwd_tol(gs, xs, w, mean, rstd, False, dt)[0], "dx")
        assert torch.isnan(bufs[2][:off]).all() and torch.isnan(bufs[2][off + T * H:]).all()


def test_no_write_outside_outputs():
    import combine_topk_ids_histogram_gb300 as ep
    for T, H in ((3, 33), (310, 64), (9, 2048), (2, 8200), (330, 1111), (330, 1112), (830, 1111),
                 (830, 1112)):
        x, w, b, gy = make(T, H, torch.bfloat16, torch.bfloat16, T)
        buf = torch.full((T * H + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
        f = torch.full((3, T + H + 64), 7.0, device="cuda")
        y = buf[64:64 + T * H].view(T, H)
        ep.layer_norm(x, w, b, out=(y, f[0, 8:8 + T], f[1, 8:8 + T]))
        assert (buf[:64] == 7).all() and (buf[64 + T * H:] == 7).all()
        assert (f[:, :8] == 7).all() and (f[:2, 8 + T:] == 7).all()
        mean, rstd = f[0, 8:8 + T].clone(), f[1, 8:8 + T].clone()
        nws = ep.layer_norm_bwd_workspace_bytes(T, H)
        ws = torch.full((nws + 256,), 7, dtype=torch.uint8, device="cuda")
        f.fill_(7)
        ep.layer_norm_bwd(gy, x, w, mean, rstd, bias=True, out=(y, f[0, 8:8 + H], f[1, 8:8 + H]),
                          workspace=ws[:nws])
        assert (buf[:64] == 7).all() and (buf[64 + T * H:] == 7).all()
        assert (f[:, :8] == 7).all() and (f[:2, 8 + H:] == 7).all() and (ws[nws:] == 7).all()


@pytest.mark.parametrize("rep", [1, 500])
def test_constant_rows_and_large_means(rep):
    """A constant row has variance 0: y = bias, and rstd = 1/sqrt(eps).  A large mean costs no digits of the
    variance.  (rep: in few rows, and in many.)"""
    import combine_topk_ids_histogram_gb300 as ep
    x = torch.zeros(4, 512, device="cuda")
    x[1] = 3.0
    x[2] = 1e4 + torch.arange(512, device="cuda") / 64
    x[3] = -1e30
    w = torch.ones(512, device="cuda")
    b = torch.full((512,), 0.25, device="cuda")
    y, mean, rstd = check_forward(ep, x.repeat(rep, 1), w, b, 1e-5, False)
    y, rstd = y[-4:], rstd[-4:]
    assert (y[:2] == 0.25).all() and (y[3] == 0.25).all()
    # in-bound at the large mean is not enough: the two-pass variance is within 1e-6 of 64 bits
    r = ref.norm(x, w, b, 1e-5, False)[2]
    assert abs(rstd[2].item() / r[2].item() - 1) < 1e-6


@pytest.mark.parametrize("T,H", [(8, 300), (1200, 300), (1200, 301)])
def test_non_finite_rows_stay_in_their_rows(T, H):
    import combine_topk_ids_histogram_gb300 as ep
    x, w, b, gy = make(T, H, torch.float32, torch.float32, 5)
    clean = ep.layer_norm(x, w, b)
    bad = x.clone()
    bad[2, 7] = float("inf")
    bad[5, H - 1] = float("nan")
    y, mean, rstd = ep.layer_norm(bad, w, b)
    rows = [r for r in range(T) if r not in (2, 5)]
    assert torch.equal(y[rows], clean[0][rows]) and torch.equal(rstd[rows], clean[2][rows])
    assert torch.isnan(y[2]).all() and torch.isnan(y[5]).all()
    dx, dw, db = ep.layer_norm_bwd(gy, bad, w, mean, rstd, bias=True)
    want = ep.layer_norm_bwd(gy, x, w, clean[1], clean[2], bias=True)
    assert torch.equal(dx[rows], want[0][rows])
    assert torch.isnan(dx[2]).all() and torch.isnan(dx[5]).all()
    assert torch.equal(db, want[2])


def test_no_tokens():
    import combine_topk_ids_histogram_gb300 as ep
    x = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(96, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = ep.layer_norm(x, w, w)
    assert y.shape == (0, 96) and mean.numel() == 0
    dw, db = torch.full((96,), 5.0, device="cuda"), torch.full((96,), 5.0, device="cuda")
    ep.layer_norm_bwd(x, x, w, mean, rstd, bias=True, out=(y, dw, db))
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("rms", [False, True])
def test_gradient_against_differences(rms):
    """<dx, v> + <dw, u> + <db, z> against central differences of the 64-bit forward form.  With step 1e-5
    the difference's own error is below 1e-8 of the gradient's magnitude."""
    import combine_topk_ids_histogram_gb300 as ep
    T, H, eps = 6, 200, 1e-5
    x, w, b, gy = make(T, H, torch.float32, torch.float32, 11)
    _, mean, rstd = ep.layer_norm(x, w, b, eps=eps, rms=rms)
    dx, dw, db = ep.layer_norm_bwd(gy, x, w, mean, rstd, rms=rms, bias=True)
    tx, tw, tb = ref.norm_bwd_tol(gy, x, w, mean, rstd, rms, torch.float32)
    g = torch.Generator().manual_seed(3)
    for _ in range(5):
        v, u, z = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((T, H), (H,), (H,)))
        loss = lambda s: (ref.norm(ref.d64(x) + s * v, ref.d64(w) + s * u, ref.d64(b) + s * z, eps, rms)[0] * ref.d64(gy)).sum()
        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = (ref.d64(dx) * v).sum() + (ref.d64(dw) * u).sum() + (ref.d64(db) * z).sum()
        # the saved statistics are fp32: their relative error of 128 * 2^-24 moves every term by as much
        mag = (ref.d64(dx).abs() * v.abs()).sum() + (ref.d64(dw).abs() * u.abs()).sum()
        tol = (tx * v.abs()).sum() + (tw * u.abs()).sum() + (tb * z.abs()).sum() + (4 * ref.ROW + 1e-8) * mag
        assert abs(got - diff) <= tol


def test_repeatable_and_on_a_side_stream():
    import combine_topk_ids_histogram_gb300 as ep
    x, w, b, gy = make(1500, 1024, torch.bfloat16, torch.bfloat16, 2)
    y, mean, rstd = ep.layer_norm(x, w, b)
    first = ep.layer_norm_bwd(gy, x, w, mean, rstd, bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, m2, r2 = ep.layer_norm(x, w, b)
        second = ep.layer_norm_bwd(gy, x, w, m2, r2, bias=True)
    s.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(first, second))


def test_refusals():
    import combine_topk_ids_histogram_gb300 as ep
    x, w, b, gy = make(4, 64, torch.bfloat16, torch.bfloat16, 1)
    y, mean, rstd = ep.layer_norm(x, w, b)
    with pytest.raises(TypeError):
        ep.layer_norm(x.double(), w, b)
    with pytest.raises(TypeError):
        ep.layer_norm(x, w.half(), b)                      # parameters in x's type or fp32
    with pytest.raises(TypeError):
        ep.layer_norm(x, w, b.float())                     # bias in the weight's type
    with pytest.raises(ValueError):
        ep.layer_norm(x, w[:32], b)
    with pytest.raises(ValueError):
        ep.layer_norm(x.t(), w[:4], None)                  # columns are not contiguous
    with pytest.raises(ValueError):
        ep.layer_norm(x[0], w, b)
    with pytest.raises(ValueError):
        ep.layer_norm(x.cpu(), w, b)
    with pytest.raises(ep.EPError):
        ep.layer_norm(x, w, b, eps=-1.0)
    with pytest.raises(ep.EPError):
        ep.layer_norm(x, w, b, eps=float("nan"))
    with pytest.raises(ValueError):
        ep.layer_norm_bwd(gy[:3], x, w, mean, rstd)
    with pytest.raises(ValueError):
        ep.layer_norm_bwd(gy, x, w, mean[:3], rstd)
    with pytest.raises(ep.EPError):
        ep.layer_norm_bwd(gy, x, w, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ep.EPError):
        ep.layer_norm(torch.zeros(1, 40000, device="cuda"), torch.zeros(40000, device="cuda"))


# ------------------------------------------------------------------------------- rows past the one-row kernel's border
def resident_rows(H, dt, aligned=True):
    """Rows up to which the forward pass takes the kernel with a CTA per row: read from the source, so that moving the border
    there cannot move these tests' cases to the other side of it unnoticed."""
    import combine_topk_ids_histogram_gb300 as ep
    src = open(os.path.join(os.path.dirname(ep.__file__), "csrc", "ep_norm.cu")).read()
    threads = int(re.search(r"constexpr int kResidentPerSm = (\d+);", src).group(1))
    threads *= torch.cuda.get_device_properties(0).multi_processor_count
    vec = (4 if dt == torch.float32 else 8) if aligned else 1
    per_row = H // vec if H // vec <= 1024 else (H // vec + 7) // 8
    return threads // ((per_row + 31) // 32 * 32)


MANY = [(9801, 256), (9803, 40), (4901, 1024), (1301, 2048), (703, 4096)]


@pytest.mark.parametrize("dt,wdt", TYPES)
@pytest.mark.parametrize("T,H", MANY)
def test_many_aligned_rows(dt, wdt, T, H):
    """The pipelined forward kernel at every shape of its groups: one warp (no named barrier, up to 21 groups) to four."""
    import combine_topk_ids_histogram_gb300 as ep
    assert T > resident_rows(H, dt)
    x, w, b, gy = make(T, H, dt, wdt, T + H)
    for bias in (b, None):
        _, mean, rstd = check_forward(ep, x, w, bias, 1e-5, False)
        _, _, rrstd = check_forward(ep, x, w, bias, 1e-5, True)
    check_backward(ep, gy, x, w, mean, rstd, False)
    check_backward(ep, gy, x, w, None, rrstd, True)


@pytest.mark.parametrize("T,H", [(9801, 300), (9801, 301), (4901, 1024), (1201, 7168)])
def test_many_rows_non_finite_and_repeated(T, H):
    """Non-finite rows stay in their rows; an infinity under RMS leaves 0 or the bias in its row's finite places; a second call
    gives the same bits."""
    import combine_topk_ids_histogram_gb300 as ep
    dt = torch.float32 if H < 1000 else torch.bfloat16
    assert T > resident_rows(H, dt, aligned=H % 4 == 0)
    x, w, b, gy = make(T, H, dt, dt, 5)
    bad = x.clone()
    bad[2, 7] = float("inf")
    bad[5, H - 1] = float("nan")
    rows = [r for r in range(T) if r not in (2, 5)]
    for rms in (False, True):
        clean, again = ep.layer_norm(x, w, b, rms=rms), ep.layer_norm(x, w, b, rms=rms)
        assert torch.equal(clean[0], again[0]) and torch.equal(clean[2], again[2])
        y, mean, rstd = ep.layer_norm(bad, w, b, rms=rms)
        assert torch.equal(y[rows], clean[0][rows]) and torch.equal(rstd[rows], clean[2][rows])
        assert torch.isnan(y[5]).all()
        if rms:
            others = [c for c in range(H) if c != 7]
            assert torch.isnan(y[2, 7]) and torch.equal(y[2, others], b[others]) and rstd[2] == 0
        else:
            assert torch.isnan(y[2]).all()
        dx, _, db = ep.layer_norm_bwd(gy, bad, w, mean, rstd, rms=rms, bias=True)
        want = ep.layer_norm_bwd(gy, x, w, clean[1], clean[2], rms=rms, bias=True)
        assert torch.equal(dx[rows], want[0][rows]) and torch.equal(db, want[2])


@pytest.mark.parametrize("rms_case", ["few", "wide"])
def test_an_infinity_under_rms(rms_case):
    import combine_topk_ids_histogram_gb300 as ep
    T, H = (4, 300) if rms_case == "few" else (3, 9000)
    x, w, b, _ = make(T, H, torch.bfloat16, torch.bfloat16, 3)
    x[1, 5] = float("-inf")
    others = [c for c in range(H) if c != 5]
    for bias in (b, None):
        y, _, rstd = ep.layer_norm(x, w, bias, rms=True)
        assert rstd[1] == 0 and torch.isnan(y[1, 5])
        assert torch.equal(y[1, others].float(), (torch.zeros_like(b) if bias is None else b)[others].float())


# 1/H is not exact at these widths; (T: in few rows, and in many)
CONSTANT = [(7168, 4, 1500), (1111, 4, 2000), (5120, 4, 2000), (40, 4, 10000), (300, 4, 10000), (9000, 4, 2000)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,few,many", CONSTANT)
@pytest.mark.parametrize("shifted", [False, True])
def test_constant_rows_of_any_width(H, few, many, dt, shifted):
    """y = bias and mean = the constant, exactly: x - mean is then the same few units for all elements, their sum (below 2^24
    units) and its H-th part are exact, and the correction by it leaves 0.  The variance is off by at most 2^-21 of the
    square of that difference."""
    import combine_topk_ids_histogram_gb300 as ep
    consts = torch.tensor([0.0, 1.0, -3.0, 0.3, 100.0, 1000.0, -1001.0, 2000.0, 4099.0, 1.7e4, -4e4, 1e-3]).to(dt).cuda()
    w, b = torch.linspace(-1.5, 1.5, H).to(dt).cuda(), torch.linspace(-2, 3, H).to(dt).cuda()
    assert few <= resident_rows(H, dt, not shifted) < many
    for T in (few, many):
        c = consts[torch.arange(T, device="cuda") % len(consts)]
        wide = torch.zeros(T, H + 13, dtype=dt, device="cuda")
        x = wide[:, 3:3 + H] if shifted else torch.empty(T, H, dtype=dt, device="cuda")
        x.copy_(c[:, None].expand(T, H))
        y, mean, rstd = ep.layer_norm(x, w, b, eps=1e-5)
        assert torch.equal(y, b.expand(T, H)), (y.float() - b.float()).abs().max()
        assert torch.equal(mean, c.float())
        want = 1e-5 ** -0.5
        tol = want * (0.5 * 2.0 ** -21 * (ref.ROW * ref.d64(c).abs()) ** 2 / 1e-5 + 4 * ref.EPS24)
        ref.assert_within(rstd, torch.full((T,), want, dtype=torch.float64), tol, "rstd")


@pytest.mark.parametrize("T,H", [(3, 7168), (1500, 7168), (3, 1111), (2000, 1111), (4, 9000), (9900, 300)])
@pytest.mark.parametrize("m", [30.0, 1000.0, -1e5])
def test_large_means_lose_nothing(T, H, m):
    """With d0 = the first pass's error of the mean, at most ROW * mean|x|: the corrected d is off by the rounding of
    x - mean (of the order of |c| + d0) and by the error of its mean, ROW * mean|d|; y, mean and rstd follow."""
    import combine_topk_ids_histogram_gb300 as ep
    g = torch.Generator().manual_seed(T + H)
    assert T < 10 or T > resident_rows(H, torch.float32, aligned=H % 4 == 0)
    x = (m + torch.randn(T, H, generator=g)).cuda()
    w, b = (1 + 0.2 * torch.randn(H, generator=g)).cuda(), torch.randn(H, generator=g).cuda()
    y, mean, rstd = ep.layer_norm(x, w, b)
    ry, rmean, rrstd = ref.norm(x, w, b, 1e-5, False)
    c, wd, bd, r = ref.d64(x) - rmean[:, None], ref.d64(w).abs(), ref.d64(b).abs(), rrstd[:, None]
    d0 = (ref.ROW * ref.d64(x).abs().mean(1))[:, None]
    of_mean = (ref.ROW + 3 * ref.EPS24) * (c.abs().mean(1, keepdim=True) + d0)
    dc = of_mean + 3 * ref.EPS24 * (c.abs() + d0)
    drel = ref.ROW * (1 + (d0 * r) ** 2) + 8 * ref.EPS24
    xh = c.abs() * r
    ty = 1.01 * (r * dc * wd + xh * wd * (drel + 4 * ref.EPS24)) + 4 * ref.EPS24 * (xh * wd + bd) + ref.EPS24 * ry.abs()
    ref.assert_within(y, ry, ty, "y")
    ref.assert_within(rstd, rrstd, rrstd * drel[:, 0], "rstd")
    ref.assert_within(mean, rmean, of_mean[:, 0] + 1.01 * ref.EPS24 * rmean.abs(), "mean")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,many", [(7168, 1500), (1110, 2000), (300, 10000)])
@pytest.mark.parametrize("rms", [False, True])
def test_statistics_do_not_depend_on_the_number_of_rows(H, many, dt, rms):
    """Rows of whole numbers and their negatives: their sum is 0 and that of their squares exact in any order, so that
    rstd is the same bits in few rows and in many."""
    import combine_topk_ids_histogram_gb300 as ep
    g = torch.Generator().manual_seed(H)
    half = torch.randint(-8, 9, (many, H // 2), generator=g) + torch.randint(-4, 5, (many, 1), generator=g)
    x = torch.cat([half, -half], 1).to(dt).cuda()
    w = torch.ones(H, dtype=dt, device="cuda")
    assert many > resident_rows(H, dt, H % 8 == 0)
    y, _, rstd = ep.layer_norm(x, w, rms=rms)
    for at in range(0, 200, 4):
        y4, _, rstd4 = ep.layer_norm(x[at:at + 4].contiguous(), w, rms=rms)
        assert torch.equal(rstd4, rstd[at:at + 4]) and torch.equal(y4, y[at:at + 4])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(4, 7168), (1000, 7168), (4, 1110), (2000, 1110), (4, 300), (3000, 300), (900, 9000)])
def test_gradient_of_a_row_of_equal_gradients_is_zero(T, H, dt):
    """With weight 1, grad_y = c and xh summing to 0, a - mean(a) and the sum of a * xh are exactly 0."""
    import combine_topk_ids_histogram_gb300 as ep
    g = torch.Generator().manual_seed(H)
    half = torch.randint(-8, 9, (T, H // 2), generator=g)
    x = torch.cat([half, -half], 1).to(dt).cuda()
    gy = ((torch.arange(T) % 7 - 3)[:, None] * torch.ones(1, H)).to(dt).cuda()
    w = torch.ones(H, dtype=dt, device="cuda")
    rstd = torch.full((T,), 0.125, device="cuda")                       # a * xh: whole eighths, exact in any order
    dx, _, _ = ep.layer_norm_bwd(gy, x, w, torch.zeros(T, device="cuda"), rstd)
    assert (dx == 0).all()


@pytest.mark.parametrize("T,H", [(1, 2048), (3, 7168), (1500, 7168), (9801, 256), (2000, 1111)])
def test_mean_near_zero_keeps_its_digits(T, H):
    """Values that are whole sixteenths below 8: their sum is exact in fp32 in any order, so that the mean is its H-th part, rounded
    once, however near 0 it is."""
    import combine_topk_ids_histogram_gb300 as ep
    g = torch.Generator().manual_seed(T)
    half = torch.randint(-127, 128, (T, H // 2), generator=g)
    x = torch.cat([half, -half, torch.zeros(T, H % 2, dtype=half.dtype)], 1)
    x[:, 0] += torch.arange(T) % 3 - 1                                  # the sum is -1, 0 or 1 sixteenth
    x = (x.clamp(-127, 127).double() / 16)
    w = torch.ones(H, device="cuda").bfloat16()
    _, mean, _ = ep.layer_norm(x.bfloat16().cuda(), w)
    want = x.sum(1) / H
    assert torch.equal(mean.cpu(), want.float())
