"""Plain 64-bit numpy/torch forms of the norm, the router and the expert products, on the CPU, and the
error bounds the GPU tests hold the kernels to.  Bounds are derived from the arithmetic, never fitted:

* u(dtype) is half an ulp of the output's type (one rounding of the fp32 result).
* A sum of n fp32 terms in any order of depth d is off by at most d * 2^-24 * sum|terms|.
"""
from __future__ import annotations

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -148}   # subnormal step
EPS24 = 2.0 ** -24


def d64(t):
    return t.detach().double().cpu()


# ------------------------------------------------------------------------------- norm
def norm(x, w, b, eps, rms):
    """y, mean, rstd in 64 bits."""
    x, w = d64(x), d64(w)
    mean = torch.zeros(x.shape[0], dtype=torch.float64) if rms else x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None] * w
    return (y if b is None else y + d64(b)), mean, rstd


# Depth of a row sum in the forward and backward kernels: at most 64 terms per thread, 5 shuffle steps,
# 32 warps, and a few single roundings; 128 covers all of them.
ROW = 128 * EPS24


def norm_tol(x, w, b, eps, rms, dtype):
    """Bounds of y, mean and rstd."""
    x, wd = d64(x), d64(w).abs()
    y, mean, rstd = norm(x, w, b, eps, rms)
    absmean = x.abs().mean(1)
    dmean = torch.zeros_like(mean) if rms else ROW * absmean
    # var is over (x - mean - dmean): + dmean^2; the squares' sum has the row sum's error
    drstd = rstd * (ROW + (dmean * rstd) ** 2)
    xh = (x - mean[:, None]).abs() * rstd[:, None]
    dxh = (rstd * dmean)[:, None] + xh * (drstd / rstd)[:, None] + 4 * EPS24 * xh
    ty = U[dtype] * y.abs() + 1.01 * dxh * wd + 4 * EPS24 * (xh * wd + (0 if b is None else d64(b).abs())) + TINY[dtype]
    return ty, dmean + EPS24 * mean.abs(), drstd + EPS24 * rstd


def norm_bwd(g, x, w, mean, rstd, rms):
    """dx, dw, db in 64 bits from the saved fp32 statistics."""
    g, x, w, r = d64(g), d64(x), d64(w), d64(rstd)[:, None]
    m = 0.0 if rms else d64(mean)[:, None]
    xh = (x - m) * r
    a = g * w
    dx = a - xh * (a * xh).mean(1, keepdim=True)
    if not rms:
        dx = dx - a.mean(1, keepdim=True)
    return r * dx, (g * xh).sum(0), g.sum(0)


def norm_bwd_tol(g, x, w, mean, rstd, rms, dtype):
    T = x.shape[0]
    dx, _, _ = norm_bwd(g, x, w, mean, rstd, rms)
    g, x, w, r = d64(g), d64(x), d64(w), d64(rstd)[:, None]
    m = 0.0 if rms else d64(mean)[:, None]
    xh = ((x - m) * r).abs()
    a = (g * w).abs()
    max_ = (a * xh).mean(1, keepdim=True)
    ma = 0.0 if rms else a.mean(1, keepdim=True)
    tx = U[dtype] * dx.abs() + r * ((ROW + 8 * EPS24) * (ma + xh * max_) + 8 * EPS24 * a) + TINY[dtype]
    # a column: at most T/16 rows per thread, 16 groups, 304/32 partial rows, 5 shuffle steps
    col = (T / 16 + 64) * EPS24
    return tx, col * (g.abs() * xh).sum(0) + 1e-30, col * g.abs().sum(0) + 1e-30


# ------------------------------------------------------------------------------- router
def select(logits, bias, K):
    """The K largest of the fp32 logit + bias, NaN first, ties to the lower id, -1 for -inf."""
    l = logits.detach().float().cpu().numpy()
    s = l if bias is None else l + bias.detach().float().cpu().numpy()
    key = np.where(np.isnan(s), np.float64(np.inf), s.astype(np.float64))
    rank = np.where(np.isnan(s), 1, 0)
    ids = np.empty((s.shape[0], K), np.int32)
    for t in range(s.shape[0]):
        order = sorted(range(s.shape[1]), key=lambda e: (-rank[t, e], -key[t, e], e))[:K]
        ids[t] = [e if s[t, e] != -np.inf else -1 for e in order]
    return ids


def probs(logits, ids, score, renorm, scale):
    """Slot probabilities in 64 bits, and 1 - sigmoid of the slots' logits."""
    l = d64(logits).numpy()
    used = ids >= 0
    v = np.take_along_axis(l, np.maximum(ids, 0), 1)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "softmax":
            pool = np.where(used, v, -np.inf) if renorm else l
            top = pool.max(1, keepdims=True)
            top = np.where(np.isinf(top), 0.0, top)
            p = np.exp(v - top) / np.exp(pool - top).sum(1, keepdims=True)
        else:
            logs = np.minimum(v, 0) - np.log1p(np.exp(-np.abs(v)))      # log sigmoid
            p = np.exp(logs)
            if renorm:
                logs = np.where(used, logs, -np.inf)
                top = logs.max(1, keepdims=True)
                top = np.where(np.isinf(top), 0.0, top)
                e = np.exp(logs - top)
                p = e / e.sum(1, keepdims=True)
        slope = np.exp(np.minimum(-v, 0) - np.log1p(np.exp(-np.abs(v))))   # 1 - sigmoid(v)
    return np.where(used, scale * p, 0.0), slope


def probs_rel(logits, ids):
    """Relative bound of a probability: expf and the divisions are good to a few ulp, the exponent's
    argument l - max is rounded once (an error of |l - max| * 2^-24 in the exponent), and the sum over up
    to 1024 experts has depth 32 + 5."""
    l = d64(logits).numpy()
    fin = np.where(np.isfinite(l), l, 0.0)
    spread = fin.max(1, keepdims=True) - fin.min(1, keepdims=True)
    return (96 + 2 * spread) * EPS24


def router_bwd(g, logits, ids, score, renorm, scale):
    """d logits in 64 bits, and the bound of its fp32 computation before the last rounding."""
    l = d64(logits).numpy()
    E = l.shape[1]
    ids = np.where((ids >= 0) & (ids < E), ids, -1)
    used = ids >= 0
    p, slope = probs(logits, ids, score, renorm, scale)
    g = np.where(used, d64(g).numpy(), 0.0)
    G = (g * p).sum(1, keepdims=True) / scale
    absG = np.abs(g * p).sum(1, keepdims=True) / scale
    out, mag = np.zeros_like(l), np.zeros_like(l)
    if score == "softmax" and not renorm:
        with np.errstate(invalid="ignore"):
            top = l.max(1, keepdims=True)
            e = np.exp(l - np.where(np.isinf(top), 0.0, top))
            tot = e.sum(1, keepdims=True)
            P = np.where(tot > 0, e / np.where(tot > 0, tot, 1), 0.0)
        out, mag = -P * scale * G, P * scale * absG
        d, m = g * p, np.abs(g * p)
    else:
        d = p * (g - G) if renorm else g * p
        m = p * (np.abs(g) + absG) if renorm else np.abs(g * p)
        if score == "sigmoid":
            d, m = d * slope, m * slope
    for t in range(l.shape[0]):
        for k in range(ids.shape[1]):
            if used[t, k]:
                out[t, ids[t, k]] += d[t, k]
                mag[t, ids[t, k]] += m[t, k]
    return out, mag * (2 * probs_rel(logits, ids) + 64 * EPS24)


# ------------------------------------------------------------------------------- expert products
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(b):
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where(b >= 128, -v, v)


def weights(codes, scales, row_scale):
    """[N, H] in 64 bits of one group."""
    N, half = codes.shape
    w = np.empty((N, 2 * half))
    w[:, 0::2], w[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    return w * np.repeat(e4m3(scales), 16, axis=1) * row_scale.astype(np.float64)[:, None]


def experts(x, w, swiglu):
    """out and its bound for rows x [R, H] and weights w [N, H].  The products of bf16 with the scaled
    codes are exact in fp32; a tensor-core step adds 16 of them to the sum with an error of at most 2^-22
    of the magnitudes it adds (it may truncate), so H/16 steps and the joins after them are off by at most
    (H/16 + 16) * 2^-22 * sum|w x|."""
    H = x.shape[1]
    y = x @ w.T
    e = (H / 16 + 16) * 2.0 ** -22 * (np.abs(x) @ np.abs(w).T)
    if swiglu:
        n = y.shape[1] // 2
        gate, up, eg, eu = y[:, :n], y[:, n:], e[:, :n], e[:, n:]
        s = gate / (1 + np.exp(-gate))
        # |silu'| <= 1.1; expf and the division are good to a few ulp
        e = 1.1 * eg * (np.abs(up) + eu) + (np.abs(s) + 1.1 * eg) * eu + 16 * EPS24 * np.abs(s * up)
        y = s * up
    return y, e + U[torch.bfloat16] * np.abs(y) * 1.01 + 1e-38


def assert_within(got, ref, tol, what):
    got, ref, tol = (torch.as_tensor(v).double().cpu().numpy() for v in (got, ref, tol))
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= tol) & ~np.isnan(ref) & ~(got == ref)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first at {i}: got {got[i]}, "
                             f"expected {ref[i]}, bound {np.broadcast_to(tol, got.shape)[i]}")
