"""Plain 64-bit forms of the grouped 16-bit products, their gradients and the low-rank adapters, with the bounds that the
GPU tests hold the kernels to.  Bounds are derived from the arithmetic, never fitted:

* Products of 16-bit values are exact in fp32.  A step of the tensor cores adds 16 of them to a sum with an error of at most
  2^-22 of the magnitudes it adds (it may truncate), so a sum of n terms is off by at most (n/16 + 16) * 2^-22 * sum|terms|.
* An output is rounded once, by at most U(type) of itself (or half the type's smallest step).
* sigmoid: the exponential and the fast division are off by 2 ulp each, under 2^-16 with the products around them.
"""
import torch

from operator_ref import TINY, U

FAST = 2.0 ** -16


def layout_of(ep, counts, shared=0, pad=1, capacity=None, seed=0):
    """A layout whose groups have these many rows (tokens in random order, one slot each)."""
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(seed))].to(torch.int32).view(-1, 1).cuda()
    if pad == 1 and capacity is None:
        return ep.dispatch_layout(ids, len(counts), fused_shared=bool(shared))
    return ep.dispatch_layout_routed(len(counts), topk_ids=ids, fused_shared=bool(shared), pad_multiple=pad,
                                     num_permuted_tokens=capacity)[0]


def extents(L):
    off = L.row_offsets.tolist()
    return [slice(a, b) for a, b in zip(off, off[1:])]


def terms(n):
    return (n / 16 + 16) * 2.0 ** -22


def rounded(y, err, dtype):
    return err + U[dtype] * (y.abs() + err) + TINY[dtype]


def linear(x, w):
    """One group: y [R, N] and the error of its sums, in 64 bits."""
    x, w = x.double(), w.double()
    return x @ w.t(), terms(x.shape[1]) * (x.abs() @ w.abs().t())


def glu(y, err):
    F = y.shape[1] // 2
    gate, up, eg, eu = y[:, :F], y[:, F:], err[:, :F], err[:, F:]
    s = gate * torch.sigmoid(gate)
    es = 1.1 * eg + 2 * FAST * s.abs()                  # |silu'| <= 1.1
    return s * up, es * (up.abs() + eu) + s.abs() * eu


def grad_gate(d, err, gate_up):
    """Gradient of (gate, up) from that of their product."""
    gate, up = gate_up.double().chunk(2, 1)
    s = torch.sigmoid(gate)
    slope = s * (1 + gate * (1 - s))
    e_slope = 4 * FAST * (1 + gate.abs())               # of s and of 1 - s, and the roundings between
    out = torch.cat([d * up * slope, d * gate * s], 1)
    e = torch.cat([err * (up * slope).abs() + (d.abs() + err) * up.abs() * e_slope,
                   err * (gate * s).abs() + (d.abs() + err) * (gate * s).abs() * 4 * FAST], 1)
    return out, e


def grad_w(g, x):
    g, x = g.double(), x.double()
    return g.t() @ x, terms(x.shape[0]) * (g.abs().t() @ x.abs())


def lora(x, a, b, scale, dtype):
    """The adapter's part for the rows of one group."""
    x, a, b = x.double(), a.double(), b.double()
    t, et = x @ a.t(), terms(x.shape[1]) * (x.abs() @ a.abs().t())
    keep = 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -22
    et = et + keep * t.abs() + 2.0 ** -37 * t.abs().max(1, keepdim=True).values
    d = scale * (t @ b.t())
    return d, scale * (et @ b.abs().t() + 2 * terms(t.shape[1]) * ((t.abs() + et) @ b.abs().t()))


def assert_within(got, want, tol, what):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    bad = ~((got - want).abs() <= tol) & ~want.isnan() & (got != want)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: got {got[i].item()}, "
                             f"expected {want[i].item()}, bound {tol[i].item()}")
