"""The router's selection, probabilities and gradient against the 64-bit definition: ties, masked experts and
rows, the types' lowest values, NaN and infinities, every score, strided logits."""
import numpy as np
import pytest
import torch

import operator_ref as ref

pytestmark = pytest.mark.gpu

MODES = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]
DT = [torch.bfloat16, torch.float16, torch.float32]
SIZES = [(1, 1, 1), (1, 8, 2), (5, 7, 7), (33, 32, 8), (9, 33, 32), (17, 64, 6), (300, 128, 8), (64, 130, 8), (70, 256, 8),
         (20, 257, 3), (12, 512, 16), (6, 1000, 10), (3, 1024, 32)]


def make(T, E, dt, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(T, E, generator=g)).to(dt).cuda()


def check(ep, l, K, bias, score, renorm, scale, seed=0):
    ids, p = ep.router_topk(l, K, bias=bias, score=score, renormalize=renorm, scale=scale)
    want = ref.select(l, bias, K)
    assert np.array_equal(ids.cpu().numpy(), want)
    rp, _ = ref.probs(l, want, score, renorm, scale)
    ref.assert_within(p, rp, ref.probs_rel(l, want) * rp + 2.0 ** -125, "probs")
    g = torch.randn(*p.shape, generator=torch.Generator().manual_seed(seed)).cuda()
    dl = ep.router_topk_bwd(g, l, ids, score=score, renormalize=renorm, scale=scale)
    rd, td = ref.router_bwd(g, l, want, score, renorm, scale)
    assert dl.dtype == l.dtype
    ref.assert_within(dl, rd, 1.01 * ref.U[l.dtype] * np.abs(rd) + td + ref.TINY[l.dtype] + 2.0 ** -120, "grad_logits")
    return ids, p, dl


@pytest.mark.parametrize("T,E,K", SIZES)
@pytest.mark.parametrize("score,renorm", MODES)
def test_sizes(T, E, K, score, renorm):
    import combine_topk_ids_histogram_gb300 as ep
    for i, dt in enumerate(DT):
        l = make(T, E, dt, 100 * i + E)
        bias = torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda() if i != 1 else None
        check(ep, l, K, bias, score, renorm, 1.0 if i else 2.5, seed=T)


@pytest.mark.parametrize("score,renorm", MODES)
def test_ties_go_to_the_lower_id(score, renorm):
    """Few distinct values, +0 beside -0."""
    import combine_topk_ids_histogram_gb300 as ep
    g = torch.Generator().manual_seed(1)
    vals = torch.tensor([-1.0, -0.0, 0.0, 0.5])
    l = vals[torch.randint(0, 4, (50, 96), generator=g)].cuda()
    check(ep, l, 12, None, score, renorm, 1.0)
    check(ep, torch.zeros(3, 40, device="cuda"), 5, None, score, renorm, 1.0)


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("dt", DT)
def test_masked_experts_and_rows(score, renorm, dt):
    """-inf is not selectable; fewer than K are left in some rows, none in others.  The type's lowest value
    is a number like any other."""
    import combine_topk_ids_histogram_gb300 as ep
    l = make(40, 64, dt, 9)
    l[:, 10:20] = float("-inf")
    l[3] = float("-inf")
    l[4] = float("-inf")
    l[4, 17] = 0.25
    l[5, 4:] = float("-inf")
    l[6] = torch.finfo(dt).min
    l[7] = float("-inf")
    l[7, 33:35] = torch.finfo(dt).min
    ids, p, dl = check(ep, l, 6, None, score, renorm, 1.5)
    assert (ids[3] == -1).all() and (p[3] == 0).all() and (dl[3] == 0).all()
    assert ids[4].tolist() == [17] + [-1] * 5
    if renorm:
        assert p[4, 0].item() == 1.5
        assert torch.equal(p[7, :2], torch.full((2,), 0.75, device="cuda"))
    # a bias of -inf switches an expert off for every token
    bias = torch.zeros(64, device="cuda")
    bias[::2] = float("-inf")
    ids, _, _ = check(ep, l, 6, bias, score, renorm, 1.0)
    assert ((ids < 0) | (ids % 2 == 1)).all()


def test_masked_slots_ignore_their_gradient():
    import combine_topk_ids_histogram_gb300 as ep
    l = make(4, 16, torch.float32, 3)
    l[:, 2:] = float("-inf")
    for score, renorm in MODES:
        ids, p = ep.router_topk(l, 4, score=score, renormalize=renorm)
        g = torch.ones(4, 4, device="cuda")
        a = ep.router_topk_bwd(g, l, ids, score=score, renormalize=renorm)
        g[:, 2:] = float("nan")
        b = ep.router_topk_bwd(g, l, ids, score=score, renormalize=renorm)
        assert torch.equal(a, b) and (a[:, 2:] == 0).all()


def test_extreme_logits():
    """Sigmoids that all underflow keep their ratios; large logits saturate."""
    import combine_topk_ids_histogram_gb300 as ep
    l = torch.full((3, 8), -300.0, device="cuda")
    l[0, 2], l[0, 5] = -299.0, -298.0
    l[1] = torch.linspace(100, 300, 8, device="cuda")
    l[2] = torch.linspace(-90, 90, 8, device="cuda")
    for score, renorm in MODES:
        check(ep, l, 3, None, score, renorm, 1.0)


def test_nan_shows_and_stays_in_its_row():
    import combine_topk_ids_histogram_gb300 as ep
    l = make(6, 32, torch.float32, 4)
    clean = {m: ep.router_topk(l, 4, score=m[0], renormalize=m[1]) for m in MODES}
    l[2, 30] = float("nan")
    l[4, 1] = float("inf")
    for m in MODES:
        ids, p = ep.router_topk(l, 4, score=m[0], renormalize=m[1])
        assert np.array_equal(ids.cpu().numpy(), ref.select(l, None, 4))
        assert ids[2, 0] == 30 and torch.isnan(p[2, 0]) and ids[4, 0] == 1
        for t in (0, 1, 3, 5):
            assert torch.equal(p[t], clean[m][1][t])


def test_nan_shows_beside_masked_experts():
    """A NaN logit is selected first and its probability is NaN, where nothing but masked experts is beside it too."""
    import combine_topk_ids_histogram_gb300 as ep
    for E in (5, 32, 40, 256):
        l = torch.full((3, E), float("-inf"), device="cuda")
        l[0, E - 2] = float("nan")
        l[1, 1], l[1, 3] = float("nan"), 0.5
        for score, renorm in MODES:
            ids, p = ep.router_topk(l, 4, score=score, renormalize=renorm)
            assert ids.tolist() == [[E - 2, -1, -1, -1], [1, 3, -1, -1], [-1] * 4]
            assert torch.isnan(p[0, 0]) and torch.isnan(p[1, 0]) and (p[0, 1:] == 0).all() and (p[2] == 0).all()


def test_strided_logits():
    import combine_topk_ids_histogram_gb300 as ep
    for off, E, width in ((0, 64, 80), (3, 60, 77), (8, 128, 160)):
        wide = make(21, width, torch.bfloat16, off)
        view = wide[:, off:off + E]
        for score, renorm in MODES:
            a = check(ep, view, 5, None, score, renorm, 1.0)
            b = check(ep, view.contiguous(), 5, None, score, renorm, 1.0)
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_ids_outside_and_repeated_in_the_backward_pass():
    """Ids outside [0, E) count as unused; slots that name the same expert add up."""
    import combine_topk_ids_histogram_gb300 as ep
    l = make(4, 20, torch.float32, 8)
    ids = torch.tensor([[3, 99, -5, 7], [2, 2, 2, 1], [20, -1, -1, -1], [19, 0, 19, 0]], dtype=torch.int32, device="cuda")
    g = torch.randn(4, 4, generator=torch.Generator().manual_seed(1)).cuda()
    for score, renorm in MODES:
        got = ep.router_topk_bwd(g, l, ids, score=score, renormalize=renorm, scale=1.25)
        want, tol = ref.router_bwd(g, l, ids.cpu().numpy(), score, renorm, 1.25)
        ref.assert_within(got, want, tol + ref.U[torch.float32] * np.abs(want) + 1e-30, f"{score} {renorm}")


@pytest.mark.parametrize("score,renorm", MODES)
def test_gradient_against_differences(score, renorm):
    """Central differences of the 64-bit probabilities with the ids held."""
    import combine_topk_ids_histogram_gb300 as ep
    T, E, K, scale = 5, 24, 4, 1.5
    l = make(T, E, torch.float32, 21, spread=1.0)
    ids, _ = ep.router_topk(l, K, score=score, renormalize=renorm, scale=scale)
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).cuda()
    dl = ref.d64(ep.router_topk_bwd(g, l, ids, score=score, renormalize=renorm, scale=scale)).numpy()
    idn, gn, h = ids.cpu().numpy(), ref.d64(g).numpy(), 1e-5
    _, td = ref.router_bwd(g, l, idn, score, renorm, scale)
    for e in range(E):
        step = torch.zeros(T, E, dtype=torch.float64)
        step[:, e] = h
        hi, _ = ref.probs(ref.d64(l) + step, idn, score, renorm, scale)
        lo, _ = ref.probs(ref.d64(l) - step, idn, score, renorm, scale)
        diff = ((hi - lo) / (2 * h) * gn).sum(1)
        # truncation h^2/6 * |third derivative| <= 1e-10 * scale * sum|g|, rounding 2^-52/h
        tol = td[:, e] + ref.U[torch.float32] * np.abs(diff) + 1e-9 * np.abs(gn).sum(1)
        assert (np.abs(dl[:, e] - diff) <= tol).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 16, 4), (33, 64, 6), (500, 256, 8)])
def test_a_bias_on_the_score_takes_two_steps(T, E, K, renorm):
    """The call's bias is added to the logit.  A router that adds it to sigmoid(logit) takes its ids from a call on those
    sums, its probabilities from the logits at these ids, and its gradient from the backward call with these ids."""
    import combine_topk_ids_histogram_gb300 as ep
    g = torch.Generator().manual_seed(E)
    l, bias = make(T, E, torch.float32, E), torch.randn(E, generator=g).cuda()
    s = torch.sigmoid(l) + bias
    ids, _ = ep.router_topk(s, K)
    want = ref.select(s, None, K)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert T == 1 or not np.array_equal(want, ref.select(l, bias, K))          # another order than the call's own bias gives
    p = torch.sigmoid(l).gather(1, ids.long())
    p = 2.5 * (p / p.sum(1, keepdim=True) if renorm else p)
    rp, _ = ref.probs(l, want, "sigmoid", renorm, 2.5)
    ref.assert_within(p, rp, ref.probs_rel(l, want) * rp, "probs")
    gp = torch.randn(T, K, generator=g).cuda()
    dl = ep.router_topk_bwd(gp, l, ids, score="sigmoid", renormalize=renorm, scale=2.5)
    rd, td = ref.router_bwd(gp, l, want, "sigmoid", renorm, 2.5)
    ref.assert_within(dl, rd, 1.01 * ref.U[l.dtype] * np.abs(rd) + td + 2.0 ** -120, "grad_logits")


def test_no_tokens_and_refusals():
    import combine_topk_ids_histogram_gb300 as ep
    l = torch.empty(0, 16, device="cuda")
    ids, p = ep.router_topk(l, 4)
    assert ids.shape == (0, 4)
    assert ep.router_topk_bwd(p, l, ids).shape == (0, 16)
    l = make(4, 16, torch.float32, 1)
    ids, p = ep.router_topk(l, 4)
    for bad in (dict(K=0), dict(K=17), dict(K=4, scale=0.0), dict(K=4, scale=float("inf")), dict(K=4, scale=float("nan"))):
        with pytest.raises(ep.EPError):
            ep.router_topk(l, **bad)
    with pytest.raises(ep.EPError):
        ep.router_topk(make(2, 40, torch.float32, 1), 33)              # K above 32
    with pytest.raises(ep.EPError):
        ep.router_topk(torch.zeros(1, 1025, device="cuda"), 2)
    with pytest.raises(ValueError):
        ep.router_topk(l, 4, score="relu")
    with pytest.raises(TypeError):
        ep.router_topk(l.double(), 4)
    with pytest.raises(ValueError):
        ep.router_topk(l, 4, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(TypeError):
        ep.router_topk(l, 4, bias=torch.zeros(16, dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        ep.router_topk_bwd(p, l, ids.long())
    with pytest.raises(ValueError):
        ep.router_topk_bwd(p[:, :3].contiguous(), l, ids)
