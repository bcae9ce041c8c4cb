"""Host-side argument checks of the norm, router and expert-product calls (no GPU: every call here returns
before any CUDA call), and the CPU reference forms against hand-worked values."""
import ctypes

import numpy as np
import torch

import operator_ref as ref


def _ep():
    import __graft_entry__ as entry
    entry._load_builder().build()
    import combine_topk_ids_histogram_gb300 as ep
    return ep


def test_norm_refusals():
    ep = _ep()
    L, bad = ep.lib(), ep.EP_ERR_INVALID_ARG
    ok = dict(x=256, ld=64, dt=0, w=256, b=256, wdt=0, T=4, H=64, eps=1e-5, rms=0, y=256, mean=256, rstd=256)

    def fwd(**kw):
        return L.ep_layer_norm(*{**ok, **kw}.values(), None)

    for kw in (dict(H=0), dict(H=32769, ld=40000), dict(T=-1), dict(T=(1 << 24) + 1), dict(ld=63), dict(dt=3), dict(dt=-1),
               dict(wdt=1), dict(dt=2, wdt=0), dict(rms=2), dict(eps=-1e-9), dict(eps=float("nan")), dict(x=None),
               dict(w=None), dict(y=None), dict(rstd=None), dict(mean=None), dict(x=257), dict(y=255), dict(rstd=258),
               dict(b=253), dict(wdt=2, w=258)):
        assert fwd(**kw) == bad, kw
    assert fwd(T=0, x=None, y=None) == ep.EP_OK
    assert L.ep_layer_norm_bwd_workspace_bytes(0, 64) > 0
    assert L.ep_layer_norm_bwd_workspace_bytes(4, 64) == 4 * 2 * 64 * 4
    assert L.ep_layer_norm_bwd_workspace_bytes(1 << 20, 7168) == 304 * 2 * 7168 * 4
    assert L.ep_layer_norm_bwd_workspace_bytes(4, 0) == 0 and L.ep_layer_norm_bwd_workspace_bytes(4, 32769) == 0
    okb = dict(g=256, ldg=64, x=256, ld=64, dt=0, w=256, wdt=0, mean=256, rstd=256, T=4, H=64, rms=0, dx=256, dw=256,
               db=256, ws=256, nws=4 * 2 * 64 * 4)

    def bwd(**kw):
        return L.ep_layer_norm_bwd(*{**okb, **kw}.values(), None)

    for kw in (dict(g=None), dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(dw=None),
               dict(ws=None), dict(nws=2047), dict(ws=264), dict(ldg=60), dict(ld=8), dict(H=0), dict(dw=258), dict(db=257),
               dict(g=255), dict(wdt=1), dict(rms=-1)):
        assert bwd(**kw) == bad, kw


def test_router_refusals():
    ep = _ep()
    L, bad = ep.lib(), ep.EP_ERR_INVALID_ARG
    ok = dict(l=256, ld=64, dt=2, b=None, T=4, E=64, K=8, score=0, renorm=1, scale=1.0, ids=256, p=256)

    def fwd(**kw):
        return L.ep_router_topk(*{**ok, **kw}.values(), None)

    for kw in (dict(l=None), dict(ids=None), dict(p=None), dict(K=0), dict(K=33), dict(K=9, E=8), dict(E=0),
               dict(E=1025, ld=2000), dict(ld=63), dict(dt=4), dict(score=2), dict(score=-1), dict(renorm=2), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(l=258), dict(b=254), dict(ids=260),
               dict(T=-1)):
        assert fwd(**kw) == bad, kw
    assert fwd(T=0, l=None, ids=None, p=None) == ep.EP_OK
    okb = dict(g=256, l=256, ld=64, dt=2, ids=256, T=4, E=64, K=8, score=1, renorm=0, scale=1.0, dl=256)

    def bwd(**kw):
        return L.ep_router_topk_bwd(*{**okb, **kw}.values(), None)

    for kw in (dict(g=None), dict(l=None), dict(ids=None), dict(dl=None), dict(K=65), dict(scale=0.0), dict(dl=264),
               dict(ld=10), dict(score=5)):
        assert bwd(**kw) == bad, kw


def test_expert_refusals():
    ep = _ep()
    L, bad = ep.lib(), ep.EP_ERR_INVALID_ARG
    lay = ep._Layout(row_offsets=256, expert_ids=256, src_info=256, row_of=256, part_tokens=256, status=256,
                     workspace=256, workspace_bytes=1 << 20, T=4, K=2, E=8, P=1, capacity=4, fused_shared=0,
                     pad_multiple=1, row_capacity=0)
    ref_ = ctypes.byref(lay)
    ok = dict(x=256, by_token=1, codes=256, scales=256, rs=256, H=64, N=32, swiglu=0, L=ref_, out=256, ws=256, nws=1 << 20)

    def call(**kw):
        return L.ep_expert_matvec(*{**ok, **kw}.values(), None)

    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(rs=None), dict(out=None), dict(x=264), dict(out=258),
               dict(codes=257), dict(ws=None), dict(ws=264), dict(nws=8 * 512 + 47), dict(H=24), dict(H=0), dict(H=32784), dict(N=0), dict(N=65537), dict(N=33, swiglu=1),
               dict(swiglu=2), dict(by_token=2), dict(L=None), dict(L=ctypes.byref(ep._Layout()))):
        assert call(**kw) == bad, kw
    # 8 rows x 256 k in fp16, and 8 scales
    assert L.ep_expert_matvec_workspace_bytes(ref_, 64) == 8 * 512 + 32 + 16
    assert L.ep_expert_matvec_workspace_bytes(ref_, 24) == 0
    lay.src_info = None
    assert call() == bad                       # token gathering needs src_info
    lay.src_info = 256
    lay.T = 0
    assert call(x=None) == ep.EP_OK


def test_reference_forms():
    """The forms that the GPU tests trust, on values worked by hand."""
    y, mean, rstd = ref.norm(torch.tensor([[1.0, 3.0]]), torch.tensor([2.0, 1.0]), torch.tensor([0.5, 0.0]), 0.0, False)
    assert mean.item() == 2 and rstd.item() == 1 and y.tolist() == [[-1.5, 1.0]]
    y, _, rstd = ref.norm(torch.tensor([[3.0, 4.0]]), torch.ones(2), None, 0.0, True)
    assert abs(rstd.item() - (2 / 25) ** 0.5) < 1e-15
    l = torch.tensor([[0.0, 1.0, float("nan"), 1.0, float("-inf")]])
    assert ref.select(l, None, 5).tolist() == [[2, 1, 3, 0, -1]]
    l = torch.tensor([[0.0, np.log(3.0), float("-inf")]])
    ids = ref.select(l, None, 2)
    assert ids.tolist() == [[1, 0]]
    p, _ = ref.probs(l, ids, "softmax", True, 2.0)
    assert np.allclose(p, [[1.5, 0.5]], atol=1e-6)
    p, slope = ref.probs(l, ids, "sigmoid", False, 1.0)
    assert np.allclose(p, [[0.75, 0.5]], atol=1e-6) and np.allclose(slope, [[0.25, 0.5]], atol=1e-6)
    codes = np.array([[0x21, 0xF7] + [0] * 6], np.uint8)
    w = ref.weights(codes, np.array([[0x40]], np.uint8), np.array([0.5], np.float32))
    assert w[0, :4].tolist() == [0.5, 1.0, 6.0, -6.0] and (w[0, 4:] == 0).all()      # scale 0x40 is 2
    assert ref.e4m3(np.array([0x01, 0x7E, 0xB8], np.uint8)).tolist() == [2.0 ** -9, 448.0, -1.0]
