"""Host-side argument checks of the grouped 16-bit products and the adapters (no GPU: every call here returns before any
CUDA call), and the 64-bit forms that the GPU tests trust on values worked by hand."""
import ctypes

import torch

import linear_ref as ref


def _ep():
    import __graft_entry__ as entry
    entry._load_builder().build()
    import combine_topk_ids_histogram_gb300 as ep
    return ep


def _layout(ep, **kw):
    return ep._Layout(**{**dict(row_offsets=256, expert_ids=256, src_info=256, row_of=256, part_tokens=256, status=256, workspace=256,
                                workspace_bytes=1 << 20, T=4, K=2, E=8, P=1, capacity=4, fused_shared=0, pad_multiple=1, row_capacity=0), **kw})


def test_linear_refusals():
    ep = _ep()
    L, bad = ep.lib(), ep.EP_ERR_INVALID_ARG
    lay = _layout(ep)
    r = ctypes.byref(lay)
    ok = dict(x=256, ld=64, w=256, K=64, N=96, dt=0, swiglu=0, L=r, out=256, gu=None)

    def fwd(**kw):
        return L.ep_expert_linear(*{**ok, **kw}.values(), None)

    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(x=264), dict(w=258), dict(out=260), dict(ld=63), dict(ld=68), dict(ld=60),
               dict(ld=1 << 31), dict(K=0), dict(K=72), dict(K=32784, ld=40000), dict(N=0), dict(N=40), dict(N=65552), dict(dt=2), dict(dt=-1),
               dict(swiglu=2), dict(swiglu=1, N=48), dict(gu=256), dict(swiglu=1, gu=264), dict(L=None),
               dict(L=ctypes.byref(ep._Layout()))):
        assert fwd(**kw) == bad, kw
    okb = dict(g=256, ldg=96, x=256, ld=64, w=256, K=64, N=96, dt=1, gu=None, L=r, gx=256, gw=256, wdt=2, acc=0)

    def bwd(**kw):
        return L.ep_expert_linear_bwd(*{**okb, **kw}.values(), None)

    for kw in (dict(g=None), dict(x=None), dict(w=None), dict(gx=None, gw=None), dict(gx=None, gu=256), dict(ldg=95), dict(ldg=100), dict(ld=56),
               dict(wdt=0), dict(wdt=3), dict(acc=2), dict(acc=1, wdt=1), dict(dt=2), dict(gx=260), dict(gw=264), dict(gu=258), dict(K=24),
               dict(N=24), dict(L=None)):
        assert bwd(**kw) == bad, kw
    lay.T = 0
    assert fwd(x=None, out=None) == ep.EP_OK
    assert bwd(g=None, x=None, gw=None) == ep.EP_OK


def test_lora_refusals():
    ep = _ep()
    L, bad = ep.lib(), ep.EP_ERR_INVALID_ARG
    lay = _layout(ep, K=1)
    r = ctypes.byref(lay)
    ok = dict(y=256, ldy=96, x=256, ldx=64, a=256, b=256, scale=None, H=64, N=96, r=16, dt=0, by=1, L=r, out=512, ldo=96)

    def call(**kw):
        return L.ep_lora_add(*{**ok, **kw}.values(), None)

    for kw in (dict(y=None), dict(x=None), dict(a=None), dict(b=None), dict(out=None), dict(y=264), dict(scale=260), dict(ldy=95), dict(ldy=100),
               dict(ldx=56), dict(ldo=92), dict(H=0), dict(H=72), dict(N=8), dict(N=100), dict(r=0), dict(r=4), dict(r=12), dict(r=136), dict(dt=2),
               dict(by=2), dict(out=256, ldo=104), dict(L=None), dict(L=ctypes.byref(_layout(ep, K=2))),
               dict(L=ctypes.byref(_layout(ep, K=1, fused_shared=1))), dict(L=ctypes.byref(_layout(ep, K=1, expert_ids=None)))):
        assert call(**kw) == bad, kw
    lay.T = 0
    assert call(x=None) == ep.EP_OK


def test_timeout_code():
    ep = _ep()
    assert "wait" in ep.strerror(ep.EP_ERR_TIMEOUT)


def test_reference_forms():
    y, err = ref.linear(torch.tensor([[1.0, 2.0]]), torch.tensor([[3.0, -1.0], [0.5, 0.25]]))
    assert y.tolist() == [[1.0, 1.0]] and (err > 0).all()
    act, _ = ref.glu(torch.tensor([[0.0, 2.0, 5.0, 3.0]]).double(), torch.zeros(1, 4).double())
    assert abs(act[0, 1].item() - 6 / (1 + torch.exp(torch.tensor(-2.0)).item())) < 1e-6 and act[0, 0] == 0
    d, _ = ref.grad_gate(torch.ones(1, 1).double(), torch.zeros(1, 1).double(), torch.tensor([[0.0, 4.0]]))
    assert d.tolist() == [[2.0, 0.0]]                    # silu'(0) = 1/2
    gu = torch.randn(1, 6, dtype=torch.float64, requires_grad=True)
    gate, up = gu.chunk(2, 1)
    c = torch.randn(1, 3, dtype=torch.float64)
    (c * gate * torch.sigmoid(gate) * up).sum().backward()
    assert torch.allclose(ref.grad_gate(c, torch.zeros_like(c), gu.detach())[0], gu.grad)
    dw, _ = ref.grad_w(torch.tensor([[1.0], [2.0]]), torch.tensor([[3.0, 0.0], [1.0, 1.0]]))
    assert dw.tolist() == [[5.0, 2.0]]
    d, _ = ref.lora(torch.tensor([[1.0, 1.0]]), torch.tensor([[2.0, 3.0]]), torch.tensor([[1.0], [-1.0]]), 0.5, torch.bfloat16)
    assert d.tolist() == [[2.5, -2.5]]
