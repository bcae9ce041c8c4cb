"""The example's MoE block: the norm, the router, the layout, the expert products and combine together, against 64-bit
torch with the same routing; its gradients against autograd in 64 bits; inside a CUDA graph; and the expert and block tests
on the bounds-checked build."""
import os
import subprocess
import sys

import pytest
import torch

import operator_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

# Each bf16 rounding of an intermediate is within 2^-9 of its value; the decode step rounds six of them one after another
# (h, logits, gate * up, y, combine's sum, the residual) and the training step's longest path about twelve.  Norms of errors
# of chained roundings add up at most.
STEP = 2.0 ** -9


def block64(x, p, ids, w13, w2):
    """The MoE branch in 64 bits for given ids (differentiable)."""
    r = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5)
    h = x * r * p["norm"]
    s = torch.sigmoid((h @ p["router"].t()).gather(1, ids))
    probs = s / s.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(p["router"].shape[0]):
        t, k = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            gate, up = (h[t] @ w13[e].t()).chunk(2, 1)
            y = (torch.nn.functional.silu(gate) * up) @ w2[e].t()
            out = out.index_add(0, t, probs[t, k, None] * y)
    return out


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("T,H,F,E,K", [(1, 256, 96, 8, 2), (7, 512, 208, 16, 4), (40, 384, 128, 8, 3)])
def test_decode_step(T, H, F, E, K):
    import combine_topk_ids_histogram_gb300 as ep
    import moe_block as M
    p = M.make_weights(H, F, E)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    q13, q2 = M.quantise(p["w13"]), M.quantise(p["w2"])
    out = M.decode_step(x, p, q13, q2, K)
    h, _, _ = ep.layer_norm(x, p["norm"], rms=True)
    ids, _ = ep.router_topk(h @ p["router"].t(), K, bias=p["bias"], score="sigmoid")
    full = [torch.stack([torch.from_numpy(ref.weights(*(v[e].cpu().numpy() for v in q))) for e in range(E)]).cuda() for q in (q13, q2)]
    p64 = {k: v.double() for k, v in p.items()}
    want = x.double() + block64(x.double(), p64, ids.long(), *full)
    assert rel(out, want) <= 6 * STEP
    # the same step in a CUDA graph, on other tokens
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        gout = M.decode_step(xs, p, q13, q2, K)
    for seed in (3, 4):
        xs.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        eager = M.decode_step(xs, p, q13, q2, K)
        torch.cuda.synchronize()
        assert torch.equal(gout, eager)


@pytest.mark.parametrize("T,H,F,E,K", [(33, 256, 96, 8, 2), (500, 128, 64, 4, 2)])
def test_train_step(T, H, F, E, K):
    import moe_block as M
    p = M.make_weights(H, F, E, seed=1)
    g = torch.Generator().manual_seed(T)
    x, go = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(2))
    out, ids, grads = M.train_step(x, go, p, K)
    x64 = x.double().requires_grad_()
    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    want = block64(x64, p64, ids.long(), p64["w13"], p64["w2"])
    want.backward(go.double())
    assert rel(out, want.detach()) <= 6 * STEP
    for name, got, w in zip(("x", "norm", "router", "w13", "w2"), grads,
                            (x64, p64["norm"], p64["router"], p64["w13"], p64["w2"])):
        assert rel(got, w.grad) <= 12 * STEP, name


def test_on_the_bounds_checked_build():
    env = dict(os.environ, EP_GB300_CHECKED="1")
    if os.environ.get("EP_GB300_CHECKED", "0") == "1":
        pytest.skip("this process runs on it already")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "tests/test_gpu_experts.py",
                        "tests/test_gpu_moe_block.py", "-k", "not bounds_checked"], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
