"""One MoE block on the library's entry points, as a decode step and as a training step.

decode_step   norm -> router logits -> experts and probabilities -> layout -> 4-bit gate/up and down products on the
              layout's rows -> combine -> residual.  Nothing is dispatched: the products take each row's token.
train_step    the same block with bf16 expert weights, forward and backward: norm, router, layout, BF16 dispatch, the
              experts (a loop of library GEMMs stands in for a grouped GEMM), combine; then the gradients of x and
              of every weight, with combine_bwd's probability gradients going back through the router.

    python examples/moe_block.py [--tokens 16] [--hidden 2048] [--width 768] [--experts 128] [--topk 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_topk_ids_histogram_gb300 as ep  # noqa: E402

SCALE = 1.0


def quantise(w: torch.Tensor):
    """Weights [G, N, H] bf16 -> the codes, block scales and row scales that expert_matvec takes: the NVFP4 dispatch of G*N
    tokens to one expert."""
    G, N, H = w.shape
    L = ep.dispatch_layout(torch.zeros(G * N, 1, dtype=torch.int32, device=w.device), 1)
    codes, scales, inv, _ = ep.dispatch_nvfp4(w.reshape(G * N, H), L)
    return codes.view(G, N, H // 2), scales.view(G, N, H // 16), inv.float().view(G, N)


def make_weights(H: int, F: int, E: int, device="cuda", seed: int = 0) -> dict:
    g = torch.Generator(device=device).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=device)
    return dict(norm=(1 + 0.1 * normal(H)).bfloat16(), router=(normal(E, H) / H ** 0.5).bfloat16(), bias=0.1 * normal(E),
                w13=(normal(E, 2 * F, H) / H ** 0.5).bfloat16(), w2=(normal(E, H, F) / F ** 0.5).bfloat16())


def decode_step(x: torch.Tensor, p: dict, w13, w2, K: int) -> torch.Tensor:
    """x [T, H] bf16 -> [T, H]; w13 and w2 are quantised."""
    h, _, _ = ep.layer_norm(x, p["norm"], rms=True)
    ids, probs = ep.router_topk(h @ p["router"].t(), K, bias=p["bias"], score="sigmoid", scale=SCALE)
    L = ep.dispatch_layout(ids, p["router"].shape[0])
    a = ep.expert_matvec(h, *w13, L, by_token=True, swiglu=True)
    y = ep.expert_matvec(a, *w2, L, by_token=False)
    return x + ep.combine(y, probs, L)


def train_step(x: torch.Tensor, grad_out: torch.Tensor, p: dict, K: int):
    """Forward and backward of the block's MoE branch (without the residual): (out, ids, grads of x, norm, router, w13, w2)."""
    E, F = p["router"].shape[0], p["w2"].shape[2]
    h, _, rstd = ep.layer_norm(x, p["norm"], rms=True)
    logits = h @ p["router"].t()
    ids, probs = ep.router_topk(logits, K, bias=p["bias"], score="sigmoid", scale=SCALE)
    L = ep.dispatch_layout(ids, E)
    rows = ep.dispatch_bf16(h, L)
    y = torch.empty_like(rows)
    off = L.row_offsets.tolist()                                   # a grouped GEMM would read the extents on the device
    saved = {}
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a < b:
            gate, up = (rows[a:b] @ p["w13"][e].t()).float().chunk(2, 1)
            act = (torch.nn.functional.silu(gate) * up).bfloat16()
            saved[e] = gate, up, act
            torch.matmul(act, p["w2"][e].t(), out=y[a:b])
    out = ep.combine(y, probs, L)

    grad_y, grad_probs = ep.combine_bwd(grad_out, y, probs, L)
    grad_rows = torch.empty_like(rows)
    gw13, gw2 = torch.zeros_like(p["w13"]), torch.zeros_like(p["w2"])
    for e, (gate, up, act) in saved.items():
        a, b = off[e], off[e + 1]
        gw2[e] = grad_y[a:b].t() @ act
        ga = (grad_y[a:b] @ p["w2"][e]).float()
        s = torch.sigmoid(gate)
        g13 = torch.cat([ga * up * s * (1 + gate * (1 - s)), ga * gate * s], 1).bfloat16()
        gw13[e] = g13.t() @ rows[a:b]
        torch.matmul(g13, p["w13"][e], out=grad_rows[a:b])
    grad_logits = ep.router_topk_bwd(grad_probs, logits, ids, score="sigmoid", scale=SCALE)
    grad_h = ep.dispatch_bwd(grad_rows, L) + grad_logits @ p["router"]
    grad_x, grad_norm, _ = ep.layer_norm_bwd(grad_h, x, p["norm"], None, rstd, rms=True)
    return out, ids, (grad_x, grad_norm, grad_logits.t() @ h, gw13, gw2)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, v in (("tokens", 16), ("hidden", 2048), ("width", 768), ("experts", 128), ("topk", 8)):
        ap.add_argument("--" + name, type=int, default=v)
    a = ap.parse_args()
    p = make_weights(a.hidden, a.width, a.experts)
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    w13, w2 = quantise(p["w13"]), quantise(p["w2"])

    def timed(name, f, n=50):
        for _ in range(5):
            f()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(n):
            f()
        end.record()
        end.synchronize()
        print(f"{name}: {begin.elapsed_time(end) / n * 1e3:.1f} us")

    timed("decode step", lambda: decode_step(x, p, w13, w2, a.topk))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode_step(x, p, w13, w2, a.topk)
    timed("decode step as a CUDA graph", graph.replay)
    g = torch.randn_like(x)
    timed("training step", lambda: train_step(x, g, p, a.topk), 5)


if __name__ == "__main__":
    main()
