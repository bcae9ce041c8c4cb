"""Measured cases of the operators around the MoE dispatch: the norm in front of it (forward and
backward), the router that makes its ids and probabilities (forward and backward), and the
experts' products with 4-bit weights on the dispatched rows.

``own = False`` computes each operator in elementary torch operations in fp32, rounded once at
the end; ``own = True`` makes the library's calls.  Both take what ``prepare`` returns.

Definitions (sums and statistics in fp32 or wider everywhere):

* norm     y = (x - mean) * rstd * w + b per row, mean = sum(x)/H, rstd = 1/sqrt(mean((x-mean)^2) + eps);
           rms: y = x * rstd * w with rstd = 1/sqrt(mean(x^2) + eps).  Backward, with xh = (x-mean)*rstd and
           a = g*w:  dx = rstd*(a - mean(a) - xh*mean(a*xh)) (rms: without mean(a)),
           dw = sum over rows of g*xh, db = sum over rows of g, both fp32.
* router   the K experts with the largest logit (+ bias), in descending order, ties to the lower id; an expert
           whose selection score is -inf is not selectable (id -1, probability 0).  softmax: p = exp(l) over the
           sum of the selected (renormalised) or of all experts; sigmoid: s = 1/(1+exp(-l)), renormalised over the
           selected or not; all times a factor.  Backward: d probs -> d logits (the ids are constants).
* experts  out[row] = W[g(row)] . x for the rows of a dispatch layout (expert-major, stable in token order), W
           stored as E2M1 codes with an E4M3 scale per 16 elements and an fp32 scale per output row;
           swiglu: W holds F gate rows then F up rows and out = silu(gate) * up.
"""
import math

import torch

own = False
BLOCK = 16                        # elements that share an E4M3 scale
EPS = 1e-5
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MOST_BYTES = 1.8e9                # what the largest case reads and writes
MOST_WEIGHTS = 4.3e9              # bytes of expert weights that a case holds
FOREIGN = 3072                    # a width that no configuration of this repository has: not drawn


def listed():
    return [
        # one token of a decode step through the norm (with bias): latency alone
        dict(name="norm_one_token", op="norm", T=1, H=2048, dtype="bf16", rms=False),
        # a prefill or training microbatch through an RMS norm, the wide hidden size of this repository
        dict(name="norm_rms_4096", op="norm", T=4096, H=7168, dtype="bf16", rms=True),
        # rows whose width no vector divides, in fp32 (a small model, a head of odd size), with gradients
        dict(name="norm_bwd_odd_f32", op="norm_bwd", T=1021, H=1111, dtype="f32", rms=False),
        # the training step's backward pass at the large microbatch
        dict(name="norm_bwd_large", op="norm_bwd", T=32768, H=7168, dtype="bf16", rms=False),
        # the router of a decode batch: 16 tokens, bf16 logits full of ties, experts masked out
        dict(name="router_decode", op="router", T=16, E=128, K=8, dtype="bf16", score="softmax", renorm=True,
             bias=False, masked=True),
        # the router of the large microbatch: sigmoid scores, a selection bias, 256 experts
        dict(name="router_large", op="router", T=32768, E=256, K=8, dtype="f32", score="sigmoid", renorm=True,
             bias=True, masked=False),
        # its gradient when probabilities come from a softmax over all experts: dense rows
        dict(name="router_bwd_dense", op="router_bwd", T=8192, E=128, K=8, dtype="bf16", score="softmax",
             renorm=False, bias=False, masked=True),
        # one token of a decode step through its eight experts' gate and up products
        dict(name="experts_one_token", op="experts", T=1, H=2048, N=1536, E=128, K=8, S=0, swiglu=True),
        # the down products of a decode batch: every expert has a few rows
        dict(name="experts_down_32", op="experts", T=32, H=768, N=2048, E=128, K=8, S=0, swiglu=False),
        # a decode batch through wide experts and a shared expert (gate and up products)
        dict(name="experts_wide_16", op="experts", T=16, H=7168, N=4096, E=256, K=8, S=1, swiglu=True),
        # few large experts, many rows each: the down products of 64 tokens
        dict(name="experts_few_64", op="experts", T=64, H=14336, N=4096, E=8, K=2, S=0, swiglu=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm_bwd", "router", "router_bwd", "experts", "experts"])
        if op in ("norm", "norm_bwd"):
            H = _log(rng, 64, 8192)
            if rng.random() < 0.7:                       # most widths are multiples of 64, some are odd
                H = max(64, H // 64 * 64)
            case = dict(op=op, T=_log(rng, 1, 32768), H=H, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                        rms=rng.random() < 0.5)
        elif op in ("router", "router_bwd"):
            E = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, 384, 512])
            case = dict(op=op, T=_log(rng, 1, 32768), E=E, K=rng.randint(2, min(E, 10)),
                        dtype=rng.choice(["bf16", "f16", "f32", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                        renorm=rng.random() < 0.6, bias=rng.random() < 0.5, masked=rng.random() < 0.5)
        else:
            E = rng.choice([8, 16, 32, 64, 128, 256])
            step = rng.choice([16, 64, 128, 128])        # most widths are multiples of 64 or 128
            H, N = (step * _log(rng, 256 // step, 14336 // step) for _ in range(2))
            swiglu = rng.random() < 0.5
            if not swiglu and rng.random() < 0.2:
                N -= rng.randint(1, 15)
            case = dict(op=op, T=_log(rng, 1, 128), H=H, N=N, E=E, K=rng.randint(1, min(E, 8)), S=rng.randint(0, 1),
                        swiglu=swiglu)
            if (E + case["S"]) * N * H * 9 / 16 > MOST_WEIGHTS or case["T"] * case["K"] > 32 * E:
                continue
        if work(case)["bytes"] <= MOST_BYTES and FOREIGN not in case.values():
            return case


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    """Normal values of the given type, drawn in pieces so that the fp32 draw stays small."""
    out = torch.empty(*shape, dtype=dtype, device=g.device)
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - s)
        flat[s:s + n] = torch.randn(n, generator=g, device=g.device).mul_(scale).to(dtype)
    return out


def _make_norm(case, g):
    T, H, dt = case["T"], case["H"], DTYPE[case["dtype"]]
    x = _normal(g, T, H, dtype=dt)
    if T > 8:
        x[:: max(1, T // 64)] *= 20                      # outlier rows
    w = (1.0 + 0.1 * torch.randn(H, generator=g, device=g.device)).to(dt)
    s = dict(x=x, w=w, b=None if case["rms"] else _normal(g, H, dtype=dt, scale=0.1))
    if case["op"] == "norm_bwd":
        s["g"] = _normal(g, T, H, dtype=dt)
    return s


def _row_pieces(T, H):
    n = max(1, (1 << 26) // H)
    return [(t, min(T, t + n)) for t in range(0, T, n)]


def _make_router(case, g):
    T, E = case["T"], case["E"]
    l = _normal(g, T, E, dtype=DTYPE[case["dtype"]])
    if case["masked"]:                                   # experts that are switched off for a token; a token with none
        l[torch.rand(T, E, generator=g, device=g.device) < 0.1] = float("-inf")
        if T > 8:
            l[T // 2 :: 97] = float("-inf")
    s = dict(l=l, bias=_normal(g, E, scale=0.5) if case["bias"] else None)
    if case["op"] == "router_bwd":
        s["g"] = _normal(g, T, case["K"])
    return s


def _make_experts(case, g):
    T, H, N, E, K, S = (case[k] for k in ("T", "H", "N", "E", "K", "S"))
    G = E + S
    dev = g.device
    bias = 0.5 * torch.randn(E, generator=g, device=dev)
    ids = torch.argsort(torch.randn(T, E, generator=g, device=dev) + bias, dim=1, descending=True, stable=True)
    ids = ids[:, :K].to(torch.int32).contiguous()
    codes = torch.randint(0, 256, (G, N, H // 2), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.randint(0x58, 0x7F, (G, N, H // BLOCK), generator=g, device=dev, dtype=torch.uint8)
    row_scale = (0.5 + torch.rand(G, N, generator=g, device=dev)) / (448 * math.sqrt(H))
    # the rows of the layout: (token, slot) pairs in expert order, stable in token order, then the shared rows
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E).tolist() + [T] * S
    tokens = torch.cat([order // K, torch.arange(T * S, device=dev)])
    return dict(ids=ids, codes=codes, scales=scales, row_scale=row_scale, tokens=tokens, counts=counts, G=G,
                x=_normal(g, T if case["swiglu"] else T * K + S * T, H, dtype=torch.bfloat16))


def _inputs(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(int(seed))
    if case["op"].startswith("norm"):
        return _make_norm(case, g)
    if case["op"].startswith("router"):
        return _make_router(case, g)
    return _make_experts(case, g)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    T = case["T"]
    if case["op"] == "norm_bwd":                         # what the forward pass saved
        s["mean"], s["rstd"] = _plain_stats(s["x"], case["rms"])
    if case["op"] == "router_bwd":
        s["ids"] = _plain_select(s["l"], s["bias"], case["K"])
    if case["op"] == "experts":                          # tables of the 4-bit and 8-bit formats
        s["pair"], s["e4m3"] = _tables(s["x"].device)
    if own:
        import combine_topk_ids_histogram_gb300 as ep
        f32 = dict(dtype=torch.float32, device=s["w" if "w" in s else "l" if "l" in s else "x"].device)
        s["ep"] = ep
        if case["op"] == "norm":
            s["out"] = (torch.empty_like(s["x"]), None if case["rms"] else torch.empty(T, **f32), torch.empty(T, **f32))
        elif case["op"] == "norm_bwd":
            H = case["H"]
            s["out"] = (torch.empty_like(s["x"]), torch.empty(H, **f32), None if case["rms"] else torch.empty(H, **f32))
            s["ws"] = torch.empty(ep.layer_norm_bwd_workspace_bytes(T, H), dtype=torch.uint8, device=f32["device"])
        elif case["op"] == "router":
            s["out"] = (torch.empty(T, case["K"], dtype=torch.int32, device=f32["device"]),
                        torch.empty(T, case["K"], **f32))
        elif case["op"] == "router_bwd":
            s["out"] = torch.empty_like(s["l"])
        else:
            s["L"] = ep.dispatch_layout(s["ids"], case["E"], fused_shared=bool(case["S"]))
            s["out"] = torch.empty(T * case["K"] + T * case["S"], case["N"] // 2 if case["swiglu"] else case["N"],
                                   dtype=torch.bfloat16, device=f32["device"])
    return s


def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(state, case, case["op"])


def _run_own(s, case, op):
    ep = s["ep"]
    if op == "norm":
        y, mean, rstd = ep.layer_norm(s["x"], s["w"], s["b"], eps=EPS, rms=case["rms"], out=s["out"])
        return (y, rstd) if mean is None else (y, rstd, mean)
    if op == "norm_bwd":
        dx, dw, db = ep.layer_norm_bwd(s["g"], s["x"], s["w"], s["mean"], s["rstd"], rms=case["rms"],
                                       bias=not case["rms"], out=s["out"], workspace=s["ws"])
        return (dx, dw) if db is None else (dx, dw, db)
    if op == "router":
        return ep.router_topk(s["l"], case["K"], bias=s["bias"], score=case["score"], renormalize=case["renorm"],
                              scale=1.5, out=s["out"])
    if op == "router_bwd":
        return ep.router_topk_bwd(s["g"], s["l"], s["ids"], score=case["score"], renormalize=case["renorm"], scale=1.5,
                                  out=s["out"])
    return ep.expert_matvec(s["x"], s["codes"], s["scales"], s["row_scale"], s["L"], by_token=case["swiglu"],
                            swiglu=case["swiglu"], out=s["out"])


def _run_plain(s, case, op):
    if op == "norm":
        y = torch.empty_like(s["x"])
        means, rstds = [], []
        for a, b in _row_pieces(*s["x"].shape):
            x = s["x"][a:b].float()
            mean = None if case["rms"] else x.mean(1)
            d = x if case["rms"] else x - mean[:, None]
            rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
            v = d * rstd[:, None] * s["w"].float()
            y[a:b] = v if case["rms"] else v + s["b"].float()
            rstds.append(rstd)
            means.append(mean)
        return (y, torch.cat(rstds)) if case["rms"] else (y, torch.cat(rstds), torch.cat(means))
    if op == "norm_bwd":
        dx = torch.empty_like(s["x"])
        dw = torch.zeros(case["H"], dtype=torch.float32, device=dx.device)
        db = torch.zeros_like(dw)
        w = s["w"].float()
        for a, b in _row_pieces(*s["x"].shape):
            x, g, rstd = s["x"][a:b].float(), s["g"][a:b].float(), s["rstd"][a:b, None]
            xh = x * rstd if case["rms"] else (x - s["mean"][a:b, None]) * rstd
            v = g * w
            d = v - xh * (v * xh).mean(1, keepdim=True)
            if not case["rms"]:
                d = d - v.mean(1, keepdim=True)
                db += g.sum(0)
            dx[a:b] = d * rstd
            dw += (g * xh).sum(0)
        return (dx, dw) if case["rms"] else (dx, dw, db)
    if op == "router":
        ids = _plain_select(s["l"], s["bias"], case["K"])
        return ids, _plain_probs(s["l"].float(), ids, case)
    if op == "router_bwd":
        return _plain_router_grad(s["g"], s["l"].float(), s["ids"], case).to(s["l"].dtype)
    return _plain_experts(s, case)


def _plain_stats(x, rms):
    means, rstds = [], []
    for a, b in _row_pieces(*x.shape):
        v = x[a:b].float()
        if not rms:
            means.append(v.mean(1))
            v = v - means[-1][:, None]
        rstds.append(1.0 / torch.sqrt((v * v).mean(1) + EPS))
    return None if rms else torch.cat(means), torch.cat(rstds)


def _plain_select(l, bias, K):
    sel = l.float() if bias is None else l.float() + bias
    v, ids = torch.sort(sel, dim=1, descending=True, stable=True)
    return torch.where(v[:, :K] == float("-inf"), -1, ids[:, :K]).to(torch.int32).contiguous()


def _plain_probs(l, ids, case):
    used = ids >= 0
    sel = torch.where(used, l.gather(1, ids.clamp(min=0).long()), float("-inf"))
    if case["score"] == "softmax":
        top = (sel if case["renorm"] else l).max(1, keepdim=True).values
        top = torch.where(top == float("-inf"), 0.0, top)
        e = torch.exp(sel - top)
        total = (e if case["renorm"] else torch.exp(l - top)).sum(1, keepdim=True)
        p = e / total
    else:
        p = 1.0 / (1.0 + torch.exp(-sel))
        if case["renorm"]:
            p = p / p.sum(1, keepdim=True)
    return torch.where(used, 1.5 * p, 0.0)


def _plain_router_grad(g, l, ids, case):
    used = ids >= 0
    at = ids.clamp(min=0).long()
    p = _plain_probs(l, ids, case)
    g = torch.where(used, g, 0.0)
    inner = (g * p).sum(1, keepdim=True)
    dl = torch.zeros_like(l)
    if case["score"] == "softmax" and not case["renorm"]:
        top = l.max(1, keepdim=True).values
        e = torch.exp(l - torch.where(top == float("-inf"), 0.0, top))
        total = e.sum(1, keepdim=True)
        dl = torch.where(total > 0, -e / total * inner, 0.0)
        return dl.scatter_add(1, at, g * p)
    if case["renorm"]:
        d = p * (g - inner / 1.5)
        if case["score"] == "sigmoid":
            d = d / (1.0 + torch.exp(l.gather(1, at)))
    else:
        d = g * p * (1.0 - p / 1.5)
    return dl.scatter_add(1, at, torch.where(used, d, 0.0))


def _tables(dev):
    """E2M1 values of both codes of a byte, and E4M3 values."""
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=dev)
    e2m1 = torch.cat([mag, -mag])
    byte = torch.arange(256, device=dev)
    pair = torch.stack([e2m1[byte & 15], e2m1[byte >> 4]], 1)
    e, m = (byte & 127) >> 3, (byte & 7).float()
    v = torch.where(e == 0, m / 512.0, torch.ldexp(1.0 + m / 8.0, e - 7))
    return pair, torch.where(byte < 128, v, -v)


def _plain_experts(s, case):
    H, N = case["H"], case["N"]
    parts, at = [], 0
    for g, n in enumerate(s["counts"]):
        if not n:
            continue
        x = (s["x"][s["tokens"][at:at + n]] if case["swiglu"] else s["x"][at:at + n]).float()
        w = s["pair"][s["codes"][g].long()].view(N, H // BLOCK, BLOCK) * s["e4m3"][s["scales"][g].long()][..., None]
        y = (x @ w.view(N, H).t()) * s["row_scale"][g]
        if case["swiglu"]:
            gate, up = y[:, :N // 2], y[:, N // 2:]
            y = gate / (1.0 + torch.exp(-gate)) * up
        parts.append(y.to(torch.bfloat16))
        at += n
    return torch.cat(parts)


def work(case):
    T, op = case["T"], case["op"]
    if op.startswith("norm"):
        H, n = case["H"], SIZE[case["dtype"]]
        params = 1 if case["rms"] else 2
        if op == "norm":
            return dict(bytes=2 * T * H * n + params * (H * n + 4 * T), flops=8 * T * H)
        return dict(bytes=3 * T * H * n + H * n + params * 4 * (T + H), flops=14 * T * H)
    if op.startswith("router"):
        E, K, n = case["E"], case["K"], SIZE[case["dtype"]]
        if op == "router":
            return dict(bytes=T * E * n + 8 * T * K + (4 * E if case["bias"] else 0), flops=4 * T * E)
        dense = case["score"] == "softmax" and not case["renorm"]
        return dict(bytes=T * E * n * (2 if dense else 1) + T * K * (8 + (0 if dense else n)), flops=4 * T * E)
    H, N, E, K, S = (case[k] for k in ("H", "N", "E", "K", "S"))
    used = E * (1 - (1 - K / E) ** T) + S                # experts that some token names (expected, as if unbiased)
    rows = T * K + S * T
    return dict(bytes=int(used * N * (H * 9 / 16 + 4)) + 2 * (T if case["swiglu"] else rows) * H
                + 2 * rows * (N // 2 if case["swiglu"] else N), flops=2 * rows * N * H)


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "norm":
        parts = [_exact_norm(s["x"][a:b].double(), s["w"].double(), s["b"]) for a, b in _row_pieces(case["T"], 4 * case["H"])]
        out = [torch.cat(v) for v in zip(*parts)]
        return tuple(out[:2]) if case["rms"] else tuple(out)
    if op == "norm_bwd":
        mean, rstd = _plain_stats(s["x"], case["rms"])   # fp32 inputs of the backward pass
        dxs, dw, db = [], 0, 0
        for a, b in _row_pieces(case["T"], 4 * case["H"]):
            r, g = rstd[a:b].double().unsqueeze(1), s["g"][a:b].double()
            xh = (s["x"][a:b].double() - (0 if mean is None else mean[a:b].double().unsqueeze(1))) * r
            v = g * s["w"].double()
            dot = torch.einsum("th,th->t", v, xh).unsqueeze(1) / case["H"]
            shift = 0 if case["rms"] else v.sum(1, keepdim=True) / case["H"]
            dxs.append(r * (v - shift - xh * dot))
            dw, db = dw + torch.einsum("th,th->h", g, xh), db + g.sum(0)
        return (torch.cat(dxs), dw) if case["rms"] else (torch.cat(dxs), dw, db)
    if op == "router":
        ids = _exact_select(s, case["K"])
        return None, _exact_probs(s["l"].double(), ids, case)
    if op == "router_bwd":
        ids, l = _exact_select(s, case["K"]), s["l"].double()
        out = torch.empty_like(l)
        for a, b in _row_pieces(case["T"], case["E"] * case["E"]):
            # the Jacobian d probs[k] / d logits[e], written out entry by entry
            p = _exact_probs(l[a:b], ids[a:b], case) / 1.5
            hit = torch.nn.functional.one_hot(ids[a:b].long() + 1, case["E"] + 1)[..., 1:].double()    # [t, K, E]
            if case["score"] == "softmax":
                share = torch.einsum("tk,tke->te", p, hit) if case["renorm"] else _exact_softmax(l[a:b])
                jac = p.unsqueeze(2) * (hit - share.unsqueeze(1))
            else:
                slope = 1 - torch.sigmoid(l[a:b])
                share = torch.einsum("tk,tke->te", p, hit).unsqueeze(1) if case["renorm"] else 0
                jac = p.unsqueeze(2) * (hit - share) * slope.unsqueeze(1)
            out[a:b] = 1.5 * torch.einsum("tk,tke->te", s["g"][a:b].double(), jac)
        return out
    T, H, N = case["T"], case["H"], case["N"]
    rows, at = [], 0
    for g, n in enumerate(s["counts"]):
        if n:
            x = s["x"][s["tokens"][at:at + n]] if case["swiglu"] else s["x"][at:at + n]
            rows.append(_exact_expert(x.double(), s["codes"][g], s["scales"][g], s["row_scale"][g].double(), case["swiglu"]))
            at += n
    return torch.cat(rows)


def _exact_norm(x, w, b):
    H = x.shape[1]
    mean = x.sum(1) / H if b is not None else torch.zeros_like(x[:, 0])
    var = ((x - mean.unsqueeze(1)) ** 2).sum(1) / H
    rstd = (var + EPS) ** -0.5
    y = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1) * w
    return (y if b is None else y + b.double()), rstd, mean


def _exact_select(s, K):
    """The selection is by the fp32 sum of logit and bias: whole numbers follow from it."""
    score = s["l"].float()
    if s["bias"] is not None:
        score = score + s["bias"]
    score = score.clone()
    ids = []
    for _ in range(K):                                   # the first of the largest, K times
        top = score.max(1, keepdim=True).values
        first = torch.where(score == top, torch.arange(score.shape[1], device=score.device), score.shape[1]).min(1).values
        ids.append(torch.where(top[:, 0] == float("-inf"), -1, first))
        score.scatter_(1, first.unsqueeze(1), float("-inf"))
    return torch.stack(ids, 1).to(torch.int32)


def _exact_softmax(l):
    return torch.nan_to_num(torch.exp(l - torch.logsumexp(l, 1, keepdim=True)), nan=0.0)


def _exact_probs(l, ids, case):
    some = ids >= 0
    v = l.gather(1, ids.clamp(min=0).long())
    if case["score"] == "softmax":
        if not case["renorm"]:
            p = _exact_softmax(l).gather(1, ids.clamp(min=0).long())
        else:
            p = _exact_softmax(v.masked_fill(~some, float("-inf")))
    else:
        p = torch.sigmoid(v)
        if case["renorm"]:
            p = p / (p * some).sum(1, keepdim=True)
    return torch.where(some, 1.5 * p, 0.0)


def _exact_expert(x, codes, scales, row_scale, swiglu):
    c = torch.stack([codes & 15, codes >> 4], 2).flatten(1)                  # element 2j is the low nibble of byte j
    e, m = (c >> 1) & 3, (c & 1).double()
    w = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e.double() - 1))
    w = torch.where(c >= 8, -w, w)
    e, m = (scales >> 3) & 15, (scales & 7).double()
    scale = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.double() - 7))
    scale = torch.where(scales >= 128, -scale, scale)
    w = w * scale.repeat_interleave(BLOCK, 1) * row_scale.unsqueeze(1)
    y = x @ w.t()
    if swiglu:
        gate, up = y.chunk(2, dim=1)
        y = gate * torch.sigmoid(gate) * up
    return y
