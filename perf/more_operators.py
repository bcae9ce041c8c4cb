"""Measured cases of the experts' 16-bit products on the rows of a dispatch layout (gated and plain, forward and
backward) and of low-rank adapters on tokens grouped by the same layout.

``own = False`` computes each operator in elementary torch operations in fp32, rounded once at the end; ``own = True``
makes the library's calls.  Both take what ``prepare`` returns.

Definitions (x, w, gradients and adapters bf16 or fp16; sums in fp32 or wider; row r belongs to group g):

* linear   y[r] = w[g] x[r], w [G, N, K].
* glu      w holds N/2 gate rows, then N/2 up rows; out = gate / (1 + exp(-gate)) * up; "save" returns (gate, up) too.
* bwd      of linear: dx[r] = w[g]^T dy[r]; dw[g] = sum over the rows of g of dy[r] x[r]^T.  "gated": x was the out of glu,
           and instead of dx the gradient of (gate, up) is returned: with da = w[g]^T dy[r] and s = 1/(1 + exp(-gate)),
           d gate = da * up * s * (1 + gate * (1 - s)), d up = da * gate * s.
* lora     out[t] = y[t] + scale[g] * B[g] (A[g] x[t]) for the adapter g of token t; out[t] = y[t] without one.
"""
import math

import torch

own = False
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MOST_FLOPS = 3.9e12               # of the largest case
MOST_WEIGHTS = 2.0e9              # elements of the largest case's weights
MOST_ELEMENTS = 5e8               # elements of the rows' matrices, together


def listed():
    return [
        # one token of a decode step through the gate and up products of its eight experts: latency, then weights
        dict(name="glu_one_token", op="glu", T=1, E=128, top=8, S=0, K=2048, N=1536, dtype="bf16", save=False),
        # a chunk of a prompt over wide experts and a shared one, few rows each: the weights have to be read
        dict(name="glu_wide_256", op="glu", T=256, E=64, top=8, S=1, K=7168, N=4096, dtype="bf16", save=False),
        # a training microbatch, many narrow experts: gate and up are kept for the backward pass
        dict(name="glu_train_8192", op="glu", T=8192, E=128, top=8, S=0, K=2048, N=1536, dtype="bf16", save=True),
        # a long prompt over a few large experts: the largest product
        dict(name="glu_large_8192", op="glu", T=8192, E=8, top=2, S=0, K=4096, N=28672, dtype="bf16", save=False),
        # the down products of the training microbatch: short sums, much output
        dict(name="linear_down_8192", op="linear", T=8192, E=128, top=8, S=0, K=768, N=2048, dtype="bf16"),
        # sizes that no tile divides, in fp16
        dict(name="linear_odd_f16", op="linear", T=1021, E=12, top=3, S=1, K=1136, N=1360, dtype="f16"),
        # the training step's way back through the down products and the activation
        dict(name="bwd_gated_8192", op="bwd", T=8192, E=128, top=8, S=0, K=768, N=2048, dtype="bf16", gated=True, dw="bf16"),
        # and through large gate and up products, weight gradients in fp32
        dict(name="bwd_large_4096", op="bwd", T=4096, E=8, top=2, S=0, K=4096, N=28672, dtype="bf16", gated=False, dw="f32"),
        # sizes that no tile divides, few rows in each expert
        dict(name="bwd_odd_f16", op="bwd", T=333, E=24, top=4, S=0, K=1136, N=720, dtype="f16", gated=True, dw="f32"),
        # one token of a decode step with its adapter
        dict(name="lora_one_token", op="lora", T=1, G=32, r=16, K=2048, N=2048, dtype="bf16", none=0.0),
        # a decode batch of many requests, most with an adapter of their own
        dict(name="lora_decode_64", op="lora", T=64, G=48, r=32, K=7168, N=4096, dtype="bf16", none=0.1),
        # prompts of a few requests
        dict(name="lora_prompt_8192", op="lora", T=8192, G=5, r=64, K=4096, N=4096, dtype="f16", none=0.2),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        op = rng.choice(["glu", "linear", "bwd", "bwd", "lora"])
        step = rng.choice([16, 64, 128, 128])            # most widths are multiples of 64 or 128
        K, N = (step * _log(rng, max(1, 128 // step), 14336 // step) for _ in range(2))
        dtype = rng.choice(["bf16", "bf16", "f16"])
        if op == "lora":
            case = dict(op=op, T=_log(rng, 1, 16384), G=_log(rng, 1, 128), r=rng.choice([8, 16, 16, 32, 64, 128]), K=K, N=N,
                        dtype=dtype, none=rng.choice([0.0, 0.1, 0.5]))
            if case["T"] * (K + 2 * N) > MOST_ELEMENTS:
                continue
            return case
        E = rng.choice([4, 8, 8, 16, 32, 60, 64, 128, 256])
        case = dict(op=op, T=_log(rng, 1, 16384), E=E, top=rng.randint(1, min(E, 8)), S=rng.randint(0, 1), K=K, N=N, dtype=dtype)
        if op == "glu":
            case["N"] = 2 * N
            case["save"] = rng.random() < 0.5
        if op == "bwd":
            case.update(gated=rng.random() < 0.5, dw=rng.choice([dtype, "f32"]))
        rows = case["T"] * (case["top"] + case["S"])
        if (work(case)["flops"] <= MOST_FLOPS and (E + case["S"]) * case["N"] * K <= MOST_WEIGHTS
                and rows * (3 * K + 2 * case["N"]) <= MOST_ELEMENTS):
            return case


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, *shape, dtype, scale=1.0):
    """Normal values of the given type, drawn in pieces so that the fp32 draw stays small."""
    out = torch.empty(*shape, dtype=dtype, device=g.device)
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - s)
        flat[s:s + n] = torch.randn(n, generator=g, device=g.device).mul_(scale).to(dtype)
    return out


def _inputs(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(int(seed))
    dev, T, K, N, dt = g.device, case["T"], case["K"], case["N"], DTYPE[case["dtype"]]
    if case["op"] == "lora":
        G, r = case["G"], case["r"]
        ids = torch.randint(0, G, (T, 1), generator=g, device=dev, dtype=torch.int32)
        ids[torch.rand(T, 1, generator=g, device=dev) < case["none"]] = -1
        return dict(ids=ids, y=_normal(g, T, N, dtype=dt), x=_normal(g, T, K, dtype=dt),
                    a=_normal(g, G, r, K, dtype=dt, scale=K ** -0.5), b=_normal(g, G, N, r, dtype=dt, scale=r ** -0.5),
                    scale=0.5 + torch.rand(G, generator=g, device=dev))
    E, top, S = case["E"], case["top"], case["S"]
    # uneven routing: some experts get several times the rows of others
    bias = 0.5 * torch.randn(E, generator=g, device=dev)
    ids = torch.argsort(torch.randn(T, E, generator=g, device=dev) + bias, dim=1, descending=True, stable=True)
    ids = ids[:, :top].to(torch.int32).contiguous()
    counts = torch.bincount(ids.flatten().long(), minlength=E).tolist() + [T] * S
    R, G = T * (top + S), E + S
    s = dict(ids=ids, counts=counts, x=_normal(g, R, K, dtype=dt), w=_normal(g, G, N, K, dtype=dt, scale=K ** -0.5))
    if case["op"] == "bwd":
        s["g"] = _normal(g, R, N, dtype=dt)
        if case["gated"]:                                # what the forward pass kept, and the x it made
            s["gu"] = _normal(g, R, 2 * K, dtype=dt)
            for a in range(0, R, 1 << 14):
                gate, up = s["gu"][a:a + (1 << 14)].float().chunk(2, 1)
                s["x"][a:a + (1 << 14)] = gate / (1 + torch.exp(-gate)) * up
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "lora":
        s["at"] = [torch.nonzero(s["ids"][:, 0] == g)[:, 0] for g in range(case["G"])]
    if own:
        import combine_topk_ids_histogram_gb300 as ep
        s["ep"] = ep
        x, N, K = s["x"], case["N"], case["K"]
        new = lambda *shape, dtype=x.dtype: torch.empty(*shape, dtype=dtype, device=x.device)
        if case["op"] == "lora":
            s["L"] = ep.dispatch_layout(s["ids"], case["G"])
            s["out"] = torch.empty_like(s["y"])
            return s
        s["L"] = ep.dispatch_layout(s["ids"], case["E"], fused_shared=bool(case["S"]))
        R = x.shape[0]
        if case["op"] == "bwd":
            s["out"] = new(R, 2 * K if case["gated"] else K), new(*s["w"].shape, dtype=DTYPE[case["dw"]])
        elif case["op"] == "glu":
            s["out"] = (new(R, N // 2), new(R, N)) if case["save"] else new(R, N // 2)
        else:
            s["out"] = new(R, N)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, case):
    ep, op = s["ep"], case["op"]
    if op == "lora":
        return ep.lora_add(s["y"], s["x"], s["a"], s["b"], s["L"], scale=s["scale"], out=s["out"])
    if op == "bwd":
        return ep.expert_linear_bwd(s["g"], s["x"], s["w"], s["L"], gate_up=s.get("gu"), out=s["out"])
    return ep.expert_linear(s["x"], s["w"], s["L"], swiglu=op == "glu", save=case.get("save", False), out=s["out"])


def _run_plain(s, case):
    op, x = case["op"], s["x"]
    if op == "lora":
        out = s["y"].clone()
        for g, t in enumerate(s["at"]):
            if t.numel():
                d = (x[t].float() @ s["a"][g].float().t()) @ s["b"][g].float().t()
                out[t] = (s["y"][t].float() + s["scale"][g] * d).to(out.dtype)
        return out
    outs = []
    dw = torch.zeros(s["w"].shape, dtype=DTYPE[case["dw"]], device=x.device) if op == "bwd" else None
    at = 0
    for g, n in enumerate(s["counts"]):
        if not n:
            continue
        xg, w = x[at:at + n].float(), s["w"][g].float()
        if op == "bwd":
            d = s["g"][at:at + n].float()
            dw[g] = d.t() @ xg
            d = d @ w
            if case["gated"]:
                gate, up = s["gu"][at:at + n].float().chunk(2, 1)
                sig = 1 / (1 + torch.exp(-gate))
                d = torch.cat([d * up * sig * (1 + gate * (1 - sig)), d * gate * sig], 1)
            outs.append((d.to(x.dtype),))
        else:
            y = xg @ w.t()
            if op == "glu":
                gate, up = y.chunk(2, 1)
                h = (gate / (1 + torch.exp(-gate)) * up).to(x.dtype)
                outs.append((h, y.to(x.dtype)) if case["save"] else (h,))
            else:
                outs.append((y.to(x.dtype),))
        at += n
    out = tuple(torch.cat(v) for v in zip(*outs))
    if op == "bwd":
        return out[0], dw
    return out if len(out) > 1 else out[0]


def work(case):
    op, T, K, N = case["op"], case["T"], case["K"], case["N"]
    if op == "lora":
        G, r = case["G"], case["r"]
        rows = T * (1 - case["none"])
        used = G * (1 - (1 - 1 / G) ** rows)             # adapters that some token names (expected)
        return dict(bytes=int(2 * (rows * K + 2 * T * N + used * r * (K + N))), flops=int(2 * rows * r * (K + N)))
    E, top, S = case["E"], case["top"], case["S"]
    rows = T * (top + S)
    used = E * (1 - (1 - top / E) ** T) + S              # experts that some token names (expected, as if unbiased)
    size = 2 * rows * (K + N) + int(2 * used * N * K)    # the rows' matrices and the weights
    if op == "linear":
        return dict(bytes=size, flops=2 * rows * N * K)
    if op == "glu":
        return dict(bytes=size - (0 if case["save"] else 2 * rows * N) + rows * N, flops=2 * rows * N * K)
    return dict(bytes=size + (8 if case["gated"] else 2) * rows * K + (4 if case["dw"] == "f32" else 2) * (E + S) * N * K,
                flops=4 * rows * N * K)


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    op, x = case["op"], s["x"]
    if op == "lora":
        out = s["y"].double()
        for g in torch.unique(s["ids"]).tolist():
            if g >= 0:
                on = s["ids"][:, 0] == g
                low = torch.einsum("tk,rk->tr", x[on].double(), s["a"][g].double())
                out[on] += s["scale"][g].double() * torch.einsum("tr,nr->tn", low, s["b"][g].double())
        return out
    ends = torch.tensor(s["counts"]).cumsum(0).tolist()
    parts = [slice(b - n, b) for b, n in zip(ends, s["counts"])]
    R, K, N = x.shape[0], case["K"], case["N"]
    f64 = dict(dtype=torch.float64, device=x.device)
    if op == "bwd":
        dx, dw = torch.empty(R, 2 * K if case["gated"] else K, **f64), torch.empty(len(parts), N, K, **f64)
        for g, p in enumerate(parts):
            d = s["g"][p].double()
            torch.matmul(d.t(), x[p].double(), out=dw[g])
            d = torch.einsum("rn,nk->rk", d, s["w"][g].double())
            if case["gated"]:
                gate, up = s["gu"][p, :K].double(), s["gu"][p, K:].double()
                sig = torch.sigmoid(gate)
                dx[p, :K] = d * up * (sig + gate * sig * torch.sigmoid(-gate))
                dx[p, K:] = d * (gate * sig)
            else:
                dx[p] = d
        return dx, dw
    y = torch.empty(R, N, **f64)
    for g, p in enumerate(parts):
        y[p] = torch.einsum("rk,nk->rn", x[p].double(), s["w"][g].double())
    if op == "linear":
        return y
    h = y[:, :N // 2] * torch.sigmoid(y[:, :N // 2]) * y[:, N // 2:]
    return (h, y) if case["save"] else h
