"""Cases that measure two groups of operators of the sparse layer, and their plain forms.

* Tokens sorted by expert and back: every assignment (token t, choice j) gets a
  row of a packed matrix ordered by expert, then t, then j; the expert outputs
  come back to token order as y[t] = base[t] + sum_j gate[t, j] * ys[row[t, j]];
  and the gradients of both.
* The product of 8-bit integers with one scale per token and one per output
  channel, y = (xq . wq) * xscale * wscale, dense and for the experts of the
  sorted rows, with the quantisation of the tokens that it starts from.

A case is a dict of plain values.  ``prepare`` makes what a program holds before
the call, ``run`` makes one pass (in elementary torch operations, or through the
package where ``own`` is set), ``exact`` gives the results in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a decoding step of 16 sequences through the full layer (E = 256, k = 8, hidden 2048): latency
        dict(name="sort decode", op="sort", T=16, k=8, E=256, D=2048, dtype="bf16"),
        # the full layer's batch: 131072 rows of 4 KB
        dict(name="sort train", op="sort", T=16384, k=8, E=256, D=2048, dtype="bf16"),
        # fp32 top-2 training with a width and a token count that fit no vector and no block
        dict(name="sort odd", op="sort", T=8191, k=2, E=64, D=1001, dtype="f32"),
        # the way back of the decoding step
        dict(name="unsort decode", op="unsort", T=16, k=8, E=256, D=2048, dtype="bf16", gates=True, base=True, pad=0),
        # the way back of the full batch onto the shared expert's output, a few padding tokens behind it
        dict(name="unsort train", op="unsort", T=16384, k=8, E=256, D=2048, dtype="bf16", gates=True, base=True, pad=5),
        # its gradient: the rows' and the gates'
        dict(name="unsort_backward train", op="unsort_backward", T=16384, k=8, E=256, D=2048, dtype="bf16", pad=0),
        # the same for the odd fp32 layer, with padding tokens
        dict(name="unsort_backward odd", op="unsort_backward", T=8191, k=2, E=64, D=1001, dtype="f32", pad=77),
        # one token through one 8-bit weight: the weight's bytes count
        dict(name="linear_i8 token", op="linear_i8", M=1, K=2048, N=2048, dtype="bf16"),
        # a ragged prompt through a width that no tile divides
        dict(name="linear_i8 ragged", op="linear_i8", M=1003, K=1000, N=1537, dtype="f32"),
        # a batch of prompts
        dict(name="linear_i8 prompt", op="linear_i8", M=16384, K=2048, N=2048, dtype="bf16"),
        # the routed SwiGLU experts in 8 bits: a decoding step and the full layer's batch
        dict(name="experts_i8 decode", op="experts_i8", T=16, k=8, E=256, D=2048, F=512, dtype="bf16"),
        dict(name="experts_i8 prompt", op="experts_i8", T=16384, k=8, E=256, D=2048, F=512, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "unsort", "unsort_backward", "linear_i8", "experts_i8"])
    if op == "linear_i8":
        return dict(op=op, M=_log(rng, 1, 16384), K=_log(rng, 64, 2048), N=_log(rng, 64, 2048),
                    dtype=rng.choice(["bf16", "f32"]))
    E = rng.choice([8, 16, 64, 100, 256])
    case = dict(op=op, T=_log(rng, 1, 16384), k=rng.randint(1, 8), E=E, D=_log(rng, 64, 2048), dtype="bf16")
    if op == "experts_i8":
        case["F"] = _log(rng, 64, 512)
        return case
    case["dtype"] = rng.choice(["bf16", "f32"]) if case["D"] <= 1024 else "bf16"
    if op != "sort":
        case["pad"] = rng.choice([0, 0, rng.randint(0, case["T"] - 1)])
    if op == "unsort":
        case["gates"], case["base"] = rng.random() < 0.7, rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs
def _route(c, g):
    """Top-k of N(0, 1) logits with a popularity bias N(0, 0.5) per expert, and softmax gates."""
    logits = torch.randn(c["T"], c["E"], device=DEV, generator=g) + 0.5 * torch.randn(c["E"], device=DEV, generator=g)
    top, selected = torch.topk(logits, c["k"], dim=1)
    return selected, torch.softmax(top, dim=1)


def _rows_i8(w):
    """Weights in 8 bits, one scale per row; rows start on multiples of 16 bytes."""
    scale = w.abs().amax(-1) / 127
    K = w.shape[-1]
    q = torch.zeros(*w.shape[:-1], (K + 15) // 16 * 16, dtype=torch.int8, device=DEV)
    q[..., :K] = torch.round(w / scale.unsqueeze(-1)).clamp(-127, 127).to(torch.int8)
    return q[..., :K], scale


def _activations(shape, g):
    """N(0, 1) with one channel in 64 eight times as large, as hidden states have."""
    x = torch.randn(shape, device=DEV, generator=g)
    loud = torch.rand(shape[-1], device=DEV, generator=g) < 1 / 64
    return x * torch.where(loud, 8.0, 1.0)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[c["dtype"]]
    s = dict(case=c, dtype=t)
    if c["op"] == "linear_i8":
        s["x"] = _activations((c["M"], c["K"]), g).to(t)
        s["wq"], s["wscale"] = _rows_i8(torch.randn(1, c["N"], c["K"], device=DEV, generator=g) * 0.02)
        return s
    T, k, E, D = c["T"], c["k"], c["E"], c["D"]
    selected, gates = _route(c, g)
    if c["op"] in ("sort", "experts_i8"):
        s["selected"] = selected
        s["x"] = _activations((T, D), g).to(t)
        if c["op"] == "experts_i8":
            s["gates"] = gates
            s["most"] = int(torch.bincount(selected.reshape(-1), minlength=E).max())  # rows of the fullest expert
            for name, shape in (("gate", (E, c["F"], D)), ("up", (E, c["F"], D)), ("down", (E, D, c["F"]))):
                s[name], s[name + "_scale"] = _rows_i8(torch.randn(shape, device=DEV, generator=g) * 0.02)
        return s
    # the way back: rows of the sorted order; the last `pad` tokens have none
    live = T - c["pad"]
    flat = selected[:live].reshape(-1)
    order = torch.sort(flat, stable=True)[1]
    row = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    row[:live] = torch.empty_like(order).scatter_(0, order, torch.arange(live * k, device=DEV)).view(live, k).int()
    s["row"], s["source"], s["gates"] = row, order, gates
    s["ys"] = torch.randn(live * k, D, device=DEV, generator=g).to(t)
    if c["op"] == "unsort":
        s["gates"] = gates if c["gates"] else None
        s["base"] = torch.randn(T, D, device=DEV, generator=g).to(t) if c["base"] else None
    else:
        s["dy"] = torch.randn(T, D, device=DEV, generator=g).to(t)
    return s


# ---------------------------------------------------------------- one pass
def _sorted(selected, E):
    """(offsets, row, source) of the stable order by expert."""
    flat = selected.reshape(-1)
    keys, order = torch.sort(flat, stable=True)
    row = torch.empty_like(order).scatter_(0, order, torch.arange(flat.numel(), device=flat.device))
    offsets = torch.searchsorted(keys, torch.arange(E + 1, device=flat.device))
    return offsets, row, order, keys


def _quantized(x):
    """Whole numbers round(127 x / max|x|) (ties to even) and scales max|x| / 127, by row; in 64 bits next to the ties."""
    most = x.float().abs().amax(-1, keepdim=True)
    q = torch.round(127 * x.double() / most.double())
    return torch.where(most > 0, q, 0).float(), most / 127


def _run_plain(s):
    c = s["case"]
    if c["op"] == "sort":
        offsets, row, source, _ = _sorted(s["selected"], c["E"])
        return dict(offsets=offsets.int(), row=row.view(c["T"], c["k"]).int(), source=source.int(),
                    xs=s["x"][source // c["k"]])
    if c["op"] == "unsort":
        row = s["row"].long()
        terms = torch.where((row >= 0).unsqueeze(-1), s["ys"][row.clamp(min=0)].float(), 0.0)
        if s["gates"] is not None:
            terms = terms * s["gates"].unsqueeze(-1)
        y = terms.sum(1)
        return (y if s["base"] is None else y + s["base"].float()).to(s["dtype"])
    if c["op"] == "unsort_backward":
        row, dy = s["row"].long(), s["dy"].float()
        dgates = (dy.unsqueeze(1) * s["ys"][row.clamp(min=0)].float()).sum(-1)
        dys = s["gates"].reshape(-1)[s["source"]].unsqueeze(-1) * dy[s["source"] // c["k"]]
        return dict(dys=dys.to(s["dtype"]), dgates=torch.where(row >= 0, dgates, 0.0))
    if c["op"] == "linear_i8":
        q, scale = _quantized(s["x"])
        return ((q @ s["wq"][0].float().T) * scale * s["wscale"]).to(s["dtype"])
    # experts_i8: the sorted rows padded to the fullest expert, one batched product per weight
    T, k, E = c["T"], c["k"], c["E"]
    offsets, row, source, keys = _sorted(s["selected"], E)
    place = keys * s["most"] + torch.arange(T * k, device=DEV) - offsets[keys]
    q, scale = _quantized(s["x"])
    xq = torch.zeros(E * s["most"], c["D"], device=DEV)
    xq[place] = q[source // k]
    xs = torch.zeros(E * s["most"], 1, device=DEV)
    xs[place] = scale[source // k]
    xq, xs = xq.view(E, s["most"], -1), xs.view(E, s["most"], 1)
    a = torch.bmm(xq, s["gate"].float().transpose(1, 2)) * xs * s["gate_scale"].unsqueeze(1)
    b = torch.bmm(xq, s["up"].float().transpose(1, 2)) * xs * s["up_scale"].unsqueeze(1)
    hq, hs = _quantized(a / (1 + torch.exp(-a)) * b)
    ys = torch.bmm(hq, s["down"].float().transpose(1, 2)) * hs * s["down_scale"].unsqueeze(1)
    ys = ys.view(E * s["most"], -1)[place][row].view(T, k, -1)
    return (ys * s["gates"].unsqueeze(-1)).sum(1).to(s["dtype"])


def _run_own(s):
    import sparse_mixture_experts_stable_b200 as moe

    c = s["case"]
    if c["op"] == "sort":
        return moe.moe_sort(s["selected"], c["E"], s["x"])
    if c["op"] == "unsort":
        return moe.moe_unsort(s["ys"], s["row"], s["gates"], base=s["base"])
    if c["op"] == "unsort_backward":
        dys, dgates = moe.moe_unsort_backward(s["dy"], s["ys"], s["row"], s["gates"])
        return dict(dys=dys, dgates=dgates)
    if c["op"] == "linear_i8":
        q, scale = moe.moe_quantize_i8(s["x"])
        return moe.moe_matmul_i8(q, scale, s["wq"], s["wscale"], out_dtype=s["dtype"])
    r = moe.moe_sort_i8(s["selected"], c["E"], s["x"])
    ys = moe.moe_expert_ffn_i8("swiglu", r["xq"], r["xscale"], r["offsets"], s["gate"], s["gate_scale"], w2=s["down"],
                               s2=s["down_scale"], w3=s["up"], s3=s["up_scale"], out_dtype=torch.float32)
    return moe.moe_unsort(ys, r["row"], s["gates"], out_dtype=s["dtype"])


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    z = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "linear_i8":
        M, K, N = c["M"], c["K"], c["N"]
        return dict(bytes=M * K * z + N * K + 4 * N + M * N * z, flops=2.0 * M * K * N)
    T, k, D, E = c["T"], c["k"], c["D"], c["E"]
    if c["op"] == "sort":
        return dict(bytes=T * D * z + T * k * (D * z + 8 + 4 + 4) + 4 * (E + 1), flops=0)
    if c["op"] == "experts_i8":
        # the experts that T * k uniform choices reach
        used = E * (1 - (1 - 1 / E) ** (T * k))
        return dict(bytes=2 * T * D * z + T * k * 12 + used * (3 * c["F"] * D + 4 * (2 * c["F"] + D)),
                    flops=2.0 * 3 * T * k * D * c["F"])
    R = (T - c["pad"]) * k
    if c["op"] == "unsort":
        return dict(bytes=R * D * z + T * D * z * (1 + c["base"]) + T * k * (4 + 4 * c["gates"]), flops=2.0 * R * D)
    return dict(bytes=2 * R * D * z + T * D * z + T * k * 12, flops=3.0 * R * D)


# ---------------------------------------------------------------- the definition in 64 bits
def _quantized64(x):
    x = x.double()
    most = x.abs().max(-1).values
    scale = most / 127
    q = torch.round(x * 127 / torch.where(most > 0, most, 1.0)[..., None])
    return q, scale


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "sort":
        n = c["T"] * c["k"]
        flat = s["selected"].reshape(-1)
        source = torch.argsort(flat * n + torch.arange(n, device=DEV))  # by expert, then by place
        row = torch.argsort(source)
        counts = torch.bincount(flat, minlength=c["E"])
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        return dict(offsets=offsets.int(), row=row.view(c["T"], c["k"]).int(), source=source.int(),
                    xs=s["x"].double().repeat_interleave(c["k"], 0)[source])
    if c["op"] == "unsort":
        y = torch.zeros(c["T"], c["D"], dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            t = (s["row"][:, j] >= 0).nonzero().squeeze(1)
            g = 1.0 if s["gates"] is None else s["gates"][t, j].double()[:, None]
            y[t] += g * s["ys"][s["row"][t, j].long()].double()
        return y if s["base"] is None else y + s["base"].double()
    if c["op"] == "unsort_backward":
        dys = torch.zeros(s["ys"].shape, dtype=torch.float64, device=DEV)
        dgates = torch.zeros(c["T"], c["k"], dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            t = (s["row"][:, j] >= 0).nonzero().squeeze(1)
            r = s["row"][t, j].long()
            dys[r] = s["gates"][t, j].double()[:, None] * s["dy"][t].double()
            dgates[t, j] = torch.einsum("td,td->t", s["dy"][t].double(), s["ys"][r].double())
        return dict(dys=dys, dgates=dgates)
    q, scale = _quantized64(s["x"])
    if c["op"] == "linear_i8":
        return torch.einsum("mk,nk->mn", q, s["wq"][0].double()) * torch.outer(scale, s["wscale"][0].double())
    y = torch.zeros(c["T"], c["D"], dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        t, j = (s["selected"] == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        a, b = (torch.einsum("md,fd->mf", q[t], s[n][e].double()) * torch.outer(scale[t], s[n + "_scale"][e].double())
                for n in ("gate", "up"))
        hq, hs = _quantized64(a * torch.sigmoid(a) * b)
        out = torch.einsum("mf,df->md", hq, s["down"][e].double()) * torch.outer(hs, s["down_scale"][e].double())
        y.index_add_(0, t, s["gates"][t, j].double()[:, None] * out)  # a token takes an expert once
    return y
