"""Workloads of the operators between a decoder layer's attention and its experts: the
residual's addition with the root-mean-square norm (optionally with an output in 8 bits),
matrix products with their epilogue, and the routing to experts.

Norm.  h = x + residual, rounded to the residual's type and kept as the new residual;
y = h / sqrt(mean(h^2) + eps) * weight.  The 8-bit output of a row is e4m3 codes of
y / scale with scale = max|y| / 448.

Product.  out = activation(x w^T + bias) * gate + residual, each part optional.  x and w
may be e4m3 codes with a scale for each row of x and of w.

Routing.  score s = sigmoid or softmax of the logits; experts are chosen by s + bias,
first the groups (by their best expert, or the sum of their two best), then the experts
inside the chosen groups; equal ones by the lower index.  The weights are the scores
themselves (without the bias), optionally divided by their sum, times a factor.  Without
a bias scores order as the logits do, and experts are compared by these.

``own`` false computes every operator from elementary torch operations; ``own`` true calls
the library.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the norm in front of a single-stream decode step: launch latency
        dict(name="norm_token", op="norm", m=1, h=7168, x="bf16", stream="bf16", codes=False),
        # the same norm in a prefill chunk of 8192 tokens
        dict(name="norm_chunk", op="norm", m=8192, h=7168, x="bf16", stream="bf16", codes=False),
        # the experts' fp32 output joins the residual, for a next layer that takes 8 bits
        dict(name="norm_codes", op="norm", m=2048, h=4096, x="fp32", stream="bf16", codes=True),
        # the attention's output projection of one decode step, with the residual: its
        # weights are read once
        dict(name="proj_token", op="linear", m=1, n=7168, k=7168, x="bf16", out="bf16", act="none",
             bias=False, gate=False, residual="bf16", wide=False),
        # the router of a decode batch: few columns, a long sum, fp32 logits
        dict(name="router_batch", op="linear", m=90, n=384, k=7168, x="bf16", out="fp32",
             act="none", bias=False, gate=False, residual="", wide=False),
        # the gate of a shared expert in a verify batch, times its up projection
        dict(name="gate_batch", op="linear", m=256, n=2048, k=7168, x="bf16", out="bf16",
             act="silu", bias=False, gate=True, residual="", wide=False),
        # odd sizes in fp16 with bias and activation, from a part of a wider projection
        dict(name="odd_gelu", op="linear", m=777, n=1411, k=1000, x="fp16", out="fp16", act="gelu",
             bias=True, gate=False, residual="fp16", wide=True),
        # the output projection of a prefill chunk: compute bound
        dict(name="proj_chunk", op="linear", m=8192, n=7168, k=7168, x="bf16", out="bf16",
             act="none", bias=False, gate=False, residual="bf16", wide=False),
        # a prefill chunk's projection with 8-bit operands
        dict(name="codes_chunk", op="linear", m=8192, n=4096, k=4096, x="e4m3", out="bf16",
             act="none", bias=True, gate=False, residual="", wide=False),
        # routing of one token
        dict(name="route_token", op="route", m=1, e=384, top_k=8, x="fp32", scoring="sigmoid",
             bias=True, groups=1, top_groups=1, best=2, renormalize=True),
        # routing of a prefill chunk
        dict(name="route_chunk", op="route", m=8192, e=384, top_k=8, x="fp32", scoring="sigmoid",
             bias=True, groups=1, top_groups=1, best=2, renormalize=True),
        # routing limited to half of the expert groups, from bf16 logits
        dict(name="route_groups", op="route", m=4096, e=256, top_k=8, x="bf16", scoring="sigmoid",
             bias=True, groups=8, top_groups=4, best=2, renormalize=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "route"])
    if op == "norm":
        m = _log(rng, 1, 8192)
        h = _log(rng, 64, min(16384, 8192 * 7168 // m))
        if rng.random() < 0.5:
            h = max(64, h - h % 64)
        return dict(op=op, m=m, h=h, x=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    stream=rng.choice(["", "bf16", "bf16", "fp16", "fp32"]),
                    codes=rng.random() < 0.4)
    if op == "route":
        e = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, rng.randrange(2, 513)])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if e % g == 0])
        top_groups = rng.randrange(1, groups + 1)
        top_k = rng.randrange(1, min(8, e // groups * top_groups) + 1)
        return dict(op=op, m=_log(rng, 1, 8192), e=e, top_k=top_k,
                    x=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    scoring=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6,
                    groups=groups, top_groups=top_groups, best=rng.choice([1, 2]),
                    renormalize=rng.random() < 0.7)
    m = _log(rng, 1, 8192)
    n = _log(rng, 64, 8192)
    k = _log(rng, 64, min(8192, 8192 * 7168 * 7168 // (m * n)))
    x = rng.choice(["bf16", "bf16", "bf16", "fp16", "e4m3"])
    if rng.random() < 0.5:
        n, k = max(64, n - n % 64), max(64, k - k % 64)
    k -= k % (16 if x == "e4m3" else 8)  # rows of operands begin at multiples of 16 bytes
    return dict(op=op, m=m, n=n, k=k, x=x,
                out=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                act=rng.choice(["none", "none", "relu", "silu", "gelu"]), bias=rng.random() < 0.4,
                gate=rng.random() < 0.2, residual=rng.choice(["", "", "bf16", "fp16", "fp32"]),
                wide=rng.random() < 0.4)


def work(case):
    m = case["m"]
    if case["op"] == "norm":
        h, out = case["h"], "fp32" if case["x"] == "fp32" and not case["stream"] else "bf16"
        row = SIZE[case["x"]] + SIZE[out]
        row += 2 * SIZE[case["stream"]] if case["stream"] else 0
        row += 1 if case["codes"] else 0
        return {"bytes": m * h * row + 2 * h + (4 * m if case["codes"] else 0), "flops": 5 * m * h}
    if case["op"] == "route":
        return {"bytes": m * case["e"] * SIZE[case["x"]] + m * case["top_k"] * 8 + 4 * case["e"],
                "flops": m * case["e"] * 10}
    n, k = case["n"], case["k"]
    size = (m + n) * k * SIZE[case["x"]] + m * n * SIZE[case["out"]]
    size += m * n * 2 if case["gate"] else 0
    size += m * n * SIZE[case["residual"]] if case["residual"] else 0
    size += 4 * n if case["bias"] else 0
    size += 4 * (m + n) if case["x"] == "e4m3" else 0
    return {"bytes": size, "flops": 2 * m * n * k}


# ---------------------------------------------------------------- prepare --
def _codes(x):
    """fp32 rows -> e4m3 codes and a scale for each row."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
    return (x / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    m, s = case["m"], {"case": case}
    if case["op"] == "norm":
        h = case["h"]
        # a stream whose channels differ in size, some of them strongly
        chan = torch.exp(0.5 * randn(h))
        s["x"] = (0.5 * randn(m, h) * chan).to(TYPES[case["x"]])
        s["weight"] = (1 + 0.2 * randn(h)).to(torch.bfloat16)
        s["residual"] = (2 * randn(m, h) * chan).to(TYPES[case["stream"]]) if case["stream"] else None
        return s
    if case["op"] == "route":
        e = case["e"]
        # some experts are liked more than others; the balance bias counters that
        liked = 0.5 * randn(e)
        s["logits"] = (1.5 * randn(m, e) + liked).to(TYPES[case["x"]])
        s["bias"] = -0.1 * liked + 0.02 * randn(e) if case["bias"] else None
        return s
    n, k = case["n"], case["k"]
    x, w = randn(m, k), randn(n, k) * (1.0 / math.sqrt(k))
    if case["x"] == "e4m3":
        s["x"], s["x_scale"] = _codes(x)
        s["w"], s["w_scale"] = _codes(w)
    else:
        s["x"], s["w"] = x.to(TYPES[case["x"]]), w.to(TYPES[case["x"]])
        s["x_scale"] = s["w_scale"] = None
    if case["wide"]:
        # x is the middle part of a projection's output, whose rows are longer
        pad = 16
        wide = torch.zeros(m, -(-(k + 2 * pad) // 16) * 16, dtype=s["x"].dtype, device="cuda")
        wide[:, pad:pad + k] = s["x"]
        s["x"] = wide[:, pad:pad + k]
    s["bias"] = 0.1 * randn(n) if case["bias"] else None
    s["gate"] = randn(m, n).to(torch.bfloat16) if case["gate"] else None
    s["residual"] = randn(m, n).to(TYPES[case["residual"]]) if case["residual"] else None
    return s


# ------------------------------------------------------------- plain forms --
def _norm_out(case):
    return torch.float32 if case["x"] == "fp32" and not case["stream"] else torch.bfloat16


def _plain_norm(s):
    case, h = s["case"], s["x"].float()
    new = None
    if s["residual"] is not None:
        new = (h + s["residual"].float()).to(s["residual"].dtype)
        h = new.float()
    # the sum in 64 bits, rounded once: a code next to a border is the same wherever the
    # sum's parts are added
    total = h.double().square().sum(-1, keepdim=True).float()
    y = h * torch.reciprocal(torch.sqrt(total * (1.0 / case["h"]) + EPS)) * s["weight"].float()
    got = {"out": y.to(_norm_out(case))}
    if new is not None:
        got["residual"] = new
    if case["codes"]:
        scale = (y.abs().amax(-1) * (1.0 / E4M3_MAX)).clamp(min=SCALE_MIN)
        codes = (y * torch.reciprocal(scale)[:, None]).to(torch.float8_e4m3fn)
        got["scales"], got["values"] = scale, codes.float() * scale[:, None]
    return got


def _activation(y, act):
    if act == "relu":
        return torch.where(y < 0, 0.0, y)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    return y


def _plain_linear(s):
    case = s["case"]
    y = torch.matmul(s["x"].float(), s["w"].float().T)
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _activation(y, case["act"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"out": y.to(TYPES[case["out"]])}


def _first(key, n):
    """Indices of the n largest along the last axis, larger first, equal ones by index."""
    return torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :n]


def _plain_route(s):
    case, k = s["case"], s["case"]["top_k"]
    logits = s["logits"].double()  # scores next to one another decide in 64 bits
    if case["scoring"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    key = logits if s["bias"] is None else score + s["bias"].double()
    if case["groups"] > 1:
        g = key.unflatten(-1, (case["groups"], -1))
        if case["best"] == 1 or g.shape[-1] == 1:
            of_group = g.amax(-1)
        else:
            value = score.unflatten(-1, (case["groups"], -1)) if s["bias"] is None else g
            of_group = torch.sort(value, dim=-1, descending=True)[0][..., :2].sum(-1)
        keep = torch.zeros_like(of_group, dtype=torch.bool)
        keep.scatter_(-1, _first(of_group, case["top_groups"]), True)
        key = torch.where(keep[..., None], g, float("-inf")).flatten(-2)
    ids = _first(key, k)
    weights = score.gather(-1, ids).float()
    if case["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": weights * 2.5}


# --------------------------------------------------------- the library's calls --
def _own(s):
    from weight_only_int4_moe_gb300 import layer
    case = s["case"]
    if case["op"] == "norm":
        r = layer.moe_add_norm(s["x"], s["weight"], s["residual"], eps=EPS,
                               out_dtype=_norm_out(case), codes=case["codes"])
        got = {"out": r.out}
        if s["residual"] is not None:
            got["residual"] = r.residual
        if case["codes"]:
            got["scales"], got["values"] = r.scales, r.codes.float() * r.scales[:, None]
        return got
    if case["op"] == "route":
        ids, weights = layer.moe_route_experts(
            s["logits"], case["top_k"], scoring=case["scoring"], bias=s["bias"],
            groups=case["groups"], top_groups=case["top_groups"], group_best=case["best"],
            renormalize=case["renormalize"], scale=2.5)
        return {"ids": ids, "weights": weights}
    if "linear" not in s:  # what a program builds once for its weights
        s["linear"] = layer.Linear(s["w"], bias=s["bias"], scale=s["w_scale"])
    return {"out": layer.moe_linear(s["x"], s["linear"], activation=case["act"], gate=s["gate"],
                                    residual=s["residual"], x_scale=s["x_scale"],
                                    out_dtype=TYPES[case["out"]])}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "linear": _plain_linear,
            "route": _plain_route}[state["case"]["op"]](state)


# ------------------------------------------------------- in 64 bits, apart --
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h, got = s["x"].double(), {}
        if s["residual"] is not None:
            h = h + s["residual"].double()
            got["residual"] = h
            h = h.float().to(s["residual"].dtype).double()  # the operator goes on with what it keeps
        y = h * (h.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() * s["weight"].double()
        got["out"] = y
        if case["codes"]:
            # a code next to a border has no value in 64 bits
            got["scales"], got["values"] = y.abs().max(-1).values / E4M3_MAX, None
        return got
    if case["op"] == "route":
        x = s["logits"].double()
        soft = case["scoring"] == "softmax"
        score = torch.softmax(x, -1) if soft else torch.special.expit(x)
        by = x if s["bias"] is None else score + s["bias"].double()
        lowest, size = torch.finfo(torch.float64).min, case["e"] // case["groups"]
        if case["groups"] > 1:
            value = by if s["bias"] is not None or case["best"] == 1 else score
            parts = value.split(size, -1)
            best = [p.topk(min(case["best"], size), -1).values.sum(-1) for p in parts]
            best, open_ = torch.stack(best, -1), torch.zeros_like(by, dtype=torch.bool)
            rows = torch.arange(case["m"], device=x.device)
            for _ in range(case["top_groups"]):
                g = best.argmax(-1)
                best[rows, g] = lowest
                open_ |= torch.arange(case["e"], device=x.device) // size == g[:, None]
            by = by.masked_fill(~open_, lowest)
        # the index counts only between equal ones
        order = torch.arange(case["e"], device=x.device).expand_as(by)
        ids = []
        for _ in range(case["top_k"]):
            top = by.max(-1, keepdim=True).values
            ids.append(order.masked_fill(by != top, case["e"]).min(-1).values)
            by = by.scatter(-1, ids[-1][:, None], -float("inf"))
        ids = torch.stack(ids, -1)
        w = torch.gather(score, 1, ids)
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return {"ids": ids.int(), "weights": 2.5 * w}
    w = s["w"].double()
    if s["w_scale"] is not None:
        w = w * s["w_scale"].double()[:, None]
    out = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
    for i in range(0, case["m"], 2048):
        r = slice(i, i + 2048)
        x = s["x"][r].double()
        if s["x_scale"] is not None:
            x = x * s["x_scale"][r].double()[:, None]
        y = torch.einsum("mk,nk->mn", x, w)
        y = y if s["bias"] is None else y + s["bias"].double()
        if case["act"] == "relu":
            y = y.clamp(min=0)
        elif case["act"] == "silu":
            y = y * torch.special.expit(y)
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        y = y if s["gate"] is None else y * s["gate"][r].double()
        out[r] = y if s["residual"] is None else y + s["residual"][r].double()
    return {"out": out}
