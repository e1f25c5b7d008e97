"""Plain forms, in 64 bits on the CPU, of the operators between attention and experts
(include/moe_layer.h), written from their definitions."""
import math

import torch

U = 2.0 ** -24  # half a step of fp32, relative


def half_step(t, dtype):
    """Half a rounding step at values t (subnormals have the smallest normal's)."""
    f = torch.finfo(dtype)
    return t.abs().clamp(min=f.tiny) * (f.eps / 2)


def add_norm(x, weight, residual, eps):
    """(h as held, y in 64 bits)."""
    h = x.float()
    if residual is not None:
        h = (h + residual.float()).to(residual.dtype)  # one fp32 addition, one rounding
    d = h.double()
    y = d / (d.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    return h, y if weight is None else y * weight.double()


def add_norm_fp32(h, weight, eps):
    """y with every operation rounded to fp32, in the header's order."""
    total = h.double().pow(2).sum(-1, keepdim=True).float()
    one = torch.ones((), dtype=torch.float32)
    q = one / torch.sqrt(total * torch.tensor(1.0 / h.shape[-1]).float() + torch.tensor(eps).float())
    y = h.float() * q
    return y if weight is None else y * weight.float()


def linear(x, w, x_scale=None, w_scale=None, bias=None, act=None, gate=None, residual=None):
    """(the result in 64 bits, a bound on its error before the last rounding)."""
    xd, wd = x.double(), w.double()
    y, size = xd @ wd.T, xd.abs() @ wd.abs().T
    # The tensor cores add the products of an instruction (16 or 32 of k) to the sum with
    # a truncation each at worst, a step of fp32 relative to what has been added up; inside
    # an instruction the terms are cut at the largest one's last place, a step a term.
    step = 2 * U
    bound = size * step * (x.shape[1] / 16 + 32)
    if x_scale is not None:
        y, bound = y * x_scale.double()[:, None], bound * x_scale.double()[:, None]
    if w_scale is not None:
        y, bound = y * w_scale.double(), bound * w_scale.double()
    bound = bound + 2 * U * y.abs()
    if bias is not None:
        y = y + bias.double()
        bound = bound + U * y.abs()
    if act == "relu":
        y = y.clamp(min=0)
    elif act == "silu":
        # slope at most 1.1; an exponential within two steps, an addition, a division
        y, bound = y * torch.special.expit(y), 1.1 * bound + 6 * U * y.abs()
    elif act == "gelu":
        # slope at most 1.13; the error function within two steps of 1
        y, bound = y * torch.special.ndtr(y), 1.13 * bound + 6 * U * y.abs()
    if gate is not None:
        g = gate.double()
        y, bound = y * g, bound * g.abs() + U * (y * g).abs()
    if residual is not None:
        y = y + residual.double()
        bound = bound + U * y.abs()
    return y, bound


def route_experts(logits, top_k, scoring="softmax", bias=None, groups=1, top_groups=None,
                  group_best=2, renormalize=True, scale=1.0):
    """(ids, weights) by lists of Python numbers, one token after the other."""
    top_groups = groups if top_groups is None else top_groups
    all_ids, all_w = [], []
    for row in logits.double().tolist():
        e_all = range(len(row))
        big = torch.finfo(torch.float32).max
        lg = [-math.inf if math.isnan(v) else min(v, big) for v in row]
        b = [0.0] * len(row) if bias is None else bias.double().tolist()
        there = [lg[e] > -math.inf and b[e] > -math.inf for e in e_all]
        if scoring == "softmax":
            top = max(lg)
            ex = [math.exp(v - top) if v > -math.inf else 0.0 for v in lg]
            total = math.fsum(ex)
            s = [v / total if total else 0.0 for v in ex]
        else:
            s = [math.exp(min(v, 0.0)) / (1 + math.exp(-abs(v))) for v in lg]
        c = lg if bias is None else [s[e] + b[e] for e in e_all]
        size = len(row) // groups
        rank = []
        for g in range(groups):
            mine = [e for e in range(g * size, (g + 1) * size) if there[e]]
            if group_best == 1 or size == 1:
                v = sorted((c[e] for e in mine), reverse=True)[:1]
            else:
                v = sorted((s[e] + b[e] for e in mine), reverse=True)[:2]
            rank.append((-sum(v) if v else math.inf, g))
        chosen = [g for _, g in sorted(rank)[:top_groups]]
        allowed = [e for e in e_all if e // size in chosen]
        order = sorted(allowed, key=lambda e: (not there[e], -c[e] if there[e] else 0.0, e))
        ids = order[:top_k]
        if not renormalize:
            w = [s[e] if there[e] else 0.0 for e in ids]
        else:
            live = [e for e in ids if there[e]]
            if scoring == "softmax":
                m = max((lg[e] for e in live), default=0.0)
                w = [math.exp(lg[e] - m) if there[e] else 0.0 for e in ids]
            else:
                m = max((min(lg[e], 0.0) for e in live), default=0.0)
                w = [math.exp(min(lg[e], 0.0) - m) / (1 + math.exp(-abs(lg[e]))) if there[e]
                     else 0.0 for e in ids]
            total = math.fsum(w)
            w = [v / total if total else 0.0 for v in w]
        all_ids.append(ids)
        all_w.append([v * scale for v in w])
    return (torch.tensor(all_ids, dtype=torch.int32).reshape(len(all_ids), top_k),
            torch.tensor(all_w, dtype=torch.float64).reshape(len(all_w), top_k))
