"""Pools and fp64 attention on the device, for batches that are too large for the
reference in numpy: codes are found by the place of every dimension, attention goes
request by request."""
import numpy as np
import torch

import kv4_reference as ref


def make_case(seed, kv, ql, hkv, group, d, ps, ramp=0.0, spread_q=2.0, extra_pages=2):
    """(pool [pages, hkv, block], tables, cu, q) on the device: random codes and scales
    of 0.1 to 0.5, slots without a token hold NaN scales.  ramp: scales of K grow by this
    factor of themselves along a sequence, so that row maxima keep moving."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_pages = [-(-int(n) // ps) for n in kv]
    pages, ng = sum(n_pages) + extra_pages, d // 32
    order = rng.permutation(pages).astype(np.int32)
    tables = np.full((len(kv), max(n_pages + [0]) + 1), -7, np.int32)
    live = np.zeros((pages, ps), bool)
    rise = np.ones((pages, ps), np.float32)
    at = 0
    for b, (n, p) in enumerate(zip(kv, n_pages)):
        ids = order[at:at + p]
        at += p
        tables[b, :p] = ids
        j = np.arange(p * ps).reshape(p, ps)
        live[ids] = j < n
        rise[ids] += ramp * j / max(int(n), 1)
    codes = torch.randint(0, 256, (pages, hkv, ps * d), dtype=torch.uint8, device="cuda", generator=g)
    scale = 0.1 + 0.4 * torch.rand(2, pages, hkv, ps, ng, device="cuda", generator=g)
    scale[0] *= torch.from_numpy(rise).cuda()[:, None, :, None]
    scale = scale.to(torch.bfloat16).to(torch.float16)
    scale.masked_fill_(~torch.from_numpy(live).cuda()[None, :, None, :, None], float("nan"))
    bytes_of = [x.reshape(pages, hkv, ps * ng).view(torch.uint8) for x in scale]
    pool = torch.cat([codes] + bytes_of, -1).contiguous()
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    q = (spread_q * torch.randn(int(cu[-1]), hkv * group, d, device="cuda", generator=g))
    return pool, tables, cu, q.to(torch.bfloat16)


def head_values(blocks, ps, d):
    """(K, V) fp64 [hkv, tokens, D] of a sequence's blocks uint8 [P, hkv, block]."""
    x = blocks.transpose(0, 1)
    hkv, c, z = x.shape[0], ps * d // 2, ps * d // 16
    out = []
    for w in (0, 1):
        rows = x[..., w * c:(w + 1) * c].reshape(hkv, -1, d // 2)
        sc = x[..., 2 * c + w * z:2 * c + (w + 1) * z].contiguous().view(torch.float16)
        bit = torch.from_numpy(ref.places(d, w == 0)).to(blocks.device)
        code = (rows[..., bit // 8].int() >> (bit % 8).int()) & 15
        out.append((code - 8).double() *
                   sc.reshape(hkv, -1, d // 32).double().repeat_interleave(32, -1))
    return out


def attention(q, pool, tables, kv, cu, ps, scale, window=0, tree=None, only=None):
    """out, lse, spread, size as kv4_reference.attention, device fp64.  only: the requests
    to compute (the others' rows stay zero)."""
    t, hq, d = q.shape
    hkv = pool.shape[1]
    dev = q.device
    out, spread = (torch.zeros(t, hq, d, dtype=torch.float64, device=dev) for _ in range(2))
    lse = torch.full((t, hq), float("-inf"), dtype=torch.float64, device=dev)
    size = torch.zeros(t, hq, dtype=torch.float64, device=dev)
    tables = torch.from_numpy(np.asarray(tables)).to(dev).long()
    for b in range(len(kv)) if only is None else only:
        n, lo, hi = int(kv[b]), int(cu[b]), int(cu[b + 1])
        m = hi - lo
        if not m or not n:
            continue
        k, v = (x[:, :n] for x in head_values(pool[tables[b, :-(-n // ps)]], ps, d))
        j = torch.arange(n, device=dev)
        p = (n - m + torch.arange(m, device=dev))[:, None]
        see = j <= p
        if window:
            see &= j > p - window
        if tree is not None:
            new = j - (n - m)
            see &= (new < 0) | (((tree[lo:hi, None] >> new.clamp(0, 63)) & 1) == 1)
        rows = q[lo:hi].double().unflatten(1, (hkv, hq // hkv)).permute(1, 2, 0, 3)
        see = see[None, None]                       # [hkv, group, m, n]
        x = scale * torch.matmul(rows.flatten(1, 2), k.transpose(1, 2)).unflatten(1, (-1, m))
        z = abs(scale) * torch.matmul(rows.flatten(1, 2).abs(), k.abs().transpose(1, 2)).amax(-1)
        x = x.masked_fill(~see, float("-inf"))
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - top.clamp(min=-1e300))
        total = e.sum(-1, keepdim=True)
        e /= total.clamp(min=1e-300)

        def put(y):                                 # [hkv, group, m, ..] -> [m, hq, ..]
            return y.movedim(2, 0).flatten(1, 2)

        out[lo:hi] = put(torch.matmul(e.flatten(1, 2), v).unflatten(1, (-1, m)))
        spread[lo:hi] = put(torch.matmul(e.flatten(1, 2), v.abs()).unflatten(1, (-1, m)))
        lse[lo:hi] = put((top + torch.log(total))[..., 0])
        size[lo:hi] = put(z.unflatten(1, (-1, m)))
        del x, e
    return out, lse, spread, size
