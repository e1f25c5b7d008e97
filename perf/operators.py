"""Workloads of the 4-bit paged cache: append (head norms, position rotation and
the cache write in one pass), attention over the cache, and page management.

The cache is a uint8 pool [layers, pages, kv heads, block].  A block holds one
page's tokens of one head: K codes [ps, D/2], V codes [ps, D/2], K scales fp16
[ps, D/32], V scales fp16 [ps, D/32]; a value is (code - 8) * scale.  In a K row,
the 32-bit word t*NG + G (t < 4, NG = D/32 groups) holds dimension
32G + 8t + 2i + h at bits 16h + 4i; in a V row, the 16-bit piece g*NG + G (g < 8)
holds dimension 32G + 4g + i at bits 4i.

``own`` false computes every operator from elementary torch operations in 32
bits; ``own`` true calls the library.
"""
import math
import random

import torch

own = False

SEVENTH = 1.0 / 7.0
SCALE_MIN, SCALE_MAX = 2.0 ** -14, 2720.0
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token of one sequence: the latency of a single-stream decode step (hidden 4096)
        dict(name="append_token", op="append", batch=1, q=1, kv=1024, hq=32, hkv=8, d=128, ps=64,
             ragged=False, half=True, lengths=1),
        # a prefill chunk of 8192 tokens of several prompts (hidden 7168: 56 heads)
        dict(name="append_chunk", op="append", batch=3, q=4096, kv=6000, hq=56, hkv=8, d=128,
             ps=64, ragged=True, half=True, lengths=2),
        # one short single-stream decode step: launch latency
        dict(name="decode_one", op="attend", batch=1, q=1, kv=777, hq=32, hkv=8, d=128, ps=64,
             ragged=False, window=0, tree=False, lse=False, lengths=3),
        # a decode batch of 90 streams of very different lengths, 7 query heads a kv head
        dict(name="decode_ragged", op="attend", batch=90, q=1, kv=8192, hq=56, hkv=8, d=128,
             ps=64, ragged=True, window=0, tree=False, lse=False, lengths=4),
        # two very long contexts: few rows, the whole GPU on each
        dict(name="decode_long", op="attend", batch=2, q=1, kv=131071, hq=64, hkv=8, d=128,
             ps=64, ragged=False, window=0, tree=False, lse=True, lengths=5),
        # a verify batch: 10 streams x 9 draft tokens of a tree
        dict(name="verify_tree", op="attend", batch=10, q=9, kv=5001, hq=56, hkv=8, d=128, ps=32,
             ragged=True, window=0, tree=True, lse=False, lengths=6),
        # a prefill chunk of 4096 tokens behind 4096 cached ones: compute bound
        dict(name="prefill_chunk", op="attend", batch=1, q=4096, kv=8192, hq=32, hkv=8, d=128,
             ps=64, ragged=False, window=0, tree=False, lse=False, lengths=7),
        # prompts and single tokens in one batch, sliding window, one kv head a query head, D = 64
        dict(name="mixed_window", op="attend", batch=24, q=500, kv=4100, hq=16, hkv=16, d=64,
             ps=16, ragged=True, window=2048, tree=False, lse=False, lengths=8),
        # a few branches of a few streams re-forked in a one-layer pool
        dict(name="fork_few", op="fork", seqs=4, children=8, kv=1000, hkv=8, d=128, ps=64,
             layers=1, pages=256, lengths=9),
        # every stream of a large batch branched in a pool of 8 layers
        dict(name="fork_many", op="fork", seqs=64, children=256, kv=8000, hkv=8, d=128, ps=64,
             layers=8, pages=9000, lengths=10),
        # a small fragmented pool made dense
        dict(name="compact_few", op="compact", seqs=16, kv=300, hkv=4, d=64, ps=16, layers=2,
             pages=500, lengths=11),
        # a large fragmented pool made dense
        dict(name="compact_many", op="compact", seqs=200, kv=4000, hkv=8, d=128, ps=64, layers=4,
             pages=10000, lengths=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "fork", "compact"])
    c = dict(op=op, lengths=rng.randrange(1 << 20))
    hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 3, 4, 7, 8])
    d = rng.choice([64, 128, 128])
    ps = rng.choice([16, 32, 64, 64])
    if op == "append":
        batch = _log(rng, 1, 200)
        q = _log(rng, 1, max(1, 8192 // batch))
        c.update(batch=batch, q=q, kv=q + _log(rng, 1, 3000), hq=min(56, hkv * group), hkv=hkv,
                 d=d, ps=ps, ragged=rng.random() < 0.6, half=rng.random() < 0.7)
        c["hq"] -= c["hq"] % hkv
    elif op == "attend":
        kind = rng.choice(["decode", "decode", "verify", "prefill"])
        batch = _log(rng, 1, {"decode": 256, "verify": 64, "prefill": 16}[kind])
        q = {"decode": 1, "verify": rng.randrange(2, 34), "prefill": _log(rng, 34, 3000)}[kind]
        hq = hkv * group
        # the plain form pads to the longest, so the padded sizes bound a drawn case
        most = min(130000, 2_000_000 // (batch * hkv), 900_000_000 // (batch * q * hq))
        if kind == "prefill":
            q = min(q, int((3.0e8 / (batch * hq)) ** 0.5))
            most = min(30000, 900_000_000 // (batch * q * hq))
        kv = q + _log(rng, 1, max(2, most - q))
        c.update(batch=batch, q=q, kv=kv, hq=hq, hkv=hkv, d=d, ps=ps, ragged=rng.random() < 0.7,
                 window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
                 tree=kind == "verify" and rng.random() < 0.6, lse=rng.random() < 0.5)
    elif op == "fork":
        seqs = _log(rng, 1, 64)
        children = _log(rng, 1, 256)
        kv, layers = _log(rng, 1, 8000), rng.randrange(1, 9)
        pages = seqs * -(-kv // ps) + children + _log(rng, 10, 500)
        if ps < 64:
            layers = min(layers, 4)
        c.update(seqs=seqs, children=children, kv=kv, hkv=min(8, hkv), d=d, ps=ps, layers=layers,
                 pages=pages)
    else:
        seqs = _log(rng, 4, 200)
        kv = _log(rng, 20, 4000)
        pages = max(64, int(seqs * (kv / 2 / ps + 1) * rng.uniform(1.3, 3.0)))
        c.update(seqs=seqs, kv=kv, hkv=min(8, hkv), d=d, ps=ps, layers=rng.randrange(1, 4),
                 pages=min(pages, 20000))
    return c


def _lengths(case):
    """(kv lengths, query lengths) of the case's requests: from the case alone."""
    r = random.Random(case["lengths"])
    kv, q = [], []
    for b in range(case.get("batch", case.get("seqs", 1))):
        full = b == 0 or not case.get("ragged", True)
        n = case["kv"] if full else r.randint(1, case["kv"])
        most = min(n, case.get("q", 1))
        # prompts beside single tokens: every third request of a ragged batch of prompts has one
        m = most if full or case.get("tree") else 1 if r.random() < 0.34 else r.randint(1, most)
        kv.append(n)
        q.append(m)
    return kv, q


def _parents(case):
    r = random.Random(case["lengths"] + 1)
    return [r.randrange(case["seqs"]) for _ in range(case["children"])]


def _used(case):
    """Sequences of a compact case that fit its pool, 70 % full at most."""
    kv, _ = _lengths(case)
    n, keep = 0, []
    for x in kv:
        p = -(-x // case["ps"])
        if n + p > 0.7 * case["pages"] and keep:
            break
        keep.append(x)
        n += p
    return keep, min(n, case["pages"])


def _token_bytes(case):  # K and V of one token and head: codes and scales
    return case["d"] + case["d"] // 8


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "append":
        _, q = _lengths(case)
        t = sum(q)
        # q, k, v, the table rows; q out and the cache rows; the rows read back as fp16
        return {"bytes": t * ((2 * case["hq"] + 2 * hkv) * d * 2 + d * 4
                              + 2 * hkv * _token_bytes(case) + 2 * hkv * d * 2),
                "flops": t * (case["hq"] + 2 * hkv) * d * 10}
    if case["op"] == "attend":
        kv, q = _lengths(case)
        w = case["window"] or (1 << 30)
        tokens = pairs = 0
        for n, m in zip(kv, q):
            tokens += min(n, m - 1 + w)
            first = n - m + 1  # cached tokens and itself, for the first query
            pairs += sum(min(first + i, w) for i in range(m))
        return {"bytes": tokens * hkv * _token_bytes(case) + 2 * sum(q) * case["hq"] * d * 2,
                "flops": 4 * d * case["hq"] * pairs}
    if case["op"] == "fork":
        kv, _ = _lengths(case)
        par = _parents(case)
        part = sum(kv[p] % case["ps"] for p in par)
        rows = sum(-(-kv[p] // case["ps"]) for p in par)
        return {"bytes": 2 * part * case["layers"] * hkv * _token_bytes(case) + rows * 4 * 6
                + case["pages"] * 4, "flops": 0}
    keep, n = _used(case)
    moved = n * (1 - n / case["pages"])
    return {"bytes": 2 * moved * case["layers"] * hkv * case["ps"] * _token_bytes(case)
            + 8 * case["pages"] + 8 * n, "flops": 0}


# ---------------------------------------------------------------- prepare --
def _pack_k(codes):
    """codes uint8 [..., D] -> bytes [..., D/2] in the K row order."""
    ng = codes.shape[-1] // 32
    n = codes.unflatten(-1, (ng, 4, 4, 2))          # G, t, i, h
    n = n.movedim((-4, -3, -2, -1), (-3, -4, -1, -2)).flatten(-4)  # t, G, h, i
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _pack_v(codes):
    ng = codes.shape[-1] // 32
    n = codes.unflatten(-1, (ng, 8, 4)).transpose(-3, -2).flatten(-3)  # g, G, i
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _nibbles(rows):
    return torch.stack((rows & 15, rows >> 4), -1).flatten(-2)


def _unpack_k(rows):
    """bytes [..., D/2] in the K row order -> codes [..., D]."""
    n = _nibbles(rows)
    n = n.unflatten(-1, (4, n.shape[-1] // 32, 2, 4))  # t, G, h, i
    return n.movedim((-4, -3, -2, -1), (-3, -4, -1, -2)).flatten(-4)


def _unpack_v(rows):
    n = _nibbles(rows)
    return n.unflatten(-1, (8, n.shape[-1] // 32, 4)).transpose(-3, -2).flatten(-3)


def _quantise(x):
    """fp32 [..., D] -> (codes uint8 [..., D], scales fp16 [..., D/32])."""
    g = x.unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) * SEVENTH).to(torch.bfloat16).float().clamp(SCALE_MIN, SCALE_MAX)
    q = torch.round(g / s[..., None]).clamp(-8, 7) + 8
    return q.to(torch.uint8).flatten(-2), s.to(torch.float16)


def _parts(pool, ps, d):
    """The four parts of every block, as views of the pool [..., block]."""
    c, s = ps * d // 2, ps * d // 32 * 2
    kc = pool[..., :c].unflatten(-1, (ps, d // 2))
    vc = pool[..., c:2 * c].unflatten(-1, (ps, d // 2))
    ks = pool[..., 2 * c:2 * c + s].view(torch.float16).unflatten(-1, (ps, d // 32))
    vs = pool[..., 2 * c + s:].view(torch.float16).unflatten(-1, (ps, d // 32))
    return kc, vc, ks, vs


def _filled(case, layers, pages, gen):
    """A pool whose every slot holds a token: keys near unit rms with a few
    stronger channels, as a head norm's weights leave them; values likewise."""
    hkv, d, ps = case["hkv"], case["d"], case["ps"]
    pool = torch.empty(layers, pages, hkv, ps * _token_bytes(case), dtype=torch.uint8, device="cuda")
    kc, vc, ks, vs = _parts(pool, ps, d)
    chan = 0.8 + 0.4 * torch.rand(hkv, 1, d, generator=gen, device="cuda")
    step = max(1, (1 << 27) // (hkv * ps * d))
    for layer in range(layers):
        for p in range(0, pages, step):
            n = min(step, pages - p)
            for code, scale, pack in ((kc, ks, _pack_k), (vc, vs, _pack_v)):
                x = torch.randn(n, hkv, ps, d, generator=gen, device="cuda") * chan
                q, s = _quantise(x)
                code[layer, p:p + n] = pack(q)
                scale[layer, p:p + n] = s
    return pool


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(kv, ps, order, width=None):
    """Page tables of sequences that take their pages from `order` in turn."""
    n = [-(-x // ps) for x in kv]
    width = width or max(max(n), 1)
    t = torch.full((len(kv), width), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(n):
        t[b, :m] = order[at:at + m]
        at += m
    return t.cuda(), at


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    d, hkv, ps = case["d"], case["hkv"], case["ps"]
    if case["op"] in ("fork", "compact"):
        s = {"case": case, "pool": _filled(case, case["layers"], case["pages"], gen)}
        order = torch.randperm(case["pages"], generator=host).to(torch.int32)
        if case["op"] == "fork":
            kv, _ = _lengths(case)
            n = case["children"]
            s["tables"], at = _tables(kv + [0] * n, ps, order, -(-case["kv"] // ps) + 1)
            s["lens"] = _ints(kv + [0] * n)
            s["parents"], s["children"] = _ints(_parents(case)), _ints(
                list(range(len(kv), len(kv) + n)))
        else:
            kv, _ = _used(case)
            s["tables"], at = _tables(kv, ps, order)
            s["lens"] = _ints(kv)
            s["tables_out"] = torch.empty_like(s["tables"])
            s["refs_out"] = torch.empty(case["pages"], dtype=torch.int32, device="cuda")
        s["refs"] = torch.zeros(case["pages"], dtype=torch.int32, device="cuda")
        s["refs"][order[:at].long().cuda()] = 1
        return s
    kv, q = _lengths(case)
    used = sum(-(-x // ps) for x in kv)
    pages = used + 3
    order = torch.randperm(pages, generator=host).to(torch.int32)
    tables, _ = _tables(kv, ps, order)
    t, hq = sum(q), case["hq"]
    cu = [0]
    for m in q:
        cu.append(cu[-1] + m)
    s = {"case": case, "tables": tables, "kv": _ints(kv), "cu": _ints(cu), "tokens": t,
         "max_q": max(q), "max_kv": max(kv)}
    pool = _filled(case, 1, pages, gen)
    # slots past a sequence's end hold whatever the memory held: NaN scales
    _, _, ks, vs = _parts(pool[0], ps, d)
    for b, n in enumerate(kv):
        if n % ps:
            p = int(order[sum(-(-x // ps) for x in kv[:b + 1]) - 1])
            ks[p, :, n % ps:] = float("nan")
            vs[p, :, n % ps:] = float("nan")
    s["pool"] = pool
    if case["op"] == "append":
        # one projection's output: q, k and v heads of a token side by side
        qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=gen, device="cuda")
        qkv *= 0.5 + torch.rand((hq + 2 * hkv) * d, generator=gen, device="cuda")
        qkv = qkv.to(torch.bfloat16)
        s["q"] = qkv[:, :hq * d].unflatten(-1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(-1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d:].unflatten(-1, (hkv, d))
        s["qw"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        s["kw"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        ang = torch.arange(max(kv), device="cuda", dtype=torch.float64)[:, None] \
            * (10000.0 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d))
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        pos = [n - m + i for n, m in zip(kv, q) for i in range(m)]
        s["positions"] = _ints(pos)
        return s
    s["q"] = (2.0 * torch.randn(t, hq, d, generator=gen, device="cuda")).to(torch.bfloat16)
    s["tree"] = None
    if case["tree"]:
        # every draft token sees itself and its ancestors; a parent is an earlier token
        r = random.Random(seed)
        words = []
        for m in q:
            seen = []
            for i in range(m):
                up = r.randrange(i) if i else None
                seen.append((1 << i) | (seen[up] if i else 0))
            words += seen
        s["tree"] = torch.tensor(words, dtype=torch.int64, device="cuda")
    return s


# ------------------------------------------------------------- plain forms --
def _head_norm(x, w):
    """x / sqrt(mean(x^2) + eps) * w over the last axis, fp32; the squares are
    added in a fixed order (halves, then eights, then neighbours), so that the
    rounding, and with it every 4-bit code, is the same wherever it is computed."""
    d = x.shape[-1]
    y = x * x
    y = (y[..., :d // 2] + y[..., d // 2:]).unflatten(-1, (-1, 8))
    for n in (4, 2, 1):
        y = y[..., :n] + y[..., n:]
    y = y[..., 0]
    while y.shape[-1] > 1:
        y = y[..., 0::2] + y[..., 1::2]
    return x * torch.reciprocal(torch.sqrt(y * (1.0 / d) + EPS)) * w


def _rotate(x, cos, sin, half):
    if half:
        a, b = x.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)


def _request_of(s):
    """For each query token: its request and its logical index in the sequence."""
    t = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    q = s["cu"][1:] - s["cu"][:-1]
    return b, (s["kv"] - q)[b] + t - s["cu"][b]


def _plain_append(s):
    case = s["case"]
    pos = s["positions"].long()
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _rotate(_head_norm(s["q"].float(), s["qw"].float()), cos, sin, case["half"])
    k = _rotate(_head_norm(s["k"].float(), s["kw"].float()), cos, sin, case["half"])
    kq, ksc = _quantise(k)
    vq, vsc = _quantise(s["v"].float())
    b, at = _request_of(s)
    page = s["tables"][b, (at // case["ps"]).long()].long()
    slot = (at % case["ps"]).long()
    kc, vc, ks, vs = _parts(s["pool"][0], case["ps"], case["d"])
    kc[page, :, slot], vc[page, :, slot] = _pack_k(kq), _pack_v(vq)
    ks[page, :, slot], vs[page, :, slot] = ksc, vsc
    back = [((c.float().unflatten(-1, (-1, 32)) - 8) * z.float()[..., None]).flatten(-2).half()
            for c, z in ((kq, ksc), (vq, vsc))]
    return {"q": q.to(torch.bfloat16), "k": back[0], "v": back[1]}


def _cached(pages, codes, scales, unpack):
    """One part of the pages [B, P] as fp32 values [B, Hkv, P * ps, D]."""
    c = unpack(codes[pages])                       # B, P, Hkv, ps, D
    x = (c.float().unflatten(-1, (-1, 32)) - 8) * scales[pages].float()[..., None]
    return x.flatten(-2).transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    case = s["case"]
    d, hq, hkv, ps = case["d"], case["hq"], case["hkv"], case["ps"]
    kc, vc, ks, vs = _parts(s["pool"][0], ps, d)
    pages = s["tables"].clamp(min=0).long()
    width = pages.shape[1] * ps
    kv, bsz, mq = s["kv"], s["kv"].numel(), s["max_q"]
    qlen = s["cu"][1:] - s["cu"][:-1]
    b, at = _request_of(s)
    i = torch.arange(s["tokens"], device="cuda") - s["cu"][b]
    q = torch.zeros(bsz, mq, hq, d, device="cuda")
    q[b, i] = s["q"].float()
    # the rows of one kv head together: [B, Hkv, rows, D]
    rows = q.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    k = _cached(pages, kc, ks, _unpack_k)
    x = torch.matmul(rows, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    del k
    x = x.unflatten(2, (mq, -1))                   # B, Hkv, mq, G, width
    j = torch.arange(width, device="cuda")
    first = kv - qlen                              # cached tokens before the new ones
    p = first[:, None] + torch.arange(mq, device="cuda")
    see = (j < kv[:, None])[:, None] & (j <= p[..., None])   # B, mq, width
    if case["window"]:
        see &= j > p[..., None] - case["window"]
    if s["tree"] is not None:
        word = torch.zeros(bsz, mq, dtype=torch.int64, device="cuda")
        word[b, i] = s["tree"]
        new = j - first[:, None]                   # index among the new tokens
        bit = (word[..., None] >> new.clamp(0, 63)[:, None]) & 1
        see &= (new < 0)[:, None] | (bit == 1)
    x = x.masked_fill(~see[:, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top.clamp(min=-3e38))
    del x
    total = e.sum(-1, keepdim=True)
    v = _cached(pages, vc, vs, _unpack_v)
    v = torch.where((j < kv[:, None])[:, None, :, None], v, 0.0)
    y = torch.matmul(e.flatten(2, 3), v).unflatten(2, (mq, -1))
    y = torch.where(total > 0, y / total, 0.0)
    out = y.permute(0, 2, 1, 3, 4).flatten(2, 3)[b, i].to(torch.bfloat16)
    if not case["lse"]:
        return {"out": out}
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).flatten(2)[b, i]
    return {"out": out, "lse": lse}


def _live_bytes(case):
    """The token that each byte of a block belongs to."""
    ps, d = case["ps"], case["d"]
    tok = torch.arange(ps, device="cuda")
    c, z = tok.repeat_interleave(d // 2), tok.repeat_interleave(d // 16)
    return torch.cat((c, c, z, z))


def _plain_fork(s):
    case = s["case"]
    ps, tables, lens, refs = case["ps"], s["tables"], s["lens"], s["refs"]
    par, kid = s["parents"].long(), s["children"].long()
    col = torch.arange(tables.shape[1], device="cuda")

    def counts(seq):  # 1 at each entry of the sequences' tables that is in use
        return (col < ((lens[seq] + ps - 1) // ps)[:, None]).to(torch.int32)

    # the children's old pages go back
    refs.index_add_(0, tables[kid].clamp(min=0).long().flatten(), -counts(kid).flatten())
    lens[kid] = 0
    # full pages are shared; a page that a sequence has only begun is copied to
    # the lowest free ones, in the children's order
    n = lens[par]
    part = n % ps
    free = torch.cumsum((refs == 0).to(torch.int64), 0)
    rank = torch.cumsum((part > 0).to(torch.int64), 0)
    new = torch.searchsorted(free, rank).to(torch.int32)
    row = torch.where(counts(par) == 1, tables[par], -1)
    last = (n // ps).long()
    old = row.gather(1, last[:, None])[:, 0].clamp(min=0).long()
    row = torch.where((col == last[:, None]) & (part > 0)[:, None], new[:, None], row)
    tables[kid] = row
    lens[kid] = n
    refs.index_add_(0, row.clamp(min=0).long().flatten(), counts(par).flatten())
    pool = s["pool"]
    dst = new.long()[part > 0]
    live = _live_bytes(case) < part[part > 0][:, None]
    pool[:, dst] = torch.where(live[None, :, None], pool[:, old[part > 0]], pool[:, dst])
    return {"tables": tables, "lens": lens, "refs": refs, "pool": pool}


def _plain_compact(s):
    tables, refs, pool = s["tables"], s["refs"], s["pool"]
    used = refs > 0
    n = used.sum()
    page = torch.arange(refs.numel(), device="cuda")
    src = page[used & (page >= n)]
    dst = page[~used & (page < n)]
    to = page.clone()
    to[src] = dst
    pool[:, dst] = pool[:, src]
    out = torch.zeros_like(refs)
    out[to[used]] = refs[used]
    moved = torch.where(tables >= 0, to[tables.clamp(min=0).long()].to(torch.int32), -1)
    return {"tables": moved, "refs": out, "used": n.to(torch.int32).reshape(1), "pool": pool}


# --------------------------------------------------------- the library's calls --
def _handles(s):
    """What a program builds once and keeps: views of its own buffers."""
    if "handles" not in s:
        from weight_only_int4_moe_gb300 import kv4
        case = s["case"]
        cache = kv4.Cache(s["pool"], case["hkv"], case["d"], case["ps"])
        if "lens" in s:
            s["handles"] = (kv4, cache, kv4.Sequences(s["tables"], s["lens"], s["refs"]))
        else:
            s["handles"] = (kv4, cache, kv4.Batch(s["cu"], s["kv"], s["tables"], s["tokens"],
                                                  s["max_q"], s["max_kv"]))
        if case["op"] == "attend":
            s["workspace"] = kv4.alloc_workspace(cache, s["handles"][2], case["hq"])
    return s["handles"]


def _own(s):
    kv4, cache, what = _handles(s)
    case = s["case"]
    if case["op"] == "append":
        q = kv4.moe_kv4_append(cache, what, s["q"], s["k"], s["v"], s["qw"], s["kw"], s["cos"],
                               s["sin"], s["positions"], eps=EPS, interleaved=not case["half"])
        k, v = kv4.moe_kv4_read(cache, what)
        return {"q": q, "k": k, "v": v}
    if case["op"] == "attend":
        out = kv4.moe_kv4_attention(s["q"], cache, what, window=case["window"], tree=s["tree"],
                                    return_lse=case["lse"], workspace=s["workspace"])
        return {"out": out[0], "lse": out[1]} if case["lse"] else {"out": out}
    if case["op"] == "fork":
        kv4.moe_kv4_free(cache, what, s["children"])
        kv4.moe_kv4_fork(cache, what, s["parents"], s["children"])
        return {"tables": s["tables"], "lens": s["lens"], "refs": s["refs"], "pool": s["pool"]}
    used = kv4.moe_kv4_compact(cache, what, tables_out=s["tables_out"], refs_out=s["refs_out"])
    return {"tables": s["tables_out"], "refs": s["refs_out"], "used": used, "pool": s["pool"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork,
            "compact": _plain_compact}[state["case"]["op"]](state)


# ------------------------------------------------------- in 64 bits, apart --
def _value(rows, scales, d, key):
    """Values in fp64 from the bytes of rows [..., D/2], by each dimension's place."""
    ng = d // 32
    dim = torch.arange(d, device=rows.device)
    g, r = dim // 32, dim % 32
    if key:
        bit = 32 * ((r // 8) * ng + g) + 16 * (r % 2) + 4 * ((r % 8) // 2)
    else:
        bit = 16 * ((r // 4) * ng + g) + 4 * (r % 4)
    code = (rows[..., bit // 8].int() >> (bit % 8).int()) & 15
    return (code - 8).double() * scales.double()[..., g]


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    d, ps, hkv, hq = case["d"], case["ps"], case["hkv"], case["hq"]
    kv, ql = _lengths(case)
    if case["op"] == "append":
        def normed(x, w):
            x, w = x.double(), w.double()
            return x * (x.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() * w

        a = torch.polar(torch.ones_like(s["cos"], dtype=torch.float64),
                        torch.atan2(s["sin"].double(), s["cos"].double()))
        a = a[s["positions"].long()][:, None] * torch.hypot(
            s["sin"].double(), s["cos"].double())[s["positions"].long()][:, None]

        def turned(x):
            h = d // 2
            z = torch.complex(x[..., :h], x[..., h:]) if case["half"] else \
                torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous())
            z = z * a
            if case["half"]:
                return torch.cat((z.real, z.imag), -1)
            return torch.view_as_real(z).flatten(-2)

        def held(x):
            g = x.reshape(*x.shape[:-1], d // 32, 32)
            z = (g.abs().max(-1).values / 7).float().to(torch.bfloat16).double()
            z = z.clamp(SCALE_MIN, SCALE_MAX)[..., None]
            return (torch.round(g / z).clamp(-8, 7) * z).reshape(x.shape)

        return {"q": turned(normed(s["q"], s["qw"])), "k": held(turned(normed(s["k"], s["kw"]))),
                "v": held(s["v"].double())}
    c, z = ps * d // 2, ps * d // 16
    out = torch.zeros(s["tokens"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], hq), float("-inf"), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(kv, ql)):
        blocks = s["pool"][0][s["tables"][b, :-(-n // ps)].long()]
        part = (blocks[..., :c], blocks[..., c:2 * c])
        scal = (blocks[..., 2 * c:2 * c + z], blocks[..., 2 * c + z:])
        j = torch.arange(n, device="cuda")
        i = torch.arange(m, device="cuda")[:, None] + (n - m)
        see = j <= i
        if case["window"]:
            see = see & (i - j < case["window"])
        if case["tree"]:
            word = s["tree"][at:at + m, None]
            see = see & ((j < n - m) | (((word >> (j - (n - m)).clamp(0, 63)) & 1) == 1))
        for h in range(hkv):
            k, v = (_value(part[w][:, h].reshape(-1, d // 2)[:n],
                           scal[w][:, h].contiguous().view(torch.float16).reshape(-1, d // 32)[:n],
                           d, w == 0) for w in (0, 1))
            for e in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][at:at + m, e].double() @ k.T / math.sqrt(d)
                x = torch.where(see, x, float("-inf"))
                lse[at:at + m, e] = torch.logsumexp(x, -1)
                out[at:at + m, e] = torch.softmax(x, -1) @ v
        at += m
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
