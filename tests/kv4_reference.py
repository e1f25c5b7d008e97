"""The 4-bit cache's operators in fp64, written from the format's description:
packing and unpacking of blocks by the place of every dimension, attention one
request and head at a time, page management as a Python model."""
import math

import numpy as np
import torch

LOG_SCALE_MIN, SCALE_MAX = -14, 2720.0


def places(d, key):
    """Bit position of every dimension's code inside its row."""
    ng = d // 32
    x = np.arange(d)
    g, r = x // 32, x % 32
    if key:
        return 32 * ((r // 8) * ng + g) + 16 * (r % 2) + 4 * ((r % 8) // 2)
    return 16 * ((r // 4) * ng + g) + 4 * (r % 4)


def pack_rows(codes, key):
    """uint8 codes [..., D] -> bytes [..., D/2]."""
    d = codes.shape[-1]
    out = np.zeros(codes.shape[:-1] + (d // 2,), np.uint8)
    for dim, bit in enumerate(places(d, key)):
        out[..., bit // 8] |= (codes[..., dim] << (bit % 8)).astype(np.uint8)
    return out


def unpack_rows(rows, d, key):
    bit = places(d, key)
    return (rows[..., bit // 8] >> (bit % 8)) & 15


def split(block, ps, d):
    """(K codes, V codes, K scales, V scales) of blocks uint8 [..., block bytes]."""
    c, s = ps * d // 2, ps * d // 16
    lead = block.shape[:-1]
    kc = block[..., :c].reshape(lead + (ps, d // 2))
    vc = block[..., c:2 * c].reshape(lead + (ps, d // 2))
    ks = np.ascontiguousarray(block[..., 2 * c:2 * c + s]).view(np.float16).reshape(lead + (ps, d // 32))
    vs = np.ascontiguousarray(block[..., 2 * c + s:]).view(np.float16).reshape(lead + (ps, d // 32))
    return kc, vc, ks, vs


def join(kc, vc, ks, vs):
    lead = kc.shape[:-2]
    flat = [kc.reshape(lead + (-1,)), vc.reshape(lead + (-1,)),
            np.ascontiguousarray(ks).view(np.uint8).reshape(lead + (-1,)),
            np.ascontiguousarray(vs).view(np.uint8).reshape(lead + (-1,))]
    return np.ascontiguousarray(np.concatenate(flat, -1))


def values(block, ps, d):
    """(K, V) fp64 [..., ps, D] of blocks."""
    kc, vc, ks, vs = split(block, ps, d)
    out = []
    for codes, scales, key in ((kc, ks, True), (vc, vs, False)):
        q = unpack_rows(codes, d, key).astype(np.float64) - 8
        out.append(q * np.repeat(scales.astype(np.float64), 32, -1))
    return out


def random_pool(rng, layers, pages, hkv, d, ps):
    """A pool of random codes and bf16 scales around 0.3."""
    shape = (layers, pages, hkv, ps)
    s = [torch.from_numpy(0.1 + 0.4 * rng.random(shape + (d // 32,))).to(torch.bfloat16)
         .to(torch.float16).numpy() for _ in range(2)]
    kc = pack_rows(rng.integers(0, 16, shape + (d,), dtype=np.uint8), True)
    vc = pack_rows(rng.integers(0, 16, shape + (d,), dtype=np.uint8), False)
    return join(kc, vc, s[0], s[1])


def visible(n, m, window, tree):
    """bool [m, n]: what each of the last m of n tokens sees."""
    j = np.arange(n)[None]
    p = (n - m + np.arange(m))[:, None]
    see = j <= p
    if window:
        see &= j > p - window
    if tree is not None:
        new = j - (n - m)
        word = np.array([int(w) & (2 ** 64 - 1) for w in tree], dtype=object)[:, None]
        bit = np.array([[new[0, c] < 0 or (int(w[0]) >> int(new[0, c])) & 1 for c in range(n)]
                        for w in word], dtype=bool).reshape(m, n)
        see &= bit
    return see


def attention(q, pool, tables, kv, cu, ps, scale, window=0, tree=None):
    """q fp64 [T, Hq, D], pool uint8 [pages, hkv, block] -> out, lse, spread
    (sum_j p_j |v_j|) and the largest |scale q.k| term sum of each row."""
    t, hq, d = q.shape
    hkv = pool.shape[1]
    out, spread = np.zeros((t, hq, d)), np.zeros((t, hq, d))
    lse, size = np.full((t, hq), -np.inf), np.zeros((t, hq))
    for b in range(len(kv)):
        n, lo, hi = int(kv[b]), int(cu[b]), int(cu[b + 1])
        m = hi - lo
        if not m or not n:
            continue
        kk, vv = values(pool[tables[b, :-(-n // ps)]], ps, d)
        see = visible(n, m, window, None if tree is None else tree[lo:hi])
        for h in range(hq):
            g = h // (hq // hkv)
            k, v = (x[:, g].reshape(-1, d)[:n] for x in (kk, vv))
            x = scale * (q[lo:hi, h] @ k.T)
            size[lo:hi, h] = (abs(scale) * (np.abs(q[lo:hi, h]) @ np.abs(k).T)).max(-1)
            x = np.where(see, x, -np.inf)
            top = x.max(-1, keepdims=True)
            e = np.where(see, np.exp(x - np.where(np.isfinite(top), top, 0)), 0)
            z = e.sum(-1)
            ok = z > 0
            p = e / np.where(ok, z, 1)[:, None]
            out[lo:hi, h] = p @ v
            spread[lo:hi, h] = p @ np.abs(v)
            with np.errstate(divide="ignore"):
                lse[lo:hi, h] = np.where(ok, top[:, 0] + np.log(z), -np.inf)
    return out, lse, spread, size


def norm_rotate(x, w, cos, sin, eps, interleaved):
    """fp64 head norm and rotation of x [T, H, D]; w, cos and sin may be None."""
    x = x.astype(np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    if cos is not None:
        c, s = cos[:, None].astype(np.float64), sin[:, None].astype(np.float64)
        y = np.empty_like(x)
        h = x.shape[-1] // 2
        a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
        u, v = a * c - b * s, b * c + a * s
        if interleaved:
            y[..., 0::2], y[..., 1::2] = u, v
        else:
            y[..., :h], y[..., h:] = u, v
        x = y
    return x


class Pages:
    """Page management as a model: tables, lens, refs and the token that every
    slot holds (any hashable; None: unwritten)."""

    def __init__(self, seqs, capacity, n_pages, ps):
        self.tables = np.full((seqs, capacity), -1, np.int32)
        self.lens = np.zeros(seqs, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.slots = [[None] * ps for _ in range(n_pages)]
        self.ps = ps

    def _take(self, n):
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        return free[:n] if len(free) >= n else None

    def reserve(self, ids, lens):
        taken = 0
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        for x, to in zip(ids, lens):
            have = -(-int(self.lens[x]) // self.ps)
            need = -(-int(to) // self.ps) - have
            if taken + need <= len(free):
                got = free[taken:taken + need]
                self.tables[x, have:have + need] = got
                self.refs[got] = 1
                self.lens[x] = to
            taken += need

    def fork(self, parents, children):
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        taken = 0
        for x, c in zip(parents, children):
            n = int(self.lens[x])
            full, part = divmod(n, self.ps)
            if part and taken + 1 > len(free):
                taken += 1
                continue
            row = self.tables[x, :full]
            self.tables[c, :full] = row
            np.add.at(self.refs, row, 1)
            if part:
                page = free[taken]
                taken += 1
                self.tables[c, full] = page
                self.refs[page] = 1
                self.slots[page][:part] = self.slots[int(self.tables[x, full])][:part]
            self.lens[c] = n

    def free(self, ids):
        for x in ids:
            n = -(-int(self.lens[x]) // self.ps)
            np.add.at(self.refs, self.tables[x, :n], -1)
            self.tables[x, :n] = -1
            self.lens[x] = 0

    def compact(self):
        used = int((self.refs > 0).sum())
        src = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(used) if self.refs[p] == 0]
        to = {s: t for s, t in zip(src, dst)}
        for s, t in to.items():
            self.slots[t] = list(self.slots[s])
            self.refs[t], self.refs[s] = self.refs[s], 0
        self.tables = np.vectorize(lambda p: to.get(int(p), int(p)), otypes=[np.int32])(self.tables)
        return used


def bf16(x):
    """fp64 or fp32 array -> the torch bf16 tensor."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def default_scale(d):
    return 1.0 / math.sqrt(d)
