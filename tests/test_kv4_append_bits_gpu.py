"""Appending, bit for bit: q, the codes and the scales against the documented arithmetic
in numpy's fp32, where every operation rounds on its own.  Nothing is allowed to differ."""
import numpy as np
import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

F = np.float32


@pytest.fixture(scope="module")
def kv4():
    from weight_only_int4_moe_gb300 import kv4 as m
    m.load_library()
    return m


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


def norm(x, w, eps):
    """x * (1 / sqrt(sum * (1/D) + eps)) * w, the sum in the documented order."""
    d = x.shape[-1]
    y = x * x
    s = (y[..., :d // 2] + y[..., d // 2:]).reshape(x.shape[:-1] + (-1, 8))
    s = ((s[..., 0] + s[..., 4]) + (s[..., 2] + s[..., 6])) + \
        ((s[..., 1] + s[..., 5]) + (s[..., 3] + s[..., 7]))
    while s.shape[-1] > 1:
        s = s[..., 0::2] + s[..., 1::2]
    r = F(1) / np.sqrt(s * F(1.0 / d) + F(eps))
    return (x * r) * w


def rotate(x, c, s, interleaved):
    c, s = c[:, None], s[:, None]
    y = np.empty_like(x)
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    u, v = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0::2], y[..., 1::2] = u, v
    else:
        y[..., :h], y[..., h:] = u, v
    return y


def quantise(x):
    """(codes uint8 [.., D], scales fp16 [.., D / 32]) of fp32 rows."""
    g = x.reshape(x.shape[:-1] + (-1, 32))
    s = ref.bf16(np.abs(g).max(-1) * F(F(1) / F(7))).float().numpy()
    s = np.minimum(np.maximum(s, F(2.0 ** -14)), F(2720))
    q = np.clip(np.rint(g / s[..., None]), -8, 7) + 8
    assert g.dtype == F and s.dtype == F
    return q.astype(np.uint8).reshape(x.shape), s.astype(np.float16)


def held(cache, tables, lens, ps, d):
    """(K codes, V codes, K scales, V scales) of all tokens in order."""
    pool = cache.pages.cpu().numpy()[0]
    parts = [[] for _ in range(4)]
    for b, n in enumerate(lens):
        blocks = pool[tables[b, :-(-n // ps)]]
        for i, x in enumerate(ref.split(blocks, ps, d)):
            x = x.transpose(0, 2, 1, 3).reshape(-1, blocks.shape[1], x.shape[-1])[:n]
            parts[i].append(x)
    kc, vc, ks, vs = (np.concatenate(p) for p in parts)
    return ref.unpack_rows(kc, d, True), ref.unpack_rows(vc, d, False), ks, vs


def run(kv4, lens, x, hq, hkv, d, ps, qw=None, kw=None, cos=None, sin=None, positions=None,
        interleaved=False, eps=1e-6):
    n_pages = [-(-n // ps) for n in lens]
    tables = np.full((len(lens), max(n_pages)), -1, np.int32)
    at = 0
    for b, p in enumerate(n_pages):
        tables[b, :p] = np.arange(at, at + p)
        at += p
    cache = kv4.Cache.empty(1, at, hkv, d, ps)
    cu = np.concatenate([[0], np.cumsum(lens)])
    batch = kv4.Batch(ints(cu), ints(lens), ints(tables), int(cu[-1]), max(lens), max(lens))

    def dev(a):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()

    parts = [p.contiguous().cuda() for p in x.split((hq, hkv, hkv), 1)]
    w = [None if a is None else a.cuda() for a in (qw, kw)]
    got = kv4.moe_kv4_append(cache, batch, *parts, *w, dev(cos), dev(sin),
                             None if positions is None else ints(positions), eps=eps,
                             interleaved=interleaved)
    assert cache.errors() == (0, 0)
    f = [p.float().numpy() for p in x.split((hq, hkv, hkv), 1)]
    if qw is not None:
        f[0] = norm(f[0], qw.float().numpy(), eps)
        f[1] = norm(f[1], kw.float().numpy(), eps)
    if cos is not None:
        place = np.concatenate([np.arange(n) for n in lens]) if positions is None else positions
        f[:2] = [rotate(y, cos[place], sin[place], interleaved) for y in f[:2]]
    want_k, want_ks = quantise(f[1])
    want_v, want_vs = quantise(f[2])
    kc, vc, ks, vs = held(cache, tables, lens, ps, d)
    differ = {
        "q": int((got.cpu() != torch.from_numpy(f[0]).to(torch.bfloat16)).sum()),
        "k codes": int((kc != want_k).sum()), "k scales": int((ks != want_ks).sum()),
        "v codes": int((vc != want_v).sum()), "v scales": int((vs != want_vs).sum())}
    assert not any(differ.values()), differ


@pytest.mark.parametrize("d,ps,interleaved", [(128, 64, False), (128, 32, True), (64, 16, False),
                                              (64, 64, True)])
def test_norm_rotation_and_codes(kv4, d, ps, interleaved):
    rng = np.random.default_rng(d + ps)
    lens, hq, hkv = [700, 1, 300, 23], 12, 4
    t = sum(lens)
    x = ref.bf16(rng.standard_normal((t, hq + 2 * hkv, d)) *
                 np.exp(2 * rng.standard_normal((t, hq + 2 * hkv, 1))))
    assert x.numel() > 1_000_000
    qw, kw = (ref.bf16(1 + 0.3 * rng.standard_normal(d)) for _ in range(2))
    ang = np.arange(5000)[:, None] * 10000.0 ** (-np.arange(d // 2) * 2 / d)
    cos, sin = np.cos(ang).astype(F), np.sin(ang).astype(F)
    run(kv4, lens, x, hq, hkv, d, ps, qw, kw, cos, sin,
        positions=rng.integers(0, 5000, t).astype(np.int32), interleaved=interleaved)
    run(kv4, lens, x, hq, hkv, d, ps, None, None, cos, sin, interleaved=interleaved)
    run(kv4, lens, x, hq, hkv, d, ps, qw, kw)


@pytest.mark.parametrize("d,ps", [(128, 64), (64, 16)])
def test_codes_at_the_middle_between_two(kv4, d, ps):
    """Quotients at and within a few units in the last place of k + 1/2, where x * (1/s)
    and x / s can fall on different sides: the rotation's cosine makes them (x = 1,
    sine 0)."""
    rng = np.random.default_rng(d)
    t, hkv, ng = 4000, 2, d // 64  # groups of a row's half
    s = ref.bf16(np.exp(rng.uniform(-6, 5, (t, ng)))).float().numpy()
    half = rng.integers(-7, 7, (t, ng, 32)).astype(F) + F(0.5)
    y = half * s[..., None]
    off = rng.integers(-4, 5, y.shape).astype(np.int32)
    y = (y.view(np.int32) + off).view(F)
    y[..., 5] = F(7) * s  # the largest, which gives the scale s
    y[..., 6] = -F(7.49) * s * (rng.random((t, ng)) < 0.5)
    cos = y.reshape(t, d // 2)
    sin = np.zeros_like(cos)
    x = torch.ones(t, 3 * hkv, d, dtype=torch.bfloat16)
    run(kv4, [t], x, hkv, hkv, d, ps, cos=cos, sin=sin)


def test_values_exactly_between_two_codes(kv4):
    """bf16 values whose quotient is k + 1/2 exactly go to the even code."""
    rng = np.random.default_rng(9)
    t, hkv, d = 500, 2, 128
    s = 2.0 ** rng.integers(-10, 8, (t, 3 * hkv, d // 32, 1))
    y = (rng.integers(-7, 7, (t, 3 * hkv, d // 32, 32)) + 0.5) * s
    y[..., 0] = 7 * s[..., 0]
    run(kv4, [t], ref.bf16(y.reshape(t, 3 * hkv, d)), hkv, hkv, d, 32)


def test_squares_below_the_normal_numbers(kv4):
    """Rows so small that their squares lose bits before they are added, eps 0."""
    rng = np.random.default_rng(3)
    t, hq, hkv, d = 400, 4, 2, 128
    x = ref.bf16(rng.standard_normal((t, hq + 2 * hkv, d)) * 2.0 ** -68)
    w = ref.bf16(1 + 0.1 * rng.standard_normal(d))
    run(kv4, [t], x, hq, hkv, d, 64, w, w, eps=0.0)
