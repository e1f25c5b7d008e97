"""The 4-bit cache on a GPU against fp64: appending, reading, attention, pages.

Tolerances are bounds, derived here before any run:
 - a bf16 output is within half an ulp of its exact value, 2^-8 |y| (2^-7 is the
   spacing), plus what precedes the rounding;
 - attention rounds each unnormalised probability p <= 1 to fp16: at most 2^-11 p,
   or 2^-25 below fp16's normals, so out moves by at most (2^-11 + the same again
   for scores off by 2^-12) * sum p|v| and by n 2^-25 max|v| over the row's sum
   (>= 1); scores are sums of D exact products in fp32, off by at most D 2^-23
   times their sum of magnitudes (1e-5 of it covers D = 128).
"""
import numpy as np
import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

HUGE = 1 << 30


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def make_batch(kv4, kv, q, tables):
    cu = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    b = kv4.Batch(cuda(cu), cuda(np.asarray(kv, np.int32)), cuda(tables), int(cu[-1]),
                  max(list(q) + [0]), max(list(kv) + [0]))
    return b, cu


def make_tables(rng, kv, ps, pages, extra=1):
    """Page tables over a random order of the pages; unused entries are junk."""
    n = [-(-int(x) // ps) for x in kv]
    assert sum(n) <= pages
    order = rng.permutation(pages).astype(np.int32)
    t = np.full((len(kv), max(n + [0]) + extra), -7, np.int32)
    at = 0
    for b, m in enumerate(n):
        t[b, :m] = order[at:at + m]
        at += m
    return t


def poison(pool, tables, kv, ps, d):
    """NaN scales in every slot that holds no token of its sequence."""
    used = np.zeros((pool.shape[0], ps), bool)
    for b, n in enumerate(kv):
        for j in range(-(-int(n) // ps)):
            used[tables[b, j], :min(ps, int(n) - j * ps)] = True
    kc, vc, ks, vs = ref.split(pool, ps, d)
    for s in (ks, vs):
        s[np.broadcast_to(~used[:, None, :, None], s.shape)] = np.nan
    return ref.join(kc, vc, ks, vs)


def check_attention(kv4, rng, kv, ql, hkv, group, d, ps, window=0, tree=False, scale=None,
                    spread_q=2.0, extra_pages=3, wide_q=False):
    pages = sum(-(-int(x) // ps) for x in kv) + extra_pages
    pool = ref.random_pool(rng, 1, pages, hkv, d, ps)[0]
    tables = make_tables(rng, kv, ps, pages)
    pool = poison(pool, tables, kv, ps, d)
    cache = kv4.Cache(cuda(pool[None]), hkv, d, ps)
    batch, cu = make_batch(kv4, kv, ql, tables)
    t, hq = int(cu[-1]), hkv * group
    q = ref.bf16(spread_q * rng.standard_normal((t, hq, d)))
    words = None
    if tree:
        words = rng.integers(0, 2 ** 63, t, dtype=np.int64) & rng.integers(-2 ** 63, 2 ** 63 - 1, t,
                                                                         dtype=np.int64)
        words[::5] = 0  # rows that see none of the new tokens
    scale = ref.default_scale(d) if scale is None else scale
    want, lse, spread, size = ref.attention(q.double().numpy(), pool, tables, kv, cu, ps, scale,
                                            window, words)
    if wide_q:  # the query heads as a part of a wider projection
        wide = torch.zeros(t, (hq + 2) * d, dtype=torch.bfloat16).cuda()
        wide[:, d:-d] = q.cuda().flatten(1)
        qd = wide[:, d:-d].unflatten(1, (hq, d))
    else:
        qd = q.cuda()
    ws = kv4.alloc_workspace(cache, batch, hq)
    args = dict(scale=scale, window=window, tree=None if words is None else cuda(words),
                return_lse=True, workspace=ws)
    out, got_lse = kv4.moe_kv4_attention(qd, cache, batch, **args)
    again, again_lse = kv4.moe_kv4_attention(qd, cache, batch, **args)
    torch.cuda.synchronize()
    head = ws[:kv4.MOE_KV4_WS_HEADER].cpu()
    assert not head.any(), "the workspace header is not as it was, or an error was reported"
    assert torch.equal(out, again) and torch.equal(got_lse, again_lse)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    n = max(list(kv) + [1])
    vmax = 8 * 0.5
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12 + 2e-5 * size[..., None]) * spread \
        + n * 2.0 ** -25 * vmax + 1e-30
    worst = np.max(np.abs(got - want) / tol) if got.size else 0.0
    assert worst <= 1.0, f"{worst} of the bound"
    got_lse = got_lse.double().cpu().numpy()
    empty = np.isneginf(lse)
    assert np.array_equal(empty, np.isneginf(got_lse))
    assert not np.any(got[empty])
    assert np.all(np.abs(got_lse - lse)[~empty] <= (1e-5 * size + 2e-6 * (1 + np.abs(lse)))[~empty])


@pytest.fixture(scope="module")
def kv4():
    from weight_only_int4_moe_gb300 import kv4 as m
    m.load_library()
    return m


# ---------------------------------------------------------------- attention --
LENGTHS = [[1], [2], [15], [16], [17], [31], [32], [33], [63], [64], [65], [127], [128], [129],
           [200], [513], [1000], [4097]]


@pytest.mark.parametrize("kv", LENGTHS, ids=lambda v: str(v[0]))
@pytest.mark.parametrize("d,ps", [(128, 64), (64, 16), (128, 32), (128, 16), (64, 64)])
def test_decode_lengths(kv4, kv, d, ps):
    rng = np.random.default_rng(kv[0] * 7 + d + ps)
    check_attention(kv4, rng, kv, [1], 2, 7, d, ps)


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 9, 16, 33, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_groups(kv4, group, d):
    rng = np.random.default_rng(group)
    check_attention(kv4, rng, [130, 1, 77], [1, 1, 1], 2, group, d, 32)


@pytest.mark.parametrize("hkv,group,d,ps", [(8, 7, 128, 64), (1, 8, 128, 64), (16, 1, 64, 16),
                                            (3, 4, 64, 32)])
def test_ragged_decode(kv4, hkv, group, d, ps):
    rng = np.random.default_rng(3)
    kv = [int(x) for x in rng.integers(1, 700, 37)]
    kv[5] = 0
    ql = [1] * 37
    ql[5] = ql[11] = 0  # requests with no tokens, and with no new ones
    check_attention(kv4, rng, kv, ql, hkv, group, d, ps)


@pytest.mark.parametrize("m", [2, 3, 5, 8, 9, 15, 16, 17, 33, 64])
@pytest.mark.parametrize("hkv,group,d,ps", [(2, 7, 128, 64), (4, 1, 64, 16), (1, 8, 128, 32)])
def test_verify_and_tree(kv4, m, hkv, group, d, ps):
    rng = np.random.default_rng(m)
    kv = [m, m + 1, m + 63, 300 + m, 129]
    ql = [m, m, m, m, min(m, 2)]
    check_attention(kv4, rng, kv, ql, hkv, group, d, ps)
    check_attention(kv4, rng, kv, ql, hkv, group, d, ps, tree=True)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200])
@pytest.mark.parametrize("d,ps", [(128, 64), (64, 16)])
def test_window(kv4, window, d, ps):
    rng = np.random.default_rng(window)
    check_attention(kv4, rng, [400, 65, 3, 900], [1, 1, 1, 1], 2, 4, d, ps, window=window)
    check_attention(kv4, rng, [400, 65, 130], [150, 65, 9], 2, 4, d, ps, window=window)
    check_attention(kv4, rng, [90, 70], [9, 33], 2, 3, d, ps, window=window, tree=True)


@pytest.mark.parametrize("m", [65, 100, 127, 128, 129, 255, 300, 600])
@pytest.mark.parametrize("hkv,group,d,ps", [(2, 7, 128, 64), (2, 1, 128, 32), (1, 8, 64, 16),
                                            (2, 4, 64, 64)])
def test_prompts(kv4, m, hkv, group, d, ps):
    rng = np.random.default_rng(m)
    check_attention(kv4, rng, [m, m + 77, m], [m, m, 1], hkv, group, d, ps, wide_q=True)


def test_prompt_beside_single_tokens(kv4):
    rng = np.random.default_rng(8)
    check_attention(kv4, rng, [700, 1, 900, 0, 64, 333], [513, 1, 1, 0, 64, 2], 4, 4, 128, 64)
    check_attention(kv4, rng, [700, 1, 900, 0, 64, 333], [513, 1, 1, 0, 64, 2], 4, 4, 64, 16,
                    window=100)


@pytest.mark.parametrize("m", [1, 5, 200])
def test_more_new_tokens_than_the_length(kv4, m):
    """The surplus first tokens see nothing: zeros and -inf."""
    rng = np.random.default_rng(1)
    hkv, d, ps = 2, 128, 64
    pool = ref.random_pool(rng, 1, 8, hkv, d, ps)[0]
    tables = np.arange(8, dtype=np.int32).reshape(1, 8)
    cache = kv4.Cache(cuda(pool[None]), hkv, d, ps)
    kv = m // 2
    batch, cu = make_batch(kv4, [kv], [m], tables)
    q = ref.bf16(rng.standard_normal((m, 6, d)))
    out, lse = kv4.moe_kv4_attention(q.cuda(), cache, batch, return_lse=True)
    out, lse = out.cpu(), lse.cpu()
    assert not out[:m - kv].any() and torch.isneginf(lse[:m - kv]).all()
    if kv:
        want, _, spread, _ = ref.attention(q[m - kv:].double().numpy(), pool, tables, [kv], [0, kv],
                                           ps, ref.default_scale(d))
        assert np.all(np.abs(out[m - kv:].double().numpy() - want) <= 2.0 ** -8 * np.abs(want)
                      + 2.0 ** -9 * spread + 1e-4)


@pytest.mark.parametrize("spread_q,scale", [(2.0, 0.0), (2.0, -0.05), (40.0, 1.0), (1e-3, 3.0)])
def test_flat_and_peaked_scores(kv4, spread_q, scale):
    """No scale, a negative one, and scores of several hundred, where one token wins."""
    rng = np.random.default_rng(2)
    check_attention(kv4, rng, [500, 70, 200], [1, 70, 3], 2, 4, 128, 64, scale=scale,
                    spread_q=spread_q)


def test_zero_scales_and_ties(kv4):
    """Equal scores everywhere average the values."""
    rng = np.random.default_rng(4)
    hkv, d, ps, n = 1, 64, 16, 48
    kc = ref.pack_rows(np.full((3, hkv, ps, d), 8, np.uint8), True)
    codes = rng.integers(0, 16, (3, hkv, ps, d), dtype=np.uint8)
    one = np.ones((3, hkv, ps, d // 32), np.float16)
    pool = ref.join(kc, ref.pack_rows(codes, False), one, one)
    cache = kv4.Cache(cuda(pool[None]), hkv, d, ps)
    batch, _ = make_batch(kv4, [n], [1], np.arange(3, dtype=np.int32)[None])
    q = ref.bf16(rng.standard_normal((1, 4, d)))
    out = kv4.moe_kv4_attention(q.cuda(), cache, batch).double().cpu().numpy()
    want = (codes.astype(np.float64) - 8).reshape(n, d).mean(0)
    assert np.all(np.abs(out - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * 8)


def test_pages_beyond_4_gib(kv4):
    """Page offsets are 64-bit: the last pages of a 5 GB pool."""
    rng = np.random.default_rng(5)
    hkv, d, ps, pages = 8, 128, 64, 70000
    n = 150
    small = ref.random_pool(rng, 1, 3, hkv, d, ps)[0]
    cache = kv4.Cache.empty(1, pages, hkv, d, ps)
    assert cache.pages.numel() > 1 << 32
    ids = np.array([[pages - 1, 65000, pages - 2]], np.int32)
    for i, p in enumerate(ids[0]):
        cache.pages[0, int(p)] = cuda(small[i])
    batch, cu = make_batch(kv4, [n], [1], ids)
    q = ref.bf16(rng.standard_normal((1, hkv * 4, d)))
    out = kv4.moe_kv4_attention(q.cuda(), cache, batch).double().cpu().numpy()
    want, _, spread, _ = ref.attention(q.double().numpy(), small, np.arange(3)[None], [n], cu, ps,
                                       ref.default_scale(d))
    assert np.all(np.abs(out - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * spread + 1e-4)
    # and written there
    k = ref.bf16(rng.standard_normal((1, hkv, d))).cuda()
    kv4.moe_kv4_append(cache, batch, None, k, k)
    back, _ = kv4.moe_kv4_read(cache, batch)
    assert torch.all((back.float() - k.float()).abs() <= 0.3)
    assert cache.errors() == (0, 0)


def test_long_context(kv4):
    rng = np.random.default_rng(6)
    check_attention(kv4, rng, [70001, 12], [1, 1], 1, 8, 128, 64)
    check_attention(kv4, rng, [20001], [9], 2, 4, 64, 32)


def test_bad_pages_are_skipped_and_reported(kv4):
    rng = np.random.default_rng(7)
    hkv, d, ps = 2, 128, 64
    pool = ref.random_pool(rng, 1, 4, hkv, d, ps)[0]
    cache = kv4.Cache(cuda(pool[None]), hkv, d, ps)
    for m in (1, 40):
        kv = 250
        tables = np.array([[0, 99, 2, 3]], np.int32)
        batch, cu = make_batch(kv4, [kv], [m], tables)
        q = ref.bf16(rng.standard_normal((m, 4, d)))
        ws = kv4.alloc_workspace(cache, batch, 4)
        out = kv4.moe_kv4_attention(q.cuda(), cache, batch, workspace=ws).double().cpu().numpy()
        flags, count = ws[:8].view(torch.int32).tolist()
        assert flags == kv4.MOE_KV4_DEVERR_PAGE and count > 0
        assert np.isfinite(out).all()
        # the same with the bad page's tokens left out
        _, vv = ref.values(pool, ps, d)
        kk, _ = ref.values(pool, ps, d)
        keep = np.r_[0:64, 128:250]
        for h in range(4):
            k, v = (x[:, h // 2].reshape(-1, d)[:kv] for x in (kk, vv))
            for i in range(m):
                see = keep[keep <= kv - m + i]
                x = (q[i, h].double().numpy() @ k[see].T) * ref.default_scale(d)
                p = np.exp(x - x.max())
                p /= p.sum()
                want, spread = p @ v[see], p @ np.abs(v[see])
                assert np.all(np.abs(out[i, h] - want) <= 2.0 ** -8 * np.abs(want)
                              + 2.0 ** -10 * spread + 1e-4)
    # a length beyond the table
    batch, cu = make_batch(kv4, [400], [1], np.array([[0, 1, 2, 3]], np.int32))
    ws = kv4.alloc_workspace(cache, batch, 4)
    out = kv4.moe_kv4_attention(q[:1].cuda(), cache, batch, workspace=ws)
    assert torch.isfinite(out).all()
    assert ws[:8].view(torch.int32).tolist()[0] == kv4.MOE_KV4_DEVERR_PAGE


def test_queries_out_of_range_are_reported(kv4):
    rng = np.random.default_rng(9)
    cache = kv4.Cache(cuda(ref.random_pool(rng, 1, 4, 2, 128, 64)), 2, 128, 64)
    for m in (1, 70):
        batch, _ = make_batch(kv4, [200], [m], np.arange(4, dtype=np.int32)[None])
        q = torch.zeros(m, 4, 128, dtype=torch.bfloat16).cuda()
        q[m // 2, 1, 5] = 1e6
        ws = kv4.alloc_workspace(cache, batch, 4)
        out = kv4.moe_kv4_attention(q, cache, batch, workspace=ws)
        assert torch.isfinite(out).all()
        assert ws[:8].view(torch.int32).tolist()[0] == kv4.MOE_KV4_DEVERR_RANGE


def test_streams_and_graphs(kv4):
    """On a stream other than the current one, and replayed from a CUDA graph whose
    lengths change between replays."""
    rng = np.random.default_rng(10)
    hkv, d, ps, group = 2, 128, 64, 4
    pool = ref.random_pool(rng, 1, 40, hkv, d, ps)[0]
    tables = rng.permutation(40).astype(np.int32).reshape(4, 10)
    cache = kv4.Cache(cuda(pool[None]), hkv, d, ps)
    kv = np.array([640, 3, 100, 65], np.int32)
    batch, cu = make_batch(kv4, kv, [1] * 4, tables)
    q = ref.bf16(rng.standard_normal((4, hkv * group, d)))
    qd = torch.zeros_like(q).cuda()
    ws = kv4.alloc_workspace(cache, batch, hkv * group)
    out = torch.empty_like(qd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv4.moe_kv4_attention(qd, cache, batch, out=out, workspace=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv4.moe_kv4_attention(qd, cache, batch, out=out, workspace=ws)
    qd.copy_(q)
    for n in ([640, 3, 100, 65], [1, 640, 64, 63], [129, 128, 127, 500]):
        batch.kv_len.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want, _, spread, _ = ref.attention(q.double().numpy(), pool, tables, n, cu, ps,
                                           ref.default_scale(d))
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * spread + 1e-4)


def test_binding_refusals(kv4):
    cache = kv4.Cache.empty(1, 4, 2, 64, 16)
    batch, _ = make_batch(kv4, [20], [1], np.arange(2, dtype=np.int32)[None])
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16).cuda()
    with pytest.raises(TypeError):
        kv4.moe_kv4_attention(q.float(), cache, batch)
    with pytest.raises(ValueError):
        kv4.moe_kv4_attention(q[:, :, :32], cache, batch)
    with pytest.raises(ValueError):
        kv4.moe_kv4_attention(q.cpu(), cache, batch)
    with pytest.raises(ValueError):
        kv4.moe_kv4_attention(q[:, :3].contiguous(), cache, batch)  # 3 heads over 2
    with pytest.raises(ValueError):
        kv4.moe_kv4_attention(torch.zeros(1, 8, 64, dtype=torch.bfloat16).cuda()[:, ::2], cache,
                              batch)  # heads apart
    with pytest.raises(ValueError):
        kv4.moe_kv4_attention(q, cache, batch, out=torch.zeros(1, 4, 64).cuda())
    with pytest.raises(RuntimeError):
        kv4.moe_kv4_attention(q, cache, batch, window=-1)
    with pytest.raises(RuntimeError):
        kv4.moe_kv4_attention(q, cache, batch, workspace=torch.zeros(64, dtype=torch.uint8).cuda())
    with pytest.raises(ValueError):
        kv4.Cache(torch.zeros(1, 4, 2, 100, dtype=torch.uint8).cuda(), 2, 64, 16)
    with pytest.raises(TypeError):
        kv4.Batch(batch.cu_q.long(), batch.kv_len, batch.tables, 1, 1, 20)
    with pytest.raises(ValueError):
        kv4.Batch(batch.cu_q, batch.kv_len, batch.tables, 5, 1, 20)
    with pytest.raises(ValueError):
        kv4.moe_kv4_append(cache, batch, q, q, q)  # 4 heads where the pool has 2
    k = q[:, :2].contiguous()
    with pytest.raises(ValueError):
        kv4.moe_kv4_append(cache, batch, q, k, k, cos=torch.zeros(9, 32).cuda())
    seqs = kv4.Sequences.empty(2, 4, 5)
    with pytest.raises(ValueError):
        kv4.moe_kv4_free(cache, seqs, torch.zeros(1, dtype=torch.int32).cuda())


# ------------------------------------------------------------ append, read --
def append_case(kv4, rng, kv, ql, hq, hkv, d, ps, norm=True, rotate=True, interleaved=False,
                positions=True, wide=False, with_q=True, layer=0, layers=1):
    pages = sum(-(-int(x) // ps) for x in kv) + 2
    pool = rng.integers(0, 256, (layers, pages, hkv, kv4.block_bytes(d, ps)), dtype=np.uint8)
    tables = make_tables(rng, kv, ps, pages)
    cache = kv4.Cache(cuda(pool), hkv, d, ps)
    batch, cu = make_batch(kv4, kv, ql, tables)
    t = int(cu[-1])
    x = ref.bf16(rng.standard_normal((t, hq + 2 * hkv, d)) * np.exp(rng.standard_normal((t, hq + 2 * hkv, 1))))
    if wide:
        buf = torch.zeros(t, (hq + 2 * hkv) * d + 16, dtype=torch.bfloat16).cuda()
        buf[:, 8:-8] = x.cuda().flatten(1)
        parts = buf[:, 8:-8].unflatten(1, (hq + 2 * hkv, d)).split((hq, hkv, hkv), 1)
    else:
        parts = [p.contiguous().cuda() for p in x.split((hq, hkv, hkv), 1)]
    qw, kw = (ref.bf16(1 + 0.2 * rng.standard_normal(d)) for _ in range(2))
    place = np.concatenate([np.arange(n - m, n) for n, m in zip(kv, ql)]) if t else np.zeros(0, int)
    pos = rng.integers(0, 5000, t).astype(np.int32) if positions else place.astype(np.int32)
    ang = np.arange(5000)[:, None] * 10000.0 ** (-np.arange(d // 2) * 2 / d)
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    got = kv4.moe_kv4_append(
        cache, batch, parts[0] if with_q else None, parts[1], parts[2],
        qw.cuda() if norm else None, kw.cuda() if norm else None,
        cuda(cos) if rotate else None, cuda(sin) if rotate else None,
        cuda(pos) if positions and rotate else None, interleaved=interleaved, layer=layer)
    assert cache.errors() == (0, 0)
    if rotate:
        c, s = cos[np.clip(pos, 0, 4999)], sin[np.clip(pos, 0, 4999)]
    else:
        c = s = None
    xs = [p.double().numpy() for p in x.split((hq, hkv, hkv), 1)]
    want_q = ref.norm_rotate(xs[0], qw.double().numpy() if norm else None, c, s, 1e-6, interleaved)
    want_k = ref.norm_rotate(xs[1], kw.double().numpy() if norm else None, c, s, 1e-6, interleaved)
    # fp32 arithmetic on values up to a few times the largest: 2^-20 of the head's largest
    slack_q = 2.0 ** -20 * np.abs(want_q).max(-1, keepdims=True) if t else 0
    if with_q:
        assert np.all(np.abs(got.double().cpu().numpy() - want_q) <= 2.0 ** -8 * np.abs(want_q)
                      + slack_q)
    else:
        assert got is None
    after = cache.pages.cpu().numpy()
    # nothing but the batch's slots of the layer changed
    mask = np.zeros((layers, pages, hkv, ps), bool)
    for b in range(len(kv)):
        for j in range(max(0, kv[b] - ql[b]), kv[b]):
            mask[layer, tables[b, j // ps], :, j % ps] = True
    for a, b in zip(ref.split(after, ps, d), ref.split(pool, ps, d)):
        same = (a.view(np.uint16) if a.dtype == np.float16 else a) == \
            (b.view(np.uint16) if b.dtype == np.float16 else b)
        assert same[~mask].all()
    kc, vc, ks, vs = ref.split(after, ps, d)
    for b in range(len(kv)):
        for i in range(ql[b]):
            j, r = kv[b] - ql[b] + i, int(cu[b]) + i
            page, slot = tables[b, j // ps], j % ps
            for codes, scales, key, want in ((kc, ks, True, want_k[r]), (vc, vs, False, xs[2][r])):
                code = ref.unpack_rows(codes[layer, page, :, slot], d, key).astype(np.float64) - 8
                sc = scales[layer, page, :, slot].astype(np.float64)
                g = np.abs(want).reshape(hkv, -1, 32).max(-1)
                # a bf16 of amax / 7, within the format's range
                assert np.all(np.abs(sc - np.clip(g / 7, 2.0 ** -14, 2720)) <= 2.0 ** -8 * sc)
                step = np.repeat(sc, 32, -1)
                # half a step, and what fp32 arithmetic before it may have moved
                assert np.all(np.abs(code * step - want) <= step * (0.5 + 2.0 ** -8 * 7)
                              + 2.0 ** -19 * np.abs(want).max())
    return cache, batch


@pytest.mark.parametrize("d,ps", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_append(kv4, d, ps, interleaved, wide):
    rng = np.random.default_rng(d + ps)
    append_case(kv4, rng, [1, 70, 0, 129, 64, 17], [1, 3, 0, 129, 1, 0], 7, 1, d, ps,
                interleaved=interleaved, wide=wide)
    append_case(kv4, rng, [5], [1], 6, 3, d, ps, interleaved=interleaved, wide=wide)


@pytest.mark.parametrize("norm,rotate,positions,with_q", [
    (False, True, True, True), (True, False, False, True), (False, False, False, True),
    (True, True, False, True), (True, True, True, False), (False, False, False, False)])
def test_append_parts(kv4, norm, rotate, positions, with_q):
    rng = np.random.default_rng(11)
    append_case(kv4, rng, [40, 9, 64], [1, 9, 30], 5, 5, 128, 32, norm=norm, rotate=rotate,
                positions=positions, with_q=with_q, layer=2, layers=4)


def test_append_in_place_and_read(kv4):
    """q_out may be q; reading returns what the slots hold, and whole sequences."""
    rng = np.random.default_rng(12)
    cache, batch = append_case(kv4, rng, [40, 65, 3], [40, 65, 3], 4, 2, 128, 32)
    k, v = kv4.moe_kv4_read(cache, batch)
    pool = cache.pages.cpu().numpy()[0]
    kk, vv = ref.values(pool, 32, 128)
    tables, at = batch.tables.cpu().numpy(), 0
    for b, n in enumerate([40, 65, 3]):
        for j in range(n):
            page, slot = tables[b, j // 32], j % 32
            assert np.array_equal(k[at].cpu().numpy(), kk[page, :, slot])
            assert np.array_equal(v[at].cpu().numpy(), vv[page, :, slot])
            at += 1
    q = ref.bf16(rng.standard_normal((108, 4, 128))).cuda()
    w = ref.bf16(1 + 0.1 * rng.standard_normal(128)).cuda()
    kx = ref.bf16(rng.standard_normal((108, 2, 128))).cuda()
    other = kv4.moe_kv4_append(cache, batch, q.clone(), kx, kx, q_weight=w)
    same = kv4.moe_kv4_append(cache, batch, q, kx, kx, q_weight=w, q_out=q)
    assert same is q and torch.equal(q, other)


def test_append_values_that_do_not_fit(kv4):
    """Infinities and large values saturate, NaN becomes 0, tiny groups keep the
    smallest scale; all but the last are reported, and the pool holds numbers."""
    hkv, d, ps = 1, 64, 16
    cache = kv4.Cache(torch.full((1, 2, hkv, kv4.block_bytes(d, ps)), 255, dtype=torch.uint8).cuda(),
                      hkv, d, ps)
    batch, _ = make_batch(kv4, [6], [6], np.array([[1]], np.int32))
    x = torch.zeros(6, hkv, d)
    x[0, 0, 3] = float("inf")
    x[1, 0, 40] = -float("inf")
    x[2, 0, 7] = float("nan")
    x[3, 0, 0], x[3, 0, 1] = 1e30, -5.0
    x[4, 0, 2] = 3e-6
    x[5] = 1.0
    x = x.to(torch.bfloat16).cuda()
    kv4.moe_kv4_append(cache, batch, None, x, x)
    k, v = kv4.moe_kv4_read(cache, batch)
    assert torch.equal(k, v)
    assert k[0, 0, 3] == 19040 and k[1, 0, 40] == -19040 and k[3, 0, 0] == 19040
    assert k[2, 0, 7] == 0 and not k[2].any() and not k[4].any()
    want = torch.tensor(1 / 7).to(torch.bfloat16).float() * 7
    assert torch.all(k[5].float() == want)
    flags, count = cache.errors()
    assert flags == kv4.MOE_KV4_DEVERR_RANGE and count > 0
    cache.clear_errors()
    assert cache.errors() == (0, 0)
    # and attention over them is finite
    out = kv4.moe_kv4_attention(torch.ones(6, 4, d, dtype=torch.bfloat16).cuda() * 0.01, cache,
                                batch)
    assert torch.isfinite(out).all()


def test_append_bad_pages_and_positions(kv4):
    hkv, d, ps = 2, 128, 16
    pool = torch.full((1, 4, hkv, kv4.block_bytes(d, ps)), 7, dtype=torch.uint8).cuda()
    cache = kv4.Cache(pool, hkv, d, ps)
    before = pool.clone()
    batch, _ = make_batch(kv4, [33, 17], [1, 1], np.array([[0, 1, -1], [4, 1 << 30, 2]], np.int32))
    x = torch.ones(2, hkv, d, dtype=torch.bfloat16).cuda()
    kv4.moe_kv4_append(cache, batch, None, x, x)
    assert torch.equal(cache.pages, before)
    assert cache.errors()[0] == kv4.MOE_KV4_DEVERR_PAGE
    k, _ = kv4.moe_kv4_read(cache, batch)
    assert not k.any()
    cache.clear_errors()
    batch, _ = make_batch(kv4, [1, 2], [1, 2], np.array([[0], [1]], np.int32))
    x = torch.ones(3, hkv, d, dtype=torch.bfloat16).cuda()
    c, s = torch.ones(8, d // 2).cuda(), torch.zeros(8, d // 2).cuda()
    q = kv4.moe_kv4_append(cache, batch, x, x, x, cos=c, sin=s,
                           positions=torch.tensor([-1, 8, 7], dtype=torch.int32).cuda())
    assert cache.errors()[0] == kv4.MOE_KV4_DEVERR_POSITION
    assert torch.equal(q, x)


# -------------------------------------------------------------------- pages --
@pytest.mark.parametrize("seed", range(6))
def test_page_calls_follow_the_model(kv4, seed):
    """Random reserves, forks, frees and compactions against the model; every slot
    keeps the token that was written to it, in every layer and head."""
    rng = np.random.default_rng(seed)
    ps = [16, 32, 64][seed % 3]
    d = [64, 128][seed % 2]
    layers, hkv, n_pages, seqs, cap = 2, 3, 90, 12, 11
    cache = kv4.Cache.empty(layers, n_pages, hkv, d, ps)
    cache.pages.zero_()
    s = kv4.Sequences.empty(seqs, cap, n_pages)
    model = ref.Pages(seqs, cap, n_pages, ps)
    token = 1

    def ids(v):
        return torch.tensor(np.asarray(v, np.int32), dtype=torch.int32).cuda()

    def write(x, lo, hi):
        """Tokens lo..hi-1 of sequence x get values of their own."""
        nonlocal token
        if hi <= lo:
            return
        n = hi - lo
        marks = np.arange(token, token + n)
        token += n
        batch, _ = make_batch(kv4, [hi], [n], s.tables[x:x + 1].cpu().numpy())
        for layer in range(layers):
            k = np.zeros((n, hkv, d), np.float32)
            # 7, 6, .. of 7 steps: exact codes that spell the mark, layer and head
            for g in range(hkv):
                for bit in range(12):
                    k[:, g, bit] = 7.0 * ((marks >> bit) & 1)
                k[:, g, 12], k[:, g, 13], k[:, g, 31] = layer, g, 7.0
            kv4.moe_kv4_append(cache, batch, None, cuda(k).to(torch.bfloat16),
                               cuda(-k).to(torch.bfloat16), layer=layer)
        for i, m in enumerate(marks):
            page = model.tables[x, (lo + i) // ps]
            model.slots[page][(lo + i) % ps] = int(m)

    for step in range(30):
        op = rng.choice(["reserve", "fork", "free", "compact"])
        if op == "reserve":
            pick = rng.permutation(seqs)[:rng.integers(1, 5)]
            to = [min(cap * ps, int(model.lens[x]) + int(rng.integers(0, 3 * ps))) for x in pick]
            old = model.lens.copy()
            kv4.moe_kv4_reserve(cache, s, ids(pick), ids(to))
            model.reserve(pick, to)
            for x in pick:
                if model.lens[x] > old[x]:
                    write(int(x), int(old[x]), int(model.lens[x]))
        elif op == "fork":
            empty = [x for x in range(seqs) if model.lens[x] == 0]
            full = [x for x in range(seqs) if model.lens[x] > 0]
            if not empty or not full:
                continue
            kids = empty[:rng.integers(1, len(empty) + 1)]
            par = [full[rng.integers(len(full))] for _ in kids]
            kv4.moe_kv4_fork(cache, s, ids(par), ids(kids))
            model.fork(par, kids)
        elif op == "free":
            pick = rng.permutation(seqs)[:rng.integers(1, 6)]
            kv4.moe_kv4_free(cache, s, ids(pick))
            model.free(pick)
        else:
            if rng.random() < 0.5:
                t, r = torch.empty_like(s.tables), torch.empty_like(s.refs)
                n = kv4.moe_kv4_compact(cache, s, tables_out=t, refs_out=r)
                s.tables.copy_(t)
                s.refs.copy_(r)
            else:
                n = kv4.moe_kv4_compact(cache, s)
            assert int(n) == model.compact()
        assert np.array_equal(s.tables.cpu().numpy(), model.tables), (step, op)
        assert np.array_equal(s.lens.cpu().numpy(), model.lens), (step, op)
        assert np.array_equal(s.refs.cpu().numpy(), model.refs), (step, op)
    flags = cache.errors()[0]
    assert flags & ~kv4.MOE_KV4_DEVERR_NO_PAGES == 0
    lens = model.lens
    assert lens.sum() > 0
    batch, _ = make_batch(kv4, lens, lens, model.tables)
    for layer in range(layers):
        k, v = (x.float().cpu().numpy() for x in kv4.moe_kv4_read(cache, batch, layer=layer))
        assert np.array_equal(k, -v)
        at = 0
        for x in range(seqs):
            for j in range(int(lens[x])):
                mark = model.slots[model.tables[x, j // ps]][j % ps]
                for g in range(hkv):
                    bits = sum(1 << b for b in range(12) if k[at, g, b] > 3.5)
                    assert bits == mark and k[at, g, 12] == layer and k[at, g, 13] == g
                at += 1


def test_page_faults_of_the_caller(kv4):
    cache = kv4.Cache.empty(1, 6, 1, 64, 16)
    s = kv4.Sequences.empty(4, 4, 6)

    def ids(*v):
        return torch.tensor(v, dtype=torch.int32).cuda()

    def state():
        return s.tables.tolist(), s.lens.tolist(), s.refs.tolist()

    kv4.moe_kv4_reserve(cache, s, ids(0, 1), ids(40, 16))
    assert s.refs.tolist() == [1, 1, 1, 1, 0, 0]
    assert s.tables.tolist()[0] == [0, 1, 2, -1] and s.tables.tolist()[1][0] == 3
    before = state()
    for call in (lambda: kv4.moe_kv4_reserve(cache, s, ids(4), ids(5)),      # no such sequence
                 lambda: kv4.moe_kv4_reserve(cache, s, ids(-1), ids(5)),
                 lambda: kv4.moe_kv4_reserve(cache, s, ids(0), ids(39)),     # shrinks
                 lambda: kv4.moe_kv4_reserve(cache, s, ids(0), ids(65)),     # beyond its table
                 lambda: kv4.moe_kv4_fork(cache, s, ids(0), ids(1)),         # not empty
                 lambda: kv4.moe_kv4_fork(cache, s, ids(2), ids(2)),         # itself
                 lambda: kv4.moe_kv4_fork(cache, s, ids(9), ids(2)),
                 lambda: kv4.moe_kv4_free(cache, s, ids(7))):
        call()
        assert cache.errors() == (kv4.MOE_KV4_DEVERR_SEQ, 1)
        assert state() == before
        cache.clear_errors()
    # too few pages: the first request that does not fit and all after it are refused
    kv4.moe_kv4_reserve(cache, s, ids(2, 3, 1), ids(16, 33, 20))
    assert cache.errors() == (kv4.MOE_KV4_DEVERR_NO_PAGES, 2)
    assert s.lens.tolist() == [40, 16, 16, 0] and s.refs.tolist() == [1, 1, 1, 1, 1, 0]
    cache.clear_errors()
    kv4.moe_kv4_reserve(cache, s, ids(1), ids(20))
    kv4.moe_kv4_fork(cache, s, ids(0), ids(3))  # its begun page finds none free
    assert cache.errors() == (kv4.MOE_KV4_DEVERR_NO_PAGES, 1)
    assert s.lens.tolist() == [40, 20, 16, 0] and s.refs.tolist() == [1] * 6
    cache.clear_errors()
    # nothing to do
    none = torch.zeros(0, dtype=torch.int32).cuda()
    kv4.moe_kv4_reserve(cache, s, none, none)
    kv4.moe_kv4_fork(cache, s, none, none)
    kv4.moe_kv4_free(cache, s, none)
    kv4.moe_kv4_copy_pages(cache, none, none)
    assert int(kv4.moe_kv4_compact(cache, s)) == 6
    assert cache.errors() == (0, 0)


@pytest.mark.parametrize("hkv,d,ps,layers", [(1, 64, 16, 1), (8, 128, 64, 3), (5, 64, 32, 2)])
def test_copy_pages(kv4, hkv, d, ps, layers):
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randint(0, 256, (layers, 12, hkv, kv4.block_bytes(d, ps)), dtype=torch.uint8,
                         device="cuda", generator=g)
    want = pool.clone()
    cache = kv4.Cache(pool, hkv, d, ps)
    src = torch.tensor([3, 3, -1, 0, 5, 200], dtype=torch.int32).cuda()
    dst = torch.tensor([4, 11, 2, 1, -1, 7], dtype=torch.int32).cuda()
    want[:, 4], want[:, 11], want[:, 1] = want[:, 3], want[:, 3], want[:, 0]
    kv4.moe_kv4_copy_pages(cache, src, dst)
    assert torch.equal(cache.pages, want)
    assert cache.errors() == (kv4.MOE_KV4_DEVERR_PAGE, 1)


def test_large_pool_bookkeeping(kv4):
    """More pages than one scanning block covers, and rows longer than a warp."""
    rng = np.random.default_rng(3)
    n_pages, ps = 20000, 16
    cache = kv4.Cache.empty(1, n_pages, 1, 64, ps)
    s = kv4.Sequences.empty(40, 700, n_pages)
    model = ref.Pages(40, 700, n_pages, ps)

    def ids(v):
        return torch.tensor(np.asarray(v, np.int32), dtype=torch.int32).cuda()

    def same():
        assert np.array_equal(s.tables.cpu().numpy(), model.tables)
        assert np.array_equal(s.refs.cpu().numpy(), model.refs)
        assert np.array_equal(s.lens.cpu().numpy(), model.lens)

    lens = rng.integers(1, 700 * ps, 30)
    kv4.moe_kv4_reserve(cache, s, ids(range(30)), ids(lens))
    model.reserve(range(30), lens)
    same()
    kv4.moe_kv4_fork(cache, s, ids([1, 2, 2, 29]), ids([30, 31, 32, 33]))
    model.fork([1, 2, 2, 29], [30, 31, 32, 33])
    same()
    gone = list(range(0, 30, 2)) + [31]
    kv4.moe_kv4_free(cache, s, ids(gone))
    model.free(gone)
    same()
    assert int(kv4.moe_kv4_compact(cache, s)) == model.compact()
    same()
