"""Attention over batches that keep every CTA (and warp) busy with many runs and long
ones, against fp64 on the device.  How the kernels cut a batch is restated in
kv4_partition, and each case asserts that its sizes reach what it is for.

Tolerances are those of test_kv4_gpu, derived there: half a bf16 ulp of the output, the
fp16 rounding of the probabilities and the fp32 error of the scores over sum p|v|, and
n 2^-25 max|v| for probabilities below fp16's normals.
"""
import numpy as np
import pytest
import torch

import kv4_gpu_reference as gref
import kv4_partition as part
import kv4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from weight_only_int4_moe_gb300 import kv4 as m
    m.load_library()
    return m


def sms():
    return min(160, torch.cuda.get_device_properties(0).multi_processor_count)


def check(kv4, seed, kv, ql, hkv, group, d, ps, window=0, tree=False, ramp=0.0, spread_q=2.0,
          only=None, repeats=1):
    pool, tables, cu, q = gref.make_case(seed, kv, ql, hkv, group, d, ps, ramp, spread_q)
    cache = kv4.Cache(pool[None], hkv, d, ps)

    def dev(x):
        return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()

    batch = kv4.Batch(dev(cu), dev(kv), dev(tables), int(cu[-1]), max(ql), max(kv))
    words = None
    if tree:
        rng = np.random.default_rng(seed + 1)
        words = torch.from_numpy(rng.integers(-2 ** 63, 2 ** 63 - 1, int(cu[-1]), dtype=np.int64)).cuda()
    scale = ref.default_scale(d)
    want, lse, spread, size = gref.attention(q, pool, tables, kv, cu, ps, scale, window, words, only)
    rows = slice(None) if only is None else torch.from_numpy(
        np.concatenate([np.arange(cu[b], cu[b + 1]) for b in only])).cuda()
    want, lse, spread, size = (x[rows] for x in (want, lse, spread, size))
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12 + 2e-5 * size[..., None]) * spread \
        + max(kv) * 2.0 ** -25 * 4 + 1e-30
    ws = kv4.alloc_workspace(cache, batch, hkv * group)
    first = None
    for _ in range(repeats):
        out, got_lse = kv4.moe_kv4_attention(q, cache, batch, window=window, tree=words,
                                             return_lse=True, workspace=ws)
        assert not ws[:kv4.MOE_KV4_WS_HEADER].any(), "the workspace header is not as it was"
        if first is None:
            first = out.clone(), got_lse.clone()
            assert torch.isfinite(out).all()
            worst = ((out[rows].double() - want).abs() / tol).max().item()
            assert worst <= 1.0, f"{worst} of the bound"
            got_lse = got_lse[rows].double()
            empty = torch.isneginf(lse)
            assert torch.equal(empty, torch.isneginf(got_lse))
            off = (got_lse - lse).abs()[~empty]
            assert torch.all(off <= (1e-5 * size + 2e-6 * (1 + lse.abs()))[~empty])
        else:
            assert torch.equal(out, first[0]) and torch.equal(got_lse, first[1])
    assert cache.errors() == (0, 0)


@pytest.mark.parametrize("d,ps,group", [(128, 64, 7), (64, 16, 8)])
def test_narrow_runs_of_odd_and_even_lengths(kv4, d, ps, group):
    """Items of up to 128 rows one after the other in a CTA, their tiles odd and even in
    number: an odd one leaves its last V tile to one of the two MMA warps, and the other
    begins the next run in the same slot of the ring."""
    rng = np.random.default_rng(d)
    ql = [int(x) for x in rng.integers(48 // group + 1, 128 // group + 1, 600)]
    kv = [m + int(x) for m, x in zip(ql, rng.integers(0, 640, 600))]
    runs = part.prefill_runs(kv, ql, 2, group, sms=sms())
    pairs = sum(a[0] % 2 == 1 and b[0] > 1 for r in runs for a, b in zip(r, r[1:]))
    assert pairs > 150 and max(len(r) for r in runs) >= 6
    check(kv4, d, kv, ql, 2, group, d, ps, repeats=5)


@pytest.mark.parametrize("d,ps,group,hkv", [(128, 64, 8, 2), (64, 16, 4, 3), (128, 16, 2, 2)])
@pytest.mark.parametrize("mode", ["", "window", "tree"])
def test_narrow_and_wide_runs_in_turn(kv4, d, ps, group, hkv, mode):
    """Requests of 49 to 128 rows between requests of more: a CTA goes from items that both
    warpgroup pairs share to items of two row tiles and back, many times."""
    rng = np.random.default_rng(d + ps + group)
    r = 420
    rows = np.where(rng.random(r) < 0.6, rng.integers(49, 129, r), rng.integers(129, 400, r))
    if mode == "tree":
        rows = np.minimum(rows, 64 * group)
    ql = [int(x) for x in -(-rows // group)]
    kv = [m + int(x) for m, x in zip(ql, rng.integers(0, 700, r))]
    window = 150 if mode == "window" else 0
    runs = part.prefill_runs(kv, ql, hkv, group, window, sms(), part.FEW_ROWS)
    turns = [(a[1] <= 128, b[1] <= 128, a[0] % 2) for x in runs for a, b in zip(x, x[1:])]
    assert max(len(x) for x in runs) >= (7 if mode else 8)
    wide = mode != "tree" or group > 2  # (64 tokens of two heads are 128 rows)
    for kind in ((True, True), (True, False), (False, True), (False, False)) if wide else ((True, True),):
        assert sum(t[:2] == kind for t in turns) > 20, kind
    assert 0.3 < np.mean([t[2] for t in turns]) < 0.7
    check(kv4, r + d, kv, ql, hkv, group, d, ps, window=window, tree=mode == "tree", repeats=2)


@pytest.mark.parametrize("d,ps,ramp", [(128, 64, 30.0), (64, 32, 0.0)])
def test_long_runs_of_wide_items(kv4, d, ps, ramp):
    """Runs of more than 40 tiles; with the ramp, row maxima that move all along."""
    kv, ql = [51200, 40001], [256, 201]
    runs = part.prefill_runs(kv, ql, 2, 4, sms=sms())
    assert np.median([max(n for n, _ in r) for r in runs if r]) >= 30
    check(kv4, d, kv, ql, 2, 4, d, ps, ramp=ramp, spread_q=0.5 if ramp else 2.0, repeats=2)


def test_long_runs_of_narrow_items(kv4):
    """Both pairs of warpgroups on the same rows for 40 tiles and more."""
    kv, ql = [65000, 30011, 48000], [9, 8, 16]
    runs = part.prefill_runs(kv * 4, ql * 4, 4, 8, sms=sms())
    assert np.median([max(n for n, _ in r) for r in runs if r]) >= 40
    check(kv4, 3, kv * 4, ql * 4, 4, 8, 128, 64, ramp=30.0, spread_q=0.5)


@pytest.mark.parametrize("requests", [1500, 2600])
def test_more_than_1024_requests_of_many_rows(kv4, requests):
    """A chunk of the prefix table stands for two or three requests."""
    rng = np.random.default_rng(requests)
    ql = [int(x) for x in rng.integers(7, 30, requests)]
    ql[5] = 120  # some of it long
    kv = [m + int(x) for m, x in zip(ql, rng.integers(0, 150, requests))]
    ql[700], kv[900] = 0, ql[900]
    only = sorted(set(range(0, requests, 7)) | {5, 699, 700, 701, 900, requests - 1})
    check(kv4, requests, kv, ql, 2, 8, 64, 16, only=only)


# ------------------------------------------------------------ few rows a request --
@pytest.mark.parametrize("group,d,ramp", [(8, 128, 0.0), (7, 64, 30.0), (16, 128, 30.0), (12, 64, 0.0)])
def test_warps_with_many_tiles(kv4, group, d, ramp):
    """Warps of the decode kernel with 30 and more tiles of an item."""
    kv = [32768 + 37 * i for i in range(24 if d == 128 else 20)]
    seg = part.decode_segments(kv, [1] * len(kv), 8, group, 1 if group <= 8 else 2, sms=sms())
    assert np.median([max(s) for s in seg if s]) >= 30
    check(kv4, group, kv, [1] * len(kv), 8, group, d, 64, ramp=ramp, spread_q=0.5 if ramp else 2.0,
          only=range(0, len(kv), 3))


@pytest.mark.parametrize("group,d,ps,m", [(7, 128, 64, 1), (4, 64, 16, 2), (16, 128, 32, 1), (6, 64, 64, 5)])
@pytest.mark.parametrize("window", [0, 70])
def test_warps_with_many_items(kv4, group, d, ps, m, window):
    """Warps of the decode kernel with three and more segments, CTAs with many items."""
    rng = np.random.default_rng(group)
    kv = [m + int(x) for x in rng.integers(0, 250, 500)]
    seg = part.decode_segments(kv, [m] * 500, 8, group, 1 if m * group <= 8 else 2, window, sms())
    assert max(len(s) for s in seg) >= 4 and np.mean([len(s) >= 3 for s in seg]) > 0.3
    check(kv4, group, kv, [m] * 500, 8, group, d, ps, window=window, repeats=2)


@pytest.mark.parametrize("requests,group", [(1500, 4), (3100, 16)])
def test_more_than_1024_requests_of_few_rows(kv4, requests, group):
    rng = np.random.default_rng(requests)
    kv = [int(x) for x in rng.integers(1, 130, requests)]
    ql = [1] * requests
    kv[17], ql[40], kv[41] = 5000, 0, 0
    ql[41] = 0
    only = sorted(set(range(0, requests, 7)) | {17, 39, 40, 41, 42, requests - 1})
    check(kv4, requests, kv, ql, 2, group, 128, 16, only=only, repeats=2)


@pytest.mark.parametrize("group", [9, 12, 16, 24, 33, 48, 64])
@pytest.mark.parametrize("d,ps", [(128, 64), (64, 16)])
def test_one_token_of_large_groups(kv4, group, d, ps):
    """Groups of 9 to 48 rows in tiles of 16 (64: the prefill kernel), their parts spread
    over several CTAs."""
    kv = [5000, 20011, 333, 12800]
    check(kv4, group, kv, [1] * 4, 2, group, d, ps, repeats=2)


def test_many_single_tokens_beside_a_prompt(kv4):
    """The usual step: both kernels, the decode kernel beside the other one."""
    rng = np.random.default_rng(4)
    kv = [int(x) for x in rng.integers(1, 3000, 90)] + [1500]
    ql = [1] * 90 + [700]
    check(kv4, 5, kv, ql, 4, 7, 128, 64, repeats=3)
    order = rng.permutation(91)
    check(kv4, 6, [kv[i] for i in order], [ql[i] for i in order], 4, 8, 64, 16, window=500, repeats=3)


def test_a_mixed_batch_in_a_graph(kv4):
    """Both kernels captured and replayed, also back to back, while lengths, new tokens and
    pages change in place."""
    hkv, group, d, ps, r = 2, 4, 128, 64, 6
    settings = [([700, 1, 900, 64, 64, 333], [513, 1, 1, 1, 64, 20]),
                ([20, 600, 800, 1, 90, 50], [1, 300, 290, 1, 4, 4]),
                ([1000, 999, 5, 7, 640, 3], [1, 597, 0, 1, 1, 0])]
    tokens, cap = 600, 16
    assert all(sum(ql) == tokens for _, ql in settings)
    cache = kv4.Cache.empty(1, 200, hkv, d, ps)
    kv_len, cu_q = torch.zeros(r, dtype=torch.int32).cuda(), torch.zeros(r + 1, dtype=torch.int32).cuda()
    tables = torch.zeros(r, cap, dtype=torch.int32).cuda()
    q = torch.zeros(tokens, hkv * group, d, dtype=torch.bfloat16).cuda()
    batch = kv4.Batch(cu_q, kv_len, tables, tokens, 597, 1000)
    ws = kv4.alloc_workspace(cache, batch, hkv * group)
    outs = [torch.empty_like(q) for _ in range(3)]

    def set_case(i):
        pool, t, cu, qq, kv, ql = gref_case(i)
        cache.pages[0, :pool.shape[0]] = pool
        kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        cu_q.copy_(torch.from_numpy(cu))
        tables.copy_(torch.from_numpy(np.ascontiguousarray(t)))
        q.copy_(qq)

    def gref_case(i):
        kv, ql = settings[i]
        pool, t, cu, qq = gref.make_case(i, kv, ql, hkv, group, d, ps)
        return pool, np.pad(t, ((0, 0), (0, cap)), constant_values=-1)[:, :cap], cu, qq, kv, ql

    set_case(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv4.moe_kv4_attention(q, cache, batch, out=outs[0], workspace=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o in outs:  # one behind the other: each starts under the one before
            kv4.moe_kv4_attention(q, cache, batch, out=o, workspace=ws)
    for i in (0, 1, 2, 1, 0):
        set_case(i)
        graph.replay()
        torch.cuda.synchronize()
        pool, t, cu, qq, kv, ql = gref_case(i)
        want, _, spread, size = gref.attention(qq, pool, t, kv, cu, ps, ref.default_scale(d))
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12 + 2e-5 * size[..., None]) * spread \
            + 1000 * 2.0 ** -25 * 4 + 1e-30
        for o in outs:
            assert ((o.double() - want).abs() / tol).max().item() <= 1.0
        assert not ws[:kv4.MOE_KV4_WS_HEADER].any()
