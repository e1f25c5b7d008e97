"""The softmax of the attention kernels where its number formats end: many tokens far
below the strongest one, and scores so large that fp32 resolves them in steps of
thousands.

A probability p relative to its row's maximum is held as 2^7 p in fp16, so its rounding
is 2^-11 p, or 2^-32 where 2^7 p is below fp16's normal numbers.
"""
import math

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


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


def sms():
    return min(160, torch.cuda.get_device_properties(0).multi_processor_count)


def blocks_of(kc, vc, scale_k, scale_v, ps):
    """uint8 [pages, hkv, block] of codes uint8 [tokens, D] (one head, a multiple of ps
    tokens) and scales."""
    n, d = kc.shape
    def rows(c, key):
        return ref.pack_rows(c, key).reshape(n // ps, 1, ps, d // 2)
    one = np.ones((n // ps, 1, ps, d // 32), np.float16)
    return ref.join(rows(kc, True), rows(vc, False), one * np.float16(scale_k),
                    one * np.float16(scale_v))


# streams, new tokens, group: one and two tiles of eight rows, the prefill kernel with
# items of up to 128 rows and of more
@pytest.mark.parametrize("streams,m,group", [(48, 1, 8), (48, 1, 16), (40, 8, 8), (20, 32, 16)])
@pytest.mark.parametrize("below", [20.5, 23.3, 25.5])
def test_many_tokens_far_below_the_strongest(kv4, streams, m, group, below):
    """One token in 4096 is strong and has value 0; the others lie 2^-below under it, and
    the output is their share."""
    d, ps, every = 128, 64, 4096
    n = 8 * every
    few = m * group <= part.FEW_ROWS
    if few:
        seg = part.decode_segments([n] * streams, [m] * streams, 1, group,
                                   1 if m * group <= 8 else 2, sms=sms())
        assert np.median([max(s) for s in seg if s]) >= 12
    else:
        runs = part.prefill_runs([n] * streams, [m] * streams, 1, group, sms=sms())
        assert np.median([max(t for t, _ in r) for r in runs if r]) >= 32
    rng = np.random.default_rng(1)
    kc = np.full((n, d), 8, np.uint8)
    vc = rng.integers(9, 16, (n, d), dtype=np.uint8)
    kc[::every, 0] = 15
    vc[::every] = 8
    # the same tokens for every stream
    pool = torch.from_numpy(blocks_of(kc, vc, 1.0, 1.0, ps)).cuda()
    cache = kv4.Cache(pool[None], 1, d, ps)
    tables = np.tile(np.arange(n // ps, dtype=np.int32), (streams, 1))
    cu = np.arange(streams + 1) * m
    batch = kv4.Batch(ints(cu), ints([n] * streams), ints(tables), streams * m, m, n)
    q = torch.zeros(streams * m, group, d)
    q[..., 0] = 4.0  # scale * 4 * 7 * log2(e) = below
    scale = below * math.log(2) / 28
    q = q.to(torch.bfloat16).cuda()
    out, lse = kv4.moe_kv4_attention(q, cache, batch, scale=scale, return_lse=True)
    want, want_lse, spread, size = gref.attention(q, pool, tables, [n] * streams, cu, ps, scale,
                                                  only=[0])
    want, want_lse, spread = want[:m], want_lse[:m], spread[:m]
    assert want.abs().max() > 1e-5
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12 + 2e-5 * below) * spread \
        + every * 2.0 ** -32 * 7
    for b in range(streams):
        off = (out[b * m:(b + 1) * m].double() - want).abs() / tol
        assert off.max().item() <= 1.0, f"{off.max().item()} of the bound"
    assert torch.all((lse[:m].double() - want_lse).abs() <= 1e-5 * below + 2e-6 * (1 + want_lse.abs()))


@pytest.mark.parametrize("m,group", [(1, 8), (1, 16), (9, 8), (40, 8)])
@pytest.mark.parametrize("winner", [0, 700, 1990])
def test_scores_of_ten_to_the_ten(kv4, m, group, winner):
    """The largest queries and keys that the format holds: the token that matches best
    wins alone, with its value exactly and the score itself as the lse."""
    d, ps, n = 128, 64, 2048
    rng = np.random.default_rng(winner + m)
    kc = rng.integers(5, 12, (n, d), dtype=np.uint8)  # some up to 4 steps, the winner 7
    vc = rng.integers(0, 16, (n, d), dtype=np.uint8)
    sign = rng.integers(0, 2, d)
    kc[winner] = np.where(sign == 1, 15, 1)
    pool = torch.from_numpy(blocks_of(kc, vc, 2720.0, 0.5, ps)).cuda()
    cache = kv4.Cache(pool[None], 1, d, ps)
    tables = np.arange(n // ps, dtype=np.int32)[None]
    batch = kv4.Batch(ints([0, m]), ints([n]), ints(tables), m, m, n)
    g = torch.Generator().manual_seed(1)
    q = torch.from_numpy(np.where(sign == 1, 1.0, -1.0)) * \
        (30000 + 30000 * torch.rand(m, group, 1, generator=g))
    q = q.to(torch.bfloat16).cuda()
    for scale in (ref.default_scale(d), 100.0):
        out, lse = kv4.moe_kv4_attention(q, cache, batch, scale=scale, return_lse=True)
        want, want_lse, _, _ = gref.attention(q, pool, tables, [n], [0, m], ps, scale)
        assert want_lse.abs().min() > 1e9
        seen = torch.arange(n - m, n).cuda() >= winner
        value = (torch.from_numpy(vc[winner].astype(np.float32)) - 8).cuda() * 0.5
        assert torch.equal(out[seen].float(), value.expand(int(seen.sum()), group, d))
        assert torch.isfinite(out).all()
        assert torch.all(((lse.double() - want_lse) / want_lse).abs()[seen] <= 2e-5)


@pytest.mark.parametrize("m,group", [(1, 8), (1, 16), (9, 8), (40, 8)])
def test_equal_scores_of_ten_to_the_ten(kv4, m, group):
    """Two tokens with the same huge score share the row."""
    d, ps, n = 64, 16, 1024
    rng = np.random.default_rng(m)
    kc = rng.integers(7, 10, (n, d), dtype=np.uint8)
    vc = rng.integers(0, 16, (n, d), dtype=np.uint8)
    kc[3] = kc[900] = 15
    pool = torch.from_numpy(blocks_of(kc, vc, 2720.0, 1.0, ps)).cuda()
    cache = kv4.Cache(pool[None], 1, d, ps)
    tables = np.arange(n // ps, dtype=np.int32)[None]
    batch = kv4.Batch(ints([0, m]), ints([n]), ints(tables), m, m, n)
    q = torch.full((m, group, d), 60000.0).to(torch.bfloat16).cuda()
    out = kv4.moe_kv4_attention(q, cache, batch, scale=1.0)
    value = ((vc[3].astype(np.float32) - 8) + (vc[900].astype(np.float32) - 8)) / 2
    assert torch.equal(out.float(), torch.from_numpy(value).cuda().expand(m, group, d))
