"""The softmax of the attention kernels where its number formats end: scores so large
that fp32 resolves them in steps of thousands."""
import numpy as np
import pytest
import torch

import kv4_gpu_reference as gref
import kv4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from weight_only_int4_moe_gb300 import kv4 as m
    m.load_library()
    return m


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


def blocks_of(kc, vc, scale_k, scale_v, ps):
    """uint8 [pages, hkv, block] of codes uint8 [tokens, D] (one head, a multiple of ps
    tokens) and scales."""
    n, d = kc.shape
    def rows(c, key):
        return ref.pack_rows(c, key).reshape(n // ps, 1, ps, d // 2)
    one = np.ones((n // ps, 1, ps, d // 32), np.float16)
    return ref.join(rows(kc, True), rows(vc, False), one * np.float16(scale_k),
                    one * np.float16(scale_v))


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
