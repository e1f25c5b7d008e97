"""The scores of the attention kernels, seen through the lse, for keys whose codes are
mostly zero beside a few large ones (a channel that stands out takes its group's whole
range) and queries of one sign: what an offset of the codes adds has to cancel.

A score is a sum of D products that are exact in fp32, so it is off by at most
D 2^-23 = 2^-16 of the sum of its terms' magnitudes; the lse adds the fp32 errors of the
maximum times log2(e), a logarithm and a product, 2^-20 of its own size and 2^-20.
"""
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


@pytest.mark.parametrize("d,ps", [(128, 64), (64, 16)])
@pytest.mark.parametrize("m,group", [(1, 1), (1, 8), (1, 16), (3, 16), (16, 8), (64, 8)])
@pytest.mark.parametrize("span", [0.0, 0.5])
def test_scores_of_keys_with_few_large_codes(kv4, d, ps, m, group, span):
    rng = np.random.default_rng(m + group)
    streams, n = 24, max(m, 3)
    pages = streams * -(-n // ps)
    shape = (pages, 2, ps, d)
    codes = np.full(shape, 8, np.uint8)
    at = rng.integers(0, 32, shape[:-1] + (d // 32, 1))
    np.put_along_axis(codes.reshape(shape[:-1] + (d // 32, 32)), at,
                      rng.choice(np.array([1, 15], np.uint8), at.shape), -1)
    one = np.full(shape[:-1] + (d // 32,), 0.75, np.float16)
    vc = ref.pack_rows(rng.integers(0, 16, shape, dtype=np.uint8), False)
    pool = torch.from_numpy(ref.join(ref.pack_rows(codes, True), vc, one, one)).cuda()
    tables = np.arange(pages, dtype=np.int32).reshape(streams, -1)
    cu = np.arange(streams + 1, dtype=np.int32) * m

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()

    cache = kv4.Cache(pool[None], 2, d, ps)
    batch = kv4.Batch(ints(cu), ints([n] * streams), ints(tables), streams * m, m, n)
    q = ref.bf16(30 * (1 + span * rng.uniform(-1, 1, (streams * m, 2 * group, d)))).cuda()
    scale = ref.default_scale(d)
    _, lse = kv4.moe_kv4_attention(q, cache, batch, scale=scale, return_lse=True)
    _, want, _, size = gref.attention(q, pool, tables, [n] * streams, cu, ps, scale)
    off = (lse.double() - want).abs() / (2.0 ** -16 * size + 2.0 ** -20 * (1 + want.abs()))
    assert off.max().item() <= 1.0, f"{off.max().item()} of the bound"
