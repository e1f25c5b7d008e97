"""Attention and append at the edges of their arguments: windows up to the largest int
and beyond."""
import numpy as np
import pytest
import torch

import kv4_gpu_reference as gref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from weight_only_int4_moe_gb300 import kv4 as m
    m.load_library()
    return m


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


# ------------------------------------------------------------------ windows --
@pytest.mark.parametrize("m", [6, 200])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2 ** 19, 2 ** 31, 2 ** 32 + 1, 10 ** 12])
@pytest.mark.parametrize("surplus", [False, True])
def test_windows_longer_than_everything(kv4, m, window, surplus):
    """They see all; also where a request has more new tokens than its length (its
    first rows see nothing)."""
    hkv, group, d, ps = 2, 4, 64, 16
    n = m // 2 if surplus else m + 50
    pool, tables, _, q = gref.make_case(m, [n], [m], hkv, group, d, ps)
    cache = kv4.Cache(pool[None], hkv, d, ps)
    batch = kv4.Batch(ints([0, m]), ints([n]), ints(tables), m, m, n)
    want, want_lse = kv4.moe_kv4_attention(q, cache, batch, return_lse=True)
    out, lse = kv4.moe_kv4_attention(q, cache, batch, window=window, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert torch.isfinite(lse[max(0, m - n):]).all()


def test_windows_below_the_ints_are_refused(kv4):
    pool, tables, _, q = gref.make_case(1, [20], [1], 1, 4, 64, 16)
    cache = kv4.Cache(pool[None], 1, 64, 16)
    batch = kv4.Batch(ints([0, 1]), ints([20]), ints(tables), 1, 1, 20)
    for window in (-1, -2 ** 31, -2 ** 32 + 5):
        with pytest.raises(RuntimeError):
            kv4.moe_kv4_attention(q, cache, batch, window=window)
