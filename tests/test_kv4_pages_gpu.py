"""Page calls whose counts pass the range of an int."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from weight_only_int4_moe_gb300 import kv4 as m
    m.load_library()
    return m


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


@pytest.mark.parametrize("each", [32769, 65538])
def test_requests_for_billions_of_pages(kv4, each):
    """65534 requests that ask for some 2^31 (2^32 - 4) pages between a request that fits and a
    small one behind them: only the first is served, all others are refused and counted."""
    n, ps, n_pages = 65536, 16, 100
    cache = kv4.Cache.empty(1, n_pages, 1, 64, ps)
    seqs = kv4.Sequences.empty(n, each, n_pages)
    to = np.full(n, each * ps)
    to[0], to[-1] = 5 * ps, 3 * ps
    assert (to // ps).sum() >= 2 ** 31
    kv4.moe_kv4_reserve(cache, seqs, ints(np.arange(n)), ints(to))
    assert cache.errors() == (kv4.MOE_KV4_DEVERR_NO_PAGES, n - 1)
    assert seqs.tables[0, :6].tolist() == [0, 1, 2, 3, 4, -1]
    assert int((seqs.lens != 0).sum()) == 1 and int(seqs.lens[0]) == 5 * ps
    assert seqs.refs.tolist() == [1] * 5 + [0] * 95
    assert not (seqs.tables[1:, 0] != -1).any() and not (seqs.tables[-1] != -1).any()


def test_a_length_near_the_largest_int(kv4):
    """A table of 2^31 / 16 entries: the page count of its longest sequence does not
    overflow, and the request fails for want of pages."""
    ps, n_pages = 16, 50
    cache = kv4.Cache.empty(1, n_pages, 1, 64, ps)
    seqs = kv4.Sequences.empty(2, 2 ** 27 + 1, n_pages)
    kv4.moe_kv4_reserve(cache, seqs, ints([0, 1]), ints([2 ** 31 - 1, 40]))
    assert cache.errors() == (kv4.MOE_KV4_DEVERR_NO_PAGES, 2)
    assert seqs.lens.tolist() == [0, 0] and not seqs.refs.any()
    cache.clear_errors()
    kv4.moe_kv4_reserve(cache, seqs, ints([1, 0]), ints([40, 2 ** 31 - 1]))
    assert cache.errors() == (kv4.MOE_KV4_DEVERR_NO_PAGES, 1)
    assert seqs.lens.tolist() == [0, 40] and seqs.refs.tolist() == [1] * 3 + [0] * 47


def test_a_pool_with_every_page_in_use(kv4):
    """Requests that need exactly what there is, and none."""
    ps, n_pages = 32, 4097
    cache = kv4.Cache.empty(1, n_pages, 1, 64, ps)
    seqs = kv4.Sequences.empty(3, n_pages, n_pages)
    kv4.moe_kv4_reserve(cache, seqs, ints([0, 1]), ints([4000 * ps, 97 * ps]))
    assert cache.errors() == (0, 0) and bool((seqs.refs == 1).all())
    kv4.moe_kv4_reserve(cache, seqs, ints([2, 0]), ints([0, 4000 * ps]))  # nothing more
    assert cache.errors() == (0, 0)
    kv4.moe_kv4_reserve(cache, seqs, ints([2]), ints([1]))
    assert cache.errors() == (kv4.MOE_KV4_DEVERR_NO_PAGES, 1)
    cache.clear_errors()
    kv4.moe_kv4_free(cache, seqs, ints([1]))
    kv4.moe_kv4_reserve(cache, seqs, ints([2]), ints([97 * ps]))
    assert cache.errors() == (0, 0)
    assert seqs.tables[2, :98].tolist() == list(range(4000, 4097)) + [-1]
