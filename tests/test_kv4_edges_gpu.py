"""Attention and append at the edges of their arguments: windows up to the largest int
and beyond, rows that no request owns, pages that a window has left behind."""
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


def close(out, want, spread, size):
    """The bound of test_kv4_gpu, for lengths of a few hundred."""
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12 + 2e-5 * size[..., None]) * spread + 1e-4
    return bool(((out.double() - want).abs() <= tol).all())


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


# ---------------------------------------------------- rows without a request --
@pytest.mark.parametrize("rotate", [False, True])
def test_rows_of_no_request(kv4, rotate):
    """A batch padded to a captured step's number of tokens: rows past cu_q's last entry
    (and before its first) are not stored, read as zeros and report nothing."""
    hkv, d, ps = 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randint(0, 64, (1, 8, hkv, kv4.block_bytes(d, ps)), dtype=torch.uint8, device="cuda",
                         generator=g)
    cache = kv4.Cache(pool, hkv, d, ps)
    before = pool.clone()
    tables = ints([[0, 1], [2, 3], [4, 5]])
    # two single tokens of sequences of 16 and 20 tokens; the row behind the first one's
    # last full page would land in its next page
    t = 6
    batch = kv4.Batch(ints([1, 2, 2, 3]), ints([16, 7, 20]), tables, t, 2, 32)
    x = torch.randn(t, hkv, d, device="cuda", generator=g).to(torch.bfloat16)
    c, s = torch.rand(32, d // 2, device="cuda"), torch.rand(32, d // 2, device="cuda")
    q = kv4.moe_kv4_append(cache, batch, x, x, x, cos=c if rotate else None, sin=s if rotate else None)
    assert cache.errors() == (0, 0)
    k, _ = kv4.moe_kv4_read(cache, batch)
    assert cache.errors() == (0, 0)
    changed = (cache.pages != before).any(-1).any(-1)[0].nonzero().flatten().tolist()
    assert changed == [0, 5]
    own = torch.tensor([1, 2], device="cuda")
    rest = torch.tensor([0, 3, 4, 5], device="cuda")
    assert not k[rest].any() and k[own].any(-1).all()
    if not rotate:
        assert torch.equal(q, x)
    assert torch.isfinite(q).all()


def test_attention_leaves_rows_of_no_request(kv4):
    hkv, group, d, ps = 2, 4, 128, 64
    pool, tables, cu, q = gref.make_case(5, [300, 90], [1, 1], hkv, group, d, ps)
    cache = kv4.Cache(pool[None], hkv, d, ps)
    q6 = torch.cat([q, torch.ones(4, hkv * group, d, dtype=torch.bfloat16, device="cuda")])
    batch = kv4.Batch(ints([0, 1, 2]), ints([300, 90]), ints(tables), 6, 3, 300)
    out = torch.full_like(q6, 7.0)
    kv4.moe_kv4_attention(q6, cache, batch, out=out)
    want, _, spread, size = gref.attention(q, pool, tables, [300, 90], cu, ps, ref.default_scale(d))
    assert close(out[:2], want, spread, size) and (out[2:] == 7).all()


@pytest.mark.parametrize("big", [False, True])
def test_row_ranges_that_are_none(kv4, big):
    """cu_q that decreases, lies outside the rows or wraps in a difference: such requests
    are left out, the others are computed."""
    hkv, group, d, ps = 2, 4, 128, 64
    m = 40 if big else 1
    kv, ql = [300, 500, 90], [m, m, m]
    pool, tables, cu, q = gref.make_case(6, kv, ql, hkv, group, d, ps)
    cache = kv4.Cache(pool[None], hkv, d, ps)
    far = 0x70000000
    # requests 1 and 3 are rows [0, m) and [m, 2 m); around them [far, -far), [m, m) after a
    # decrease, [2 m, far) and [far, wrapped)
    bounds = [far, 0, m, m, 2 * m, far, -2 ** 31 + 16]
    lens = [300, 300, 77, 500, 90, 90]
    t6 = ints(np.stack([tables[0], tables[0], tables[1], tables[1], tables[2], tables[2]]))
    batch = kv4.Batch(ints(bounds), ints(lens), t6, 3 * m, m, 500)
    out = torch.full_like(q, 7.0)
    ws = kv4.alloc_workspace(cache, batch, hkv * group)
    kv4.moe_kv4_attention(q, cache, batch, out=out, workspace=ws)
    want, _, spread, size = gref.attention(q, pool, tables, kv, cu, ps, ref.default_scale(d), only=[0, 1])
    assert close(out[:2 * m], want[:2 * m], spread[:2 * m], size[:2 * m])
    assert (out[2 * m:] == 7).all()
    assert not ws[:kv4.MOE_KV4_WS_HEADER].any()


# ------------------------------------------------ pages a window has left behind --
@pytest.mark.parametrize("ps", [16, 32])
@pytest.mark.parametrize("m,group", [(1, 4), (1, 16), (5, 4), (150, 4)])
@pytest.mark.parametrize("window", [1, 37, 64, 100, 130])
def test_pages_before_the_window_are_not_needed(kv4, ps, m, group, window):
    """Their entries may be anything, also pages of NaN: nothing read there reaches a result
    and nothing is reported."""
    hkv, d, kv = 2, 128, [517, 333, 1024]
    pool, tables, cu, q = gref.make_case(window, kv, [m] * 3, hkv, group, d, ps)
    cache = kv4.Cache(pool[None], hkv, d, ps)
    want, _, spread, size = gref.attention(q, pool, tables, kv, cu, ps, ref.default_scale(d), window)
    other = min(set(range(pool.shape[0])) - set(tables.flatten().tolist()))  # all its scales are NaN
    for b, n in enumerate(kv):
        gone = tables[b, :max(0, n - m - window + 1) // ps]
        gone[:] = np.where(np.arange(len(gone)) % 3 == 2, -1, other)
    batch = kv4.Batch(ints(cu), ints(kv), ints(tables), int(cu[-1]), m, max(kv))
    ws = kv4.alloc_workspace(cache, batch, hkv * group)
    out = kv4.moe_kv4_attention(q, cache, batch, window=window, workspace=ws)
    assert close(out, want, spread, size)
    assert ws[:8].view(torch.int32).tolist() == [0, 0]
