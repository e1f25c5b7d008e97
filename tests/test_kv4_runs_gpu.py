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
