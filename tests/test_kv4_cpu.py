"""The 4-bit cache's C ABI without a GPU: the header and the binding agree, sizes,
and arguments that are refused on the host before anything is launched."""
import ctypes
import os
import re

import numpy as np
import pytest

import kv4_reference as ref
from weight_only_int4_moe_gb300 import kv4, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_kv4.h")
P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 4)


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"^(?:int|size_t)\s+(moe_kv4_[a-z0-9_]+)\s*\(", text, flags=re.M))


def test_header_binding_and_library_agree():
    assert declared() == set(kv4.EXPORTED)
    lib = kv4.load_library()
    for name in kv4.EXPORTED:
        assert hasattr(lib, name)
    defs = dict(re.findall(r"^#define\s+(MOE_KV4_[A-Z0-9_]+)\s+(0x[0-9a-fA-F]+|\d+)u?\b",
                           open(HEADER).read(), flags=re.M))
    for name, v in defs.items():
        assert getattr(kv4, name) == int(v, 0), name
    flags = [int(v, 0) for k, v in defs.items() if "DEVERR" in k]
    flags += [ops.MOE_DEVERR_BAD_EXPERT_ID, ops.MOE_DEVERR_TIMEOUT, ops.MOE_DEVERR_BOUNDS,
              ops.MOE_DEVERR_RANGE]
    assert len(set(flags)) == len(flags) and all(f & (f - 1) == 0 for f in flags)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64])
def test_sizes(d, ps):
    lib = kv4.load_library()
    sh = kv4.Shape(3, 7, 5, d, ps)
    block = ps * (d + 2 * (d // 32) * 2)
    assert lib.moe_kv4_block_bytes(ctypes.byref(sh)) == block == kv4.block_bytes(d, ps)
    assert block % 16 == 0
    assert lib.moe_kv4_pool_bytes(ctypes.byref(sh)) == 3 * 7 * 5 * block
    assert lib.moe_kv4_workspace_bytes(ctypes.byref(sh), 35) >= kv4.MOE_KV4_WS_HEADER
    assert lib.moe_kv4_scratch_bytes(ctypes.byref(sh), 10) > 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("key", [True, False])
def test_every_code_has_a_place_of_its_own(d, key):
    bits = ref.places(d, key)
    assert sorted(bits) == list(range(0, 4 * d, 4))
    codes = np.random.default_rng(0).integers(0, 16, (3, d), dtype=np.uint8)
    assert np.array_equal(ref.unpack_rows(ref.pack_rows(codes, key), d, key), codes)


@pytest.mark.parametrize("bad", [(0, 1, 1, 64, 16), (1, 0, 1, 64, 16), (1, 1, 0, 64, 16),
                                 (1, 1, 257, 64, 16), (1, 1, 1, 96, 16), (1, 1, 1, 256, 16),
                                 (1, 1, 1, 64, 8), (1, 1, 1, 64, 48), (1, 1, 1, 64, 128),
                                 (1, (1 << 20) + 1, 1, 64, 16), (1025, 1, 1, 64, 16)])
def test_unsupported_pools(bad):
    lib = kv4.load_library()
    sh = ctypes.byref(kv4.Shape(*bad))
    assert lib.moe_kv4_block_bytes(sh) == 0 and lib.moe_kv4_pool_bytes(sh) == 0
    assert lib.moe_kv4_workspace_bytes(sh, 1) == 0 and lib.moe_kv4_scratch_bytes(sh, 1) == 0
    b = ctypes.byref(kv4._Batch(1, 1, 1, 1, 1, 1 << 20, 1 << 20, 1 << 20))
    assert lib.moe_kv4_read(P, 0, sh, b, P, P, None, None) == -2
    q = ctypes.byref(kv4._Seqs(1, 1, 1 << 20, 1 << 20, 1 << 20))
    assert lib.moe_kv4_free(sh, q, P, 1, None, None) == -2


def _append(**kw):
    sh = kv4.Shape(2, 8, 2, 64, 16)
    b = kv4._Batch(2, 5, 3, 9, 4, 1 << 20, 1 << 20, 1 << 20)
    a = dict(q=P, qs=256, k=P, ks=128, v=P, vs=128, qw=P, kw=P, eps=1e-6, cos=P, sin=P, pos=None,
             max_pos=16, inter=0, hq=4, out=P, pages=P, layer=0, shape=ctypes.byref(sh),
             batch=ctypes.byref(b), err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return kv4.load_library().moe_kv4_append(*a.values())


def test_append_refusals():
    for name in ("k", "v", "out", "pages", "sin"):
        assert _append(**{name: None}) == -1, name
    assert _append(shape=None) == -1 and _append(batch=None) == -1
    for kw in (dict(layer=2), dict(layer=-1), dict(hq=0), dict(hq=-1), dict(max_pos=0),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(inter=2),
               dict(qs=248), dict(ks=120), dict(vs=132), dict(qs=260)):
        assert _append(**kw) == -2, kw
    for name in ("q", "k", "v", "qw", "kw", "cos", "sin", "out", "pages"):
        assert _append(**{name: ODD}) == -3, name
    none = ctypes.byref(kv4._Batch(0, 0, 0, 0, 0, None, None, None))
    assert _append(batch=none, k=None, pages=None) == 0  # nothing to do
    for bad in (kv4._Batch(-1, 0, 0, 0, 0), kv4._Batch(0, 1, 1, 1, 1), kv4._Batch(1, -1, 0, 0, 0),
                kv4._Batch(1, (1 << 20) + 1, 1, 1, 1), kv4._Batch(65537, 1, 1, 1, 1),
                kv4._Batch(1, 1, -1, 1, 1), kv4._Batch(1, 1, 1, 1, -1)):
        assert _append(batch=ctypes.byref(bad)) == -2


def _attend(**kw):
    sh = kv4.Shape(2, 8, 2, 64, 16)
    b = kv4._Batch(2, 5, 3, 9, 4, 1 << 20, 1 << 20, 1 << 20)
    a = dict(q=P, qs=256, hq=4, pages=P, layer=0, shape=ctypes.byref(sh), batch=ctypes.byref(b),
             scale=0.1, window=0, tree=None, out=P, lse=None, ws=P, n=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return kv4.load_library().moe_kv4_attention(*a.values())


def test_attention_refusals():
    for name in ("q", "out", "pages", "ws"):
        assert _attend(**{name: None}) == -1, name
    wide = ctypes.byref(kv4._Batch(2, 70, 65, 90, 4, 1 << 20, 1 << 20, 1 << 20))
    for kw in (dict(hq=3), dict(hq=0), dict(hq=130), dict(window=-1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(layer=2), dict(qs=248), dict(qs=260),
               dict(tree=P, batch=wide)):
        assert _attend(**kw) == -2, kw
    for name in ("q", "out", "ws", "pages", "tree"):
        assert _attend(**{name: ODD}) == -3, name
    assert _attend(lse=ctypes.c_void_p((1 << 20) + 2)) == -3
    assert _attend(n=100) == -4
    none = ctypes.byref(kv4._Batch(3, 0, 0, 0, 0, None, None, None))
    assert _attend(batch=none, q=None, out=None) == 0


def test_scales_whose_power_of_two_overflows():
    assert _attend(scale=3e38) == -2 and _attend(scale=-3e38) == -2


def test_page_refusals():
    lib = kv4.load_library()
    sh = ctypes.byref(kv4.Shape(1, 100, 2, 64, 16))
    q = ctypes.byref(kv4._Seqs(4, 5, 1 << 20, 1 << 20, 1 << 20))
    big = 1 << 30
    assert lib.moe_kv4_reserve(sh, q, None, P, 1, P, big, None, None) == -1
    assert lib.moe_kv4_reserve(sh, q, P, P, 1, None, big, None, None) == -1
    assert lib.moe_kv4_reserve(sh, q, P, P, 1, P, 64, None, None) == -4
    assert lib.moe_kv4_reserve(sh, q, P, P, 1, ODD, big, None, None) == -3
    assert lib.moe_kv4_reserve(sh, q, P, P, 65537, P, big, None, None) == -2
    assert lib.moe_kv4_reserve(sh, q, P, P, -1, P, big, None, None) == -2
    assert lib.moe_kv4_reserve(sh, q, None, None, 0, None, 0, None, None) == 0
    assert lib.moe_kv4_fork(None, sh, q, P, P, 1, P, big, None, None) == -1
    assert lib.moe_kv4_fork(ODD, sh, q, P, P, 1, P, big, None, None) == -3
    assert lib.moe_kv4_free(sh, q, None, 1, None, None) == -1
    assert lib.moe_kv4_compact(P, sh, q, P, P, None, P, big, None, None) == -1
    assert lib.moe_kv4_compact(P, sh, q, P, P, P, P, 64, None, None) == -4
    for s in (kv4._Seqs(0, 5, 1 << 20, 1 << 20, 1 << 20), kv4._Seqs(4, 0, 1 << 20, 1 << 20, 1 << 20),
              kv4._Seqs(65537, 5, 1 << 20, 1 << 20, 1 << 20)):
        assert lib.moe_kv4_free(sh, ctypes.byref(s), P, 1, None, None) == -2
    s = ctypes.byref(kv4._Seqs(4, 5, 1 << 20, None, 1 << 20))
    assert lib.moe_kv4_free(sh, s, P, 1, None, None) == -1
    assert lib.moe_kv4_copy_pages(P, sh, P, P, 101, None, None) == -2
    assert lib.moe_kv4_copy_pages(P, sh, None, P, 1, None, None) == -1
    assert lib.moe_kv4_copy_pages(P, sh, None, None, 0, None, None) == 0
