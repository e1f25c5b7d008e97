"""Thin Python binding of the 4-bit paged key/value cache (``include/moe_kv4.h``):
appending with head norms and position rotation, attention over the cache, and
page management.  Argument checks and marshalling only; the work is done by the
CUDA library that ``ops`` loads, and calls raise where that is missing.

A program keeps three kinds of objects, all over its own device tensors: a
``Cache`` (the page pool of all layers), a ``Batch`` for each shape of step (whose
tensors it may update in place between calls), and ``Sequences`` for page
management.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import ops

MOE_KV4_DEVERR_PAGE = 0x10
MOE_KV4_DEVERR_POSITION = 0x20
MOE_KV4_DEVERR_RANGE = 0x40
MOE_KV4_DEVERR_NO_PAGES = 0x80
MOE_KV4_DEVERR_SEQ = 0x100
MOE_KV4_WS_HEADER = 8192

EXPORTED = [
    "moe_kv4_block_bytes", "moe_kv4_pool_bytes", "moe_kv4_append", "moe_kv4_read",
    "moe_kv4_workspace_bytes", "moe_kv4_attention", "moe_kv4_scratch_bytes", "moe_kv4_reserve",
    "moe_kv4_fork", "moe_kv4_free", "moe_kv4_compact", "moe_kv4_copy_pages",
]


class Shape(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("cu_q", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("tables", ctypes.c_void_p)]


class _Seqs(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int32), ("table_stride", ctypes.c_int32),
                ("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("refs", ctypes.c_void_p)]


_lib = None


def load_library():
    """The CUDA library with this module's signatures declared."""
    global _lib
    if _lib is None:
        lib = ops.load_library()
        p, i, i64, f, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
        sig = {
            "moe_kv4_block_bytes": ([p], sz),
            "moe_kv4_pool_bytes": ([p], sz),
            "moe_kv4_append": ([p, i64, p, i64, p, i64, p, p, f, p, p, p, i, i, i, p, p, i, p, p,
                                p, p], i),
            "moe_kv4_read": ([p, i, p, p, p, p, p, p], i),
            "moe_kv4_workspace_bytes": ([p, i], sz),
            "moe_kv4_attention": ([p, i64, i, p, i, p, p, f, i, p, p, p, p, sz, p], i),
            "moe_kv4_scratch_bytes": ([p, i], sz),
            "moe_kv4_reserve": ([p, p, p, p, i, p, sz, p, p], i),
            "moe_kv4_fork": ([p, p, p, p, p, i, p, sz, p, p], i),
            "moe_kv4_free": ([p, p, p, i, p, p], i),
            "moe_kv4_compact": ([p, p, p, p, p, p, p, sz, p, p], i),
            "moe_kv4_copy_pages": ([p, p, p, p, i, p, p], i),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


class _Here:
    """No-op context: the tensors' device is already the current one."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(device):
    """Makes the device that holds a call's tensors the current one."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _raw_stream(stream, device):
    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def _ints(t, what, device, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        raise TypeError(f"{what}: expected an int32 tensor")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor on {device}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")
    return t


def _rows(t, what, device, tokens, dim, heads=None):
    """(pointer, token stride, heads) of bf16 [tokens, heads, dim] whose heads are
    contiguous; the tokens may be further apart (a part of a projection)."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{what}: expected bf16, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what}: expected a tensor on {device}")
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != dim or \
            (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{what}: expected [{tokens}, {heads or 'heads'}, {dim}], got "
                         f"{tuple(t.shape)}")
    n = t.shape[1]
    if tokens and (t.stride(2) != 1 or (n > 1 and t.stride(1) != dim)):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return t.data_ptr(), (t.stride(0) if tokens > 1 else n * dim), n


def _like(t, what, device, dtype, shape):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor on {device}")
    return t


def block_bytes(head_dim: int, page_size: int) -> int:
    """Bytes of one page of one head."""
    return page_size * (head_dim + head_dim // 8)


class Cache:
    """A page pool: uint8 [layers, n_pages, kv_heads, block_bytes] device memory
    of the caller.  ``errors`` reads the device error words that append, read and
    the page calls accumulate (``moe_kv4_attention`` has its own in its workspace)."""

    def __init__(self, pages: torch.Tensor, kv_heads: int, head_dim: int, page_size: int):
        if pages.dtype != torch.uint8 or pages.dim() != 4:
            raise TypeError("pages: expected uint8 [layers, n_pages, kv_heads, block_bytes]")
        if not pages.is_cuda or not pages.is_contiguous():
            raise ValueError("pages: expected a contiguous CUDA tensor")
        self.shape = Shape(pages.shape[0], pages.shape[1], kv_heads, head_dim, page_size)
        lib = load_library()
        self.ref = ctypes.byref(self.shape)
        if lib.moe_kv4_pool_bytes(self.ref) != pages.numel() or pages.shape[2] != kv_heads:
            raise ValueError(f"pages {tuple(pages.shape)} does not fit kv_heads {kv_heads}, "
                             f"head_dim {head_dim}, page_size {page_size}, or these are not "
                             "supported")
        self.pages = pages
        self.device = pages.device
        self.err = torch.zeros(2, dtype=torch.int32, device=pages.device)
        self._scratch = None

    @classmethod
    def empty(cls, layers, n_pages, kv_heads, head_dim, page_size, device="cuda"):
        """A pool of uninitialised pages."""
        pages = torch.empty((layers, n_pages, kv_heads, block_bytes(head_dim, page_size)),
                            dtype=torch.uint8, device=device)
        return cls(pages, kv_heads, head_dim, page_size)

    def errors(self):
        """(flags, count) accumulated so far; waits for the device."""
        flags, count = self.err.tolist()
        return flags & 0xFFFFFFFF, count

    def clear_errors(self):
        self.err.zero_()

    def scratch(self, n):
        """Device scratch for page calls of up to n requests, kept between calls
        (calls that share it run one after the other on one stream)."""
        need = load_library().moe_kv4_scratch_bytes(self.ref, n)
        if need == 0:
            raise ValueError(f"{n} requests in one call are not supported")
        if self._scratch is None or self._scratch.numel() < need:
            self._scratch = torch.empty(need, dtype=torch.uint8, device=self.device)
        return self._scratch


class Batch:
    """The requests of one step: cu_q int32 [R + 1] (where each request's new
    tokens begin), kv_len int32 [R] (lengths with the new tokens), tables int32
    [R, capacity] (page ids), the number of new tokens and upper bounds on a
    request's new tokens and length.  The tensors may change between calls."""

    def __init__(self, cu_q, kv_len, tables, tokens: int, max_q: int, max_kv: int):
        dev = kv_len.device
        if dev.type != "cuda":
            raise ValueError("kv_len: expected a CUDA tensor")
        r = kv_len.numel()
        _ints(kv_len, "kv_len", dev, (r,))
        _ints(cu_q, "cu_q", dev, (r + 1,))
        if tables.dtype != torch.int32 or tables.dim() != 2 or tables.shape[0] != r:
            raise ValueError(f"tables: expected int32 [{r}, capacity]")
        _ints(tables, "tables", dev)
        if tokens < 0 or max_q < 0 or max_kv < 0 or tokens > r * max_q:
            raise ValueError(f"{tokens} tokens in {r} requests of at most {max_q}")
        self.cu_q, self.kv_len, self.tables, self.tokens = cu_q, kv_len, tables, tokens
        self.device = dev
        self.struct = _Batch(r, tokens, max_q, max_kv, tables.shape[1], cu_q.data_ptr(),
                             kv_len.data_ptr(), tables.data_ptr())
        self.ref = ctypes.byref(self.struct)


class Sequences:
    """What page management works on: tables int32 [S, capacity] (-1 past a
    sequence's pages), lens int32 [S], refs int32 [n_pages]."""

    def __init__(self, tables, lens, refs):
        dev = tables.device
        if tables.dim() != 2:
            raise ValueError("tables: expected [sequences, capacity]")
        _ints(tables, "tables", dev)
        _ints(lens, "lens", dev, (tables.shape[0],))
        _ints(refs, "refs", dev)
        if dev.type != "cuda":
            raise ValueError("expected CUDA tensors")
        self.tables, self.lens, self.refs, self.device = tables, lens, refs, dev
        self.struct = _Seqs(tables.shape[0], tables.shape[1], tables.data_ptr(), lens.data_ptr(),
                            refs.data_ptr())
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, seqs, capacity, n_pages, device="cuda"):
        """Empty sequences over a pool whose pages are all free."""
        return cls(torch.full((seqs, capacity), -1, dtype=torch.int32, device=device),
                   torch.zeros(seqs, dtype=torch.int32, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device))


def _same(cache, other):
    if other.device != cache.device:
        raise ValueError(f"the cache is on {cache.device}, the batch or sequences on "
                         f"{other.device}")


# ------------------------------------------------------------------- tokens --
def moe_kv4_append(cache: Cache, batch: Batch, q, k, v, q_weight=None, k_weight=None, cos=None,
                   sin=None, positions=None, eps: float = 1e-6, interleaved: bool = False,
                   layer: int = 0, q_out=None, stream=None):
    """Head norm (where a weight bf16 [D] is given) and rotation (where cos and sin
    fp32 [max_pos, D/2] are given) of the batch's new q, k heads, bf16 [tokens,
    heads, D]; k and v go into the cache, q is returned (bf16, contiguous).  q may
    be None."""
    _same(cache, batch)
    dev, d, t = cache.device, cache.shape.head_dim, batch.tokens
    kp, ks, _ = _rows(k, "k", dev, t, d, cache.shape.kv_heads)
    vp, vs, _ = _rows(v, "v", dev, t, d, cache.shape.kv_heads)
    qp, qs, hq = (None, 0, 0) if q is None else _rows(q, "q", dev, t, d)
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
    else:
        _like(q_out, "q_out", dev, torch.bfloat16, (t, hq, d))
    for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _like(w, what, dev, torch.bfloat16, (d,))
    max_pos = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin are given together")
    if cos is not None:
        max_pos = cos.shape[0]
        _like(cos, "cos", dev, torch.float32, (max_pos, d // 2))
        _like(sin, "sin", dev, torch.float32, (max_pos, d // 2))
    if positions is not None:
        _ints(positions, "positions", dev, (t,))
    with _on(dev):
        rc = load_library().moe_kv4_append(
            qp, qs, kp, ks, vp, vs, None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(), eps,
            None if cos is None else cos.data_ptr(), None if sin is None else sin.data_ptr(),
            None if positions is None else positions.data_ptr(), max_pos, int(bool(interleaved)),
            hq, None if q_out is None else q_out.data_ptr(), cache.pages.data_ptr(), layer,
            cache.ref, batch.ref, cache.err.data_ptr(), _raw_stream(stream, dev))
    ops._check(rc, "moe_kv4_append")
    return q_out


def moe_kv4_read(cache: Cache, batch: Batch, layer: int = 0, k_out=None, v_out=None, stream=None):
    """(k, v) of the batch's new tokens as the cache holds them, fp16 [tokens,
    kv_heads, D]."""
    _same(cache, batch)
    shape = (batch.tokens, cache.shape.kv_heads, cache.shape.head_dim)
    out = []
    for t, what in ((k_out, "k_out"), (v_out, "v_out")):
        if t is None:
            t = torch.empty(shape, dtype=torch.float16, device=cache.device)
        out.append(_like(t, what, cache.device, torch.float16, shape))
    with _on(cache.device):
        rc = load_library().moe_kv4_read(
            cache.pages.data_ptr(), layer, cache.ref, batch.ref, out[0].data_ptr(),
            out[1].data_ptr(), cache.err.data_ptr(), _raw_stream(stream, cache.device))
    ops._check(rc, "moe_kv4_read")
    return out[0], out[1]


def alloc_workspace(cache: Cache, batch: Batch | None, q_heads: int) -> torch.Tensor:
    """A workspace for attention with this cache and number of query heads (any
    batch), its header zeroed."""
    n = load_library().moe_kv4_workspace_bytes(cache.ref, q_heads)
    if n == 0:
        raise ValueError(f"{q_heads} query heads over {cache.shape.kv_heads} kv heads are not "
                         "supported")
    ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
    ws[:MOE_KV4_WS_HEADER].zero_()
    return ws


def moe_kv4_attention(q, cache: Cache, batch: Batch, scale: float | None = None, window: int = 0,
                      tree=None, layer: int = 0, out=None, lse=None, return_lse: bool = False,
                      workspace=None, stream=None):
    """Causal attention of the batch's new tokens, q bf16 [tokens, q_heads, D], over
    their sequences: out bf16 [tokens, q_heads, D], with return_lse (or an lse
    tensor) also the fp32 log-sum-exp [tokens, q_heads].  window: only the last
    tokens (0: all).  tree: int64 [tokens], bit i set where the i-th new token of
    the request is seen.  scale defaults to 1 / sqrt(D)."""
    _same(cache, batch)
    dev, d, t = cache.device, cache.shape.head_dim, batch.tokens
    qp, qs, hq = _rows(q, "q", dev, t, d)
    if out is None:
        out = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
    else:
        _like(out, "out", dev, torch.bfloat16, (t, hq, d))
    if lse is not None:
        _like(lse, "lse", dev, torch.float32, (t, hq))
    elif return_lse:
        lse = torch.empty((t, hq), dtype=torch.float32, device=dev)
    if tree is not None:
        _like(tree, "tree", dev, torch.int64, (t,))
    if workspace is None:
        workspace = alloc_workspace(cache, batch, hq)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {dev}")
    with _on(dev):
        rc = load_library().moe_kv4_attention(
            qp, qs, hq, cache.pages.data_ptr(), layer, cache.ref, batch.ref,
            1.0 / math.sqrt(d) if scale is None else scale, window,
            None if tree is None else tree.data_ptr(), out.data_ptr(),
            None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
            _raw_stream(stream, dev))
    ops._check(rc, "moe_kv4_attention")
    return out if lse is None else (out, lse)


# -------------------------------------------------------------------- pages --
def _ids(t, what, cache, n=None):
    _ints(t, what, cache.device)
    if t.dim() != 1 or (n is not None and t.numel() != n):
        raise ValueError(f"{what}: expected [{'n' if n is None else n}], got {tuple(t.shape)}")
    return t.data_ptr() if t.numel() else None


def _pool_of(cache, seqs):
    _same(cache, seqs)
    if seqs.refs.numel() != cache.shape.n_pages:
        raise ValueError(f"refs has {seqs.refs.numel()} entries for {cache.shape.n_pages} pages")


def moe_kv4_reserve(cache: Cache, seqs: Sequences, ids, new_lens, stream=None):
    """Sequences ids grow to new_lens tokens: the lowest free pages are entered in
    their tables."""
    _pool_of(cache, seqs)
    n = ids.numel()
    ip, lp = _ids(ids, "ids", cache), _ids(new_lens, "new_lens", cache, n)
    s = cache.scratch(n)
    with _on(cache.device):
        rc = load_library().moe_kv4_reserve(cache.ref, seqs.ref, ip, lp, n, s.data_ptr(), s.numel(),
                                            cache.err.data_ptr(),
                                            _raw_stream(stream, cache.device))
    ops._check(rc, "moe_kv4_reserve")


def moe_kv4_fork(cache: Cache, seqs: Sequences, parents, children, stream=None):
    """Empty sequences children become copies of parents: full pages are shared,
    a begun page is copied."""
    _pool_of(cache, seqs)
    n = parents.numel()
    pp, cp = _ids(parents, "parents", cache), _ids(children, "children", cache, n)
    s = cache.scratch(n)
    with _on(cache.device):
        rc = load_library().moe_kv4_fork(cache.pages.data_ptr(), cache.ref, seqs.ref, pp, cp, n,
                                         s.data_ptr(), s.numel(), cache.err.data_ptr(),
                                         _raw_stream(stream, cache.device))
    ops._check(rc, "moe_kv4_fork")


def moe_kv4_free(cache: Cache, seqs: Sequences, ids, stream=None):
    """Sequences ids give their pages back and become empty."""
    _pool_of(cache, seqs)
    n = ids.numel()
    ip = _ids(ids, "ids", cache)
    with _on(cache.device):
        rc = load_library().moe_kv4_free(cache.ref, seqs.ref, ip, n, cache.err.data_ptr(),
                                         _raw_stream(stream, cache.device))
    ops._check(rc, "moe_kv4_free")


def moe_kv4_compact(cache: Cache, seqs: Sequences, tables_out=None, refs_out=None, n_used=None,
                    stream=None):
    """Moves the pages in use to the lowest indices.  The new tables and refs are
    written in place, or to tables_out and refs_out.  Returns the number of pages
    in use (device int32 [1])."""
    _pool_of(cache, seqs)
    dev = cache.device
    tables_out = seqs.tables if tables_out is None else \
        _ints(tables_out, "tables_out", dev, tuple(seqs.tables.shape))
    refs_out = seqs.refs if refs_out is None else \
        _ints(refs_out, "refs_out", dev, tuple(seqs.refs.shape))
    if n_used is None:
        n_used = torch.empty(1, dtype=torch.int32, device=dev)
    else:
        _ints(n_used, "n_used", dev, (1,))
    s = cache.scratch(0)
    with _on(dev):
        rc = load_library().moe_kv4_compact(
            cache.pages.data_ptr(), cache.ref, seqs.ref, tables_out.data_ptr(),
            refs_out.data_ptr(), n_used.data_ptr(), s.data_ptr(), s.numel(), cache.err.data_ptr(),
            _raw_stream(stream, dev))
    ops._check(rc, "moe_kv4_compact")
    return n_used


def moe_kv4_copy_pages(cache: Cache, src, dst, stream=None):
    """Page dst[i] becomes a copy of page src[i] in every layer (negative ids:
    skipped)."""
    n = src.numel()
    sp, dp = _ids(src, "src", cache), _ids(dst, "dst", cache, n)
    with _on(cache.device):
        rc = load_library().moe_kv4_copy_pages(cache.pages.data_ptr(), cache.ref, sp, dp, n,
                                               cache.err.data_ptr(),
                                               _raw_stream(stream, cache.device))
    ops._check(rc, "moe_kv4_copy_pages")
