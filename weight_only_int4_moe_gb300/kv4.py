"""Thin Python binding of the 4-bit paged key/value cache (``include/moe_kv4.h``):
appending with head norms and position rotation, attention over the cache, and
page management.  Argument checks and marshalling only; the work is done by the
CUDA library that ``ops`` loads, and calls raise where that is missing.

A program keeps three kinds of objects, all over its own device tensors: a
``Cache`` (the page pool of all layers), a ``Batch`` for each shape of step (whose
tensors it may update in place between calls), and ``Sequences`` for page
management.

Calls run on `stream`, or on the current one.  What a call makes for itself (outputs
that are not given, a workspace, scratch) is made on that stream; the caller orders its
own tensors, and reads of the results, with it.
"""
from __future__ import annotations

import ctypes

import torch

from . import ops

MOE_KV4_DEVERR_PAGE = 0x10
MOE_KV4_DEVERR_POSITION = 0x20
MOE_KV4_DEVERR_RANGE = 0x40
MOE_KV4_DEVERR_NO_PAGES = 0x80
MOE_KV4_DEVERR_SEQ = 0x100
MOE_KV4_WS_HEADER = 8192
MAX_REQUESTS = 65536  # of one page call

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
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_INT_MAX = 2 ** 31 - 1  # (ctypes would wrap what lies beyond)


def _on(index):
    """Makes the device that holds a call's tensors the current one."""
    return _HERE if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


def _raw_stream(stream, index):
    """The cudaStream_t of `stream`, or of the device's current one."""
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """Uninitialised memory for a call on `stream` (None: the device's current one).
    It comes from that stream's memory, so that nothing still running elsewhere uses it,
    and the current stream, where the caller goes on with it, is recorded."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


# The checks below run before every launch and are kept short: a single-token step
# is bound by what the host does per call (a tensor's get_device() costs a third
# of comparing its .device).
def _ints(t, what, index, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype is not _I32:
        raise TypeError(f"{what}: expected an int32 tensor")
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor on cuda:{index}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")
    return t


def _rows(t, what, index, tokens, dim, heads=None):
    """(pointer, token stride, heads) of bf16 [tokens, heads, dim] whose heads are
    contiguous; the tokens may be further apart (a part of a projection)."""
    if t.dtype is not _BF16:
        raise TypeError(f"{what}: expected bf16, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{what}: expected a tensor on cuda:{index}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim or \
            (heads is not None and shape[1] != heads):
        raise ValueError(f"{what}: expected [{tokens}, {heads or 'heads'}, {dim}], got "
                         f"{tuple(shape)}")
    n = shape[1]
    st, sh, sd = t.stride()
    if tokens and (sd != 1 or (n > 1 and sh != dim)):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return t.data_ptr(), (st if tokens > 1 else n * dim), n


def _like(t, what, index, dtype, shape):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what}: expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor on cuda:{index}")
    return t.data_ptr()


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
        self.pages, self.pages_ptr = pages, pages.data_ptr()
        self.device, self.index = pages.device, pages.get_device()
        self.err = torch.zeros(2, dtype=torch.int32, device=pages.device)
        self.err_ptr = self.err.data_ptr()
        self._scratch = None

    @classmethod
    def empty(cls, layers, n_pages, kv_heads, head_dim, page_size, device="cuda"):
        """A pool of uninitialised pages."""
        pages = torch.empty((layers, n_pages, kv_heads, block_bytes(head_dim, page_size)),
                            dtype=torch.uint8, device=device)
        return cls(pages, kv_heads, head_dim, page_size)

    def errors(self):
        """(flags, count) accumulated so far; waits for the device (all its streams)."""
        torch.cuda.synchronize(self.device)
        flags, count = self.err.tolist()
        return flags & 0xFFFFFFFF, count

    def clear_errors(self):
        self.err.zero_()

    def scratch(self, stream=None):
        """(pointer, bytes) of the device scratch of page calls, for any number of
        requests: taken by the first call, on its stream, and kept (calls that share it
        run one after the other)."""
        if self._scratch is None:
            n = load_library().moe_kv4_scratch_bytes(self.ref, MAX_REQUESTS)
            self._scratch = _empty(n, torch.uint8, self.device, stream)
        return self._scratch.data_ptr(), self._scratch.numel()


class Batch:
    """The requests of one step: cu_q int32 [R + 1] (where each request's new
    tokens begin), kv_len int32 [R] (lengths with the new tokens), tables int32
    [R, capacity] (page ids), the number of new tokens and upper bounds on a
    request's new tokens and length.  The tensors may change between calls."""

    def __init__(self, cu_q, kv_len, tables, tokens: int, max_q: int, max_kv: int):
        if not kv_len.is_cuda:
            raise ValueError("kv_len: expected a CUDA tensor")
        dev, r = kv_len.get_device(), kv_len.numel()
        _ints(kv_len, "kv_len", dev, (r,))
        _ints(cu_q, "cu_q", dev, (r + 1,))
        if tables.dtype != torch.int32 or tables.dim() != 2 or tables.shape[0] != r:
            raise ValueError(f"tables: expected int32 [{r}, capacity]")
        _ints(tables, "tables", dev)
        if tokens < 0 or max_q < 0 or max_kv < 0 or tokens > r * max_q:
            raise ValueError(f"{tokens} tokens in {r} requests of at most {max_q}")
        self.cu_q, self.kv_len, self.tables, self.tokens = cu_q, kv_len, tables, tokens
        self.index = dev
        self.struct = _Batch(r, tokens, max_q, max_kv, tables.shape[1], cu_q.data_ptr(),
                             kv_len.data_ptr(), tables.data_ptr())
        self.ref = ctypes.byref(self.struct)


class Sequences:
    """What page management works on: tables int32 [S, capacity] (-1 past a
    sequence's pages), lens int32 [S], refs int32 [n_pages]."""

    def __init__(self, tables, lens, refs):
        if not tables.is_cuda or tables.dim() != 2:
            raise ValueError("tables: expected a CUDA tensor [sequences, capacity]")
        dev = tables.get_device()
        _ints(tables, "tables", dev)
        _ints(lens, "lens", dev, (tables.shape[0],))
        _ints(refs, "refs", dev)
        self.tables, self.lens, self.refs, self.index = tables, lens, refs, dev
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
    if other.index != cache.index:
        raise ValueError(f"the cache is on cuda:{cache.index}, the batch or sequences on "
                         f"cuda:{other.index}")


# ------------------------------------------------------------------- tokens --
def moe_kv4_append(cache: Cache, batch: Batch, q, k, v, q_weight=None, k_weight=None, cos=None,
                   sin=None, positions=None, eps: float = 1e-6, interleaved: bool = False,
                   layer: int = 0, q_out=None, stream=None):
    """Head norm (where a weight bf16 [D] is given) and rotation (where cos and sin
    fp32 [max_pos, D/2] are given) of the batch's new q, k heads, bf16 [tokens,
    heads, D]; k and v go into the cache, q is returned (bf16, contiguous).  q may
    be None."""
    _same(cache, batch)
    dev, d, t, hkv = cache.index, cache.shape.head_dim, batch.tokens, cache.shape.kv_heads
    kp, ks, _ = _rows(k, "k", dev, t, d, hkv)
    vp, vs, _ = _rows(v, "v", dev, t, d, hkv)
    if q is None:
        qp = op = q_out = None
        qs = hq = 0
    else:
        qp, qs, hq = _rows(q, "q", dev, t, d)
        if q_out is None:
            q_out = _empty((t, hq, d), _BF16, cache.device, stream)
            op = q_out.data_ptr()
        else:
            op = _like(q_out, "q_out", dev, _BF16, (t, hq, d))
    qw = None if q_weight is None else _like(q_weight, "q_weight", dev, _BF16, (d,))
    kw = None if k_weight is None else _like(k_weight, "k_weight", dev, _BF16, (d,))
    max_pos, cp, sp = 0, None, None
    if cos is not None and sin is not None:
        max_pos = cos.shape[0]
        cp = _like(cos, "cos", dev, _F32, (max_pos, d // 2))
        sp = _like(sin, "sin", dev, _F32, (max_pos, d // 2))
    elif cos is not None or sin is not None:
        raise ValueError("cos and sin are given together")
    pp = None if positions is None else _ints(positions, "positions", dev, (t,)).data_ptr()
    with _on(dev):
        rc = (_lib or load_library()).moe_kv4_append(
            qp, qs, kp, ks, vp, vs, qw, kw, eps, cp, sp, pp, max_pos, 1 if interleaved else 0, hq,
            op, cache.pages_ptr, layer, cache.ref, batch.ref, cache.err_ptr,
            _raw_stream(stream, dev))
    if rc:
        ops._check(rc, "moe_kv4_append")
    return q_out


def moe_kv4_read(cache: Cache, batch: Batch, layer: int = 0, k_out=None, v_out=None, stream=None):
    """(k, v) of the batch's new tokens as the cache holds them, fp16 [tokens,
    kv_heads, D]."""
    _same(cache, batch)
    shape = (batch.tokens, cache.shape.kv_heads, cache.shape.head_dim)
    dev = cache.index
    if k_out is None:
        k_out = _empty(shape, torch.float16, cache.device, stream)
    if v_out is None:
        v_out = _empty(shape, torch.float16, cache.device, stream)
    kp = _like(k_out, "k_out", dev, torch.float16, shape)
    vp = _like(v_out, "v_out", dev, torch.float16, shape)
    with _on(dev):
        rc = (_lib or load_library()).moe_kv4_read(cache.pages_ptr, layer, cache.ref, batch.ref, kp,
                                                   vp, cache.err_ptr, _raw_stream(stream, dev))
    if rc:
        ops._check(rc, "moe_kv4_read")
    return k_out, v_out


def alloc_workspace(cache: Cache, batch: Batch | None, q_heads: int, stream=None) -> torch.Tensor:
    """A workspace for attention with this cache and number of query heads (any
    batch), its header zeroed on `stream` (None: the current one), on which, or after
    which, its calls run."""
    n = load_library().moe_kv4_workspace_bytes(cache.ref, q_heads)
    if n == 0:
        raise ValueError(f"{q_heads} query heads over {cache.shape.kv_heads} kv heads are not "
                         "supported")
    ws = _empty(n, torch.uint8, cache.device, stream)
    if stream is None:
        ws[:MOE_KV4_WS_HEADER].zero_()
    else:
        with torch.cuda.stream(stream):
            ws[:MOE_KV4_WS_HEADER].zero_()
    return ws


def moe_kv4_attention(q, cache: Cache, batch: Batch, scale: float | None = None, window: int = 0,
                      tree=None, layer: int = 0, out=None, lse=None, return_lse: bool = False,
                      workspace=None, stream=None):
    """Causal attention of the batch's new tokens, q bf16 [tokens, q_heads, D], over
    their sequences: out bf16 [tokens, q_heads, D], with return_lse (or an lse
    tensor) also the fp32 log-sum-exp [tokens, q_heads].  window: only the last
    tokens (0: all).  tree: int64 [tokens], bit i set where the i-th new token of
    the request is seen.  scale defaults to 1 / sqrt(D).  Without a workspace the call
    takes one for itself (its error words are lost with it)."""
    _same(cache, batch)
    dev, d, t = cache.index, cache.shape.head_dim, batch.tokens
    qp, qs, hq = _rows(q, "q", dev, t, d)
    if out is None:
        out = _empty((t, hq, d), _BF16, cache.device, stream)
        op = out.data_ptr()
    else:
        op = _like(out, "out", dev, _BF16, (t, hq, d))
    if lse is None and return_lse:
        lse = _empty((t, hq), _F32, cache.device, stream)
    lp = None if lse is None else _like(lse, "lse", dev, _F32, (t, hq))
    tp = None if tree is None else _like(tree, "tree", dev, torch.int64, (t,))
    if workspace is None:
        workspace = alloc_workspace(cache, batch, hq, stream)
    elif workspace.get_device() != dev or workspace.dtype is not torch.uint8 or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on cuda:{dev}")
    with _on(dev):
        rc = (_lib or load_library()).moe_kv4_attention(
            qp, qs, hq, cache.pages_ptr, layer, cache.ref, batch.ref,
            d ** -0.5 if scale is None else scale, min(max(window, -1), _INT_MAX), tp, op, lp,
            workspace.data_ptr(),
            workspace.numel(), _raw_stream(stream, dev))
    if rc:
        ops._check(rc, "moe_kv4_attention")
    return out if lse is None else (out, lse)


# -------------------------------------------------------------------- pages --
def _ids(t, what, cache, n=None):
    _ints(t, what, cache.index)
    if len(t.shape) != 1 or (n is not None and t.numel() != n):
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
    sp, sb = cache.scratch(stream)
    with _on(cache.index):
        rc = (_lib or load_library()).moe_kv4_reserve(
            cache.ref, seqs.ref, ip, lp, n, sp, sb, cache.err_ptr,
            _raw_stream(stream, cache.index))
    if rc:
        ops._check(rc, "moe_kv4_reserve")


def moe_kv4_fork(cache: Cache, seqs: Sequences, parents, children, stream=None):
    """Empty sequences children become copies of parents: full pages are shared,
    a begun page is copied."""
    _pool_of(cache, seqs)
    n = parents.numel()
    pp, cp = _ids(parents, "parents", cache), _ids(children, "children", cache, n)
    sp, sb = cache.scratch(stream)
    with _on(cache.index):
        rc = (_lib or load_library()).moe_kv4_fork(
            cache.pages_ptr, cache.ref, seqs.ref, pp, cp, n, sp, sb, cache.err_ptr,
            _raw_stream(stream, cache.index))
    if rc:
        ops._check(rc, "moe_kv4_fork")


def moe_kv4_free(cache: Cache, seqs: Sequences, ids, stream=None):
    """Sequences ids give their pages back and become empty."""
    _pool_of(cache, seqs)
    n = ids.numel()
    ip = _ids(ids, "ids", cache)
    with _on(cache.index):
        rc = (_lib or load_library()).moe_kv4_free(cache.ref, seqs.ref, ip, n, cache.err_ptr,
                                                   _raw_stream(stream, cache.index))
    if rc:
        ops._check(rc, "moe_kv4_free")


def moe_kv4_compact(cache: Cache, seqs: Sequences, tables_out=None, refs_out=None, n_used=None,
                    stream=None):
    """Moves the pages in use to the lowest indices.  The new tables and refs are
    written in place, or to tables_out and refs_out.  Returns the number of pages
    in use (device int32 [1])."""
    _pool_of(cache, seqs)
    dev = cache.index
    tables_out = seqs.tables if tables_out is None else \
        _ints(tables_out, "tables_out", dev, seqs.tables.shape)
    refs_out = seqs.refs if refs_out is None else \
        _ints(refs_out, "refs_out", dev, seqs.refs.shape)
    if n_used is None:
        n_used = _empty(1, _I32, cache.device, stream)
    else:
        _ints(n_used, "n_used", dev, (1,))
    sp, sb = cache.scratch(stream)
    with _on(dev):
        rc = (_lib or load_library()).moe_kv4_compact(
            cache.pages_ptr, cache.ref, seqs.ref, tables_out.data_ptr(), refs_out.data_ptr(),
            n_used.data_ptr(), sp, sb, cache.err_ptr, _raw_stream(stream, dev))
    if rc:
        ops._check(rc, "moe_kv4_compact")
    return n_used


def moe_kv4_copy_pages(cache: Cache, src, dst, stream=None):
    """Page dst[i] becomes a copy of page src[i] in every layer (negative ids:
    skipped)."""
    n = src.numel()
    sp, dp = _ids(src, "src", cache), _ids(dst, "dst", cache, n)
    with _on(cache.index):
        rc = (_lib or load_library()).moe_kv4_copy_pages(
            cache.pages_ptr, cache.ref, sp, dp, n, cache.err_ptr,
            _raw_stream(stream, cache.index))
    if rc:
        ops._check(rc, "moe_kv4_copy_pages")
