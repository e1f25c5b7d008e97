"""Thin Python binding of the operators between attention and experts
(``include/moe_layer.h``): the residual's addition with the norm, matrix products with
their epilogue, and the routing to experts.  Argument checks and marshalling only; the
work is done by the CUDA library that ``ops`` loads, and calls raise where that is
missing.

Calls run on `stream`, or on the current one.  Outputs that are not given are made on
that stream; the caller orders its own tensors, and reads of the results, with it.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import ops
from .kv4 import _INT_MAX, _empty, _like, _raw_stream

MOE_T_BF16 = 0
MOE_T_F32 = 1
MOE_T_F16 = 2
MOE_T_E4M3 = 3
ACTIVATIONS = {"none": 0, None: 0, "relu": 1, "silu": 2, "gelu": 3}
SCORES = {"softmax": 0, "sigmoid": 1}

KERNELS = {0: None, 1: "split", 2: "pairs_128", 3: "pairs_128_sums", 4: "pairs_256"}  # of moe_linear

EXPORTED = ["moe_add_norm", "moe_linear", "moe_linear_last_kernel", "moe_route_experts"]

_TYPES = {torch.bfloat16: MOE_T_BF16, torch.float32: MOE_T_F32, torch.float16: MOE_T_F16}
_OPERANDS = {torch.bfloat16: MOE_T_BF16, torch.float16: MOE_T_F16,
             torch.float8_e4m3fn: MOE_T_E4M3}
_F32, _I32, _E4M3 = torch.float32, torch.int32, torch.float8_e4m3fn
_lib = None


def load_library():
    """The CUDA library with this module's signatures declared."""
    global _lib
    if _lib is None:
        lib = ops.load_library()
        p, i, i64, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        sig = {
            "moe_add_norm": ([p, i, i64, p, i, i64, p, i, f, i, i, p, i64, p, i, i64, p, i64, p, p], i),
            "moe_linear": ([p, i64, p, p, i64, p, i, p, i, p, i, i64, p, i, i64, p, i, i64, i, i, i, p,
                            p], i),
            "moe_linear_last_kernel": ([], i),
            "moe_route_experts": ([p, i, i64, p, i, i, i, i, i, i, i, i, f, p, p, p], i),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


# The checks below run before every launch and are kept short: a single-token step is
# bound by what the host does per call.
_here = torch._C._cuda_getDevice


def _device_of(t, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    return t.get_device()


def _matrix(t, what, index, shape, types):
    """(pointer, type, row stride) of a matrix whose rows are contiguous."""
    kind = types.get(t.dtype)
    if kind is None:
        raise TypeError(f"{what}: {t.dtype} is not supported")
    if t.get_device() != index:
        raise ValueError(f"{what}: expected a tensor on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected {tuple(shape)}, got {tuple(t.shape)}")
    rows, cols = t.stride()
    if cols != 1 and shape[1] > 1 and shape[0]:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    # (torch may say any stride for a single row; empty matrices have no rows to step)
    return t.data_ptr(), kind, rows if shape[0] > 1 else shape[1]


def _vector(t, what, index, n, dtype=_F32):
    if t.dtype is not dtype or t.shape != (n,):
        raise ValueError(f"{what}: expected {dtype} [{n}], got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor on cuda:{index}")
    return t.data_ptr()


def _call(fn, name, index, args):
    """fn(*args) with the tensors' device as the current one."""
    if _here() == index:
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc:
        ops._check(rc, name)


class Normed(NamedTuple):
    """What moe_add_norm returns; None for what was not asked for."""
    out: torch.Tensor | None
    residual: torch.Tensor | None
    codes: torch.Tensor | None
    scales: torch.Tensor | None


def moe_add_norm(x, weight=None, residual=None, eps: float = 1e-6, out_dtype=torch.bfloat16,
                 codes: bool | torch.Tensor = False, out=None, residual_out=None, scales=None,
                 stream=None) -> Normed:
    """The root-mean-square norm of h = x + residual over the last axis of x [rows,
    hidden] (bf16, fp16 or fp32), times weight [hidden].  h is rounded to the residual's
    type and returned as `residual` (residual_out may be the residual itself).  `out` is
    of out_dtype (None, with no out given: not wanted).  codes=True (or an e4m3 tensor):
    also e4m3 `codes` with a scale for each row, `scales` fp32 [rows]."""
    dev = _device_of(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x: expected [rows, hidden], got {tuple(x.shape)}")
    shape = x.shape
    rows, hidden = shape
    if rows > _INT_MAX or hidden > _INT_MAX:
        raise ValueError(f"x: {tuple(shape)} is too large")
    xp, xt, xs = _matrix(x, "x", dev, shape, _TYPES)
    rp, rt, rs, np_, ns = None, 0, 0, None, hidden
    if residual is not None:
        rp, rt, rs = _matrix(residual, "residual", dev, shape, _TYPES)
        if residual_out is None:
            residual_out = _empty(shape, residual.dtype, residual.device, stream)
            np_ = residual_out.data_ptr()
        else:
            if residual_out.dtype is not residual.dtype:
                raise TypeError(f"residual_out: expected {residual.dtype}, got {residual_out.dtype}")
            np_, _, ns = _matrix(residual_out, "residual_out", dev, shape, _TYPES)
    elif residual_out is not None:
        raise ValueError("residual_out: there is no residual")
    wp, wt = None, 0
    if weight is not None:
        wt = _TYPES.get(weight.dtype)
        if wt is None:
            raise TypeError(f"weight: {weight.dtype} is not supported")
        wp = _vector(weight, "weight", dev, hidden, weight.dtype)
    op, ot, os = None, 0, hidden
    if out is not None:
        op, ot, os = _matrix(out, "out", dev, shape, _TYPES)
    elif out_dtype is not None:
        ot = _TYPES.get(out_dtype)
        if ot is None:
            raise TypeError(f"out_dtype: {out_dtype} is not supported")
        out = _empty(shape, out_dtype, x.device, stream)
        op = out.data_ptr()
    cp, cs, sp = None, 0, None
    if codes is not False and codes is not None:
        if codes is True:
            codes = _empty(shape, _E4M3, x.device, stream)
        cp, _, cs = _matrix(codes, "codes", dev, shape, {_E4M3: 0})
        if scales is None:
            scales = _empty((rows,), _F32, x.device, stream)
        sp = _vector(scales, "scales", dev, rows)
    elif scales is not None:
        raise ValueError("scales: there are no codes")
    else:
        codes = None
    args = (xp, xt, xs, rp, rt, rs, wp, wt, eps, rows, hidden, np_, ns, op, ot, os, cp, cs, sp,
            _raw_stream(stream, dev))
    _call((_lib or load_library()).moe_add_norm, "moe_add_norm", dev, args)
    return Normed(out, residual_out, codes, scales)


class Linear:
    """The weights of a product, built once: weight [N, K] in bf16, fp16 or e4m3 codes
    (rows contiguous, beginning at multiples of 16 bytes), bias [N] (kept in fp32) and, for
    codes, scale fp32 [N].  It is made on the current stream, on which, or after which, its
    calls run.  ``errors`` reads the device error word of its calls."""

    def __init__(self, weight: torch.Tensor, bias=None, scale=None):
        dev = _device_of(weight, "weight")
        if weight.dim() != 2:
            raise ValueError(f"weight: expected [N, K], got {tuple(weight.shape)}")
        self.weight, self.index, self.device = weight, dev, weight.device
        self.N, self.K = weight.shape
        if self.N > _INT_MAX or self.K > _INT_MAX:
            raise ValueError(f"weight: {tuple(weight.shape)} is too large")
        self.ptr, self.type, self.stride = _matrix(weight, "weight", dev, weight.shape, _OPERANDS)
        self.dtype = weight.dtype
        self.scale, self.scale_ptr, self.bias, self.bias_ptr = scale, None, None, None
        if scale is not None:
            self.scale_ptr = _vector(scale, "scale", dev, self.N)
        if bias is not None:
            if bias.dtype not in _TYPES:
                raise TypeError(f"bias: {bias.dtype} is not supported")
            self.bias = bias.float().contiguous()
            self.bias_ptr = _vector(self.bias, "bias", dev, self.N)
        if self.ptr % 16 or (self.N > 1 and self.stride * weight.element_size() % 16):
            raise ValueError("weight: rows must begin at multiples of 16 bytes")
        self.err = torch.zeros(1, dtype=_I32, device=weight.device)
        self.err_ptr = self.err.data_ptr()

    def errors(self) -> int:
        """The device error flags accumulated so far; waits for the device."""
        torch.cuda.synchronize(self.device)
        return int(self.err.item()) & 0xFFFFFFFF

    def clear_errors(self):
        self.err.zero_()


def moe_linear(x, linear: Linear, activation=None, gate=None, residual=None, x_scale=None,
               out=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """activation(x weight^T [* x_scale * scale] + bias) * gate + residual, [M, N] of
    out's type or out_dtype (bf16, fp16 or fp32), summed in fp32 and rounded once.  x
    [M, K] has the weight's type; x_scale fp32 [M] (for codes).  gate and residual
    [M, N] are bf16, fp16 or fp32; out may be either of them.  activation: "relu",
    "silu", "gelu" or None."""
    dev = linear.index
    if x.dim() != 2:
        raise ValueError(f"x: expected [M, {linear.K}], got {tuple(x.shape)}")
    if x.dtype is not linear.dtype:
        raise TypeError(f"x: expected {linear.dtype}, got {x.dtype}")
    m = x.shape[0]
    if m > _INT_MAX:
        raise ValueError(f"x: {tuple(x.shape)} is too large")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation: {activation!r} is not one of {list(ACTIVATIONS)}")
    xp, _, xs = _matrix(x, "x", dev, (m, linear.K), _OPERANDS)
    shape = (m, linear.N)
    sp = None if x_scale is None else _vector(x_scale, "x_scale", dev, m)
    gp, gt, gs = (None, 0, 0) if gate is None else _matrix(gate, "gate", dev, shape, _TYPES)
    rp, rt, rs = (None, 0, 0) if residual is None else \
        _matrix(residual, "residual", dev, shape, _TYPES)
    if out is None:
        ot, os = _TYPES.get(out_dtype), linear.N
        if ot is None:
            raise TypeError(f"out_dtype: {out_dtype} is not supported")
        out = _empty(shape, out_dtype, linear.device, stream)
        op = out.data_ptr()
    else:
        op, ot, os = _matrix(out, "out", dev, shape, _TYPES)
    args = (xp, xs, sp, linear.ptr, linear.stride, linear.scale_ptr, linear.type, linear.bias_ptr,
            act, gp, gt, gs, rp, rt, rs, op, ot, os, m, linear.N, linear.K, linear.err_ptr,
            _raw_stream(stream, dev))
    _call((_lib or load_library()).moe_linear, "moe_linear", dev, args)
    return out


def moe_linear_last_kernel() -> str | None:
    """Which of its kernels (KERNELS) this thread's last moe_linear launched."""
    return KERNELS[(_lib or load_library()).moe_linear_last_kernel()]


def moe_route_experts(logits, top_k: int, scoring: str = "softmax", bias=None, groups: int = 1,
                      top_groups: int | None = None, group_best: int = 2, renormalize: bool = True,
                      scale: float = 1.0, topk_ids=None, topk_weights=None, stream=None):
    """(topk_ids int32 [M, top_k], topk_weights fp32 [M, top_k]) from router logits
    [M, E] (fp32, bf16 or fp16): the experts with the largest score + bias among the
    top_groups best groups (all by default), and their scores, renormalised to their sum,
    times scale.  scoring: "softmax" or "sigmoid".  group_best: groups compare by their
    best expert (1) or the sum of their two best (2)."""
    dev = _device_of(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits: expected [M, E], got {tuple(logits.shape)}")
    m, e = shape = logits.shape
    top_groups = groups if top_groups is None else top_groups
    if m > _INT_MAX or e > _INT_MAX:
        raise ValueError(f"logits: {tuple(shape)} is too large")
    how = (top_k, groups, top_groups, group_best)
    if max(how) > _INT_MAX or min(how) < -_INT_MAX:
        raise ValueError(f"(top_k, groups, top_groups, group_best): {how} is out of range")
    kind = SCORES.get(scoring)
    if kind is None:
        raise ValueError(f"scoring: {scoring!r} is not one of {list(SCORES)}")
    lp, lt, ls = _matrix(logits, "logits", dev, shape, _TYPES)
    bp = None if bias is None else _vector(bias, "bias", dev, e)
    size = (m, top_k)
    if topk_ids is None:
        topk_ids = _empty(size, _I32, logits.device, stream)
    else:
        _like(topk_ids, "topk_ids", dev, _I32, size)
    if topk_weights is None:
        topk_weights = _empty(size, _F32, logits.device, stream)
    else:
        _like(topk_weights, "topk_weights", dev, _F32, size)
    args = (lp, lt, ls, bp, m, e, top_k, kind, groups, top_groups, group_best,
            1 if renormalize else 0, scale, topk_ids.data_ptr(), topk_weights.data_ptr(),
            _raw_stream(stream, dev))
    _call((_lib or load_library()).moe_route_experts, "moe_route_experts", dev, args)
    return topk_ids, topk_weights


def moe_int4_forward_hidden(x, experts: ops.PackedWeights, router: Linear, scoring: str = "softmax",
                            bias=None, groups: int = 1, top_groups: int | None = None,
                            group_best: int = 2, renormalize: bool = True, scale: float = 1.0,
                            out=None, workspace=None, stream=None):
    """The expert layer from the tokens alone: router logits in fp32 (moe_linear; router's
    bias, if it has one, is added to them), their routing (moe_route_experts) and
    moe_int4_forward.  x bf16 [M, hidden].  Returns (out, topk_ids, topk_weights)."""
    shape = experts.shape
    if (router.N, router.K) != (shape.E, shape.hidden):
        raise ValueError(f"router: expected [{shape.E}, {shape.hidden}], got "
                         f"[{router.N}, {router.K}]")
    logits = moe_linear(x, router, out_dtype=_F32, stream=stream)
    ids, weights = moe_route_experts(logits, shape.top_k, scoring, bias, groups, top_groups, group_best,
                                     renormalize, scale, stream=stream)
    if out is None:
        out = _empty((x.shape[0], shape.hidden), shape.torch_out_dtype, x.device, stream)
    if workspace is None:
        n = max(ops.moe_int4_workspace_bytes(x.shape[0], shape), 256)
        workspace = _empty((n,), torch.uint8, x.device, stream)
        ops.moe_int4_clear_errors(workspace, stream)
    experts.forward(x, ids, weights, out=out, workspace=workspace, stream=stream)
    return out, ids, weights
