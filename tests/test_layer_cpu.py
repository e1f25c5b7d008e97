"""The C ABI of the operators between attention and experts without a GPU: the header
and the binding agree, and arguments are refused on the host before anything is
launched."""
import ctypes
import os
import re

import pytest
import torch

import layer_reference as ref
from weight_only_int4_moe_gb300 import layer, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_layer.h")
P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)
HALF = ctypes.c_void_p((1 << 20) + 8)
NULL, SHAPE, ALIGN = -1, -2, -3


def test_header_binding_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^(?:int|size_t)\s+(moe_[a-z0-9_]+)\s*\(", text, flags=re.M))
    assert names == set(layer.EXPORTED)
    lib = layer.load_library()
    for name in names:
        assert hasattr(lib, name)
    defs = dict(re.findall(r"^#define\s+(MOE_[A-Z0-9_]+)\s+(\d+)\b", text, flags=re.M))
    for name in ("MOE_T_BF16", "MOE_T_F32", "MOE_T_F16", "MOE_T_E4M3"):
        assert int(defs[name]) == getattr(layer, name)
    assert (ops.MOE_OUT_BF16, ops.MOE_OUT_F32) == (layer.MOE_T_BF16, layer.MOE_T_F32)
    for name, v in layer.ACTIVATIONS.items():
        assert int(defs["MOE_ACT_" + (name or "none").upper()]) == v
    for name, v in layer.SCORES.items():
        assert int(defs["MOE_SCORE_" + name.upper()]) == v


NORM = dict(x=P, x_type=0, x_stride=256, residual=P, residual_type=0, residual_stride=256, weight=P,
            weight_type=0, eps=1e-6, rows=4, hidden=256, residual_out=P, residual_out_stride=256,
            out=P, out_type=0, out_stride=256, codes=P, codes_stride=256, scales=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), SHAPE), (dict(rows=(1 << 20) + 1), SHAPE), (dict(hidden=0), SHAPE),
    (dict(hidden=32769, x_stride=40000, residual_stride=40000, residual_out_stride=40000,
          out_stride=40000, codes_stride=40000), SHAPE),
    (dict(eps=-1e-6), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(x_type=3), SHAPE), (dict(residual_type=3), SHAPE), (dict(weight_type=-1), SHAPE),
    (dict(out_type=3), SHAPE), (dict(x_stride=255), SHAPE), (dict(residual_stride=0), SHAPE),
    (dict(residual_out_stride=-256), SHAPE), (dict(out_stride=255), SHAPE),
    (dict(codes_stride=255), SHAPE), (dict(residual=None), SHAPE),
    (dict(scales=None), NULL), (dict(codes=None), NULL), (dict(x=None), NULL),
    (dict(x=ODD), ALIGN), (dict(residual=ODD), ALIGN), (dict(residual_out=ODD), ALIGN),
    (dict(weight=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(scales=ODD), ALIGN),
    (dict(rows=0, x=None), 0), (dict(residual_out=None, out=None, codes=None, scales=None), 0),
])
def test_add_norm_refuses(change, code):
    assert layer.load_library().moe_add_norm(*{**NORM, **change}.values()) == code


LINEAR = dict(x=P, x_stride=64, x_scale=P, w=P, w_stride=64, w_scale=P, type=0, bias=P, act=0,
              gate=P, gate_type=0, gate_stride=48, residual=P, residual_type=0, residual_stride=48,
              out=P, out_type=0, out_stride=48, M=4, N=48, K=60, err=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), SHAPE), (dict(M=(1 << 20) + 1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE),
    (dict(N=(1 << 20) + 1), SHAPE), (dict(K=(1 << 20) + 1), SHAPE), (dict(type=1), SHAPE),
    (dict(type=4), SHAPE), (dict(act=4), SHAPE), (dict(act=-1), SHAPE), (dict(x_stride=59), SHAPE),
    (dict(w_stride=-64), SHAPE), (dict(gate_stride=47), SHAPE), (dict(gate_type=3), SHAPE),
    (dict(residual_type=3), SHAPE), (dict(residual_stride=0), SHAPE), (dict(out_type=3), SHAPE),
    (dict(out_stride=47), SHAPE), (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(x=HALF), ALIGN), (dict(w=HALF), ALIGN), (dict(x_stride=68), ALIGN),
    (dict(w_stride=60), ALIGN), (dict(type=3, x_stride=72), ALIGN), (dict(x_scale=ODD), ALIGN),
    (dict(w_scale=ODD), ALIGN), (dict(bias=ODD), ALIGN), (dict(gate=ODD), ALIGN),
    (dict(residual=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(err=ODD), ALIGN),
    (dict(M=0, x=None, out=None), 0),
])
def test_linear_refuses(change, code):
    assert layer.load_library().moe_linear(*{**LINEAR, **change}.values()) == code


ROUTE = dict(logits=P, type=1, stride=64, bias=P, M=4, E=64, top_k=8, scoring=1, groups=8,
             top_groups=4, group_best=2, renormalize=1, scale=1.0, ids=P, weights=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), SHAPE), (dict(M=(1 << 20) + 1), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1032, stride=1032), SHAPE), (dict(type=3), SHAPE), (dict(stride=63), SHAPE),
    (dict(scoring=2), SHAPE), (dict(groups=0), SHAPE), (dict(groups=7), SHAPE),
    (dict(groups=64), SHAPE), (dict(top_groups=0), SHAPE), (dict(top_groups=9), SHAPE),
    (dict(group_best=3), SHAPE), (dict(group_best=0), SHAPE), (dict(renormalize=2), SHAPE),
    (dict(top_k=0), SHAPE), (dict(top_k=33), SHAPE), (dict(top_groups=1, top_k=9), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL),
    (dict(logits=HALF, type=0, bias=ODD), ALIGN), (dict(logits=ODD), ALIGN), (dict(ids=ODD), ALIGN),
    (dict(weights=ODD), ALIGN), (dict(M=0, logits=None), 0),
])
def test_route_experts_refuses(change, code):
    assert layer.load_library().moe_route_experts(*{**ROUTE, **change}.values()) == code


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        layer.moe_add_norm(x)
    with pytest.raises(ValueError):
        layer.Linear(x)
    with pytest.raises(ValueError):
        layer.moe_route_experts(x, 2)


def test_reference_routing():
    """The tests' own reference: by hand."""
    inf = float("inf")
    one = torch.tensor([[0.0, 3.0, 1.0, 3.0]])
    ids, w = ref.route_experts(one, 3)
    assert ids.tolist() == [[1, 3, 2]] and abs(w.sum() - 1) < 1e-15 and w[0, 0] == w[0, 1]
    ids, w = ref.route_experts(one, 2, scoring="sigmoid", bias=torch.tensor([9.0, 0, 0, -inf]),
                               renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 1]] and w[0, 0] == 1.0
    # groups {0, 1} and {2, 3}: the best alone, the two best together, one masked
    two = torch.tensor([[4.0, -9.0, 3.0, 3.0]])
    assert ref.route_experts(two, 1, "sigmoid", None, 2, 1, 1)[0].tolist() == [[0]]
    assert ref.route_experts(two, 1, "sigmoid", None, 2, 1, 2)[0].tolist() == [[2]]
    gone = torch.tensor([[-inf, float("nan"), -inf, 1.0]])
    ids, w = ref.route_experts(gone, 2, "softmax", None, 2, 1)
    assert ids.tolist() == [[3, 2]] and w.tolist() == [[1.0, 0.0]]
    ids, w = ref.route_experts(torch.full((1, 4), -inf), 2, "sigmoid")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


def test_header_is_plain_c(tmp_path):
    """The header by itself in a pedantic C11 program that links the library and is refused
    its arguments."""
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    layer.load_library()
    lib = ops.library_path()
    src, exe = tmp_path / "use.c", tmp_path / "use"
    src.write_text("""#include "moe_layer.h"
#include <stdio.h>
int main(void) {
    printf("%d\\n", moe_add_norm(0, MOE_T_BF16, 8, 0, 0, 0, 0, 0, 1e-6f, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0));
    printf("%d\\n", moe_linear(0, 8, 0, 0, 8, 0, MOE_T_E4M3, 0, MOE_ACT_SILU, 0, 0, 0, 0, 0, 0, 0,
                              MOE_T_F32, 8, 1, 8, 8, 0, 0));
    printf("%d\\n", moe_route_experts(0, MOE_T_F32, 8, 0, 0, 8, 2, MOE_SCORE_SIGMOID, 1, 1, 1, 1, 1.0f, 0, 0,
                                     0));
    return 0;
}
""")
    r = subprocess.run([gcc, "-std=c11", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), lib, "-Wl,-rpath," + os.path.dirname(lib),
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [SHAPE, NULL, 0]
