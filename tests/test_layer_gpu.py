"""The operators between attention and experts on the GPU against plain forms in 64
bits, with tolerances from the roundings that the operators make."""
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF16, FP16, FP32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
INF = float("inf")


@pytest.fixture(scope="module")
def layer():
    from weight_only_int4_moe_gb300 import layer as m
    m.load_library()
    return m


def rng(seed):
    return torch.Generator().manual_seed(seed)


def strided(t, extra=16, offset=16):
    """t's values as a part of a wider buffer on the GPU, the rest of it NaN."""
    rows, cols = t.shape
    wide = torch.full((rows, cols + offset + extra), 127, dtype=torch.uint8) if t.dtype == E4M3 else \
        torch.full((rows, cols + offset + extra), float("nan"), dtype=t.dtype)
    wide = wide.view(t.dtype) if t.dtype == E4M3 else wide
    wide = wide.cuda()
    part = wide[:, offset:offset + cols]
    part.copy_(t.cuda())
    return part


def within(got, want, bound, dtype):
    """|got - want| within half a step of the type beyond `bound`."""
    got, want = got.double().cpu(), want
    room = bound + ref.half_step(want.abs() + bound, dtype)
    worst = ((got - want).abs() / room).max().item() if got.numel() else 0.0
    assert worst <= 1.0, worst


# ------------------------------------------------------------------- norm --
# rows x hidden: a thread, a warp, several; whole vectors and odd ends; more than one
# vector a thread; the largest
SIZES = [(1, 1), (3, 7), (5, 8), (2, 250), (4, 256), (7, 264), (3, 1411), (2, 7168), (2, 8200),
         (2, 9001), (1, 16392), (1, 32768), (1, 32761), (33, 128), (20, 1003), (9, 4095), (10, 5),
         (17, 1), (9, 8190), (5, 8188), (3, 32763)]


@pytest.mark.parametrize("rows,hidden", SIZES)
@pytest.mark.parametrize("x_type,res_type,w_type,out_type", [
    (BF16, BF16, BF16, BF16), (FP32, BF16, FP32, FP16), (FP16, FP32, FP16, FP32),
    (BF16, None, None, FP32), (FP32, FP16, BF16, BF16), (FP16, None, BF16, FP16)])
def test_add_norm(layer, rows, hidden, x_type, res_type, w_type, out_type):
    g = rng(rows * 40000 + hidden)
    x = (torch.randn(rows, hidden, generator=g) * torch.randn(1, hidden, generator=g).exp()).to(x_type)
    r = None if res_type is None else (3 * torch.randn(rows, hidden, generator=g)).to(res_type)
    w = None if w_type is None else (1 + 0.3 * torch.randn(hidden, generator=g)).to(w_type)
    h, y = ref.add_norm(x, w, r, 1e-6)
    got = layer.moe_add_norm(x.cuda(), None if w is None else w.cuda(), None if r is None else r.cuda(),
                             out_dtype=out_type, codes=True)
    if r is None:
        assert got.residual is None
    else:
        assert got.residual.dtype == res_type and torch.equal(got.residual.cpu(), h)
    # three roundings under the root count half; root, reciprocal and two products
    within(got.out, y, 6 * ref.U * y.abs(), out_type)
    assert got.out.dtype == out_type
    # the same bits as the operations in order; the codes of exactly these numbers
    y32 = ref.add_norm_fp32(h, w, 1e-6)
    assert torch.equal(got.out.cpu(), y32.to(out_type))
    scale = (y32.abs().amax(-1) * (1.0 / 448)).clamp(min=2.0 ** -100)
    assert torch.equal(got.scales.cpu(), scale)
    codes = (y32 * (1 / scale)[:, None]).to(E4M3)
    assert torch.equal(got.codes.cpu().view(torch.uint8), codes.view(torch.uint8))
    # and what they stand for: half a step of e4m3 (2^-4 relative, 2^-10 at least)
    values = got.codes.cpu().double() * got.scales.cpu().double()[:, None]
    room = 2.0 ** -4 * y.abs() + 2.0 ** -10 * scale.double()[:, None]
    assert ((values - y).abs() <= room * (1 + 1e-5)).all()


@pytest.mark.parametrize("hidden,offset", [(264, 16), (264, 3), (131, 8)])
def test_add_norm_of_parts_of_wider_rows(layer, hidden, offset):
    g = rng(hidden + offset)
    x, r = (torch.randn(6, hidden, generator=g).to(BF16) for _ in range(2))
    w = torch.randn(hidden, generator=g).to(BF16)
    xs, rs = strided(x, 16, offset), strided(r, 24, offset)
    out = torch.zeros(6, hidden + 40, dtype=BF16, device="cuda")
    codes = torch.zeros(6, hidden + 8, dtype=torch.uint8, device="cuda").view(E4M3)
    got = layer.moe_add_norm(xs, w.cuda(), rs, out=out[:, 8:8 + hidden], residual_out=rs,
                             codes=codes[:, :hidden])
    h, _ = ref.add_norm(x, w, r, 1e-6)
    y = ref.add_norm_fp32(h, w, 1e-6).to(BF16)
    assert torch.equal(out[:, 8:8 + hidden].cpu(), y) and got.residual is rs
    assert torch.equal(rs.cpu(), h)
    assert not out[:, :8].any() and not out[:, 8 + hidden:].any()
    assert not codes.view(torch.uint8)[:, hidden:].any()


def test_add_norm_in_place(layer):
    g = rng(1)
    x, r = (torch.randn(50, 512, generator=g).to(BF16).cuda() for _ in range(2))
    want = layer.moe_add_norm(x, None, r)
    got = layer.moe_add_norm(x, None, r, out=x, residual_out=r)
    assert got.out is x and got.residual is r
    assert torch.equal(x, want.out) and torch.equal(r, want.residual)


@pytest.mark.parametrize("size,eps", [(1e25, 1e-6), (3e30, 0.0), (1e-20, 0.0), (1e-30, 0.0), (1e-20, 1e-6)])
def test_add_norm_of_very_large_and_small_values(layer, size, eps):
    """Squares beyond fp32's range, or below it: the norm itself is an ordinary number."""
    x = torch.randn(4, 700, generator=rng(2)) * size
    _, y = ref.add_norm(x, None, None, eps)
    got = layer.moe_add_norm(x.cuda(), eps=eps, out_dtype=FP32).out
    within(got, y, 6 * ref.U * y.abs(), FP32)


@pytest.mark.parametrize("hidden", [64, 100, 9000])
def test_add_norm_rows_that_are_not_numbers(layer, hidden):
    """NaN and infinities stay in their rows; a row of zeros is zeros with codes of zero."""
    x = torch.randn(6, hidden, generator=rng(3))
    x[1, 5], x[2, 7], x[3], x[4, 3] = float("nan"), INF, 0.0, -INF
    x[4, 9] = INF
    got = layer.moe_add_norm(x.cuda(), out_dtype=FP32, codes=True)
    out = got.out.cpu()
    fine = [0, 5]
    alone = layer.moe_add_norm(x[fine].cuda(), out_dtype=FP32, codes=True)
    assert torch.equal(out[fine], alone.out.cpu())
    assert torch.equal(got.codes.view(torch.uint8)[fine], alone.codes.view(torch.uint8))
    assert out[1].isnan().all()
    for row, at in ((2, [7]), (4, [3, 9])):
        bad = torch.zeros(hidden, dtype=torch.bool)
        bad[at] = True
        assert torch.equal(out[row].isnan(), bad) and not out[row][~bad].any()
        assert torch.equal(got.codes[row].float().isnan().cpu(), bad)
    assert not out[3].any() and not got.codes[3].view(torch.uint8).any()
    assert got.scales[3].item() == 2.0 ** -100


def test_add_norm_outputs_that_are_not_wanted(layer):
    x = torch.randn(3, 256, generator=rng(4)).cuda()
    r = torch.randn(3, 256, generator=rng(5)).cuda()
    got = layer.moe_add_norm(x, out_dtype=None, codes=True)
    assert got.out is None and got.residual is None and got.codes is not None
    both = layer.moe_add_norm(x, codes=True)
    assert torch.equal(got.codes.view(torch.uint8), both.codes.view(torch.uint8))
    got = layer.moe_add_norm(x, None, r, out_dtype=None)
    assert got.out is None and got.codes is None and torch.equal(got.residual, x + r)
    empty = layer.moe_add_norm(x[:0], codes=True)
    assert empty.out.shape == (0, 256) and empty.scales.shape == (0,)


# ----------------------------------------------------------------- linear --
def codes_of(t):
    scale = t.abs().amax(-1) / 448
    return (t / scale[:, None]).to(E4M3), scale


def operands(m, n, k, dtype, seed):
    g = rng(seed)
    x, w = torch.randn(m, k, generator=g), torch.randn(n, k, generator=g) / k ** 0.5
    if dtype == E4M3:
        (x, sx), (w, sw) = codes_of(x), codes_of(w)
        return x, w, sx, sw
    return x.to(dtype), w.to(dtype), None, None


def gpu(t):
    return None if t is None else t.cuda()


def check_linear(layer, m, n, k, dtype, seed=0, act=None, bias=None, gate=None, residual=None,
                 out_dtype=FP32, wide=False):
    x, w, sx, sw = operands(m, n, k, dtype, seed)
    g = rng(seed + 1)
    b = None if bias is None else torch.randn(n, generator=g).to(bias)
    gt = None if gate is None else torch.randn(m, n, generator=g).to(gate)
    r = None if residual is None else torch.randn(m, n, generator=g).to(residual)
    pad = -k % 16
    put = (lambda t: strided(t, 16 + pad)) if wide or pad else gpu
    lin = layer.Linear(put(w), gpu(b), gpu(sw))
    got = layer.moe_linear(put(x), lin, act, gpu(gt), gpu(r), gpu(sx), out_dtype=out_dtype)
    want, bound = ref.linear(x, w, sx, sw, b, act, gt, r)
    assert got.dtype == out_dtype and got.shape == (m, n) and lin.errors() == 0
    within(got, want, bound, out_dtype)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 255, 256, 257, 300, 513])
@pytest.mark.parametrize("n,k", [(1, 8), (40, 64), (128, 72), (129, 640), (384, 4100)])
def test_linear_sizes(layer, m, n, k):
    check_linear(layer, m, n, k, BF16, seed=m + n)


@pytest.mark.parametrize("dtype", [FP16, E4M3])
@pytest.mark.parametrize("m,n,k", [(1, 300, 1000), (7, 1, 16), (40, 257, 129), (200, 130, 2050),
                                   (600, 515, 333), (1, 7168, 7168)])
def test_linear_types(layer, dtype, m, n, k):
    check_linear(layer, m, n, k, dtype, seed=m + k, wide=m > 1)


@pytest.mark.parametrize("k", [1, 3, 63, 64, 65, 127, 128, 129, 500, 513, 1023])
def test_linear_odd_sums(layer, k):
    """Sums that end inside a stage; what lies behind them in a row is NaN."""
    check_linear(layer, 20, 150, k, BF16, seed=k, wide=True)
    check_linear(layer, 20, 150, k, E4M3, seed=k, wide=True)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("m,n,k", [(1, 130, 9000), (90, 384, 7168), (200, 700, 5000), (2500, 520, 3000),
                                   (1300, 3001, 1700), (700, 5000, 800)])
def test_linear_long_sums_of_fp32_results(layer, dtype, m, n, k):
    """What a long product's single sum would lose shows in a result that stays fp32: no sum
    takes more than 12 stages (48 instructions, each cuts a step at most), and the sums are
    added up in fp32 (K / 384 of them at most, 64 elements a stage at least)."""
    x, w, sx, sw = operands(m, n, k, dtype, k)
    pad = -k % 16
    put = (lambda t: strided(t, 16 + pad)) if pad else gpu
    r = torch.randn(m, n, generator=rng(1))
    lin = layer.Linear(put(w), None, gpu(sw))
    got = layer.moe_linear(put(x), lin, None, None, r.cuda(), gpu(sx), out_dtype=FP32)
    assert lin.errors() == 0
    xd, wd = x.double().cuda(), w.double().cuda()
    y, size = xd @ wd.T, xd.abs() @ wd.abs().T
    if sx is not None:
        scale = sx.double().cuda()[:, None] * sw.double().cuda()
        y, size = y * scale, size * scale
    # a sum's share of the products, and 32 steps inside an instruction
    bound = size * 2 * ref.U * (48 + 32 + k / 384) + 4 * ref.U * y.abs()
    worst = ((got.double() - y - r.double().cuda()).abs() / (bound + ref.U * (y.abs() + r.abs().cuda()))).max()
    assert worst.item() <= 1.0
    # and over all elements: truncations of random sums are far below their bound
    rms = ((got.double() - y - r.double().cuda()).pow(2).mean() / y.pow(2).mean()).sqrt().item()
    assert rms <= 48 * 2 * ref.U


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu"])
@pytest.mark.parametrize("m,n,k", [(3, 200, 520), (90, 130, 2000), (300, 260, 130)])
@pytest.mark.parametrize("bias,gate,residual,out", [
    (BF16, None, BF16, BF16), (FP32, BF16, None, FP32), (None, FP16, FP16, FP16),
    (FP16, FP32, FP32, BF16)])
def test_linear_epilogue(layer, act, m, n, k, bias, gate, residual, out):
    check_linear(layer, m, n, k, BF16, 5, act, bias, gate, residual, out)
    check_linear(layer, m, n, k, E4M3, 6, act, bias, gate, residual, out)


@pytest.mark.parametrize("m,n,k", [(5, 300, 2048), (300, 333, 512), (2100, 1300, 256)])
def test_linear_of_parts_and_in_place(layer, m, n, k):
    """Output, gate and residual inside wider rows; the output over the residual or gate;
    nothing else is written."""
    x, w, _, _ = operands(m, n, k, BF16, 9)
    r, gt = (torch.randn(m, n, generator=rng(s)).to(BF16) for s in (1, 2))
    lin = layer.Linear(w.cuda())
    want = layer.moe_linear(x.cuda(), lin, "silu", gt.cuda(), r.cuda())
    for over in (0, 1):
        rs, gs = strided(r, 5, 3), strided(gt, 7, 2)
        out = (rs, gs)[over]
        whole = out._base.clone()
        got = layer.moe_linear(strided(x), lin, "silu", gs, rs, out=out)
        assert got is out and torch.equal(got, want)
        at = out.storage_offset()
        whole[:, at:at + n] = want
        assert torch.equal(whole.view(torch.int16), out._base.view(torch.int16))


def test_linear_repeats_its_bits(layer):
    for m, n, k in ((90, 384, 7168), (1, 7168, 4096), (700, 512, 512)):
        x, w, _, _ = operands(m, n, k, BF16, 3)
        x, lin = x.cuda(), layer.Linear(w.cuda())
        first = layer.moe_linear(x, lin, out_dtype=FP32)
        for _ in range(5):
            assert torch.equal(layer.moe_linear(x, lin, out_dtype=FP32), first)


def test_linear_rows_do_not_meet(layer):
    """A row or column that is not a number stays the only one."""
    x, w, _, _ = operands(140, 200, 333, BF16, 4)
    x[3, 7], x[130, 0], w[11, 5], w[199, 1] = float("nan"), INF, float("nan"), -INF
    put = lambda t: strided(t, 16 + 3)  # noqa: E731
    got = layer.moe_linear(put(x), layer.Linear(put(w)), out_dtype=FP32).cpu()
    bad = torch.zeros(140, 200, dtype=torch.bool)
    bad[[3, 130]] = True
    bad[:, [11, 199]] = True
    assert torch.equal(got.isfinite(), ~bad)


@pytest.mark.parametrize("m,n,k,dtype,out", [(3, 40, 70000, FP16, FP16), (140, 130, 40000, BF16, FP32),
                                             (5, 20, 1 << 20, E4M3, FP16)])
def test_linear_very_long_sums(layer, m, n, k, dtype, out):
    check_linear(layer, m, n, k, dtype, 3, out_dtype=out)


def test_linear_most_rows(layer):
    """The largest M, more row tiles than a grid's second dimension has at 16 rows each."""
    m, n, k = 1 << 20, 3, 16
    x = torch.randn(m, k, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF16)
    w = torch.randn(n, k, generator=rng(2)).to(BF16).cuda()
    lin = layer.Linear(w)
    got = layer.moe_linear(x, lin, out_dtype=FP32)
    want = x.double() @ w.double().T
    bound = (x.double().abs() @ w.double().abs().T) * 2 * ref.U * 33 + ref.U * want.abs()
    assert ((got.double() - want).abs() <= bound).all() and lin.errors() == 0


def test_offsets_beyond_32_bits(layer):
    """Matrices of more than 2^31 elements: the last rows are those of a small call."""
    g = torch.Generator("cuda").manual_seed(5)
    m, h = 540_000, 4096  # 2.2e9 elements
    tail = slice(m - 40, m)
    x = torch.zeros(m, h, dtype=BF16, device="cuda")
    r = torch.zeros(m, h, dtype=BF16, device="cuda")
    x[tail], r[tail] = torch.randn(40, h, generator=g, device="cuda"), torch.randn(40, h, generator=g, device="cuda")
    got = layer.moe_add_norm(x, None, r, codes=True, residual_out=r)
    again = layer.moe_add_norm(r[tail], out_dtype=BF16, codes=True)
    assert torch.equal(got.out[tail], again.out) and torch.equal(got.scales[tail], again.scales)
    assert torch.equal(got.codes.view(torch.uint8)[tail], again.codes.view(torch.uint8))
    assert not got.out[:8].any() and not got.codes.view(torch.uint8)[m // 2].any()
    del got, r
    w = torch.randn(4200, 64, generator=g, device="cuda").to(BF16)
    lin = layer.Linear(w)
    out = layer.moe_linear(x[:, :64], lin, residual=None)  # rows 8 KB apart, 2.27e9 results
    assert torch.equal(out[tail], layer.moe_linear(x[tail, :64].contiguous(), lin))
    del out
    ids, wts = layer.moe_route_experts(x[:, :1024], 4)  # rows of a wider matrix
    one = layer.moe_route_experts(x[tail, :1024].contiguous(), 4)
    assert torch.equal(ids[tail], one[0]) and torch.equal(wts[tail], one[1])
    assert lin.errors() == 0


def test_first_calls_in_a_capture():
    """Nothing that a kernel's first call sets up keeps it out of a captured graph."""
    import os
    import subprocess
    import sys
    code = """
import torch
from weight_only_int4_moe_gb300 import layer
x, w = (torch.randn(r, 768, device="cuda").to(torch.bfloat16) for r in (300, 640))
y, v = (torch.randn(r, 768, device="cuda").to(torch.bfloat16) for r in (4000, 3008))
a, b = layer.Linear(w), layer.Linear(v)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    p = layer.moe_linear(x, a, out_dtype=torch.float32)
    q, r = layer.moe_linear(y, b), layer.moe_linear(y, b, out_dtype=torch.float32)
    s, t = layer.moe_add_norm(p, residual=p), layer.moe_route_experts(p[:, :256], 8, "sigmoid")
g.replay()
torch.cuda.synchronize()
assert torch.equal(p, layer.moe_linear(x, a, out_dtype=torch.float32))
assert torch.equal(q, layer.moe_linear(y, b))
assert torch.equal(r, layer.moe_linear(y, b, out_dtype=torch.float32))
assert torch.equal(s.out, layer.moe_add_norm(p, residual=p).out)
assert torch.equal(t[0], layer.moe_route_experts(p[:, :256], 8, "sigmoid")[0])
assert a.errors() == b.errors() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_linear_without_rows(layer):
    lin = layer.Linear(torch.zeros(64, 64, dtype=BF16, device="cuda"))
    assert layer.moe_linear(torch.zeros(0, 64, dtype=BF16, device="cuda"), lin).shape == (0, 64)


def test_linear_refuses(layer):
    w = torch.zeros(64, 72, dtype=BF16, device="cuda")
    x = torch.zeros(4, 72, dtype=BF16, device="cuda")
    lin = layer.Linear(w)
    for bad in (x.half(), x.float()):
        with pytest.raises(TypeError):
            layer.moe_linear(bad, lin)
    with pytest.raises(ValueError):
        layer.moe_linear(x[:, :64], lin)
    with pytest.raises(ValueError):
        layer.moe_linear(x.T.contiguous().T, lin)
    with pytest.raises(ValueError):
        layer.moe_linear(x, lin, "tanh")
    with pytest.raises(ValueError):
        layer.moe_linear(x, lin, residual=x)
    with pytest.raises(TypeError):
        layer.moe_linear(x, lin, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        layer.moe_linear(x.cpu(), lin)
    with pytest.raises(RuntimeError):  # rows at multiples of 8 bytes
        layer.moe_linear(torch.zeros(4, 76, dtype=BF16, device="cuda")[:, :72], lin)
    with pytest.raises(ValueError):
        layer.Linear(torch.zeros(64, 76, dtype=BF16, device="cuda")[:, :72])
    with pytest.raises(ValueError):
        layer.Linear(w, bias=torch.zeros(72, device="cuda"))
    with pytest.raises(TypeError):
        layer.Linear(w.float())


# ---------------------------------------------------------------- routing --
def check_route(layer, logits, top_k, bias=None, **how):
    want, weights = ref.route_experts(logits, top_k, bias=bias, **how)
    ids, w = layer.moe_route_experts(logits.cuda(), top_k, bias=gpu(bias), **how)
    assert torch.equal(ids.cpu(), want)
    # an exponential's argument is rounded (its size counts), exponential and division
    # within two steps, a sum of 5 additions after up to 32 in a lane
    finite = logits.double()[logits.double().abs() < 1e4]
    size = (finite.max() - finite.min()).item() if finite.numel() else 0.0
    room = (60 + 2 * size) * ref.U * weights.abs() + 1e-37
    assert ((w.cpu().double() - weights).abs() <= room).all()


@pytest.mark.parametrize("e", [1, 2, 8, 31, 32, 33, 64, 100, 128, 256, 300, 384, 512, 640, 1024])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_sizes(layer, e, scoring, with_bias):
    g = rng(e)
    logits = 2 * torch.randn(37, e, generator=g)
    bias = 0.05 * torch.randn(e, generator=g) if with_bias else None
    for k in {1, min(8, e), min(32, e)}:
        for renormalize in (True, False):
            check_route(layer, logits, k, bias, scoring=scoring, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("e,groups", [(256, 8), (64, 32), (60, 4), (384, 12), (1024, 2), (8, 8), (96, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("best", [1, 2])
def test_route_groups(layer, e, groups, scoring, with_bias, best):
    g = rng(e + groups)
    logits = 1.5 * torch.randn(50, e, generator=g)
    bias = 0.1 * torch.randn(e, generator=g) if with_bias else None
    for top_groups in {1, (groups + 1) // 2, groups}:
        k = min(6, e // groups * top_groups)
        check_route(layer, logits, k, bias, scoring=scoring, groups=groups, top_groups=top_groups,
                    group_best=best)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_route_logits_of_16_bits_and_strided(layer, dtype):
    g = rng(7)
    logits = torch.randn(200, 161, generator=g).to(dtype)  # many equal ones
    bias = (0.02 * torch.randn(161, generator=g)).to(dtype).float()
    for b in (None, torch.zeros(161), bias):
        check_route(layer, logits, 8, b, scoring="sigmoid")
    want = layer.moe_route_experts(logits.cuda(), 8, "sigmoid", bias.cuda())
    got = layer.moe_route_experts(strided(logits, 3, 1), 8, "sigmoid", bias.cuda())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_near_ties(layer, scoring):
    """Scores that fp32 cannot tell apart, or orders wrongly, in every order; equal ones by
    the lower index."""
    g = rng(11)
    e = 96
    rows = []
    for i in range(64):
        base = [12.0, 0.3, -4.0, 16.5][i % 4]
        near = base + torch.arange(e) * (abs(base) * 2.0 ** -23)
        rows.append(near[torch.randperm(e, generator=g)])
    logits = torch.stack(rows).float()
    steps = torch.randint(0, 3, (e,), generator=g) * 2.0 ** -26
    for bias in (torch.zeros(e), steps.float(), 8 + torch.zeros(e)):
        check_route(layer, logits, 8, bias, scoring=scoring)
        check_route(layer, logits, 8, bias, scoring=scoring, groups=8, top_groups=3)
        check_route(layer, logits, 8, bias, scoring=scoring, groups=8, top_groups=3, group_best=1)
    check_route(layer, logits, 8, None, scoring=scoring, groups=8, top_groups=3)
    equal = torch.zeros(5, e)
    check_route(layer, equal, 32, torch.zeros(e), scoring=scoring, groups=4, top_groups=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_experts(layer, scoring, renormalize, groups):
    """Logits of -inf, NaN and +inf, rows that leave nothing or one, biases that take an
    expert out: ids stay distinct and in range, the weights of what is not there are 0."""
    g = rng(13)
    e, k = 64, 8
    logits = torch.randn(12, e, generator=g)
    logits[0] = -INF
    logits[1] = float("nan")
    logits[2] = -INF
    logits[2, 37] = -50.0
    logits[3, ::2] = -INF
    logits[4, 10:] = float("nan")
    logits[5, 3], logits[5, 40] = INF, INF
    logits[6] = INF
    logits[7] = torch.finfo(torch.float32).min
    logits[8, :16] = -INF
    logits[9] = -120.0 + 0.1 * torch.arange(e)  # sigmoids that fp32 does not hold
    bias = 0.1 * torch.randn(e, generator=g)
    masks = bias.clone()
    masks[5:20], masks[33], masks[50] = -INF, float("nan"), INF
    for b in (None, bias, masks):
        for top_groups in {1, groups}:
            how = dict(scoring=scoring, renormalize=renormalize, groups=groups, top_groups=top_groups)
            check_route(layer, logits, k, b, **how)
            ids, w = layer.moe_route_experts(logits.cuda(), k, bias=gpu(b), **how)
            assert w.isfinite().all() and ids.min() >= 0 and ids.max() < e
            assert (ids.sort(-1)[0].diff(dim=-1) > 0).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
def test_route_infinite_biases(layer, scoring, best):
    """Biases of +inf in more groups than are chosen, and in fewer: such groups and experts
    are equal, by the lower index."""
    g = rng(15)
    logits = torch.randn(6, 96, generator=g)
    for at in ([4, 20, 21, 38, 43, 50, 70, 77, 95], [21, 50], [90]):
        bias = torch.randn(96, generator=g)
        bias[at] = INF
        for top_groups in (1, 6, 16):
            check_route(layer, logits, min(6 * top_groups, 26), bias, scoring=scoring, groups=16,
                        top_groups=top_groups, group_best=best)


def test_route_agrees_with_the_plain_router(layer):
    from weight_only_int4_moe_gb300 import ops
    logits = torch.randn(300, 384, generator=rng(17)).cuda()
    ids, w = ops.moe_route(logits, 8)
    got = layer.moe_route_experts(logits, 8)
    assert torch.equal(got[0], ids) and (got[1] - w).abs().max() <= 8 * ref.U


def test_route_many_tokens_and_none(layer):
    logits = torch.randn(70000, 16, generator=rng(19)).cuda()
    ids, _ = layer.moe_route_experts(logits, 3, scoring="sigmoid")
    assert torch.equal(ids.long(), torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :3])
    ids, w = layer.moe_route_experts(logits[:0], 3)
    assert ids.shape == w.shape == (0, 3)


def test_route_refuses(layer):
    x = torch.zeros(2, 64, device="cuda")
    with pytest.raises(RuntimeError):
        layer.moe_route_experts(x, 65)
    with pytest.raises(RuntimeError):
        layer.moe_route_experts(x, 8, groups=5)
    with pytest.raises(ValueError):
        layer.moe_route_experts(x, 8, scoring="tanh")
    with pytest.raises(ValueError):
        layer.moe_route_experts(x, 8, bias=torch.zeros(63, device="cuda"))
    with pytest.raises(TypeError):
        layer.moe_route_experts(x.double(), 8)
