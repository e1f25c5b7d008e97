"""The kernels of large products (two SMs a tile) against 64 bits, each case with the kernel
that it is about; their sums in parts; and all kernels at the same time on several streams."""
import threading

import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF16, FP16, FP32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def layer():
    from weight_only_int4_moe_gb300 import layer as m
    m.load_library()
    return m


def operands(m, n, k, dtype, seed):
    """(x, w, their scales) on the GPU; rows are parts of wider ones (of NaN) where they would
    not begin at multiples of 16 bytes."""
    g = torch.Generator("cuda").manual_seed(seed)
    got = []
    for rows, scale in ((m, 1.0), (n, k ** -0.5)):
        t = torch.randn(rows, k, generator=g, device="cuda") * scale
        s = None
        if dtype == E4M3:
            s = t.abs().amax(-1) / 448
            t = t / s[:, None]
        wide = torch.full((rows, -(-k // 16) * 16 + (16 if k % 16 else 0)), float("nan"), device="cuda").to(dtype)
        wide[:, :k] = t.to(dtype)
        got += [wide[:, :k], s]
    return got[0], got[2], got[1], got[3]


def random(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def within(got, want, bound, dtype):
    """|got - want| within half a step of the type beyond `bound`."""
    room = bound + ref.half_step(want.abs() + bound, dtype)
    worst = ((got.double() - want).abs() / room).max().item()
    assert worst <= 1.0, worst


# bias, activation, gate, residual, result
PLAIN = (None, None, None, None, BF16)
GATED = (BF16, "silu", BF16, FP32, BF16)
GELU = (FP32, "gelu", None, FP16, FP16)
RELU = (None, "relu", FP16, BF16, FP32)
STREAM = (None, None, None, BF16, BF16)

# M and N end inside tiles: 8200 = 32 x 256 + 8 and 2600 = 20 x 128 + 40 rows (the second block of
# the last tiles has none of x's, or the first one 40), 4950 = 19 x 256 + 86 columns (the second
# block's lie past the end); more tiles than pairs of SMs; up to 18 lines of k (1152 elements, 2304
# codes) the next tile's gate and residual are asked for ahead
CASES = [
    ("pairs_256", 4000, 3008, 768, BF16, PLAIN),
    ("pairs_256", 8200, 4950, 1024, BF16, GATED),
    ("pairs_256", 8200, 4951, 2048, BF16, GATED),
    ("pairs_256", 6000, 6000, 264, FP16, GELU),
    ("pairs_256", 8200, 4950, 700, FP16, RELU),
    ("pairs_256", 8200, 4950, 2048, E4M3, GATED),
    ("pairs_256", 8200, 4951, 4096, E4M3, STREAM),
    ("pairs_256", 4000, 3008, 1111, E4M3, GELU),
    ("pairs_128", 2600, 2100, 1000, BF16, GATED),
    ("pairs_128", 2600, 2101, 2048, BF16, GELU),
    ("pairs_128", 4200, 3900, 1000, FP16, STREAM),
    ("pairs_128", 2600, 2100, 768, BF16, RELU),
    ("pairs_128", 2600, 2100, 2048, E4M3, GATED),
    ("pairs_128", 2600, 2101, 4096, E4M3, PLAIN),
    ("pairs_128_sums", 1300, 3900, 1024, BF16, RELU),
    ("pairs_128_sums", 1300, 3901, 7168, FP16, (FP16, "silu", FP32, FP32, FP32)),
    ("pairs_128_sums", 1300, 3900, 4100, E4M3, RELU),
]


@pytest.mark.parametrize("kernel,m,n,k,dtype,how", CASES)
def test_pairs_against_64_bits(layer, kernel, m, n, k, dtype, how):
    x, w, sx, sw = operands(m, n, k, dtype, m + n + k)
    bias, act, gate, residual, out = how
    b = None if bias is None else random((n,), bias, 1)
    gt = None if gate is None else random((m, n), gate, 2)
    r = None if residual is None else random((m, n), residual, 3)
    lin = layer.Linear(w, b, sw)
    got = layer.moe_linear(x, lin, act, gt, r, sx, out_dtype=out)
    assert layer.moe_linear_last_kernel() == kernel and lin.errors() == 0
    want, bound = ref.linear(x.float(), w.float(), sx, sw, b, act, gt, r)
    within(got, want, bound, out)


@pytest.mark.parametrize("kernel,m,n,k,out,pads", [
    ("pairs_256", 8200, 4950, 2048, BF16, (8, 5)), ("pairs_256", 4000, 3008, 768, FP32, (8,)),
    ("pairs_128", 2600, 2100, 2048, BF16, (8, 5)), ("pairs_128_sums", 1300, 3900, 3000, FP32, (8, 5))])
def test_pairs_of_parts_and_in_place(layer, kernel, m, n, k, out, pads):
    """Gate and residual inside wider rows, at even and odd places; the output over either;
    nothing else is written."""
    x, w, _, _ = operands(m, n, k, BF16, 5)
    lin = layer.Linear(w)
    gt, r = random((m, n), out, 1), random((m, n), out, 2)
    want, bound = ref.linear(x.float(), w.float(), act="silu", gate=gt, residual=r)
    for pad, over in ((pad, over) for pad in pads for over in (0, 1)):
        wide = [torch.full((m, n + 2 * pad), float("nan"), dtype=out, device="cuda") for _ in range(2)]
        parts = [t[:, pad:pad + n] for t in wide]
        for part, t in zip(parts, (gt, r)):
            part.copy_(t)
        got = layer.moe_linear(x, lin, "silu", parts[0], parts[1], out=parts[over])
        assert layer.moe_linear_last_kernel() == kernel and lin.errors() == 0
        within(got, want, bound, out)
        assert wide[over][:, :pad].isnan().all() and wide[over][:, pad + n:].isnan().all()
        assert torch.equal(parts[1 - over], (gt, r)[1 - over])


@pytest.mark.parametrize("kernel,m,n,k,dtype", [
    ("pairs_128_sums", 1300, 3900, 7168, BF16), ("pairs_128_sums", 1300, 3900, 14336, E4M3),
    ("pairs_128_sums", 600, 8000, 7168, FP16), ("split", 90, 384, 7168, BF16), ("split", 2, 2048, 14336, E4M3),
    ("split", 256, 2048, 7168, BF16)])
def test_sums_in_parts_are_exact(layer, kernel, m, n, k, dtype):
    """A sum of 48 instructions: each cuts it at its last place, at most 2^-23 of what it has grown
    to, sqrt(i / 48) of the part for random terms, evenly: 2^-23 / sqrt 3 sum_i sqrt(i / 48) = 2.3e-6
    of the part at most, however the cuts go together, and so of the whole; its parts are added up
    with 2^-24 each.  One sum of 448 instructions has 7.9e-6 (measured)."""
    x, w, sx, sw = operands(m, n, k, dtype, k)
    lin = layer.Linear(w, None, sw)
    got = layer.moe_linear(x, lin, x_scale=sx, out_dtype=FP32).double()
    assert layer.moe_linear_last_kernel() == kernel and lin.errors() == 0
    want = x.double() @ w.double().T
    if sx is not None:
        want = want * sx.double()[:, None] * sw.double()
    assert ((got - want).pow(2).mean() / want.pow(2).mean()).sqrt().item() <= 2.5e-6


def test_all_kernels_at_the_same_time(layer):
    """Threads with a stream each: the kernels of large products beside each other and beside the
    small ones', norms and routings."""
    sizes = [("pairs_256", 4000, 3008, 768, BF16, BF16), ("pairs_128", 2600, 2100, 1000, BF16, BF16),
             ("pairs_128_sums", 1300, 3900, 1024, BF16, FP32), ("pairs_256", 8200, 4950, 2048, E4M3, BF16),
             ("split", 90, 384, 4096, BF16, FP32), ("split", 1, 7168, 2048, BF16, BF16),
             ("split", 300, 640, 512, FP16, FP16)]
    data, want = [], []
    for i, (kernel, m, n, k, dtype, out) in enumerate(sizes):
        x, w, sx, sw = operands(m, n, k, dtype, i)
        data.append((x, sx, layer.Linear(w, None, sw)))
        y = layer.moe_linear(x, data[i][2], x_scale=sx, out_dtype=out)
        assert layer.moe_linear_last_kernel() == kernel
        exact = x[:64].double() @ w.double().T
        if sx is not None:
            exact = exact * sx[:64].double()[:, None] * sw.double()
        assert ((y[:64].double() - exact).norm() / exact.norm()).item() <= 4e-3
        want.append((y, layer.moe_add_norm(y, codes=True).codes, *layer.moe_route_experts(y[:, :256], 8, "sigmoid")))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            kernel, _, _, _, _, out = sizes[i]
            x, sx, lin = data[i]
            stream = torch.cuda.Stream()
            for _ in range(15):
                y = layer.moe_linear(x, lin, x_scale=sx, out_dtype=out, stream=stream)
                codes = layer.moe_add_norm(y, codes=True, stream=stream).codes
                got = (y, codes, *layer.moe_route_experts(y[:, :256], 8, "sigmoid", stream=stream))
                stream.synchronize()
                if layer.moe_linear_last_kernel() != kernel or not all(
                        torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want[i])):
                    bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert all(lin.errors() == 0 for _, _, lin in data)
