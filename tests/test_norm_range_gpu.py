"""Rows whose root mean square, or its reciprocal, leaves the normal numbers of fp32: the norm
itself is an ordinary number."""
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def layer():
    from weight_only_int4_moe_gb300 import layer as m
    m.load_library()
    return m


@pytest.mark.parametrize("hidden", [8, 100, 700, 1024, 9000, 32768])
@pytest.mark.parametrize("size", [1e-44, 1e-41, 1e-38, 1e-33, 1e33, 1e37, 5e37])
@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_rows_at_the_ends_of_the_range(layer, hidden, size, dtype):
    g = torch.Generator().manual_seed(hidden)
    x = (torch.randn(5, hidden, generator=g, dtype=torch.float64).clamp(-4, 4) * size).to(dtype)
    x[1, 1:] = 0  # one number of the row
    x[:, 0] = size
    w = 1 + 0.1 * torch.randn(hidden, generator=g)
    _, y = ref.add_norm(x, w, None, 0.0)
    got = layer.moe_add_norm(x.cuda(), w.cuda(), eps=0.0, out_dtype=FP32, codes=True)
    # three roundings under the root count half; root, reciprocal and two products, half a step of
    # fp32 at the end; a y that is no normal number itself is off by its own steps
    out, room = got.out.cpu().double(), 7 * ref.U * y.abs() + 2.0 ** -148
    values = got.codes.cpu().double() * got.scales.cpu().double()[:, None]
    # (bf16 does not hold 1e-44: a row of zeros and eps 0 are 0 / 0)
    there = ~y.isnan()
    assert torch.equal(there, x.any(-1, keepdim=True).expand(5, hidden))
    assert torch.equal(out.isnan(), ~there) and torch.equal(values.isnan(), ~there)
    assert ((out - y).abs() <= room)[there].all()
    room = (2.0 ** -4 * y.abs() + 2.0 ** -10 * got.scales.cpu().double()[:, None]) * (1 + 1e-5)
    assert ((values - y).abs() <= room)[there].all()


@pytest.mark.parametrize("size", [1e-42, 4e37])
def test_residual_at_the_ends_of_the_range(layer, size):
    """The sum that is kept is the sum, whatever the norm does with it."""
    g = torch.Generator().manual_seed(1)
    x, r = ((torch.randn(4, 520, generator=g, dtype=torch.float64).clamp(-4, 4) * size).float() for _ in range(2))
    h, y = ref.add_norm(x, None, r, 0.0)
    got = layer.moe_add_norm(x.cuda(), None, r.cuda(), eps=0.0, out_dtype=FP32)
    assert torch.equal(got.residual.cpu(), h)
    assert ((got.out.cpu().double() - y).abs() <= 7 * ref.U * y.abs() + 2.0 ** -148).all()
