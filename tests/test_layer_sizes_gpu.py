"""Sizes beyond 32 bits are refused by the binding, and not taken modulo 2^32."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
MANY = 2 ** 32 + 1  # 1 in 32 bits


@pytest.fixture(scope="module")
def layer():
    from weight_only_int4_moe_gb300 import layer as m
    m.load_library()
    return m


def rows(n, cols, dtype=BF16):
    """n rows that are one and the same."""
    return torch.zeros(1, cols, dtype=dtype, device="cuda").expand(n, cols)


@pytest.mark.parametrize("n,error", [((1 << 20) + 1, RuntimeError), (MANY, ValueError)])
def test_more_rows_than_a_call_takes(layer, n, error):
    x = rows(n, 16)
    one = layer.Linear(torch.zeros(16, 16, dtype=BF16, device="cuda"))
    with pytest.raises(error):
        layer.moe_add_norm(x, out=rows(n, 16))
    with pytest.raises(error):
        layer.moe_linear(x, one, out=rows(n, 16))
    with pytest.raises(error):
        layer.moe_route_experts(x, 2)
    if n > 2 ** 31:
        with pytest.raises(ValueError):
            layer.Linear(x)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("name", ["top_k", "groups", "top_groups", "group_best"])
def test_numbers_beyond_32_bits(layer, name, sign):
    how = dict(top_k=2, groups=2, top_groups=1, group_best=1)
    logits = torch.zeros(3, 8, device="cuda")
    layer.moe_route_experts(logits, **how)
    how[name] += sign * 2 ** 32
    with pytest.raises(ValueError):
        layer.moe_route_experts(logits, **how)
