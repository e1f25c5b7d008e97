"""Groups that rank by the sum of their two best experts' scores, where the biases make the two
terms much larger than their sum: what fp32 decides is bounded by the terms, not by the sum."""
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
INF = float("inf")
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module")
def layer():
    from weight_only_int4_moe_gb300 import layer as m
    m.load_library()
    return m


def check(layer, logits, bias, top_k, **how):
    want, weights = ref.route_experts(logits, top_k, bias=bias, **how)
    ids, w = layer.moe_route_experts(logits.cuda(), top_k, bias=bias.cuda(), **how)
    assert torch.equal(ids.cpu(), want)
    # exponentials of |x| <= 20 (their argument's rounding counts) and divisions within two
    # steps, a sum of up to 37 additions
    assert ((w.cpu().double() - weights).abs() <= 100 * ref.U * weights.abs()).all()


def test_two_groups_by_hand(layer):
    """u = 2^-13: the sums differ by 2.7e-5, the terms' rounding by 1.2e-4."""
    u = 2.0 ** -13
    logits = 4 * u * torch.tensor([[0.51, 0, 0, 0, 0.49, 0.24, 0, 0]])
    bias = torch.tensor([1024.0, -1024.0, -5000.0, -5000.0] * 2)
    want, _ = ref.route_experts(logits, 2, "sigmoid", bias, 2, 1, 2)
    assert want.tolist() == [[4, 5]]
    check(layer, logits, bias, 2, scoring="sigmoid", groups=2, top_groups=1)


def near_groups(tokens, groups, size, seed):
    """Logits a, e - a and lower ones in each group: with equal biases the groups' sums of two
    sigmoids differ by some e / 4."""
    g = torch.Generator().manual_seed(seed)
    x = -3 + 0.1 * torch.randn(tokens, groups, size, generator=g)
    a = 0.5 * torch.randn(tokens, groups, generator=g)
    x[:, :, 0] = a
    x[:, :, 1] = 1e-4 * torch.randn(tokens, groups, generator=g) - a
    return x.flatten(1)


@pytest.mark.parametrize("large", [4.0, 16.0, 100.0, 1000.0, 1e4, 1e6])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_terms_that_cancel(layer, large, scoring):
    groups, size = 8, 8
    logits = near_groups(400, groups, size, int(large))
    one = torch.full((size,), -10 * large)
    one[0], one[1] = large, -large
    for top_groups in (1, 3, 7):
        check(layer, logits, one.repeat(groups), 2, scoring=scoring, groups=groups, top_groups=top_groups)
    # each group at a size of its own, either sign first
    sizes = large * 2.0 ** -torch.arange(groups) * torch.tensor([1.0, -1.0] * (groups // 2))
    bias = torch.full((groups, size), -10 * large)
    bias[:, 0], bias[:, 1] = sizes, -sizes
    check(layer, logits, bias.flatten(), 2, scoring=scoring, groups=groups, top_groups=3)


@pytest.mark.parametrize("e,groups", [(256, 8), (96, 3), (64, 32), (384, 12)])
def test_terms_that_cancel_in_other_layouts(layer, e, groups):
    size = e // groups
    logits = near_groups(200, groups, size, e)
    one = torch.full((size,), -5000.0)
    one[0], one[1] = 300.0, -300.0
    for top_groups in {1, groups // 2}:
        check(layer, logits, one.repeat(groups), 2, scoring="sigmoid", groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("mask", [-1e9, -1e30, LOWEST])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
def test_masks_that_are_large_numbers(layer, mask, scoring, best):
    """Biases that take experts out by a large negative number: whole groups, all but one of a
    group, and groups beside others that -inf takes out (which come after them).  The sum of two
    of the type's lowest value is below fp32."""
    groups, size = 8, 8
    logits = near_groups(60, groups, size, 5)
    for case in range(4):
        bias = 0.01 * torch.randn(groups, size, generator=torch.Generator().manual_seed(case))
        bias[5] = mask
        if case >= 1:
            bias[2, 1:] = mask
        if case >= 2:
            bias[0], bias[3] = -INF, mask
        if case == 3:
            bias[1:5] = -INF
            bias[6:, :7] = mask
        for top_groups in (1, 3, 4, 6):
            check(layer, logits, bias.flatten(), 6, scoring=scoring, groups=groups, top_groups=top_groups,
                  group_best=best)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_sums_beyond_fp32(layer, scoring):
    """Two biases near the largest number, in more groups than are chosen; one group has +inf."""
    groups, size = 4, 4
    logits = near_groups(30, groups, size, 9)
    big = torch.tensor([3.0e38, 2.0e38, 2.5e38, 1.5e38])
    for at in (None, 3):
        bias = torch.zeros(groups, size)
        bias[:, 0] = big
        bias[:, 1] = torch.tensor([1.0e38, 3.0e38, 2.0e38, 3.2e38])
        if at is not None:
            bias[at, 2] = INF
        for top_groups in (1, 2, 3):
            check(layer, logits, bias.flatten(), 2, scoring=scoring, groups=groups, top_groups=top_groups)
            check(layer, logits, -bias.flatten().clamp(max=3e38), 2, scoring=scoring, groups=groups,
                  top_groups=top_groups)
