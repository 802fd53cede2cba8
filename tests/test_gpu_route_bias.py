"""GPU: routing with biases at the ends of fp32's range, where a group's score
of two candidates leaves it: masks of the type's lowest value, and +inf, which
counts as the largest finite value."""
import math

import pytest
import torch

import step_reference as ref
from gpu_util import note

pytestmark = pytest.mark.gpu

LOW, HIGH = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
# experts, groups: whole power-of-two lanes of the 16 (64, 256, 512), other groups (96), none (40, 1000)
SHAPES = [(64, 8), (256, 4), (512, 2), (96, 3), (40, 1), (1000, 1)]


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


def _check(dt, e, k, groups, stay, bias, score, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(37, e, generator=g, device="cuda")
    b = bias.cuda()
    ex, we = torch.empty(37, k, dtype=torch.int32, device="cuda"), torch.empty(37, k, device="cuda")
    dt.dt_moe_route([x], [ex], [we], bias=b, groups=groups, topk_groups=stay, score=score)
    want, w, err = ref.route(x, k, bias=b.clamp(max=HIGH), groups=groups, topk_groups=stay, score=score)
    assert torch.equal(ex.long().cpu(), want), (ex.long().cpu() != want).nonzero()[:4]
    ref.assert_close(we, w, err, "weights")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", SHAPES)
def test_experts_masked_by_the_lowest_value(dt, e, groups, score):
    """All groups but the first are masked: the second group that stays is the first masked one, and it fills the slots that
    the first leaves."""
    note(f"route masked by the lowest value, {e} in {groups} {score}")
    per = e // groups
    bias = torch.full((e,), LOW)
    bias[:5] = 0.25
    bias[5:per] = -math.inf
    _check(dt, e, 8, groups, min(2, groups), bias, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", SHAPES)
@pytest.mark.parametrize("top", [3e38, math.inf])
def test_groups_that_are_forced(dt, e, groups, score, top):
    """Two experts of the last group are forced, one of the first: the sum of two decides between the groups."""
    note(f"route forced {top}, {e} in {groups} {score}")
    per = e // groups
    bias = torch.zeros(e)
    bias[2] = top
    bias[3] = 2e38
    bias[e - 1] = bias[e - per] = top
    _check(dt, e, 2, groups, 1, bias, score)


@pytest.mark.parametrize("e,groups", SHAPES)
def test_plus_infinity_is_the_largest_finite_value(dt, e, groups):
    note(f"route +inf beside the largest value, {e} in {groups}")
    bias = torch.zeros(e)
    bias[1], bias[4], bias[e - 1] = HIGH, math.inf, HIGH
    _check(dt, e, 3, groups, groups, bias, "sigmoid")
    if groups > 1:
        _check(dt, e, 3, groups, groups - 1, bias, "softmax")
