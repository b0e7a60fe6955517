"""The router by groups where FP32 is at its end: sums whose parts cancel, biases of the
type's lowest value, distinct logits of equal scores, scores far below 1, and the gradient
entry by entry, against the definition in float64."""
import math

import numpy as np
import pytest
import torch

from all_movement_amd import moe
from tests import moe_plain as plain
from tests import moe_plain_groups as groups_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
INF = float("inf")
LOWEST = torch.finfo(torch.float32).min
# One workgroup with a wave to each token and with four tokens to a wave; three launches
# with either (more than 256 experts or 16 groups: always a wave to each).
TOKENS = [7, 21, 200, 2400]
# (E, groups, top): groups of whole lanes and of parts of them, in rows of lanes (up to
# 256 experts and 16 groups) and in waves.
SHAPES = [(4, 2, 1), (60, 5, 2), (64, 8, 3), (256, 8, 4), (256, 64, 9), (300, 5, 2), (512, 8, 3)]


def weight_tol(E):
    """exp's argument rounded (half a step of up to 70), exp within 2 steps, E + 8 steps of
    additions, quotient and scale 3: (2 * 35 + 4 + 3 + E + 8) * 2^-23 at most, as the sum has
    the same errors."""
    return (96 + E) * 2.0 ** -23


def check(some, T, k, kind, bias=None, groups=1, top=1, best=2, renorm=True, scale=1.0):
    """T tokens that take the rows of ``some`` in turn; experts and weights of each."""
    n, E = some.shape
    print("bounds", T, E, k, kind, groups, top, best, renorm, scale, flush=True)
    at = torch.arange(T) % n
    r = moe.route_grouped(some[at].to(DEV), k, scores=kind,
                          bias=None if bias is None else bias.to(DEV), groups=groups,
                          top_groups=top, group_best=best, renormalize=renorm, scale=scale)
    experts, weights, _, _, _ = groups_of.route(
        some.float().numpy(), k, kind, None if bias is None else bias.numpy(), groups, top, best,
        renorm, 1.0)
    weights *= scale  # last: times scores of e^-700 first it would leave float64
    assert np.array_equal(r.experts.cpu().numpy(), experts[at.numpy()])
    want, got = weights[at.numpy()], r.weights.cpu().numpy()
    # Half of the smallest number where a weight is below the normal ones.
    assert np.all(np.abs(got - want) <= weight_tol(E) * want + 2.0 ** -150)
    return r


# ---------------------------------------------------------------- groups

def cancelling(n, E, groups, B, kind, seed):
    """Tokens whose groups' two best sums are near +B and -B and add up to nearly the same:
    they differ by what FP32 loses of each."""
    gen = torch.Generator().manual_seed(seed)
    size = E // groups
    bias = torch.full((groups, size), -4.0 * B)
    bias[:, 0] = B * (1 + torch.arange(groups) / groups)
    bias[:, 1] = -bias[:, 0]
    base = torch.randn(n, 1, size, generator=gen) * 0.5
    off = B * 2.0 ** -23 * (4 if kind == "sigmoid" else E)
    l = base + off * torch.randn(n, groups, size, generator=gen)
    return l.reshape(n, E), bias.reshape(E)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("E,groups,top", SHAPES)
def test_group_sums_that_cancel(kind, T, E, groups, top):
    for B in (4.0, 64.0, 1000.0):
        l, bias = cancelling(min(T, 80), E, groups, B, kind, E)
        check(l, T, 2, kind, bias, groups, top)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("E,groups,top", SHAPES)
@pytest.mark.parametrize("B", [4.0, 1000.0])
def test_large_biases_of_both_signs(kind, T, E, groups, top, B):
    gen = torch.Generator().manual_seed(E + T)
    l = torch.randn(min(T, 50), E, generator=gen)
    bias = torch.where(torch.rand(E, generator=gen) < 0.5, -B, B)
    for best in (1, 2):
        check(l, T, 2, kind, bias, groups, top, best)
        check(l, T, 2, kind, bias * torch.rand(E, generator=gen), groups, top, best)


def test_four_experts_that_cancel():
    l = torch.tensor([[-0.428161740, 0.256157368, 0.254069805, -0.426022798]])
    for T in TOKENS:
        r = check(l, T, 2, "sigmoid", torch.tensor([64.0, -64.0, 64.0, -64.0]), 2, 1)
        assert bool((r.experts == torch.tensor([0, 1], device=DEV)).all())


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("E,groups,top", SHAPES)
def test_biases_of_the_lowest_value(kind, T, E, groups, top):
    """As a mask on whole groups and on single experts: they come last, but they come."""
    gen = torch.Generator().manual_seed(E)
    l = torch.randn(min(T, 25), E, generator=gen)
    size = E // groups
    k = min(16, top * size)
    for low in (LOWEST, -2.0 ** 127):
        bias = torch.randn(E, generator=gen) * 0.01
        bias[size:] = low  # all but the first group
        for best in (1, 2):
            r = check(l, T, k, kind, bias, groups, top, best)
            assert bool((r.experts >= 0).all())
            check(l, T, k, kind, bias, groups, groups, best)
        bias[1::2] = low
        check(l, T, k, kind, bias, groups, top)


# Logits of each kind that have equal scores in 64 bits: past 37 a sigmoid is 1, below -745
# it is 0, near 0 it is 1/2; softmax beside 0 has exp(l), 1 or 0.
LEVELS = {"sigmoid": [38.0, 40.0, 41.0, 55.0, 300.0, 1.0, -800.0, -900.0, LOWEST],
          "softmax": [0.0, -1e-17, -2e-17, -1.0, -800.0, -801.0, -900.0, LOWEST]}


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("E,groups,top", SHAPES)
def test_distinct_logits_of_equal_scores(kind, T, E, groups, top):
    """Groups of equal scores go by their number, without a bias too; experts by logits."""
    gen = torch.Generator().manual_seed(E)
    n, size = min(T, 60), E // groups
    levels = torch.tensor(LEVELS[kind])
    l = levels[torch.randint(0, len(levels), (n, E), generator=gen)]
    l[n // 2:] -= 1000  # a best logit of each group that is not the token's largest
    l[n // 2:].clamp_(min=LOWEST)
    at = torch.randint(0, len(levels), (n - n // 2, groups), generator=gen)
    l[n // 2:].view(-1, groups, size)[:, :, -1] = levels[at]
    if kind == "sigmoid":
        l[n // 4:n // 2] = torch.tensor([1e-17, 2e-17, -3e-17, 0.0])[
            torch.randint(0, 4, (n // 2 - n // 4, E), generator=gen)]
    for best in (1, 2):
        check(l, T, min(3, top * size), kind, None, groups, top, best, renorm=False)


def test_two_saturated_groups():
    l = torch.tensor([[40.0, 50.0], [40.0, 41.0]])
    for T in TOKENS:
        r = check(l, T, 1, "sigmoid", None, 2, 1, 1)
        assert bool((r.experts == 0).all())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T", TOKENS)
def test_groups_by_their_best_logit(dt, T):
    """Ordinary logits without a bias, many of them alike."""
    gen = torch.Generator().manual_seed(T)
    l = (torch.randn(min(T, 150), 96, generator=gen) * 8).round().div(4).to(dt)
    for kind in ("sigmoid", "softmax"):
        check(l, T, 5, kind, None, 12, 4, 1)
        check(l * 8, T, 5, kind, None, 12, 4, 1)


# ---------------------------------------------------------------- weights

@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("E,groups,top", [(60, 1, 1), (60, 5, 2), (256, 1, 1), (256, 8, 4),
                                          (300, 1, 1), (300, 5, 2)])
@pytest.mark.parametrize("scale", [2.0 ** -100, 1.0, 2.0 ** 100])
def test_weights_of_small_scores(T, E, groups, top, scale):
    """Scores far below 1, and scales of the whole range: a weight is as near as others."""
    gen = torch.Generator().manual_seed(E)
    l = torch.randn(min(T, 60), E, generator=gen)
    for far in (42.0, 62.0, 69.0, 85.0, 100.0):
        for renorm in (True, False):
            check(l - far, T, 6, "sigmoid", None, groups, top, 1, renorm, scale)
            m = l - far
            m[:, 0] = 0.0  # softmax: one above all others
            check(m, T, 6, "softmax", None, groups, top, 1, renorm, scale)
    m = l - 700.0
    check(m, T, 6, "sigmoid", None, groups, top, 1, True, scale)
    m[:, 0] = 0.0
    bias = torch.zeros(E)
    bias[0] = -2.0  # its group does without it
    check(m, T, 6, "softmax", bias, groups, top, 1, True, scale)
    # Masked by the lowest value: their scores are 0.
    m[:, 1:] = LOWEST
    check(m, T, 6, "softmax", None, groups, top, 1, True, scale)
