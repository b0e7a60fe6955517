"""The router by groups where FP32 is at its end: sums whose parts cancel, biases of the
type's lowest value, distinct logits of equal scores, scores far below 1, and the gradient
entry by entry, against the definition in float64."""

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


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("E,groups,top", SHAPES)
def test_logits_about_zero(kind, T, E, groups, top):
    """All alike, alike but for a few, and small ones that 64 bits tell apart."""
    gen = torch.Generator().manual_seed(E)
    n, size = min(T, 60), E // groups
    l = torch.zeros(n, E)
    some = torch.tensor([0.0, -0.0, 2.0 ** -16, 2.0 ** -15, 1e-4, -1e-4, 1e-17, 1e-12])
    for first, m in ((n // 4, 2), (n // 2, 6), (3 * n // 4, 8)):
        l[first:] = some[:m][torch.randint(0, m, (n - first, E), generator=gen)]
    check(l, T, min(3, top * size), kind, None, groups, top, 1, renorm=False)


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


# ---------------------------------------------------------------- the gradient

def gradient(logits, experts, dweights, kind, renorm, scale):
    """The gradient in float64, and for each entry the magnitudes that errors go with: its
    score's slope times the sum of the magnitudes in its bracket."""
    T, E = logits.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        l = logits[t].astype(np.float64)
        s = groups_of.scores(l, kind)
        slots = np.nonzero(experts[t] >= 0)[0]
        at, g = experts[t][slots], dweights[t][slots].astype(np.float64)
        total = s[at].sum() if renorm else 1.0
        u = s[at] / total if total > 0 else np.zeros(len(at))
        if kind == "softmax" and not renorm:
            ds = np.zeros(E)
            ds[at] = g
            out[t] = s * scale * (ds - u @ g)
            size[t] = s * scale * (np.abs(ds) + u @ np.abs(g))
            continue
        slope = scale * u
        if kind == "sigmoid":
            slope = slope * (1 / (1 + np.exp(l[at])))
        if renorm:
            out[t, at] = slope * ((g[:, None] - g) @ u)
            size[t, at] = slope * (np.abs(g[:, None] - g) @ u)
        else:
            out[t, at] = slope * g
            size[t, at] = np.abs(slope * g)
    return out, size


def check_gradient(l, rows, k, kind, bias, groups, top, renorm, scale, gen):
    """The gradient of rows, l's values on the GPU; what the tolerance is for each entry."""
    dt, (T, E) = l.dtype, l.shape
    r = moe.route_grouped(rows, k, scores=kind, bias=bias, groups=groups, top_groups=top,
                          renormalize=renorm, scale=scale)
    experts = r.experts.cpu().numpy()
    dw = torch.randn(T, k, generator=gen)
    got = moe.route_grouped_backward(rows, r.experts, r.weights, dw.to(DEV), scores=kind,
                                     renormalize=renorm, scale=scale).double().cpu().numpy()
    want, size = gradient(l.float().numpy(), experts, dw.numpy(), kind, renorm, scale)
    oracle = groups_of.route_back(l.float().numpy(), experts, np.where(experts < 0, 0, dw.numpy()),
                                  kind, renorm, scale)
    # The oracle's sums of terms up to 2 scale g cancel: (k + 2) 2^-53 of that, 1e-14 at most.
    most = scale * dw.abs().max().item()
    assert np.all(np.abs(want - oracle) <= 1e-14 * most + 1e-14 * size)
    # The slope has a weight's or a score's error and 8 steps more (1 - s: exp within 2, a
    # sum, a quotient; products); the bracket a weight's, and 2 steps a term.
    tol = (2 * weight_tol(E) + (2 * k + 12) * 2.0 ** -23) * size
    if kind == "softmax" and not renorm:  # a score below the normal numbers counts as 0
        tol += 2.0 ** -126 * 2 * most
    tol += plain.step(dt) * np.abs(want)
    tol += torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    worst = np.max(np.abs(got - want) - tol)
    assert worst <= 0, worst
    return want, size, tol


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,groups,top,pad", [
    (3, 5, 2, 1, 1, 0), (70, 64, 4, 8, 2, 0), (70, 100, 5, 5, 2, 0), (40, 256, 8, 8, 4, 0),
    (40, 130, 8, 2, 1, 1), (30, 300, 8, 4, 2, 0), (30, 512, 8, 8, 4, 0), (30, 512, 8, 8, 4, 3),
    (20, 1001, 16, 7, 3, 0), (20, 1024, 16, 8, 4, 0)])
def test_gradient_entry_by_entry(dt, kind, renorm, T, E, k, groups, top, pad):
    gen = torch.Generator().manual_seed(E)
    l = (torch.randn(T, E, generator=gen) * 3).to(dt)
    l[1, E // 2:] = -INF
    rows = torch.zeros(T, E + pad, dtype=dt, device=DEV)[:, :E]  # pad: rows that are no pieces
    rows.copy_(l)
    bias = (torch.randn(E, generator=gen) * 0.05).to(DEV)
    want, size, tol = check_gradient(l, rows, k, kind, bias, groups, top, renorm, 2.5, gen)
    # What the tolerance can see: nearly every entry that is not 0.
    seen = size > 0
    if dt is not torch.float16:
        assert np.mean(np.abs(want[seen]) > tol[seen]) > 0.9


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 100])
@pytest.mark.parametrize("E", [48, 512])
def test_gradient_of_small_scores(kind, renorm, scale, E):
    gen = torch.Generator().manual_seed(E)
    for far in (40.0, 60.0, 80.0):
        l = torch.randn(20, E, generator=gen) - far
        if kind == "softmax":
            l[:, 1] = 0.0
        check_gradient(l, l.to(DEV), 6, kind, None, 1, 1, renorm, scale, gen)
