"""The router by groups and its gradient against the definition in float64."""
import numpy as np
import pytest
import torch

from all_movement_amd import moe
from tests import moe_plain as plain
from tests import moe_plain_groups as groups_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
INF, NAN = float("inf"), float("nan")
# Scores in FP32 at worst: exp's argument is rounded once (half a step of up to 20 in
# these tests), exp within 2 steps, the sums E + 8 steps of additions, quotient and
# scale within 3 steps: (20 + 20 + 10 + E + 8) * 2^-23 at most.


def weight_tol(E):
    return (64 + E) * 2.0 ** -23


def check(logits, k, kind="sigmoid", bias=None, groups=1, top=None, best=2, renorm=True, scale=1.0):
    top = groups if top is None else top
    T, E = logits.shape
    print("groups", T, E, k, kind, bias is not None, groups, top, best, renorm, scale, logits.dtype,
          flush=True)
    r = moe.route_grouped(logits.to(DEV) if not logits.is_cuda else logits, k, scores=kind,
                          bias=None if bias is None else bias.to(DEV), groups=groups,
                          top_groups=top, group_best=best, renormalize=renorm, scale=scale)
    got = [t.cpu().numpy() for t in r]
    want = groups_of.route(logits.float().cpu().numpy(), k, kind,
                           None if bias is None else bias.numpy(), groups, top, best, renorm, scale)
    for i in (0, 2, 3, 4):
        assert np.array_equal(got[i], want[i]), i
    assert np.array_equal(np.isnan(got[1]), np.isnan(want[1]))
    ok = ~np.isnan(want[1])
    assert np.all(np.abs(got[1] - want[1])[ok] <= weight_tol(E) * want[1][ok] + 1e-37)
    return r


SIZES = [(1, 1, 1, 1, 1), (3, 8, 2, 2, 1), (16, 256, 8, 8, 4), (37, 100, 5, 5, 2), (300, 256, 8, 8, 4),
         (129, 160, 6, 8, 3), (1000, 18, 3, 6, 3), (100, 1000, 16, 10, 4), (64, 512, 16, 64, 7),
         (65, 64, 16, 64, 20), (300, 1024, 8, 32, 8), (700, 6, 2, 1, 1), (1025, 3, 1, 3, 2),
         (49, 96, 4, 3, 1), (257, 44, 7, 4, 4), (9, 256, 8, 8, 4), (33, 120, 6, 10, 4),
         (2400, 256, 8, 8, 4), (2500, 96, 4, 3, 1), (3001, 60, 5, 12, 5)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("kind,best,renorm,biased,scale", [
    ("sigmoid", 2, True, True, 2.5), ("sigmoid", 1, False, True, 1.0), ("softmax", 1, False, False, 16.0),
    ("softmax", 2, True, True, 1.0), ("sigmoid", 2, True, False, 0.3)])
@pytest.mark.parametrize("T,E,k,groups,top", SIZES)
def test_against_definition(dt, kind, best, renorm, biased, scale, T, E, k, groups, top):
    gen = torch.Generator().manual_seed(T * 31 + E)
    l = (torch.randn(T, E, generator=gen) * 2).to(dt)
    bias = torch.randn(E, generator=gen) * (0.1 if kind == "sigmoid" else 0.3 / E) if biased else None
    check(l, k, kind, bias, groups, top, best, renorm, scale)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [5, 20, 900, 2400])
@pytest.mark.parametrize("biased", [True, False])
def test_ties_and_masks(T, kind, biased):
    gen = torch.Generator().manual_seed(9)
    l = torch.randint(-2, 3, (T, 72), generator=gen).float()
    l[l == 0] *= torch.where(torch.rand(int((l == 0).sum()), generator=gen) < 0.5, -1.0, 1.0)
    l[:, 3] = -INF                   # an expert that is off
    l[1] = -INF                      # a token without experts
    l[2] = -INF
    l[2, [5, 71]] = 1.0              # fewer experts than slots
    l[3] = torch.finfo(torch.float32).min  # masked by the lowest value: all alike
    l[4, :24] = -INF                 # groups without experts
    l[4, 36:] = -INF
    bias = torch.zeros(72) if biased else None
    r = check(l, 4, kind, bias, 6, 2)
    assert r.experts[1].tolist() == [-1] * 4
    assert sorted(r.experts[2].tolist()) == [-1, -1, 5, 71]
    assert all(24 <= e < 36 for e in r.experts[4].tolist())
    if bias is not None:
        bias[::2] = 0.25             # equal sums of unequal parts
        bias[7], bias[40:44] = -INF, -INF
        check(l, 4, kind, bias, 6, 3, 1)
        bias[9] = INF
        check(l, 4, kind, bias, 6, 2, 2)


def test_every_token_without_experts():
    for T in (6, 20, 300, 2400):
        r = check(torch.full((T, 40), -INF), 8, "softmax", None, 4, 2)
        assert r.counts.sum().item() == 0 and bool((r.order == -1).all())
        r = check(torch.full((T, 40), -INF), 8, "sigmoid", torch.zeros(40), 4, 2)
        assert r.counts.sum().item() == 0


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("times", [1, 3, 100, 350])
def test_logits_that_are_no_numbers(kind, biased, times):
    l = torch.randn(7, 20, generator=torch.Generator().manual_seed(1))
    l[0, 4] = NAN
    l[1, 7] = INF
    l[2, [3, 9]] = NAN
    l[3, [2, 5]] = INF
    l[4, 3], l[4, 16] = NAN, -INF
    l[5, :5], l[5, 11] = -INF, NAN
    l = l.repeat(times, 1)
    bias = torch.randn(20, generator=torch.Generator().manual_seed(2)) * 0.1 if biased else None
    for groups, top in ((1, 1), (4, 2), (5, 1)):
        for renorm in (True, False):
            check(l, 3, kind, bias, groups, top, 2, renorm)
    if biased:
        bias[6] = NAN
        check(l, 3, kind, bias, 4, 2)


@pytest.mark.parametrize("T", [7, 21, 200, 2400])
@pytest.mark.parametrize("E,groups,top", [(64, 1, 1), (64, 8, 3), (256, 8, 4), (100, 5, 2)])
def test_sums_that_only_64_bits_tell_apart(T, E, groups, top):
    """Biases that bring every score to the same number, up to their own rounding."""
    for seed in range(4):
        gen = torch.Generator().manual_seed(seed)
        for kind in ("sigmoid", "softmax"):
            l = torch.randn(1, E, generator=gen)
            s = groups_of.scores(l[0].double().numpy(), kind)
            bias = torch.from_numpy(0.75 - s).float()
            apart = np.diff(np.sort(s + bias.double().numpy()))
            assert apart.min() > 1e-14 and np.median(apart) < 1e-7
            check(l.repeat(T, 1), 6, kind, bias, groups, top)


def test_no_tokens():
    r = moe.route_grouped(torch.empty(0, 12, device=DEV), 3, groups=4, top_groups=2)
    assert r.counts.tolist() == [0] * 12 and r.order.numel() == 0
    assert moe.route_grouped_backward(torch.empty(0, 12, device=DEV), r.experts, r.weights,
                                      r.weights).shape == (0, 12)


@pytest.mark.parametrize("dt", DTYPES)
def test_strided_logits(dt):
    wide = torch.full((500, 41), 100.0, device=DEV, dtype=dt)
    wide[:, :32] = torch.randn(500, 32, device=DEV)
    bias = torch.randn(32) * 0.1
    check(wide[:, :32], 4, "sigmoid", bias, 4, 2)
    r = moe.route_grouped(wide[:, :32], 4, groups=4, top_groups=2)
    dw = torch.randn(500, 4, device=DEV)
    got = moe.route_grouped_backward(wide[:, :32], r.experts, r.weights, dw)
    assert torch.equal(got, moe.route_grouped_backward(wide[:, :32].contiguous(), r.experts,
                                                       r.weights, dw))


def test_one_group_without_a_bias_is_the_router():
    l = torch.randn(3000, 200, device=DEV)
    a = moe.route(l, 6, renormalize=False)
    b = moe.route_grouped(l, 6, scores="softmax", renormalize=False)
    assert all(torch.equal(x, y) for i, (x, y) in enumerate(zip(a, b)) if i != 1)
    assert bool(((a.weights - b.weights).abs() <= weight_tol(200) * a.weights).all())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,groups,top", [
    (1, 1, 1, 1, 1), (5, 64, 2, 8, 2), (300, 100, 5, 5, 2), (33, 1024, 16, 8, 4), (9, 130, 8, 2, 1),
    (4100, 48, 8, 4, 2)])
def test_gradient(dt, kind, renorm, T, E, k, groups, top):
    gen = torch.Generator().manual_seed(E)
    l = (torch.randn(T, E, generator=gen) * 2).to(dt)
    if T > 2 and E > k:
        l[1::13] = -INF
        l[2::13, 1:] = -INF
        l[0, E // 2] = -INF
    l = l.to(DEV)
    bias = (torch.randn(E, generator=gen) * 0.05).to(DEV)
    scale = 2.5
    r = moe.route_grouped(l, k, scores=kind, bias=bias, groups=groups, top_groups=top,
                          renormalize=renorm, scale=scale)
    dw = torch.randn(T, k, generator=gen).to(DEV)
    dw[r.experts < 0] = NAN  # an empty slot's gradient is not read
    got = moe.route_grouped_backward(l, r.experts, r.weights, dw, scores=kind, renormalize=renorm,
                                     scale=scale).double().cpu().numpy()
    dw = np.nan_to_num(dw.cpu().numpy())
    want = groups_of.route_back(l.float().cpu().numpy(), r.experts.cpu().numpy(), dw, kind, renorm,
                                scale)
    # The weights and scores within weight_tol, the bracket within 2 k + 4 steps of its
    # magnitudes, all of them at most scale * 2 * size.
    size = np.abs(dw).max()
    tol = (2 * weight_tol(E) + (2 * k + 4) * 2.0 ** -23) * scale * 2 * size
    tol = tol + plain.step(dt) * np.abs(want) + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    assert np.all(np.abs(got - want) <= tol)
    assert np.all(got[~np.isfinite(l.float().cpu().numpy())] == 0)
    if k == 1 and renorm:
        assert np.all(got == 0)
    if kind == "sigmoid" or renorm:
        rest = np.ones((T, E), bool)
        e = r.experts.cpu().numpy()
        rest[np.nonzero(e >= 0)[0], e[e >= 0]] = False
        assert np.all(got[rest] == 0)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(kind, renorm):
    gen = torch.Generator().manual_seed(12)
    l = torch.randn(3, 12, generator=gen)
    bias = torch.randn(12, generator=gen) * 0.1
    dw = torch.randn(3, 4, generator=gen)
    args = (4, kind, bias.numpy(), 3, 2, 2, renorm, 2.0)
    r = moe.route_grouped(l.to(DEV), 4, scores=kind, bias=bias.to(DEV), groups=3, top_groups=2,
                          renormalize=renorm, scale=2.0)
    got = moe.route_grouped_backward(l.to(DEV), r.experts, r.weights, dw.to(DEV), scores=kind,
                                     renormalize=renorm, scale=2.0).cpu()
    h = 1e-5
    for t in range(3):
        for e in range(12):
            f = []
            for s in (h, -h):
                m = l.double().numpy().copy()
                m[t, e] += s
                x, w, _, _, _ = groups_of.route(m, *args)
                assert np.array_equal(x, r.experts.cpu().numpy())
                f.append((w * dw.numpy()).sum())
            assert abs((f[0] - f[1]) / (2 * h) - got[t, e].item()) < 1e-5


def test_saturated_scores():
    """Scores that round to 1, and weights that underflow to 0: no NaN comes of them."""
    l = torch.tensor([[40.0, 30.0, 50.0, -120.0], [-120.0] * 4, [100.0, 100.0, -100.0, 0.0]])
    for renorm in (True, False):
        r = moe.route_grouped(l.to(DEV), 2, renormalize=renorm)
        assert r.experts.tolist() == [[2, 0], [0, 1], [0, 1]]
        g = moe.route_grouped_backward(l.to(DEV), r.experts, r.weights,
                                       torch.ones(3, 2, device=DEV), renormalize=renorm)
        assert bool(torch.isfinite(g).all()) and bool(torch.isfinite(r.weights).all())


@pytest.mark.parametrize("T", [12, 3000])
def test_graph_streams_and_given_outputs(T):
    l = torch.randn(T, 48, device=DEV)
    bias = torch.randn(48, device=DEV) * 0.1
    k, kw = 4, dict(bias=bias, groups=6, top_groups=2, scale=2.5)
    dw = torch.randn(T, k, device=DEV)
    ws = torch.empty(moe.route_workspace(T, 48, k), dtype=torch.uint8, device=DEV)
    out = moe.route_grouped(l, k, workspace=ws, **kw)
    grad = torch.empty_like(l)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.route_grouped(l, k, workspace=ws, out=out, **kw)
        moe.route_grouped_backward(l, out.experts, out.weights, dw, scale=2.5, out=grad)
    for i in range(3):
        l.normal_()
        g.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        want = moe.route_grouped(l, k, stream=side, **kw)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert torch.equal(grad, moe.route_grouped_backward(l, want.experts, want.weights, dw,
                                                            scale=2.5))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,top", [(300, 4, 2), (512, 8, 3), (256, 64, 9), (1000, 10, 4), (128, 32, 7),
                                          (60, 20, 5)])
def test_more_experts_or_groups_than_a_row_of_lanes_has(kind, E, groups, top):
    """The form with a wave to each token: numbers, near sums, masks, many tokens."""
    gen = torch.Generator().manual_seed(E)
    l = torch.randn(700, E, generator=gen) * 2
    l[3, 4], l[4, 7], l[5, [3, 9]] = NAN, INF, NAN
    l[6] = -INF
    l[7, : E // 2] = -INF
    l[8] = torch.finfo(torch.float32).min
    bias = torch.randn(E, generator=gen) * (0.1 if kind == "sigmoid" else 0.3 / E)
    for b in (bias, None):
        for best in (1, 2):
            check(l, 5, kind, b, groups, top, best)
    s = groups_of.scores(l[20].double().numpy(), kind)
    check(l[20:21].repeat(9, 1), 5, kind, torch.from_numpy(0.75 - s).float(), groups, top)
    bias[5], bias[6] = NAN, -INF
    check(l[:40], 5, kind, bias, groups, top)


@pytest.mark.parametrize("T", [8, 30, 2000, 2310])
def test_all_alike(T):
    """Every logit and bias the same: the lowest numbers, in order."""
    for E, groups, top in ((64, 8, 2), (256, 8, 4), (160, 8, 3), (512, 8, 4)):
        r = check(torch.zeros(T, E), 6, "sigmoid", torch.zeros(E), groups, top)
        assert bool((r.experts.cpu() == torch.arange(6)).all())
