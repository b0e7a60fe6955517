"""The router and its gradient against the definition in float64."""
import numpy as np
import pytest
import torch

from all_movement_amd import moe
from tests import moe_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
# p = exp(l - top) / sum in FP32: l - top is rounded once (half a step of up to
# 20 in these tests), exp within 2 steps, the sum's terms likewise, E + 8 steps
# of additions, the quotient within 2 steps: (20 + 20 + 10 + E + 8) * 2^-23 at most.


def weight_tol(E):
    return (64 + E) * 2.0 ** -23


def check(logits, k, renorm):
    T, E = logits.shape
    print("route", T, E, k, renorm, logits.dtype, flush=True)
    r = moe.route(logits.to(DEV) if not logits.is_cuda else logits, k, renormalize=renorm)
    got = [t.cpu().numpy() for t in r]
    want = plain.route(logits.float().cpu().numpy(), k, renorm)
    assert np.array_equal(got[0], want[0])
    assert np.array_equal(got[2], want[2])
    assert np.array_equal(got[3], want[3])
    assert np.array_equal(got[4], want[4])
    assert np.array_equal(np.isnan(got[1]), np.isnan(want[1]))
    ok = ~np.isnan(want[1])
    assert np.all(np.abs(got[1] - want[1])[ok] <= weight_tol(E) * want[1][ok] + 1e-37)
    return r


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (8, 64, 2), (37, 100, 5), (128, 256, 8),
                                   (129, 256, 8), (1000, 17, 3), (200, 1000, 16), (64, 512, 16),
                                   (65, 64, 16), (700, 5, 2), (1025, 3, 1)])
def test_against_definition(dt, renorm, T, E, k):
    gen = torch.Generator().manual_seed(T * 31 + E)
    check((torch.randn(T, E, generator=gen) * 2).to(dt), k, renorm)


@pytest.mark.parametrize("T", [5, 900])
@pytest.mark.parametrize("renorm", [True, False])
def test_ties_and_masks(T, renorm):
    gen = torch.Generator().manual_seed(9)
    l = torch.randint(-2, 3, (T, 70), generator=gen).float()
    l[l == 0] *= torch.where(torch.rand(int((l == 0).sum()), generator=gen) < 0.5, -1.0, 1.0)
    l[:, 3] = -float("inf")          # an expert that is off
    l[1] = -float("inf")             # a token without experts
    l[2] = -float("inf")
    l[2, [5, 69]] = 1.0              # fewer experts than slots
    l[3] = torch.finfo(torch.float32).min  # masked by the lowest value: all alike
    l[4] = torch.finfo(torch.float32).min
    l[4, 66] = 0.0
    r = check(l, 4, renorm)
    assert r.experts[1].tolist() == [-1] * 4 and r.experts[3].tolist() == [0, 1, 2, 3]
    assert r.experts[2].tolist() == [5, 69, -1, -1] and r.experts[4].tolist() == [66, 0, 1, 2]


def test_every_token_without_experts():
    r = check(torch.full((300, 40), -float("inf")), 8, True)
    assert r.counts.sum().item() == 0 and bool((r.order == -1).all())


def test_logits_that_are_no_numbers():
    l = torch.randn(6, 20, generator=torch.Generator().manual_seed(1))
    l[0, 4] = float("nan")
    l[1, 7] = float("inf")
    l[2, [3, 9]] = float("nan")
    l[3, [2, 5]] = float("inf")
    for renorm in (True, False):
        r = check(l, 3, renorm)
        assert r.experts[2, :2].tolist() == [3, 9] and r.experts[3, :2].tolist() == [2, 5]


def test_no_tokens():
    r = moe.route(torch.empty(0, 12, device=DEV), 3)
    assert r.counts.tolist() == [0] * 12 and r.order.numel() == 0
    assert moe.route_backward(torch.empty(0, 12, device=DEV), r.experts, r.weights,
                              r.weights).shape == (0, 12)


def test_strided_logits():
    wide = torch.full((500, 40), 100.0, device=DEV)
    wide[:, :30] = torch.randn(500, 30, device=DEV)
    check(wide[:, :30], 4, True)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 64, 2), (300, 100, 5), (33, 1024, 16), (9, 130, 8)])
def test_gradient(dt, renorm, T, E, k):
    gen = torch.Generator().manual_seed(E)
    l = (torch.randn(T, E, generator=gen) * 2).to(dt)
    if T > 2 and E > k:
        l[1] = -float("inf")
        l[2, 1:] = -float("inf")
        l[0, E // 2] = -float("inf")
    l = l.to(DEV)
    r = moe.route(l, k, renormalize=renorm)
    dw = torch.randn(T, k, generator=gen).to(DEV)
    dw[r.experts < 0] = float("nan")  # an empty slot's gradient is not read
    got = moe.route_backward(l, r.experts, r.weights, dw, renormalize=renorm).double().cpu().numpy()
    want = plain.route_back(l.float().cpu().numpy(), r.experts.cpu().numpy(),
                            r.weights.cpu().numpy(), dw.cpu().numpy(), renorm)
    # q within weight_tol, the bracket within (k + 4) steps of its magnitudes.
    size = np.abs(np.nan_to_num(dw.cpu().numpy())).max()
    tol = (weight_tol(E) + (k + 4) * 2.0 ** -23) * size * 3 + plain.step(dt) * np.abs(want)
    tol = tol + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    assert np.all(np.abs(got - want) <= tol)
    assert np.all(got[~np.isfinite(l.float().cpu().numpy())] == 0)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(64, 3), (250, 8), (700, 16)])
def test_gradient_of_many_tokens(renorm, E, k):
    """More tokens than waves: nothing of a token is left for the next; some
    tokens have empty slots, some no expert at all."""
    gen = torch.Generator().manual_seed(E + k)
    T = 20011
    l = torch.randn(T, E, generator=gen) * 2
    l[::7] = -float("inf")
    l[3::11, 2:] = -float("inf")
    l = l.to(DEV)
    r = moe.route(l, k, renormalize=renorm)
    dw = torch.randn(T, k, generator=gen).to(DEV)
    dw[r.experts < 0] = float("nan")
    got = moe.route_backward(l, r.experts, r.weights, dw, renormalize=renorm).double().cpu().numpy()
    want = plain.route_back(l.cpu().numpy(), r.experts.cpu().numpy(), r.weights.cpu().numpy(),
                            dw.cpu().numpy(), renorm)
    size = np.abs(np.nan_to_num(dw.cpu().numpy())).max()
    tol = (weight_tol(E) + (k + 4) * 2.0 ** -23) * size * 3 + plain.step(torch.float32) * np.abs(want)
    assert np.all(np.abs(got - want) <= tol + torch.finfo(torch.float32).smallest_normal)


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    gen = torch.Generator().manual_seed(12)
    l = torch.randn(3, 10, generator=gen)
    dw = torch.randn(3, 4, generator=gen)
    r = moe.route(l.to(DEV), 4, renormalize=renorm)
    got = moe.route_backward(l.to(DEV), r.experts, r.weights, dw.to(DEV), renormalize=renorm).cpu()
    h = 1e-5
    for t in range(3):
        for e in range(10):
            f = []
            for s in (h, -h):
                m = l.double().numpy().copy()
                m[t, e] += s
                x, w, _, _, _ = plain.route(m, 4, renorm)
                assert np.array_equal(x, r.experts.cpu().numpy())
                f.append((w * dw.numpy()).sum())
            assert abs((f[0] - f[1]) / (2 * h) - got[t, e].item()) < 1e-5


def test_graph_and_given_outputs():
    l = torch.randn(3000, 48, device=DEV)
    k = 4
    ws = torch.empty(moe.route_workspace(3000, 48, k), dtype=torch.uint8, device=DEV)
    out = moe.route(l, k, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.route(l, k, workspace=ws, out=out)
    for i in range(3):
        l.normal_()
        g.replay()
        torch.cuda.synchronize()
        want = moe.route(l, k)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_order_is_the_exchange_gather_list():
    """a2av_run_indexed over the router's order puts the rows in expert order."""
    from all_movement_amd import a2av
    T, E, k, H = 50, 6, 2, 16
    x = torch.randn(T, H, device=DEV)
    r = moe.route(torch.randn(T, E, device=DEV), k)
    ex = a2av.Exchange(1, T * H * 4, T * k * H * 4, 1)
    got = torch.empty(T * k, H, device=DEV)
    sig = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    sc = (r.counts.sum().to(torch.int32) * H).view(1, 1)
    rc = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    ex.run(x, got, sig, sc, rc, 1, a2av.FP32, index=r.order.view(1, -1), row_elems=H, check=True)
    ex.close()
    assert torch.equal(got, x[r.order.long()])
