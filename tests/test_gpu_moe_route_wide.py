"""The router of 257 to 512 experts, which take eight logits per lane: few tokens
(one workgroup) and the gradient, at row lengths of whole pieces and others."""
import pytest
import torch

from all_movement_amd import moe
from tests import moe_plain as plain
from tests.test_gpu_moe_route import DTYPES, DEV, check, weight_tol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 257, 1), (16, 512, 8), (13, 300, 16), (9, 511, 3),
                                   (200, 512, 8), (77, 301, 5)])
def test_wide_routers(dt, renorm, T, E, k):
    gen = torch.Generator().manual_seed(T + E)
    l = (torch.randn(T, E, generator=gen) * 2).to(dt)
    l[:, 5] = -float("inf")
    if T > 4:
        l[2] = -float("inf")
        l[3, 2:] = -float("inf")
    r = check(l, k, renorm)
    l = l.to(DEV)
    dw = torch.randn(T, k, generator=gen).to(DEV)
    dw[r.experts < 0] = float("nan")  # an empty slot's gradient is not read
    got = moe.route_backward(l, r.experts, r.weights, dw, renormalize=renorm).double().cpu()
    want = torch.from_numpy(plain.route_back(l.float().cpu().numpy(), r.experts.cpu().numpy(),
                                             r.weights.cpu().numpy(), dw.cpu().numpy(), renorm))
    size = dw.nan_to_num().abs().max().item()
    # The weights' error, and k + 4 steps of the bracket's magnitudes.
    tol = (weight_tol(E) + (k + 4) * 2.0 ** -23) * size * 3 + plain.step(dt) * want.abs()
    tol = tol + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    assert bool(((got - want).abs() <= tol).all())
    assert bool((got[(l == -float("inf")).cpu()] == 0).all())
