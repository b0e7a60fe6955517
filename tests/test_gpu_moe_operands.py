"""Operands at the border of what the operators take."""
import math

import pytest
import torch

from all_movement_amd import moe
from tests import moe_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_columns_of_one_buffer_as_input_and_output():
    gen = torch.Generator().manual_seed(1)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.randn(90, 160, generator=gen).to(dt).to(DEV)
        y, out = buf[:, :64], buf[:30, 64:128]
        place = torch.randperm(90, generator=gen).to(torch.int32).view(30, 3).to(DEV)
        w = torch.rand(30, 3, generator=gen).to(DEV)
        want = moe.combine(y.contiguous(), place, w)
        edge = buf[:, 128:].clone()
        assert torch.equal(moe.combine(y, place, w, out=out), want)
        assert torch.equal(buf[:, 128:], edge) and torch.equal(buf[:30, 64:128], want)
    buf = torch.randn(70, 104, generator=gen).to(torch.bfloat16).to(DEV)
    wt = torch.randn(2, 40, 64, generator=gen).to(torch.bfloat16).to(DEV)
    c = torch.tensor([30, 40], dtype=torch.int32, device=DEV)
    want = moe.gmm(buf[:, :64].contiguous(), wt, c)
    before = buf[:, :64].clone()
    moe.gmm(buf[:, :64], wt, c, out=buf[:, 64:])
    assert torch.equal(buf[:, 64:], want) and torch.equal(buf[:, :64], before)


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(20, 3), (128, 4), (700, 16)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_gradient_of_masked_logits_beside_ones_that_are_no_numbers(dt, renorm, E, k, bad):
    gen = torch.Generator().manual_seed(E)
    l = torch.randn(9, E, generator=gen).to(dt)
    clean = l.clone()
    l[1, 4] = bad
    l[1, [0, 7, E - 1]] = -math.inf
    l[3] = -math.inf
    l[3, 2] = bad
    l[5, 1], l[5, 2] = math.nan, math.inf
    l[5, 3:] = -math.inf
    l = l.to(DEV)
    r = moe.route(l, k, renormalize=renorm)
    dw = torch.randn(9, k, generator=gen).to(DEV)
    d = moe.route_backward(l, r.experts, r.weights, dw, renormalize=renorm)
    assert bool((d[l == -math.inf] == 0).all())
    assert bool(torch.isnan(d[[1, 3, 5], [4, 2, 1]]).all())
    rest = [0, 2, 4, 6, 7, 8]
    want = plain.route_back(clean[rest].float().numpy(), r.experts[rest].cpu().numpy(),
                            r.weights[rest].cpu().numpy(), dw[rest].cpu().numpy(), renorm)
    # as in the router's tests: the weights' error and that of the bracket
    tol = ((64 + E) + (k + 4)) * 2.0 ** -23 * dw.abs().max().item() * 3
    want = torch.from_numpy(want)
    off = (d[rest].double().cpu() - want).abs()
    assert bool((off <= tol + plain.step(dt) * want.abs() +
                 torch.finfo(dt).smallest_normal * torch.finfo(dt).eps).all())
