"""The 8-bit paths of examples/moe_layer.py: router by groups, exchange of codes and
scales, products and their gradients together, against a dense float64 layer."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_layer",
                                              os.path.join(ROOT, "examples", "moe_layer.py"))
layer = importlib.util.module_from_spec(spec)
spec.loader.exec_module(layer)

# A code is off by at most 2^-4 of its value, evenly spread: 2^-4 / sqrt(3) in the mean
# square, and independent from value to value, so that a product of two such operands is
# off by sqrt(2) times that, 0.051 of its 2-norm.  The output has two products (the
# activation's slope is at most 1.1): 0.051 sqrt(1.1^2 + 1) = 0.076.  A gradient has the
# forward pass's error in it and two products more: 0.11.  Twice that for chance.
OUT, GRAD = 0.15, 0.22


def run(P, T, E, H, F, seed):
    x, logits, w1, w2, dout = layer.inputs(P, T, E, H, F, seed=seed)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(seed)).to(x.device)
    return x, logits, bias, w1, w2, dout


@pytest.mark.parametrize("P,T,E,H,F,k,groups,top", [
    (1, 5, 4, 128, 40, 2, 2, 1), (2, 33, 6, 64, 96, 3, 2, 2), (4, 96, 8, 256, 512, 2, 4, 2)])
def test_expert_parallel(P, T, E, H, F, k, groups, top):
    x, logits, bias, w1, w2, _ = run(P, T, E, H, F, P)
    out, routes = layer.expert_parallel_8(x, logits, bias, w1, w2, k, groups, top, 2.5)
    want = layer.dense_8(*[t.double().cpu() for t in (x, logits, w1, w2)],
                         torch.stack([r.experts for r in routes]), 2.5)
    assert layer.relative(out, want) < OUT


@pytest.mark.parametrize("T,E,H,F,k,groups,top", [(7, 4, 32, 24, 2, 2, 2), (130, 8, 96, 200, 3, 4, 2)])
def test_training_step(T, E, H, F, k, groups, top):
    x, logits, bias, w1, w2, dout = run(1, T, E, H, F, T)
    got, r = layer.training_step_8(x[0], logits[0], bias, w1, w2, dout[0], k, groups, top, 2.5)
    leaves = [t.double().cpu().requires_grad_() for t in (x[0], logits[0], w1, w2)]
    want = layer.dense_8(*leaves, r.experts, 2.5)
    grads = torch.autograd.grad(want, leaves, dout[0].double().cpu())
    assert layer.relative(got[0], want.detach()) < OUT
    for g, w in zip(got[1:], grads):
        assert layer.relative(g, w) < GRAD
