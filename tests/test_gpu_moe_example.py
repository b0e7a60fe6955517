"""The layer of examples/moe_layer.py: router, exchange, products, return and their
gradients together, against a dense float64 layer."""
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

# Each value is rounded to bf16 a handful of times on its way (rows of h, of the
# activation, of y, the result; the gradients twice as often), each by at most
# half a step, 2^-8 of it: 5 and 10 such errors in a 2-norm stay under 8 and 16
# half steps whatever their signs.
OUT, GRAD = 8 * 2.0 ** -8, 16 * 2.0 ** -8


@pytest.mark.parametrize("P,T,E,H,F,k", [(1, 5, 4, 32, 40, 2), (2, 33, 6, 64, 96, 3),
                                         (4, 96, 8, 256, 512, 2)])
def test_expert_parallel(P, T, E, H, F, k):
    x, logits, w1, w2, _ = layer.inputs(P, T, E, H, F, seed=P)
    got = layer.expert_parallel(x, logits, w1, w2, k)
    want = layer.dense(*[t.double().cpu() for t in (x, logits, w1, w2)], k, True)
    assert layer.relative(got, want) < OUT


def test_expert_parallel_in_4_bits():
    """A code is off by at most a quarter of its value (0.5 against 0.25 or 0.75
    apart, the small ones of a block): rows and weights of both products, and the
    rounding errors are as good as random: the layer stays within 1/2."""
    x, logits, w1, w2, _ = layer.inputs(2, 40, 4, 128, 256, seed=9)
    got = layer.expert_parallel(x, logits, w1, w2, 2, mx4=True)
    want = layer.dense(*[t.double().cpu() for t in (x, logits, w1, w2)], 2, True)
    assert layer.relative(got, want) < 0.5


@pytest.mark.parametrize("T,E,H,F,k", [(7, 4, 32, 24, 2), (130, 8, 96, 200, 3)])
def test_training_step(T, E, H, F, k):
    x, logits, w1, w2, dout = layer.inputs(1, T, E, H, F, seed=T)
    got = layer.training_step(x[0], logits[0], w1, w2, dout[0], k)
    leaves = [t.double().cpu().requires_grad_() for t in (x[0], logits[0], w1, w2)]
    want = layer.dense(*leaves, k, False)
    grads = torch.autograd.grad(want, leaves, dout[0].double().cpu())
    assert layer.relative(got[0], want.detach()) < OUT
    for g, w in zip(got[1:], grads):
        assert layer.relative(g, w) < GRAD
