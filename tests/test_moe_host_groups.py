"""CPU tests of the host checks of the router by groups (nothing is enqueued; the
addresses are never read)."""
import ctypes

import pytest
import torch

from all_movement_amd import a2av, moe
from tests import moe_plain as plain
from tests import moe_plain_groups as groups_of

OK, NULL, INVALID, DTYPE = a2av.OK, a2av.ERR_NULLPTR, a2av.ERR_INVALID_ARGS, a2av.ERR_UNSUPPORTED_DTYPE
A = [0x10000000 * (i + 1) for i in range(12)]  # far apart, aligned
FWD, BACK = "a2av_moe_route_grouped", "a2av_moe_route_grouped_backward"
GOOD = {
    FWD: dict(logits=A[0], stride=64, bias=A[6], tokens=40, E=64, k=4, groups=8, top=2, best=2,
              scores=1, renorm=1, scale=2.5, dtype=a2av.FP32, experts=A[1], weights=A[2],
              counts=A[3], order=A[4], place=A[5], ws=None, ws_bytes=0, stream=None),
    BACK: dict(logits=A[0], stride=64, tokens=100, E=64, k=4, scores=1, renorm=1, scale=2.5,
               dtype=a2av.FP32, experts=A[1], weights=A[2], dweights=A[3], dlogits=A[4],
               stream=None),
}


def call(name, **change):
    return getattr(moe.lib(), name)(*{**GOOD[name], **change}.values())


@pytest.mark.parametrize("name,arg", [(FWD, a) for a in ("logits", "experts", "weights", "counts",
                                                         "order", "place")] +
                         [(BACK, a) for a in ("logits", "experts", "weights", "dweights", "dlogits")])
def test_null(name, arg):
    assert call(name, **{arg: None}) == NULL
    assert call(name, **{arg: None, "dtype": 77}) == NULL


@pytest.mark.parametrize("name", [FWD, BACK])
@pytest.mark.parametrize("dtype", [-1, a2av.INT8, 4])
def test_dtype(name, dtype):
    assert call(name, dtype=dtype) == DTYPE


@pytest.mark.parametrize("change", [
    dict(groups=0), dict(groups=-1), dict(groups=65, E=65, stride=65), dict(groups=7), dict(top=0),
    dict(top=9), dict(k=16, groups=32, top=7), dict(best=0), dict(best=3), dict(scores=2),
    dict(scores=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=1e-40), dict(bias=A[6] + 2), dict(bias=A[3] + 4),
    dict(E=0), dict(E=1025, groups=1, top=1, stride=1025), dict(k=17), dict(k=0), dict(stride=63),
    dict(tokens=-1), dict(tokens=2 ** 30), dict(tokens=5000, ws=A[8], ws_bytes=4),
    dict(logits=A[0] + 2), dict(place=A[0] + 400), dict(experts=A[2] + 8)])
def test_invalid(change):
    assert call(FWD, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(scores=2), dict(scale=0.0), dict(scale=float("nan")), dict(E=1025, stride=1025), dict(k=65),
    dict(stride=3), dict(dlogits=A[0] + 4), dict(weights=A[2] + 2)])
def test_invalid_backward(change):
    assert call(BACK, **change) == INVALID


def test_workspace_is_the_routers():
    n = ctypes.c_int64()
    assert moe.lib().a2av_moe_route_workspace(100000, 64, 4, ctypes.byref(n)) == OK and n.value > 0
    assert call(FWD, tokens=100000, ws=None, ws_bytes=n.value, logits=A[9]) == NULL
    assert call(BACK, tokens=0, logits=None, experts=None, weights=None, dweights=None,
                dlogits=None) == OK


def test_python_refuses():
    l, b = torch.zeros(4, 16), torch.zeros(16)
    for f, what in ((lambda: moe.route_grouped(l, 2), "must live on a GPU"),
                    (lambda: moe.route_grouped(l, 2, scores="relu"), "scores must be"),
                    (lambda: moe.route_grouped(l, 2, bias=b[:8]), "bias must be"),
                    (lambda: moe.route_grouped(l, 2, bias=b.double()), "bias must be"),
                    (lambda: moe.route_grouped(l.double(), 2), "must be one of"),
                    (lambda: moe.route_grouped(l, 2, bias=b.clone().requires_grad_()), "gradient"),
                    (lambda: moe.route_grouped(l.clone().requires_grad_(), 2), "gradient"),
                    (lambda: moe.route_grouped_backward(l, torch.zeros(4, 2, dtype=torch.int32),
                                                        torch.zeros(4, 2), torch.zeros(4, 2),
                                                        scores="none"), "scores must be")):
        with pytest.raises(ValueError, match=what):
            f()


def test_the_oracle_with_one_group_is_the_routers():
    gen = torch.Generator().manual_seed(0)
    l = torch.randn(9, 20, generator=gen).numpy()
    l[2, 5:] = -float("inf")
    for renorm in (True, False):
        a = plain.route(l, 6, renorm)
        b = groups_of.route(l, 6, "softmax", None, 1, 1, 1, renorm, 1.0)
        assert all((abs(x - y) < 1e-12).all() for x, y in zip(a, b))
