"""CPU tests of the operators' host checks: every refusal returns before
anything is enqueued, so they need no GPU (the addresses are never read)."""
import ctypes
import os
import re

import pytest
import torch

from all_movement_amd import a2av, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, INVALID, DTYPE = a2av.OK, a2av.ERR_NULLPTR, a2av.ERR_INVALID_ARGS, a2av.ERR_UNSUPPORTED_DTYPE
A = [0x10000000 * (i + 1) for i in range(12)]  # far apart, aligned

GOOD = {
    "a2av_moe_route": dict(logits=A[0], stride=64, tokens=40, E=64, k=2, renorm=1,
                           dtype=a2av.FP32, experts=A[1], weights=A[2], counts=A[3], order=A[4],
                           place=A[5], ws=None, ws_bytes=0, stream=None),
    "a2av_moe_route_backward": dict(logits=A[0], stride=64, tokens=100, E=64, k=2, renorm=1,
                                    dtype=a2av.FP32, experts=A[1], weights=A[2], dweights=A[3],
                                    dlogits=A[4], stream=None),
    "a2av_moe_gmm": dict(x=A[0], x_stride=64, x_rows=10, w=A[1], counts=A[2], index=None, y=A[3],
                         y_stride=32, rows=10, E=4, N=32, K=64, dtype=a2av.BF16, status=A[4],
                         stream=None),
    "a2av_moe_gmm_dx": dict(dy=A[0], dy_stride=32, w=A[1], counts=A[2], dx=A[3], dx_stride=64,
                            rows=10, E=4, N=32, K=64, dtype=a2av.BF16, status=A[4], stream=None),
    "a2av_moe_gmm_dw": dict(dy=A[0], dy_stride=32, x=A[1], x_stride=64, x_rows=10, counts=A[2],
                            index=None, dw=A[3], rows=10, E=4, N=32, K=64, dtype=a2av.BF16,
                            dw_dtype=a2av.FP32, status=A[4], stream=None),
    "a2av_moe_combine": dict(y=A[0], y_stride=64, y_rows=20, place=A[1], weights=A[2], out=A[3],
                             out_stride=64, tokens=10, k=2, width=64, dtype=a2av.BF16, status=A[4],
                             stream=None),
    "a2av_moe_combine_backward": dict(dout=A[0], dout_stride=64, y=A[1], y_stride=64, y_rows=20,
                                      place=A[2], weights=A[3], dy=A[4], dy_stride=64,
                                      dweights=A[5], tokens=10, k=2, width=64, dtype=a2av.BF16,
                                      status=A[6], stream=None),
    "a2av_moe_mx4_quantize": dict(x=A[0], x_stride=64, rows=10, cols=64, dtype=a2av.BF16,
                                  codes=A[1], scales=A[2], stream=None),
    "a2av_moe_mx4_dequantize": dict(codes=A[1], scales=A[2], rows=10, cols=64, dtype=a2av.BF16,
                                    x=A[0], x_stride=64, stream=None),
    "a2av_moe_gmm_mx4": dict(xc=A[0], xs=A[1], x_rows=10, wc=A[2], ws=A[3], counts=A[4], index=None,
                             y=A[5], y_stride=32, rows=10, E=4, N=32, K=64, dtype=a2av.BF16,
                             status=A[6], stream=None),
}


def call(name, **change):
    args = {**GOOD[name], **change}
    return getattr(moe.lib(), name)(*args.values())


def test_every_declared_function_is_exported():
    text = open(os.path.join(ROOT, "include", "a2av_moe.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(a2av_moe_[a-z0-9_]+)\s*\(", text))
    assert names == set(moe.MOE_EXPORTS)
    assert all(hasattr(moe.lib(), n) for n in names)


REQUIRED = {
    "a2av_moe_route": ["logits", "experts", "weights", "counts", "order", "place"],
    "a2av_moe_route_backward": ["logits", "experts", "weights", "dweights", "dlogits"],
    "a2av_moe_gmm": ["x", "w", "counts", "y"],
    "a2av_moe_gmm_dx": ["dy", "w", "counts", "dx"],
    "a2av_moe_gmm_dw": ["dy", "x", "counts", "dw"],
    "a2av_moe_combine": ["y", "place", "out"],
    "a2av_moe_combine_backward": ["dout", "y", "place", "dy", "dweights"],
    "a2av_moe_mx4_quantize": ["x", "codes", "scales"],
    "a2av_moe_mx4_dequantize": ["codes", "scales", "x"],
    "a2av_moe_gmm_mx4": ["xc", "xs", "wc", "ws", "counts", "y"],
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in REQUIRED.items() for a in args])
def test_null(name, arg):
    assert call(name, **{arg: None}) == NULL
    # NULLPTR comes before the dtype and the sizes
    assert call(name, **{arg: None, "dtype": 77}) == NULL


@pytest.mark.parametrize("name", sorted(GOOD))
@pytest.mark.parametrize("dtype", [-1, a2av.INT8, 4, 77])
def test_dtype(name, dtype):
    assert call(name, dtype=dtype) == DTYPE


@pytest.mark.parametrize("name", ["a2av_moe_gmm", "a2av_moe_gmm_dx", "a2av_moe_gmm_dw"])
def test_products_take_16_bits(name):
    assert call(name, dtype=a2av.FP32) == DTYPE


def test_dw_types():
    assert call("a2av_moe_gmm_dw", dw_dtype=a2av.FP16) == DTYPE


BAD = {
    "a2av_moe_route": [dict(tokens=-1), dict(E=0), dict(E=1025, stride=2000), dict(k=0), dict(k=17),
                       dict(k=3, E=2), dict(stride=63), dict(tokens=2 ** 31), dict(tokens=2 ** 30 + 1),
                       dict(tokens=5000, ws=A[8], ws_bytes=4), dict(logits=A[0] + 2),
                       dict(order=A[4] + 1), dict(experts=A[2] + 8), dict(place=A[0] + 400)],
    "a2av_moe_route_backward": [dict(E=1025, stride=2000), dict(k=65), dict(stride=3),
                                dict(dlogits=A[0] + 4), dict(weights=A[2] + 2)],
    "a2av_moe_gmm": [dict(E=0), dict(E=4097), dict(N=0), dict(K=0), dict(rows=-1), dict(x_rows=9),
                     dict(x_stride=63), dict(y_stride=31), dict(rows=2 ** 30 + 1, x_rows=2 ** 30 + 1),
                     dict(y=A[0] + 100), dict(y=A[1] + 2), dict(x=A[0] + 1), dict(counts=A[2] + 2),
                     dict(status=A[3] + 4), dict(N=2 ** 31 - 1, K=2 ** 31 - 1, E=4096,
                                                 x_stride=2 ** 31 - 1, y_stride=2 ** 31 - 1)],
    "a2av_moe_gmm_dx": [dict(E=0), dict(dy_stride=31), dict(dx_stride=63), dict(dx=A[1] + 64)],
    "a2av_moe_gmm_dw": [dict(x_rows=3), dict(dw=A[0] + 64), dict(dw=A[3] + 2), dict(K=0)],
    "a2av_moe_combine": [dict(k=0), dict(k=65), dict(width=0), dict(y_stride=63),
                         dict(out_stride=63), dict(out=A[0] + 128), dict(weights=A[2] + 1),
                         dict(tokens=-1), dict(y_rows=2 ** 31)],
    "a2av_moe_combine_backward": [dict(dy=A[1] + 64), dict(dy=A[0]), dict(dweights=A[3]),
                                  dict(dy_stride=1), dict(k=65)],
    "a2av_moe_mx4_quantize": [dict(cols=0), dict(rows=-1), dict(x_stride=63), dict(codes=A[1] + 8),
                              dict(scales=A[1] + 5), dict(x=A[0] + 1)],
    "a2av_moe_mx4_dequantize": [dict(cols=0), dict(x_stride=63), dict(codes=A[1] + 8),
                                dict(x=A[1] + 32)],
    "a2av_moe_gmm_mx4": [dict(E=0), dict(x_rows=9), dict(y_stride=31), dict(xc=A[0] + 8),
                         dict(wc=A[2] + 4), dict(y=A[2] + 16), dict(K=0)],
}


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in BAD.items() for c in cs])
def test_invalid(name, change):
    assert call(name, **change) == INVALID


def test_calls_without_rows_do_nothing():
    assert call("a2av_moe_gmm", rows=0, x_rows=0, x=None, y=None) == OK
    assert call("a2av_moe_gmm_dx", rows=0, dy=None, dx=None) == OK
    assert call("a2av_moe_combine", tokens=0, out=None, place=None) == OK
    assert call("a2av_moe_mx4_quantize", rows=0, x=None, codes=None, scales=None) == OK
    assert call("a2av_moe_gmm_mx4", rows=0, x_rows=0, xc=None, xs=None, y=None) == OK
    assert call("a2av_moe_route_backward", tokens=0, logits=None, experts=None, weights=None,
                dweights=None, dlogits=None) == OK


def test_workspace():
    n = ctypes.c_int64()
    f = moe.lib().a2av_moe_route_workspace
    assert f(100, 64, 2, None) == NULL
    assert f(-1, 64, 2, ctypes.byref(n)) == INVALID
    assert f(40, 64, 2, ctypes.byref(n)) == OK and n.value == 0
    assert f(100000, 64, 2, ctypes.byref(n)) == OK and n.value > 0
    assert call("a2av_moe_route", tokens=100000, ws=None, ws_bytes=n.value, logits=A[9]) == NULL


def test_python_refuses_what_it_would_have_to_copy():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    c = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must live on a GPU"):
        moe.gmm(x, w, c)
    with pytest.raises(ValueError, match="contiguous"):
        moe.gmm(x, w.transpose(1, 2).contiguous().transpose(1, 2), c)
    with pytest.raises(ValueError, match="contiguous"):
        moe.gmm(torch.zeros(16, 4, dtype=torch.bfloat16).t(), w, c)
    with pytest.raises(ValueError, match="contiguous rows"):
        moe.mx4_quantize(torch.zeros(1, 16, dtype=torch.bfloat16).expand(4, 16))
    with pytest.raises(ValueError, match="int32"):
        moe.gmm(x, w, c.long())
    with pytest.raises(ValueError, match="columns"):
        moe.gmm(x[:, :8], w, c)
    with pytest.raises(ValueError, match="one of"):
        moe.mx4_quantize(torch.zeros(4, 16, dtype=torch.float64))
    with pytest.raises(TypeError):
        moe.mx4_quantize([1.0])
