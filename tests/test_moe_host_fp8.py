"""CPU tests of the host checks of the 8-bit operators: every refusal returns
before anything is enqueued (the addresses are never read)."""
import pytest
import torch

from all_movement_amd import a2av, moe

OK, NULL, INVALID, DTYPE = a2av.OK, a2av.ERR_NULLPTR, a2av.ERR_INVALID_ARGS, a2av.ERR_UNSUPPORTED_DTYPE
A = [0x10000000 * (i + 1) for i in range(12)]  # far apart, aligned

GOOD = {
    "a2av_moe_fp8_quantize": dict(x=A[0], x_stride=200, rows=10, cols=200, dtype=a2av.BF16,
                                  codes=A[1], scales=A[2], stream=None),
    "a2av_moe_fp8_dequantize": dict(codes=A[1], scales=A[2], rows=10, cols=200, dtype=a2av.BF16,
                                    x=A[0], x_stride=200, stream=None),
    "a2av_moe_fp8_quantize_weights": dict(w=A[0], E=3, N=130, K=200, dtype=a2av.FP32, codes=A[1],
                                          scales=A[2], stream=None),
    "a2av_moe_fp8_dequantize_weights": dict(codes=A[1], scales=A[2], E=3, N=130, K=200,
                                            dtype=a2av.FP16, w=A[0], stream=None),
    "a2av_moe_gmm_fp8": dict(xc=A[0], xs=A[1], x_rows=10, wc=A[2], ws=A[3], counts=A[4], index=None,
                             y=A[5], y_stride=32, rows=10, E=4, N=32, K=200, dtype=a2av.BF16,
                             status=A[6], stream=None),
    "a2av_moe_gmm_fp8_dx": dict(yc=A[0], ys=A[1], wc=A[2], ws=A[3], counts=A[4], dx=A[5],
                                dx_stride=200, rows=10, E=4, N=32, K=200, dtype=a2av.BF16,
                                status=A[6], stream=None),
}
REQUIRED = {
    "a2av_moe_fp8_quantize": ["x", "codes", "scales"],
    "a2av_moe_fp8_dequantize": ["codes", "scales", "x"],
    "a2av_moe_fp8_quantize_weights": ["w", "codes", "scales"],
    "a2av_moe_fp8_dequantize_weights": ["codes", "scales", "w"],
    "a2av_moe_gmm_fp8": ["xc", "xs", "wc", "ws", "counts", "y"],
    "a2av_moe_gmm_fp8_dx": ["yc", "ys", "wc", "ws", "counts", "dx"],
}
BIG = 2 ** 30 + 1
BAD = {
    "a2av_moe_fp8_quantize": [dict(cols=0), dict(rows=-1), dict(rows=BIG), dict(cols=BIG, x_stride=BIG),
                              dict(x_stride=199), dict(x_stride=2 ** 31), dict(codes=A[1] + 8),
                              dict(scales=A[2] + 2), dict(x=A[0] + 1), dict(codes=A[0] + 16),
                              dict(scales=A[1] + 2556)],
    "a2av_moe_fp8_dequantize": [dict(cols=0), dict(x_stride=199), dict(codes=A[1] + 8),
                                dict(scales=A[2] + 1), dict(x=A[1] + 2558), dict(x=A[2] + 38)],
    "a2av_moe_fp8_quantize_weights": [dict(E=0), dict(E=4097), dict(N=0), dict(K=0), dict(N=BIG),
                                      dict(K=BIG), dict(N=2 ** 30, K=2 ** 30, E=4096),
                                      dict(w=A[0] + 2), dict(codes=A[1] + 4), dict(scales=A[2] + 2),
                                      dict(codes=A[0] + 3 * 130 * 200 * 4 // 16 * 16 - 16),
                                      dict(scales=A[1] + 3 * 130 * 256 - 4)],
    "a2av_moe_fp8_dequantize_weights": [dict(E=0), dict(N=0), dict(K=0), dict(w=A[0] + 1),
                                        dict(codes=A[1] + 8), dict(w=A[2] + 22),
                                        dict(w=A[1] + 3 * 130 * 256 - 2)],
    "a2av_moe_gmm_fp8": [dict(E=0), dict(E=4097), dict(N=0), dict(K=0), dict(rows=-1), dict(x_rows=9),
                         dict(y_stride=31), dict(rows=BIG, x_rows=BIG), dict(xc=A[0] + 8),
                         dict(wc=A[2] + 4), dict(xs=A[1] + 2), dict(ws=A[3] + 1), dict(y=A[2] + 16),
                         dict(y=A[3] + 14), dict(counts=A[4] + 2), dict(status=A[5] + 4),
                         dict(y=A[1] + 38)],
    "a2av_moe_gmm_fp8_dx": [dict(E=0), dict(dx_stride=199), dict(dx=A[0] + 1278), dict(N=0),
                            dict(dx=A[2] + 4 * 32 * 256 - 2), dict(wc=A[2] + 8), dict(rows=-1)],
}


def call(name, **change):
    return getattr(moe.lib(), name)(*{**GOOD[name], **change}.values())


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in REQUIRED.items() for a in args])
def test_null(name, arg):
    assert call(name, **{arg: None}) == NULL
    assert call(name, **{arg: None, "dtype": 77}) == NULL


@pytest.mark.parametrize("name", sorted(GOOD))
@pytest.mark.parametrize("dtype", [-1, a2av.INT8, 4, 77])
def test_dtype(name, dtype):
    assert call(name, dtype=dtype) == DTYPE


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in BAD.items() for c in cs])
def test_invalid(name, change):
    assert call(name, **change) == INVALID


def test_calls_without_rows_do_nothing():
    assert call("a2av_moe_fp8_quantize", rows=0, x=None, codes=None, scales=None) == OK
    assert call("a2av_moe_fp8_dequantize", rows=0, x=None, codes=None, scales=None) == OK
    assert call("a2av_moe_gmm_fp8", rows=0, x_rows=0, xc=None, xs=None, y=None) == OK
    assert call("a2av_moe_gmm_fp8_dx", rows=0, yc=None, ys=None, dx=None) == OK


def test_python_refuses():
    x, w = torch.zeros(4, 200, dtype=torch.bfloat16), torch.zeros(2, 130, 200, dtype=torch.bfloat16)
    xc, xs = torch.zeros(4, 256, dtype=moe.E4M3), torch.zeros(4, 4, dtype=torch.uint8)
    wc, ws = torch.zeros(2, 130, 256, dtype=moe.E4M3), torch.zeros(2, 2, 4, dtype=torch.uint8)
    yc, ys = torch.zeros(4, 256, dtype=moe.E4M3), torch.zeros(4, 4, dtype=torch.uint8)
    c = torch.zeros(2, dtype=torch.int32)
    for f in (lambda: moe.fp8_quantize(x), lambda: moe.fp8_dequantize(xc, xs, 200),
              lambda: moe.fp8_quantize_weights(w), lambda: moe.fp8_dequantize_weights(wc, ws, 200),
              lambda: moe.gmm_fp8(xc, xs, wc, ws, c), lambda: moe.gmm_fp8_dx(yc, ys, wc, ws, c)):
        with pytest.raises(ValueError, match="must live on a GPU"):
            f()
    for f in (lambda: moe.fp8_dequantize(xc.view(torch.uint8), xs, 200),
              lambda: moe.gmm_fp8(xc, xs.int(), wc, ws, c),
              lambda: moe.gmm_fp8(xc, xs, wc, ws, c.long()),
              lambda: moe.fp8_quantize(x.double()), lambda: moe.fp8_quantize_weights(w.double())):
        with pytest.raises(ValueError, match="must be"):
            f()
    for f in (lambda: moe.fp8_dequantize(xc, xs, 300), lambda: moe.gmm_fp8(xc[:, :128], xs, wc, ws, c),
              lambda: moe.gmm_fp8_dx(yc, ys, wc, ws, c, cols=300), lambda: moe.gmm_fp8(xc, xs, wc, ws[:1], c),
              lambda: moe.fp8_quantize_weights(w[0]), lambda: moe.gmm_fp8(xc, xs, wc[0], ws, c),
              lambda: moe.fp8_quantize_weights(w.transpose(1, 2))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        moe.fp8_quantize_weights([1.0])
    for f in (lambda: moe.fp8_quantize(x.requires_grad_()),
              lambda: moe.fp8_quantize_weights(w.requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            f()
