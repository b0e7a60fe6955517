"""CPU tests of what the operators accept and refuse as operands: shared bytes of
strided rows, against a count of the bytes one by one."""
import random
from types import SimpleNamespace

import pytest
import torch

from all_movement_amd import a2av, moe
from tests.test_moe_host import A, INVALID, call


def _bytes(at, rows, stride, width):
    return {at + r * stride + b for r in range(rows) for b in range(width)}


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would be launched")
def test_an_output_may_interleave_with_another_operand_but_share_no_byte():
    """x and y of one buffer: refused exactly if they share a byte."""
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(6000):
        rows, x_rows = rng.randint(1, 7), 0
        x_rows = rows + rng.randint(0, 3)
        K, N = rng.randint(1, 9), rng.randint(1, 9)
        xs = K + rng.choice([0, 1, 5, 12, 30])
        ys = xs if rng.random() < 0.4 and xs >= N else N + rng.choice([0, 2, 9, 31])
        y = A[0] + 2 * rng.randint(-rows * ys - 3, x_rows * xs + 3)
        shared = bool(_bytes(A[0], x_rows, 2 * xs, 2 * K) & _bytes(y, rows, 2 * ys, 2 * N))
        got = call("a2av_moe_gmm", x=A[0], x_stride=xs, x_rows=x_rows, y=y, y_stride=ys, rows=rows,
                   N=N, K=K, w=A[8], status=None)
        assert (got == INVALID) == shared, (rows, x_rows, K, N, xs, ys, y - A[0])
        seen[shared] += 1
    assert min(seen) > 500


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would be launched")
def test_halves_of_one_buffer_are_accepted():
    half = dict(y=A[0], y_stride=128, out=A[0] + 128, out_stride=128, width=64)
    assert call("a2av_moe_combine", **half) != INVALID
    assert call("a2av_moe_combine", **{**half, "out": A[0] + 126}) == INVALID
    # Far rows: strides and extents of the largest sizes.
    far = dict(rows=2 ** 30, cols=2 ** 30, x=A[0], x_stride=2 ** 31 - 1, dtype=a2av.FP32)
    assert call("a2av_moe_mx4_dequantize", **{**far, "codes": A[1], "scales": A[2]}) == INVALID


def test_a_gradient_is_not_lost_in_silence():
    """No call records a gradient: operands that want one are refused while
    gradients are recorded."""
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    c, p = torch.zeros(2, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    f = torch.zeros(4, 2)

    def g(t):
        return t.clone().requires_grad_()
    calls = [lambda: moe.gmm(g(x), w, c), lambda: moe.gmm(x, g(w), c),
             lambda: moe.gmm_dx(g(x[:, :8].contiguous()), w, c),
             lambda: moe.gmm_dw(x, g(x), c), lambda: moe.route(g(f), 1),
             lambda: moe.route_backward(f, p[:, :1].contiguous(), g(f[:, :1].contiguous()),
                                        f[:, :1].contiguous()),
             lambda: moe.combine(g(x), p, f), lambda: moe.combine(x, p, g(f)),
             lambda: moe.combine_backward(x, g(x), p, f), lambda: moe.mx4_quantize(g(x)),
             lambda: moe.combine(x, p, f, out=g(x))]
    for one in calls:
        with pytest.raises(ValueError, match="gradient"):
            one()
        with torch.no_grad(), pytest.raises(ValueError, match="must live on a GPU"):
            one()


def test_a_stream_of_another_device_is_refused():
    here, there = torch.device("cuda:0"), torch.device("cuda:1")
    with pytest.raises(ValueError, match="stream"):
        moe._elsewhere(here, SimpleNamespace(device=there))
    assert moe._elsewhere(here, SimpleNamespace(device=here))
