"""The microscaled 4-bit format: codes and scales equal to the definition's, and
the grouped product on them against float64."""
import math

import numpy as np
import pytest
import torch

from all_movement_amd import a2av, moe
from tests import moe_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def rows_of(dt, rows, cols, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen) * torch.randn(rows, 1, generator=gen).mul(3).exp()
    return x.to(dt)


def check(x):
    codes, scales = moe.mx4_quantize(x.to(DEV))
    want_c, want_s, want_v = plain.mx4(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), plain.pack(want_c))
    for dt in DTYPES:
        v = moe.mx4_dequantize(codes, scales, x.shape[1], dt).cpu()
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want_v).to(torch.float32).to(dt)
        assert torch.equal(v.nan_to_num(nan=9.0), want.nan_to_num(nan=9.0))
        assert torch.equal(torch.signbit(v), torch.signbit(want)) or not bool(
            torch.isfinite(want).all())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (5, 31), (7, 64), (130, 160),
                                       (2, 7168), (9, 523)])
def test_codes_and_values(dt, rows, cols):
    check(rows_of(dt, rows, cols, rows * 1000 + cols))


def test_ties_zeros_and_the_ends_of_the_range():
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.9, 6.0, 4.0, 0.0, -0.0]
    block = []
    for m in mids:
        block += [m, -m]
    block += [math.nextafter(0.25, 0), math.nextafter(0.25, 1), 2.0, 3.0, 1.0, 7.99]
    rows = [[v * s for v in block] for s in (1.0, 2.0 ** -100, 2.0 ** 100)]
    rows += [[0.0] * 32, [-0.0] * 32, [2.0 ** -126] * 32, [2.0 ** -149] * 31 + [2.0 ** -130],
             [3.4028234e38] + [1.0] * 31, [2.0 ** -124] + [2.0 ** -126] * 31]
    check(torch.tensor(rows, dtype=torch.float64).to(torch.float32))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_blocks_that_are_no_numbers(bad):
    x = rows_of(torch.float32, 3, 96, 1)
    x[1, 40] = bad
    check(x)
    codes, scales = moe.mx4_quantize(x.to(DEV))
    assert scales[1, 1].item() == 255 and bool((codes[1, 16:32] == 0).all())
    v = moe.mx4_dequantize(codes, scales, 96)
    assert bool(torch.isnan(v[1, 32:64]).all()) and int(torch.isnan(v).sum()) == 32


def test_strided_rows():
    x = rows_of(torch.bfloat16, 6, 64, 2).to(DEV)
    for pad in (8, 1):
        s = torch.full((6, 64 + pad), 1e30, dtype=x.dtype, device=DEV)[:, :64]
        s.copy_(x)
        a, b = moe.mx4_quantize(s), moe.mx4_quantize(x)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        o = torch.full((6, 64 + pad), 5.0, dtype=x.dtype, device=DEV)
        moe.mx4_dequantize(*a, 64, x.dtype, out=o[:, :64])
        assert torch.equal(o[:, :64], moe.mx4_dequantize(*b, 64, x.dtype))
        assert bool((o[:, 64:] == 5).all())


def product(counts, N, K, dt, tokens=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    E, rows = len(counts), sum(counts)
    x = torch.randn(tokens or rows, K, generator=gen).to(DEV)
    w = (torch.randn(E * N, K, generator=gen) / math.sqrt(K)).to(DEV)
    xc, xs = moe.mx4_quantize(x)
    wc, ws = moe.mx4_quantize(w)
    B = xs.shape[1]
    wc, ws = wc.view(E, N, 16 * B), ws.view(E, N, B)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    index = None
    if tokens:
        index = torch.randint(0, tokens, (rows,), generator=gen).to(torch.int32).to(DEV)
    print("mx4", counts, N, K, dt, tokens, flush=True)
    y = moe.gmm_mx4(xc, xs, wc, ws, c, index=index, dtype=dt, check=True)
    want, mag = plain.gmm(plain.unpack_values(xc, xs, K), plain.unpack_values(wc, ws, K), c, index)
    plain.check_sums(y, want, mag, K)
    return xc, xs, wc, ws, c, y


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts,N,K", [
    ([1], 1, 1), ([1], 16, 32), ([0, 2, 0, 3], 40, 64), ([130, 1, 0, 260], 136, 288),
    ([17, 40], 129, 1000), ([64, 9], 256, 2049), ([5, 7, 20, 3], 72, 544)])
def test_product(dt, counts, N, K):
    product(counts, N, K, dt, seed=N + K)


@pytest.mark.parametrize("K", [512, 1024, 1536, 2560])
@pytest.mark.parametrize("counts,N,tokens", [([300, 0, 200], 520, None), ([40, 3, 0, 77], 130, 90),
                                             ([2, 1], 48, None)])
def test_product_of_whole_scale_groups(counts, N, K, tokens):
    product(counts, N, K, torch.bfloat16, tokens, seed=K + N)


def test_product_in_rounds_of_whole_tiles():
    product([520, 300], 16640, 512, torch.float16, seed=3)


@pytest.mark.parametrize("counts,N,K,tokens", [([9, 0, 30], 64, 256, 11), ([200, 77], 200, 416, 100)])
def test_product_of_gathered_rows(counts, N, K, tokens):
    product(counts, N, K, torch.bfloat16, tokens, seed=tokens)


def test_product_with_scales_of_the_whole_range():
    """Scales whose product is an ordinary number; a scale of NaN makes its rows NaN."""
    xc, xs, wc, ws, c, _ = product([3, 4], 48, 128, torch.float32)
    xs[:] = 7
    ws[:] = 245
    y = moe.gmm_mx4(xc, xs, wc, ws, c, dtype=torch.float32)
    want, mag = plain.gmm(plain.unpack_values(xc, xs, 128), plain.unpack_values(wc, ws, 128), c)
    plain.check_sums(y, want, mag, 128)
    xs[2, 1] = 255
    y = moe.gmm_mx4(xc, xs, wc, ws, c, dtype=torch.float32)
    assert bool(torch.isnan(y[2]).all()) and int(torch.isnan(y).sum()) == 48


def test_product_refuses_counts_and_index():
    xc, xs, wc, ws, c, y = product([3, 4], 48, 128, torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(y, 2.0)
    bad = torch.tensor([4, 4], dtype=torch.int32, device=DEV)
    moe.gmm_mx4(xc, xs, wc, ws, bad, out=out, status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS and bool((out == 2).all())
    status.zero_()
    index = torch.tensor([0, 1, 2, 7, 4, -3, 6], dtype=torch.int32, device=DEV)
    z = moe.gmm_mx4(xc, xs, wc, ws, c, index=index, status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS
    assert bool((z[[3, 5]] == 0).all()) and torch.equal(z[[0, 1, 2, 4, 6]], y[[0, 1, 2, 4, 6]])
