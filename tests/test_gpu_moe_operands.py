"""Operands at the border of what the operators take: interleaved views, logits
that are no numbers beside masked ones, indexes outside x in every kernel."""
import math

import pytest
import torch

from all_movement_amd import a2av, moe
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


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())


# Sizes that take each forward kernel: few rows per expert (16 and 32 rows to a
# tile), 128 x 128 tiles with four and with two stages, 256 x 256 tiles cut and
# whole, loads by way of registers in 64 x 64 and 128 x 128 tiles, short rows.
KERNELS = [([3, 5], 32, 64), ([20, 9], 72, 77), ([30, 40], 40, 1000), ([100, 60], 264, 640),
           ([30 + 3 * i for i in range(24)], 2176, 512), ([300, 200], 264, 640),
           ([520, 300], 16640, 640), ([90, 70], 64, 203), ([2048], 4199, 203), ([60, 60], 24, 5)]


def bad_index(counts, tokens, spread, gen):
    """An index whose bad entries lie in the rows that one wave loads (or all
    over), and the same with them on row `tokens` (zeros)."""
    rows = sum(counts)
    index = torch.randint(1, tokens, (rows,), generator=gen).to(torch.int32)
    at = list(range(0, rows, 5)) if spread else [rows // 3]
    fixed = index.clone()
    for i, a in enumerate(at):
        index[a] = (-1, tokens, 2 ** 31 - 1, -2 ** 31)[i % 4]
        fixed[a] = tokens
    return index.to(DEV), fixed.to(DEV)


@pytest.mark.parametrize("counts,N,K", KERNELS)
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("finite", [True, False])
def test_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite):
    gen = torch.Generator().manual_seed(N + K)
    E, tokens, dt = len(counts), 50, torch.bfloat16
    x = torch.randn(tokens, K, generator=gen).to(dt).to(DEV)
    x[0] = math.nan  # nobody's row
    x0 = torch.cat([x, torch.zeros_like(x[:1])])
    w = torch.randn(E, N, K, device=DEV, dtype=dt)
    dy = torch.randn(sum(counts), N, device=DEV, dtype=dt)
    if not finite:  # zeros times these are NaN
        w[E - 1, N // 2, K - 1] = math.inf
        w[0, 0, 0] = math.nan
        dy[sum(counts) // 3, N - 1] = math.inf
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    index, fixed = bad_index(counts, tokens, spread, gen)
    print("bad index", counts[:4], N, K, spread, finite, flush=True)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = moe.gmm(x, w, c, index=index, status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS
    assert same(y, moe.gmm(x0, w, c, index=fixed, check=True))
    status.zero_()
    dw = moe.gmm_dw(dy, x, c, index=index, status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS
    assert same(dw, moe.gmm_dw(dy, x0, c, index=fixed, check=True))


# The 4-bit kernels: whole scale groups (K of 512) and others.
@pytest.mark.parametrize("counts,N,K", [
    ([3, 5], 32, 64), ([30, 40], 40, 1000), ([20, 9], 72, 1024), ([100, 60], 264, 1536),
    ([30 + 3 * i for i in range(24)], 2176, 1024), ([300, 200], 264, 2560),
    ([520, 300], 16640, 1024), ([90, 70], 64, 416)])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("finite", [True, False])
def test_4_bit_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite):
    gen = torch.Generator().manual_seed(N + K)
    E, tokens, B = len(counts), 50, (K + 31) // 32
    xc, xs = moe.mx4_quantize(torch.randn(tokens, K, generator=gen).to(DEV))
    xs[0] = 255  # nobody's row
    zc, zs = moe.mx4_quantize(torch.zeros(1, K, device=DEV))
    x0c, x0s = torch.cat([xc, zc]), torch.cat([xs, zs])
    wc, ws = moe.mx4_quantize(torch.randn(E * N, K, device=DEV))
    wc, ws = wc.view(E, N, 16 * B), ws.view(E, N, B)
    if not finite:
        ws[E - 1, N // 2, B - 1] = 255
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    index, fixed = bad_index(counts, tokens, spread, gen)
    print("bad index, 4 bits", counts[:4], N, K, spread, finite, flush=True)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = moe.gmm_mx4(xc, xs, wc, ws, c, index=index, status=status, dtype=torch.float32)
    assert status.item() == a2av.ERR_INVALID_ARGS
    assert same(y, moe.gmm_mx4(x0c, x0s, wc, ws, c, index=fixed, check=True, dtype=torch.float32))


@pytest.mark.parametrize("counts,N,K", [([20] * 8, 1024, 520), ([500], 250, 1024), ([300], 61, 397)])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("finite", [True, False])
def test_streamed_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite):
    test_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite)


@pytest.mark.parametrize("counts,N,K", [([20] * 8, 2048, 1024), ([50] * 8, 2048, 1056),
                                        ([2000], 256, 512)])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("finite", [True, False])
def test_streamed_4_bit_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite):
    test_4_bit_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite)
