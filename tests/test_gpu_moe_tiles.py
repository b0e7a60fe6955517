"""The tile kernels of the forward products, at widths that the streaming kernel of
few workgroups leaves to them: ends of rows, strides, alignments, short rows, rows
that are no numbers, indexes outside x."""
import pytest
import torch

from all_movement_amd import moe
from tests import test_gpu_moe_operands as operands
from tests.test_gpu_moe_kernels import check, test_4_bit_rows as check_4_bits, whole
from tests.test_gpu_moe_mx4 import product

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts,N,K,tokens", [
    ([100, 0, 60], 2568, 640, None), ([100, 0, 60], 2568, 1600, 90),   # 128 x 128, four stages
    ([90, 0, 70], 2571, 203, 50), ([90, 0, 70], 2571, 1003, None),     # by way of registers
    ([90, 50], 2600, 5, None), ([90, 50], 2601, 1, 33),                # short rows
    ([300, 200], 1032, 328, 77)])                                      # 256 x 256, cut
def test_wide_products(dt, counts, N, K, tokens):
    check(counts, N, K, dt, tokens, ("fwd",))


@pytest.mark.parametrize("counts,N,K,tokens", [
    ([100, 0, 60], 2568, 512, None), ([100, 0, 60], 2568, 1536, 90), ([100, 0, 60], 2568, 2560, None),
    ([300, 200], 2568, 416, 77), ([300, 200], 2568, 1120, None), ([300, 200], 2568, 2880, 90),
    ([300, 200], 2568, 2560, 77), ([120, 130], 4104, 1536, None), ([120, 130], 4104, 2560, 90)])
def test_wide_4_bit_products(counts, N, K, tokens):
    check_4_bits(counts, N, K, tokens)


@pytest.mark.parametrize("K,tokens", [(1, None), (32, 90), (288, None), (1000, 50), (2049, None)])
def test_wide_4_bit_products_of_any_length(K, tokens):
    for dt in (torch.float32, torch.bfloat16):
        product([300, 200], 2568, K, dt, tokens, seed=K)


def among_nan(t, pad, before):
    """t with rows `pad` further apart, NaN between and around them, `before` + 1
    elements behind an aligned address."""
    rows, width = t.numel() // t.shape[-1], t.shape[-1]
    flat = torch.full((rows * (width + pad) + before + 9,), float("nan"), dtype=t.dtype, device=DEV)
    v = flat[before + 1:before + 1 + rows * (width + pad)]
    return v.view(*t.shape[:-1], width + pad)[..., :width].copy_(t)


@pytest.mark.parametrize("K", [200 - t for t in range(8)] + [15 - t for t in range(8)] + [4, 521])
def test_row_ends_of_every_length(K):
    """Rows that end inside a piece of 8, at odd addresses, among NaN."""
    gen = torch.Generator(device=DEV).manual_seed(K)
    dt, counts = torch.bfloat16, [90, 0, 70]
    x, w = whole(gen, 160, K, dt=dt), whole(gen, 3, 2571, K, dt=dt)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    want = torch.cat([x[:90].double() @ w[0].double().t(), x[90:].double() @ w[2].double().t()])
    for before in (0, 3, 6):
        print("K", K, "before", before, flush=True)
        y = moe.gmm(among_nan(x, 5, before), among_nan(w, 0, before), c, check=True)
        assert torch.equal(y, want.float().to(dt))


@pytest.mark.parametrize("pad", [8, 3])
def test_strided_rows(pad):
    gen = torch.Generator(device=DEV).manual_seed(pad)
    dt = torch.bfloat16
    x, w = whole(gen, 160, 136, dt=dt), whole(gen, 2, 2568, 136, dt=dt)
    c = torch.tensor([90, 70], dtype=torch.int32, device=DEV)
    want = moe.gmm(x, w, c, check=True)
    out = torch.full((160, 2568 + pad), 5.0, dtype=dt, device=DEV)
    y = moe.gmm(among_nan(x, pad, 7), w, c, out=out[:, :2568], check=True)
    assert torch.equal(y, want) and bool((out[:, 2568:] == 5).all())


@pytest.mark.parametrize("K", [136, 203])
def test_rows_that_are_no_numbers_stay_where_they_are(K):
    gen = torch.Generator(device=DEV).manual_seed(K)
    x, w = whole(gen, 230, K, dt=torch.bfloat16), whole(gen, 3, 2568, K, dt=torch.bfloat16)
    c = torch.tensor([90, 70, 60], dtype=torch.int32, device=DEV)  # and ten rows past them
    out = torch.full((230, 2568), 7.0, dtype=x.dtype, device=DEV)
    good = moe.gmm(x, w, c)[:220]
    x[100], x[220:] = float("nan"), float("nan")
    w[2], w[0, 9] = float("inf"), float("nan")
    y = moe.gmm(x, w, c, out=out, check=True)
    assert bool((y[220:] == 7).all()) and bool(torch.isnan(y[100]).all())
    assert bool(torch.isnan(y[:90, 9]).all())
    keep = torch.ones(220, 2568, dtype=torch.bool, device=DEV)
    keep[100], keep[160:], keep[:90, 9] = False, False, False
    assert torch.equal(y[:220][keep], good[keep])


@pytest.mark.parametrize("counts,N,K", [([100, 60], 2568, 640), ([300, 200], 1032, 640),
                                        ([90, 70], 2571, 203), ([90, 70], 2600, 5)])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("finite", [True, False])
def test_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite):
    operands.test_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite)


@pytest.mark.parametrize("counts,N,K", [([100, 60], 2568, 1536), ([300, 200], 2568, 2560),
                                        ([300, 200], 2568, 416), ([120, 130], 4104, 1536)])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("finite", [True, False])
def test_4_bit_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite):
    operands.test_4_bit_rows_outside_x_are_rows_of_zeros(counts, N, K, spread, finite)


def test_gathered_rows_past_4_gib():
    gen = torch.Generator(device=DEV).manual_seed(9)
    x, w = whole(gen, 600, 320, dt=torch.bfloat16), whole(gen, 2, 2568, 320, dt=torch.bfloat16)
    c = torch.tensor([100, 60], dtype=torch.int32, device=DEV)
    index = torch.randint(0, 600, (160,), generator=gen, device=DEV, dtype=torch.int32)
    index[:8] = 599
    wide = torch.empty(599 * 2 ** 22 + 320, dtype=x.dtype, device=DEV)
    far = wide.as_strided((600, 320), (2 ** 22, 1)).copy_(x)
    assert torch.equal(moe.gmm(far, w, c, index=index, check=True), moe.gmm(x, w, c, index=index))
    far = wide.as_strided((90, 320), (2 ** 24, 1)).copy_(x[:90])
    c = torch.tensor([50, 40], dtype=torch.int32, device=DEV)
    assert torch.equal(moe.gmm(far, w, c, check=True), moe.gmm(x[:90], w, c))
