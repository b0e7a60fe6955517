"""The weighted return of rows and its gradients against float64."""
import pytest
import torch

from all_movement_amd import a2av, moe
from tests import moe_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def make(T, k, H, dt, dropped, seed, offset=0):
    gen = torch.Generator().manual_seed(seed)
    kept = torch.rand(T * k, generator=gen) >= dropped
    rows = int(kept.sum())
    place = torch.full((T * k,), -1, dtype=torch.int32)
    place[kept] = torch.randperm(rows, generator=gen).to(torch.int32)

    def randn(n, m):
        return torch.randn(n * m + offset, generator=gen).to(dt).to(DEV)[offset:].view(n, m)
    return (randn(max(rows, 1), H), place.view(T, k).to(DEV),
            (torch.rand(T, k, generator=gen) - 0.3).to(DEV), randn(T, H))


def expect(y, place, w, dout):
    y, w, dout, place = y.double().cpu(), w.double().cpu(), dout.double().cpu(), place.cpu().long()
    here = place >= 0
    rows = y[place.clamp(min=0)] * here[:, :, None]
    out = (rows * w[:, :, None]).sum(1)
    mag = (rows * w[:, :, None]).abs().sum(1)
    dy = torch.zeros_like(y)
    dy[place[here]] = (w[:, :, None] * dout[:, None, :])[here]
    dw = (rows * dout[:, None, :]).sum(2)
    dmag = (rows * dout[:, None, :]).abs().sum(2)
    return out, mag, dy, dw, dmag


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 2, 7168), (16, 2, 256), (33, 3, 1023), (7, 8, 40),
                                   (300, 1, 24), (5, 64, 16), (12, 9, 2050), (2, 17, 4104)])
@pytest.mark.parametrize("dropped", [0.0, 0.4])
def test_against_float64(dt, T, k, H, dropped):
    y, place, w, dout = make(T, k, H, dt, dropped, T * 100 + k)
    print("combine", T, k, H, dt, dropped, flush=True)
    out, mag, dy, dw, dmag = expect(y, place, w, dout)
    plain.check_sums(moe.combine(y, place, w, check=True), out, mag, k)
    gy, gw = moe.combine_backward(dout, y, place, w, check=True)
    named = torch.zeros(y.shape[0], dtype=torch.bool)
    named[place[place >= 0].cpu().long()] = True
    plain.check_sums(gy[named.to(DEV)], dy[named], dy[named].abs(), 1)
    plain.check_sums(gw, dw, dmag, H)
    assert bool((gw[place < 0] == 0).all())


@pytest.mark.parametrize("offset", [1, 2, 4])
def test_addresses_of_every_alignment(offset):
    for dt in DTYPES:
        y, place, w, dout = make(9, 3, 64, dt, 0.2, offset, offset)
        out, mag, dy, dw, dmag = expect(y, place, w, dout)
        plain.check_sums(moe.combine(y, place, w), out, mag, 3)
        gy, gw = moe.combine_backward(dout, y, place, w)
        plain.check_sums(gw, dw, dmag, 64)
        plain.check_sums(gy, dy, dy.abs(), 1)


def test_without_weights_is_the_gradient_of_the_gather():
    y, place, _, dout = make(40, 2, 72, torch.bfloat16, 0.3, 5)
    ones = torch.ones(40, 2, device=DEV)
    assert torch.equal(moe.combine(y, place), moe.combine(y, place, ones))
    gy, gw = moe.combine_backward(dout, y, place)
    assert gw is None and torch.equal(gy, moe.combine_backward(dout, y, place, ones)[0])


def test_tokens_without_rows_and_strides():
    y, place, w, dout = make(6, 2, 24, torch.float32, 0.0, 7)
    place[2] = -1
    y[place[3].long()] = float("nan")  # stays in its token
    w[2] = float("nan")                # an empty slot's weight is not read
    for pad in (4, 1):
        ys = torch.full((y.shape[0], 24 + pad), float("nan"), device=DEV)[:, :24]
        ys.copy_(y)
        buf = torch.full((6, 24 + pad), 9.0, device=DEV)
        out = moe.combine(ys, place, w, out=buf[:, :24])
        assert bool((out[2] == 0).all()) and bool(torch.isnan(out[3]).all())
        assert int(torch.isnan(out).sum()) == 24 and bool((buf[:, 24:] == 9).all())
        assert torch.equal(out.nan_to_num(), moe.combine(y, place, w).nan_to_num())


def test_rows_that_no_slot_names_are_left():
    y, place, w, dout = make(6, 2, 32, torch.bfloat16, 0.0, 8)
    place[4, 1] = -1
    dy = torch.full_like(y, 6.0)
    dw = torch.empty(6, 2, device=DEV)
    moe.combine_backward(dout, y, place, w, out=(dy, dw))
    named = set(place[place >= 0].tolist())
    for r in range(y.shape[0]):
        assert bool((dy[r] == 6).all()) == (r not in named)


def test_places_are_checked_on_the_device():
    y, place, w, dout = make(6, 2, 32, torch.bfloat16, 0.0, 9)
    good = place.clone()
    good[1, 0] = good[5, 1] = -1
    place[1, 0], place[5, 1] = y.shape[0], -2
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert torch.equal(moe.combine(y, place, w, status=status), moe.combine(y, good, w, check=True))
    assert status.item() == a2av.ERR_INVALID_ARGS
    with pytest.raises(ValueError, match="INVALID_ARGS"):
        moe.combine_backward(dout, y, place, w, check=True)


def test_no_tokens_and_no_rows():
    y = torch.empty(0, 16, device=DEV)
    assert moe.combine(y, torch.empty(0, 2, dtype=torch.int32, device=DEV)).shape == (0, 16)
    none = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    w = torch.rand(3, 2, device=DEV)
    assert bool((moe.combine(y, none, w, check=True) == 0).all())
    dy, dw = moe.combine_backward(torch.randn(3, 16, device=DEV), y, none, w, check=True)
    assert dy.shape == (0, 16) and bool((dw == 0).all())


def test_gradient_against_differences():
    y, place, w, dout = make(4, 2, 16, torch.float32, 0.2, 10)
    dy, dw = moe.combine_backward(dout, y, place, w)
    f = lambda a, b: (expect(a, place, b, dout)[0] * dout.double().cpu()).sum().item()  # noqa: E731
    h = 0.25  # bilinear
    for t, j in [(0, 0), (3, 1)]:
        d = torch.zeros_like(w)
        d[t, j] = h
        diff = (f(y, w.double() + d) - f(y, w.double() - d)) / (2 * h)
        assert abs(diff - dw[t, j].item()) < 1e-5 * (1 + abs(diff))
    for r, c in [(0, 0), (y.shape[0] - 1, 15)]:
        d = torch.zeros_like(y)
        d[r, c] = h
        diff = (f(y.double() + d, w) - f(y.double() - d, w)) / (2 * h)
        assert abs(diff - dy[r, c].item()) < 1e-5 * (1 + abs(diff))


def test_graph():
    y, place, w, dout = make(50, 3, 128, torch.bfloat16, 0.1, 11)
    out = moe.combine(y, place, w)
    back = moe.combine_backward(dout, y, place, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.combine(y, place, w, out=out)
        moe.combine_backward(dout, y, place, w, out=back)
    for _ in range(3):
        y.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe.combine(y, place, w))
        assert torch.equal(back[0], moe.combine_backward(dout, y, place, w)[0])
