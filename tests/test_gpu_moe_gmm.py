"""The products grouped by expert against float64, over sizes, raggedness,
types, strides and alignments, with the device-side refusals."""
import pytest
import torch

from all_movement_amd import a2av, moe
from tests import moe_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(gen, rows, E, N, K, dt, counts, tokens=None, offset=0):
    """x, w, dy (views `offset` elements into their storage) and the counts."""
    def randn(*shape):
        n = 1
        for s in shape:
            n *= s
        flat = torch.randn(n + offset, generator=gen).to(dt).to(DEV)
        return flat[offset:].view(*shape)
    x = randn(tokens or rows, K)
    w = randn(E, N, K) if K < 64 else (randn(E, N, K) * 0.125)
    if offset:
        w0 = torch.empty(E * N * K + offset, dtype=dt, device=DEV)[offset:].view(E, N, K)
        w0.copy_(w)
        w = w0
    return x, w, randn(rows, N), torch.tensor(counts, dtype=torch.int32, device=DEV)


def check_all(gen, counts, N, K, dt, tokens=None, offset=0, extra=0):
    E, used = len(counts), sum(counts)
    rows = used + extra
    x, w, dy, c = make(gen, max(rows, 1), E, N, K, dt, counts, tokens, offset)
    index = None
    if tokens:
        index = torch.randint(0, tokens, (max(rows, 1),), generator=gen).to(torch.int32).to(DEV)
    print("rows", rows, "E", E, "N", N, "K", K, dt, "tokens", tokens, "offset", offset, flush=True)
    y0 = torch.full((max(rows, 1), N), 7.0, dtype=dt, device=DEV)
    y = moe.gmm(x, w, c, index=index, out=y0, check=True)
    want, mag = plain.gmm(x, w, c, index)
    plain.check_sums(y[:used], want, mag, K)
    assert bool((y[used:] == 7).all()), "rows past the counts were written"
    dx0 = torch.full((max(rows, 1), K), 7.0, dtype=dt, device=DEV)
    dx = moe.gmm_dx(dy, w, c, out=dx0, check=True)
    want, mag = plain.gmm_dx(dy, w, c)
    plain.check_sums(dx[:used], want, mag, N)
    assert bool((dx[used:] == 7).all())
    for odt in (dt, torch.float32):
        dw = moe.gmm_dw(dy, x, c, index=index, out_dtype=odt, check=True)
        want, mag = plain.gmm_dw(dy, x, c, index)
        plain.check_sums(dw, want, mag, max(counts) if counts else 0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 8),
    ([1], 1, 1),
    ([0, 1, 0], 16, 64),
    ([3, 0, 5, 1], 72, 136),
    ([130, 0, 1, 257], 264, 200),
    ([128, 128], 128, 128),
    ([17, 31, 0, 0, 64, 2], 320, 512),
    ([300], 512, 1000),
    ([5, 9], 33, 65),
    ([129, 1, 70], 131, 77),
    ([64, 3], 130, 259),
])
def test_against_float64(dt, counts, N, K):
    check_all(torch.Generator().manual_seed(N * 7 + K), counts, N, K, dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,N,K,tokens", [
    ([4, 0, 7, 5], 64, 128, 8), ([200, 3, 150], 136, 264, 177), ([9, 2], 31, 45, 5)])
def test_gathered_rows(dt, counts, N, K, tokens):
    check_all(torch.Generator().manual_seed(tokens), counts, N, K, dt, tokens=tokens, extra=3)


@pytest.mark.parametrize("offset", [1, 4, 8])
def test_addresses_of_every_alignment(offset):
    check_all(torch.Generator().manual_seed(offset), [40, 0, 90], 64, 96, torch.bfloat16,
              offset=offset)


def test_many_experts():
    gen = torch.Generator().manual_seed(3)
    counts = torch.randint(0, 3, (500,), generator=gen).tolist()
    check_all(gen, counts, 24, 40, torch.bfloat16)


def test_no_rows():
    w = torch.randn(3, 16, 32, device=DEV, dtype=torch.bfloat16)
    c = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 32, device=DEV, dtype=torch.bfloat16)
    assert moe.gmm(x, w, c).shape == (0, 16)
    dy = torch.empty(0, 16, device=DEV, dtype=torch.bfloat16)
    assert moe.gmm_dx(dy, w, c).shape == (0, 32)
    assert bool((moe.gmm_dw(dy, x, c, check=True) == 0).all())


def test_strided_rows():
    gen = torch.Generator().manual_seed(11)
    for pad in (8, 3):
        x, w, dy, c = make(gen, 70, 2, 40, 48, torch.bfloat16, [30, 40])
        xs = torch.full((70, 48 + pad), float("nan"), dtype=x.dtype, device=DEV)[:, :48]
        ds = torch.full((70, 40 + pad), float("nan"), dtype=x.dtype, device=DEV)[:, :40]
        xs.copy_(x)
        ds.copy_(dy)
        ys = torch.full((70, 40 + pad), 5.0, dtype=x.dtype, device=DEV)
        moe.gmm(xs, w, c, out=ys[:, :40])
        assert torch.equal(ys[:, :40], moe.gmm(x, w, c)) and bool((ys[:, 40:] == 5).all())
        gs = torch.full((70, 48 + pad), 5.0, dtype=x.dtype, device=DEV)
        moe.gmm_dx(ds, w, c, out=gs[:, :48])
        assert torch.equal(gs[:, :48], moe.gmm_dx(dy, w, c)) and bool((gs[:, 48:] == 5).all())
        assert torch.equal(moe.gmm_dw(ds, xs, c), moe.gmm_dw(dy, x, c))


def test_rows_do_not_leak_into_each_other():
    """NaN rows (and infinite weights of another expert) stay where they are."""
    gen = torch.Generator().manual_seed(5)
    x, w, dy, c = make(gen, 12, 3, 32, 64, torch.bfloat16, [5, 4, 3])
    good = moe.gmm(x, w, c)
    x[6] = float("nan")
    w[2] = float("inf")
    y = moe.gmm(x, w, c)
    keep = [0, 1, 2, 3, 4, 5, 7, 8]
    assert torch.equal(y[keep], good[keep])
    assert bool(torch.isnan(y[6]).all())
    dx = moe.gmm_dx(dy, w, c)
    assert bool(torch.isfinite(dx[:9].float()).all())
    dw = moe.gmm_dw(dy, x, c)
    assert bool(torch.isfinite(dw[[0, 2]].float()).all()) and bool(torch.isnan(dw[1]).all())


@pytest.mark.parametrize("counts", [[5, -1, 3], [9, 9, 0], [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]])
def test_counts_are_checked_on_the_device(counts):
    gen = torch.Generator().manual_seed(1)
    x, w, dy, c = make(gen, 12, 3, 32, 64, torch.bfloat16, counts)
    out = torch.full((12, 32), 3.0, dtype=x.dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.gmm(x, w, c, out=out, status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS and bool((out == 3).all())
    with pytest.raises(ValueError, match="INVALID_ARGS"):
        moe.gmm_dx(dy, w, c, check=True)
    dw = torch.full((3, 32, 64), 3.0, dtype=x.dtype, device=DEV)
    with pytest.raises(ValueError, match="INVALID_ARGS"):
        moe.gmm_dw(dy, x, c, out=dw, check=True)
    assert bool((dw == 3).all())


def test_bad_index_entries_count_as_zero_rows():
    gen = torch.Generator().manual_seed(2)
    x, w, dy, c = make(gen, 6, 2, 32, 64, torch.bfloat16, [3, 3], tokens=4)
    index = torch.tensor([0, 4, 1, -1, 2, 3], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = moe.gmm(x, w, c, index=index, status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS
    x0 = torch.cat([x, torch.zeros_like(x[:1])])
    fixed = torch.tensor([0, 4, 1, 4, 2, 3], dtype=torch.int32, device=DEV)
    assert torch.equal(y, moe.gmm(x0, w, c, index=fixed, check=True))
    status.zero_()
    dw = moe.gmm_dw(dy, x, c, index=index, status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS
    assert torch.equal(dw, moe.gmm_dw(dy, x0, c, index=fixed, check=True))


def test_gradients_against_differences():
    """dx and dw are the derivatives of sum(y * dy): central differences of the
    float64 form, which the forward product is checked against."""
    gen = torch.Generator().manual_seed(4)
    x, w, dy, c = make(gen, 5, 2, 8, 16, torch.bfloat16, [2, 3])
    dx, dw = moe.gmm_dx(dy, w, c).double().cpu(), moe.gmm_dw(dy, x, c, out_dtype=torch.float32)
    f = lambda a, b: (plain.gmm(a, b, c)[0] * dy.double().cpu()).sum()  # noqa: E731
    x64, w64, h = x.double().cpu(), w.double().cpu(), 0.5  # bilinear: any step is exact
    for r, k in [(0, 0), (3, 7), (4, 15)]:
        d = torch.zeros_like(x64)
        d[r, k] = h
        diff = (f(x64 + d, w64) - f(x64 - d, w64)) / (2 * h)
        assert abs(diff - dx[r, k]) <= 2 ** -8 * abs(diff) + 1e-4
    for e, n, k in [(0, 0, 0), (1, 7, 3)]:
        d = torch.zeros_like(w64)
        d[e, n, k] = h
        diff = (f(x64, w64 + d) - f(x64, w64 - d)) / (2 * h)
        assert abs(diff - dw[e, n, k].item()) <= 1e-4 * (1 + abs(diff))


def test_another_stream_and_graph():
    gen = torch.Generator().manual_seed(6)
    x, w, dy, c = make(gen, 100, 4, 64, 128, torch.bfloat16, [40, 0, 50, 10])
    want = [moe.gmm(x, w, c), moe.gmm_dx(dy, w, c), moe.gmm_dw(dy, x, c)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [moe.gmm(x, w, c, stream=side), moe.gmm_dx(dy, w, c, stream=side),
           moe.gmm_dw(dy, x, c, stream=side)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.gmm(x, w, c, out=out[0])
        moe.gmm_dx(dy, w, c, out=out[1])
        moe.gmm_dw(dy, x, c, out=out[2])
    for n in ([40, 0, 50, 10], [0, 90, 0, 10], [25, 25, 25, 25]):
        c.copy_(torch.tensor(n, dtype=torch.int32))
        x.mul_(0.5)
        g.replay()
        torch.cuda.synchronize()
        want = [moe.gmm(x, w, c), moe.gmm_dx(dy, w, c), moe.gmm_dw(dy, x, c)]
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("counts,N,K", [([520, 300], 16640, 136), ([1100, 0, 3], 2048, 16640),
                                        ([700, 90], 1000, 8456), ([5000], 4096, 264)])
def test_rounds_of_whole_tiles_and_cut_ones(counts, N, K):
    """More tiles than CUs, in one direction or another, and a part of a round."""
    check_all(torch.Generator().manual_seed(N), counts, N, K, torch.bfloat16)


@pytest.mark.parametrize("K", [64, 128, 192, 256, 320, 72, 200])
def test_lengths_around_the_stages(K):
    gen = torch.Generator().manual_seed(K)
    check_all(gen, [200, 0, 310], 264, K, torch.float16)
    check_all(gen, [K, 3 * K, 1, 2], 136, 264, torch.bfloat16, tokens=50)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_every_product_is_in_the_sums_that_are_stored(dt):
    """One step of the reduction, tiles of every kind: the last products end right
    before their sums are stored."""
    gen = torch.Generator().manual_seed(21)
    for counts, N, K in [([64, 3], 130, 259), ([40, 64], 72, 72), ([300], 264, 64), ([9], 48, 32),
                         ([64], 264, 264), ([30, 20], 40, 64)]:
        check_all(gen, counts, N, K, dt)


@pytest.mark.parametrize("N,K", [(64 + t, 200 - t) for t in range(1, 8)]
                         + [(8 + t, 8 - t) for t in range(1, 8)]
                         + [(8 - t, 8 + t) for t in range(1, 8)] + [(7, 5), (129, 521)])
def test_row_ends_of_every_length(N, K):
    """Rows that end inside a piece of 8 elements, with NaN before and after them."""
    gen = torch.Generator().manual_seed(N * 1000 + K)
    x, w, dy, c = make(gen, 160, 3, N, K, torch.bfloat16, [90, 0, 70])

    def among_nan(t, pad):
        flat = torch.full((t[..., 0].numel() * (t.shape[-1] + pad) + 22,), float("nan"),
                          dtype=t.dtype, device=DEV)[11:-11]
        v = flat.view(*t.shape[:-1], t.shape[-1] + pad)[..., :t.shape[-1]]
        return v.copy_(t)
    xn, wn, dyn = among_nan(x, 5), among_nan(w, 0), among_nan(dy, 9)
    print("N", N, "K", K, flush=True)
    plain.check_sums(moe.gmm(xn, wn, c, check=True), *plain.gmm(x, w, c), K)
    plain.check_sums(moe.gmm_dx(dyn, wn, c, check=True), *plain.gmm_dx(dy, w, c), N)
    plain.check_sums(moe.gmm_dw(dyn, xn, c, check=True), *plain.gmm_dw(dy, x, c), 90)


def test_far_rows_take_the_plain_loads():
    """A stride of which 256 rows pass 4 GiB: the same values as close together."""
    gen = torch.Generator().manual_seed(8)
    x, w, dy, c = make(gen, 3, 1, 64, 128, torch.bfloat16, [3])
    far = torch.empty(2 ** 24 * 2 + 128, dtype=torch.bfloat16, device=DEV)
    xf = far.as_strided((3, 128), (2 ** 24, 1))
    xf.copy_(x)
    assert torch.equal(moe.gmm(xf, w, c), moe.gmm(x, w, c))
    assert torch.equal(moe.gmm_dw(dy, xf, c), moe.gmm_dw(dy, x, c))
