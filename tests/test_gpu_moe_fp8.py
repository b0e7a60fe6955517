"""The 8-bit format: codes and scales equal to the definition's, and the grouped
products on them against float64."""
import math

import numpy as np
import pytest
import torch

from all_movement_amd import a2av, moe
from tests import moe_plain as plain
from tests import moe_plain8 as plain8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def rows_of(dt, rows, cols, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen) * torch.randn(rows, 1, generator=gen).mul(3).exp()
    return x.to(dt)


def bytes_of(t):
    return t.cpu().view(torch.uint8).numpy()


def same_values(v, want, dt):
    with np.errstate(over="ignore"):
        want = torch.from_numpy(want).to(torch.float32).to(dt)
    v = v.cpu()
    assert torch.equal(v.nan_to_num(nan=9.0), want.nan_to_num(nan=9.0))
    assert torch.equal(torch.signbit(v), torch.signbit(want)) or not bool(
        torch.isfinite(want).all())


def check(x):
    codes, scales = moe.fp8_quantize(x.to(DEV))
    want_c, want_s, want_v = plain8.quantize(x.double().numpy())
    assert np.array_equal(bytes_of(scales), want_s)
    assert np.array_equal(bytes_of(codes), want_c)
    for dt in DTYPES:
        same_values(moe.fp8_dequantize(codes, scales, x.shape[1], dt), want_v, dt)
    return codes, scales


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (5, 127), (7, 256), (130, 640),
                                       (2, 7168), (9, 523), (33, 12), (4, 1540), (300, 8)])
def test_codes_and_values(dt, rows, cols):
    check(rows_of(dt, rows, cols, rows * 1000 + cols))


def test_ties_zeros_and_the_ends_of_the_range():
    grid = list(plain8.GRID)
    mids = [(a + b) / 2 for a, b in zip(grid, grid[1:])]
    near = [float(np.nextafter(np.float32(m), np.float32(d))) for m in mids[:40] for d in (0, 500)]
    block = (mids + [-m for m in mids] + near + grid + [-0.0, 448.0])
    rows = []
    for at in range(0, len(block), 127):
        part = block[at:at + 127]
        part = [448.0] + part + [0.0] * (127 - len(part))
        rows += [[v * s for v in part] for s in (1.0, 2.0 ** -100, 2.0 ** 100)]
    for top in (448.0, 449.0, 1.75, 1.7500001, 2.0, 1.0):
        rows.append([top] + [1.0] * 127)
    rows += [[0.0] * 128, [-0.0] * 128, [2.0 ** -126] * 128, [2.0 ** -149] * 127 + [2.0 ** -130],
             [3.4028234e38] + [1.0] * 127, [2.0 ** -118] + [2.0 ** -126] * 127,
             [1.75 * 2.0 ** -119] * 128, [1.76 * 2.0 ** -119] * 128]
    check(torch.tensor(rows, dtype=torch.float64).to(torch.float32))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_blocks_that_are_no_numbers(bad):
    x = rows_of(torch.float32, 3, 384, 1)
    x[1, 140] = bad
    codes, scales = check(x)
    assert scales[1, 1].item() == 255
    v = moe.fp8_dequantize(codes, scales, 384)
    assert bool(torch.isnan(v[1, 128:256]).all()) and int(torch.isnan(v).sum()) == 128


def test_strided_rows():
    x = rows_of(torch.bfloat16, 6, 256, 2).to(DEV)
    for pad in (8, 1):
        s = torch.full((6, 256 + pad), 1e30, dtype=x.dtype, device=DEV)[:, :256]
        s.copy_(x)
        a, b = moe.fp8_quantize(s), moe.fp8_quantize(x)
        assert np.array_equal(bytes_of(a[0]), bytes_of(b[0])) and torch.equal(a[1], b[1])
        o = torch.full((6, 256 + pad), 5.0, dtype=x.dtype, device=DEV)
        moe.fp8_dequantize(*a, 256, x.dtype, out=o[:, :256])
        assert torch.equal(o[:, :256], moe.fp8_dequantize(*b, 256, x.dtype))
        assert bool((o[:, 256:] == 5).all())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (2, 128, 128), (3, 129, 256), (2, 300, 523),
                                   (1, 127, 640), (2, 5, 1100)])
def test_weights(dt, E, N, K):
    w = rows_of(dt, E * N, K, E + N + K).view(E, N, K)
    codes, scales = moe.fp8_quantize_weights(w.to(DEV))
    back = {d: moe.fp8_dequantize_weights(codes, scales, K, d) for d in DTYPES}
    for e in range(E):
        c, s, v = plain8.quantize(w[e].double().numpy(), 128)
        assert np.array_equal(bytes_of(scales[e]), s)
        assert np.array_equal(bytes_of(codes[e]), c)
        for d in DTYPES:
            same_values(back[d][e], v, d)


def test_a_weight_block_that_is_no_number():
    w = rows_of(torch.bfloat16, 400, 300, 5).view(2, 200, 300)
    w[1, 130, 129] = math.inf
    codes, scales = moe.fp8_quantize_weights(w.to(DEV))
    v = moe.fp8_dequantize_weights(codes, scales, 300)
    assert scales[1, 1, 1].item() == 255
    assert bool(torch.isnan(v[1, 128:, 128:256]).all()) and int(torch.isnan(v).sum()) == 72 * 128


# ---------------------------------------------------------------- products

def operands(counts, N, K, tokens=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    E, rows = len(counts), sum(counts)
    x = torch.randn(tokens or rows, K, generator=gen).to(DEV)
    w = (torch.randn(E, N, K, generator=gen) / math.sqrt(K)).to(DEV)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    index = None
    if tokens:
        index = torch.randint(0, tokens, (rows,), generator=gen).to(torch.int32).to(DEV)
    dy = torch.randn(rows, N, generator=gen).to(DEV)
    return moe.fp8_quantize(x), moe.fp8_quantize_weights(w), c, index, moe.fp8_quantize(dy)


def factors(scales, blocks):
    return torch.exp2(scales[..., :blocks].double() - 127)


def wanted(mode, codes, scales, wc, ws, counts, cols, index=None):
    """The instruction's sums, their magnitudes, and a check of them against plain float64."""
    v = torch.from_numpy(plain8.VALUES).to(DEV)
    x, w = v[codes.view(torch.uint8).long()], v[wc.view(torch.uint8).long()]
    E, N, C = w.shape
    B, strips = C // 128, -(-N // 128)
    xs, w_s = factors(scales, x.shape[1] // 128), factors(ws, B)
    if index is not None:
        x, xs = x[index.long()], xs[index.long()]
    out, mags, at = [], [], 0
    for e, m in enumerate(counts):
        if not m:
            continue
        if mode == "fwd":
            we, se = w[e], w_s[e].repeat_interleave(128, 0)[:N]
        else:
            we = torch.zeros(C, strips * 128, dtype=torch.float64, device=DEV)
            we[:, :N] = w[e].T
            we, se = we[:cols], w_s[e].T.repeat_interleave(128, 0)[:cols]
        r, rs = x[at:at + m], xs[at:at + m]
        cut = plain8.cut_products(r, rs, we, se)
        xv, wv = r * rs.repeat_interleave(128, 1), we * se.repeat_interleave(128, 1)
        exact = xv @ wv.T
        assert bool(((cut - exact).abs() <= plain8.CUT * plain8.tops(xv, wv)
                     + 1e-12 * exact.abs()).all())
        out.append(cut)
        mags.append(xv.abs() @ wv.abs().T)
        at += m
    return torch.cat(out).cpu(), torch.cat(mags).cpu()


def both(counts, N, K, dt, tokens=None, seed=0):
    (xc, xs), (wc, ws), c, index, (yc, ys) = operands(counts, N, K, tokens, seed)
    print("fp8", counts[:8], N, K, dt, tokens, flush=True)
    y = moe.gmm_fp8(xc, xs, wc, ws, c, index=index, dtype=dt, check=True)
    plain.check_sums(y, *wanted("fwd", xc, xs, wc, ws, counts, K, index), K)
    dx = moe.gmm_fp8_dx(yc, ys, wc, ws, c, cols=K, dtype=dt, check=True)
    plain.check_sums(dx, *wanted("dx", yc, ys, wc, ws, counts, K), N)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts,N,K", [
    ([1], 1, 1), ([1], 16, 128), ([0, 2, 0, 3], 40, 64), ([130, 1, 0, 260], 136, 288),
    ([17, 40], 129, 1000), ([64, 9], 256, 2049), ([5, 7, 20, 3], 72, 544), ([3, 0, 0], 523, 1001)])
def test_products(dt, counts, N, K):
    both(counts, N, K, dt, seed=N + K)


@pytest.mark.parametrize("counts,N,K,tokens", [
    ([9, 0, 30], 64, 256, 11), ([200, 77], 200, 416, 100), ([300, 0, 200], 520, 512, 90),
    ([700], 1100, 384, 50), ([40, 3, 0, 77], 130, 1536, None), ([2, 1], 48, 2560, None),
    ([1] * 70, 33, 140, 20)])
def test_products_of_gathered_rows(counts, N, K, tokens):
    both(counts, N, K, torch.bfloat16, tokens, seed=N)


def test_products_in_rounds_of_whole_tiles():
    both([520, 300], 16640, 512, torch.float16, seed=3)


def whole(shape, gen):
    """Whole numbers of -8..8 as codes, scales of 1: their sums are exact."""
    return torch.randint(-8, 9, shape, generator=gen).float()


def whole_numbers(counts, N, K, tokens=None):
    """Every sum is a whole number below 2^24: equal to float64's."""
    gen = torch.Generator().manual_seed(N + K)
    E, rows = len(counts), sum(counts)
    x, w, dy = whole((tokens or rows, K), gen), whole((E, N, K), gen), whole((rows, N), gen)
    x[:, 0], w[:, :, 0], dy[:, 0] = 8, 8, 8

    def coded(t, tall):
        C, S = -(-t.shape[-1] // 128) * 128, plain8.pitch(t.shape[-1])
        c = torch.zeros(*t.shape[:-1], C)
        c[..., :t.shape[-1]] = t
        strips = -(-t.shape[-2] // tall)
        s = torch.full((*t.shape[:-2], strips, S), 127, dtype=torch.uint8)
        return c.to(torch.float8_e4m3fn).to(DEV), s.to(DEV)

    (xc, xs), (wc, ws), (yc, ys) = coded(x, 1), coded(w, 128), coded(dy, 1)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    index = torch.randint(0, tokens, (rows,), generator=gen).to(torch.int32) if tokens else None
    print("whole", counts[:8], N, K, tokens, flush=True)
    y = moe.gmm_fp8(xc, xs, wc, ws, c, index=None if index is None else index.to(DEV),
                    dtype=torch.float32, check=True)
    assert torch.equal(y.cpu().double(), plain.gmm(x, w, c, index)[0])
    dx = moe.gmm_fp8_dx(yc, ys, wc, ws, c, cols=K, dtype=torch.float32, check=True)
    assert torch.equal(dx.cpu().double(), plain.gmm_dx(dy, w, c)[0])


@pytest.mark.parametrize("counts,N,K,tokens", [
    ([1, 0, 5], 100, 4000, None), ([12] * 16, 256, 2048, 40), ([31, 17, 40, 2], 257, 1024, None),
    ([260, 150, 390], 384, 1280, 333), ([1000, 24], 640, 900, None), ([513], 300, 7168, None),
    ([2100, 5], 2300, 256, None), ([520, 300], 16640, 512, None),
    ([64] * 5, 2304, 128, None), ([16], 4096, 8192, None)])
def test_whole_numbers(counts, N, K, tokens):
    whole_numbers(counts, N, K, tokens)


@pytest.mark.parametrize("counts,N", [
    ([4] * 8, 2048), ([100], 2048), ([70, 0, 30, 60, 64, 64, 90, 64], 2048), ([300] * 3, 900),
    ([513], 1500)])
@pytest.mark.parametrize("K", [128, 500, 640, 2304])
def test_every_kernel(counts, N, K):
    """The streaming products by four and eight waves, small tiles of two stages and of
    four, large tiles, with one stage, an odd number and an even one."""
    whole_numbers(counts, N, K, 37)


def test_scales_of_the_whole_range():
    """Scales whose product is an ordinary number; a scale of NaN makes its rows NaN."""
    (xc, xs), (wc, ws), c, _, (yc, ys) = operands([3, 4], 48, 256)
    xs[:], ws[:], ys[:] = 7, 245, 7
    y = moe.gmm_fp8(xc, xs, wc, ws, c, dtype=torch.float32)
    plain.check_sums(y, *wanted("fwd", xc, xs, wc, ws, [3, 4], 256), 256)
    dx = moe.gmm_fp8_dx(yc, ys, wc, ws, c, dtype=torch.float32)
    plain.check_sums(dx, *wanted("dx", yc, ys, wc, ws, [3, 4], 256), 48)
    xs[2, 1] = 255
    y = moe.gmm_fp8(xc, xs, wc, ws, c, dtype=torch.float32)
    assert bool(torch.isnan(y[2]).all()) and int(torch.isnan(y).sum()) == 48
    ws[1, 0, 1] = 255  # columns 128.. of the second expert
    dx = moe.gmm_fp8_dx(yc, ys, wc, ws, c, dtype=torch.float32)
    assert bool(torch.isnan(dx[3:, 128:]).all()) and int(torch.isnan(dx).sum()) == 4 * 128


@pytest.mark.parametrize("rows", [4, 200])
def test_codes_of_nan_beside_a_tile(rows):
    """Rows and experts beside the ones in use hold NaN: none of it shows."""
    (xc, xs), (wc, ws), c, _, (yc, ys) = operands([rows, 0, rows], 200, 256)
    (wc[1].view(torch.uint8))[:] = 0x7f
    ws[1] = 255
    want = [moe.gmm_fp8(xc, xs, wc, ws, c), moe.gmm_fp8_dx(yc, ys, wc, ws, c)]
    assert all(bool(torch.isfinite(t).all()) for t in want)
    more = [torch.cat([b, torch.full_like(b[:5], 0x7f)]).view(a.dtype)
            for a, b in ((a, a.view(torch.uint8)) for a in (xc, xs, yc, ys))]
    y = torch.full((2 * rows + 5, 200), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.gmm_fp8(more[0], more[1], wc, ws, c, out=y, check=True)
    dx = torch.full((2 * rows + 5, 256), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.gmm_fp8_dx(more[2], more[3], wc, ws, c, out=dx, check=True)
    for got, w in ((y, want[0]), (dx, want[1])):
        assert torch.equal(got[:2 * rows], w) and bool((got[2 * rows:] == 3).all())


@pytest.mark.parametrize("counts", [[3, 4], [300, 400], [5000, 3000]])
def test_counts_and_index_outside(counts):
    (xc, xs), (wc, ws), c, _, (yc, ys) = operands(counts, 48, 256)
    rows = sum(counts)
    y = moe.gmm_fp8(xc, xs, wc, ws, c)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for bad in ([counts[0] + 1, counts[1]], [-1, 2]):
        bad = torch.tensor(bad, dtype=torch.int32, device=DEV)
        out = torch.full_like(y, 2.0)
        moe.gmm_fp8(xc, xs, wc, ws, bad, out=out, status=status)
        assert status.item() == a2av.ERR_INVALID_ARGS and bool((out == 2).all())
        status.zero_()
        out = torch.full((rows, 256), 2.0, dtype=torch.bfloat16, device=DEV)
        moe.gmm_fp8_dx(yc, ys, wc, ws, bad, out=out, status=status)
        assert status.item() == a2av.ERR_INVALID_ARGS and bool((out == 2).all())
        status.zero_()
    index = torch.arange(rows, dtype=torch.int32, device=DEV)
    index[1], index[4] = rows, -3
    z = moe.gmm_fp8(xc, xs, wc, ws, c, index=index, status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS
    keep = [i for i in range(rows) if i not in (1, 4)]
    assert bool((z[[1, 4]] == 0).all()) and torch.equal(z[keep], y[keep])


def test_strided_and_unaligned_outputs():
    for rows, N in ((6, 72), (400, 264)):
        (xc, xs), (wc, ws), c, _, (yc, ys) = operands([rows, 3], N, 260)
        for dt in DTYPES:
            y = moe.gmm_fp8(xc, xs, wc, ws, c, dtype=dt)
            dx = moe.gmm_fp8_dx(yc, ys, wc, ws, c, cols=260, dtype=dt)
            for pad in (1, 8):
                o = torch.full((rows + 3, N + pad), 7.0, dtype=dt, device=DEV)
                moe.gmm_fp8(xc, xs, wc, ws, c, out=o[:, 1:N + 1] if pad > 1 else o[:, :N], dtype=dt)
                got = o[:, 1:N + 1] if pad > 1 else o[:, :N]
                assert torch.equal(got, y) and int((o == 7).sum()) >= (rows + 3) * pad
                o = torch.full((rows + 3, 260 + pad), 7.0, dtype=dt, device=DEV)
                moe.gmm_fp8_dx(yc, ys, wc, ws, c, cols=260, out=o[:, :260], dtype=dt)
                assert torch.equal(o[:, :260], dx) and bool((o[:, 260:] == 7).all())


def test_streams_and_replayed_graphs():
    (xc, xs), (wc, ws), c, index, (yc, ys) = operands([40, 300, 0, 9], 256, 640, 64)
    x = moe.fp8_dequantize(xc, xs, 640)
    want = (moe.gmm_fp8(xc, xs, wc, ws, c, index=index), moe.gmm_fp8_dx(yc, ys, wc, ws, c))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.gmm_fp8(xc, xs, wc, ws, c, index=index, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, scales = moe.fp8_quantize(x)
        y = moe.gmm_fp8(codes, scales, wc, ws, c, index=index)
        dx = moe.gmm_fp8_dx(yc, ys, wc, ws, c)
    for _ in range(3):
        y.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
        c2 = moe.gmm_fp8(xc, xs, wc, ws, c, index=index)  # the program's own work between
        assert torch.equal(c2, want[0])


def test_gradient_against_differences():
    """dx of gmm_fp8_dx for the linear map that gmm_fp8 is: <dy, y(x + d) - y(x)> = <dx, d>,
    exactly, for whole numbers."""
    gen = torch.Generator().manual_seed(4)
    counts, N, K = [5, 0, 140], 130, 256
    one = dict(dtype=torch.uint8, device=DEV)
    w = whole((3, N, K), gen).to(DEV).to(torch.float8_e4m3fn)
    ws = torch.full((3, 2, 4), 127, **one)
    x, d = whole((145, K), gen).to(DEV), whole((145, K), gen).to(DEV)
    dy = torch.zeros(145, 256, device=DEV)
    dy[:, :N] = whole((145, N), gen).to(DEV)
    xs, ys = torch.full((145, 4), 127, **one), torch.full((145, 4), 127, **one)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)

    def y(v):
        return moe.gmm_fp8(v.to(torch.float8_e4m3fn), xs, w, ws, c, dtype=torch.float32).double()

    dx = moe.gmm_fp8_dx(dy.to(torch.float8_e4m3fn), ys, w, ws, c, dtype=torch.float32).double()
    # x + d in -16..16 is held exactly by E4M3
    left = (dy[:, :N].double() * (y(x + d) - y(x))).sum()
    assert left.item() == (dx * d.double()).sum().item()


def test_rows_of_x_past_4_GiB():
    """Gathered rows that no 32-bit offset reaches, in the tile kernel and the streaming one."""
    gen = torch.Generator().manual_seed(6)
    K, N, far = 4096, 640, (1 << 20) + 5000
    one = dict(dtype=torch.uint8, device=DEV)
    x = torch.zeros(far, K, **one)
    some = torch.randint(0, far, (900,), generator=gen)
    some[:4] = torch.tensor([far - 1, 0, 1 << 20, (1 << 20) - 1])
    values = whole((900, K), gen)
    x[some.to(DEV)] = values.to(DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    values = x[some.to(DEV)].view(torch.float8_e4m3fn).float().cpu()  # of rows drawn twice
    w = whole((2, N, K), gen)
    wc, ws = w.to(DEV).to(torch.float8_e4m3fn), torch.full((2, 5, 32), 127, **one)
    xs = torch.full((far, 32), 127, **one)
    for counts in ([500, 400], [3, 1]):
        rows = sum(counts)
        index = some[:rows].to(torch.int32).to(DEV)
        c = torch.tensor(counts, dtype=torch.int32, device=DEV)
        y = moe.gmm_fp8(x.view(torch.float8_e4m3fn), xs, wc, ws, c, index=index,
                        dtype=torch.float32, check=True)
        assert torch.equal(y.cpu().double(), plain.gmm(values[:rows], w, c)[0])


def test_a_gradient_of_rows_past_16_MiB():
    """Rows of dy longer than a tile's 32-bit offsets allow: 17 million values."""
    N, K, rows = 17_000_000, 10, 3
    one = dict(dtype=torch.uint8, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(7)
    C = -(-N // 128) * 128
    dy = torch.zeros(rows, C, device=DEV)
    dy[:, :N] = torch.randint(-1, 2, (rows, N), generator=gen, device=DEV).float()
    w = torch.zeros(1, N, 128, device=DEV, dtype=torch.bfloat16)
    w[:, :, :K] = torch.randint(-1, 2, (1, N, K), generator=gen, device=DEV)
    strips = C // 128
    ys = torch.full((rows, -(-strips // 4) * 4), 127, **one)
    ws = torch.full((1, strips, 4), 127, **one)
    c = torch.tensor([rows], dtype=torch.int32, device=DEV)
    dx = moe.gmm_fp8_dx(dy.to(torch.float8_e4m3fn), ys, w.to(torch.float8_e4m3fn), ws, c, cols=K,
                        dtype=torch.float32, check=True)
    want = torch.zeros(rows, K, dtype=torch.float64, device=DEV)
    for at in range(0, N, 1 << 20):
        part = slice(at, min(N, at + (1 << 20)))
        want += dy[:, part].double() @ w[0, part, :K].double()
    assert torch.equal(dx.double(), want)


@pytest.mark.parametrize("counts", [[2], [700, 5]])
def test_an_empty_x(counts):
    """x without rows: every index lies outside it, every row is a row of zeros."""
    (_, _), (wc, ws), c, _, _ = operands(counts, 130, 256)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    index = torch.zeros(sum(counts), dtype=torch.int32, device=DEV)
    y = moe.gmm_fp8(torch.empty(0, 256, dtype=moe.E4M3, device=DEV),
                    torch.empty(0, 4, dtype=torch.uint8, device=DEV), wc, ws, c, index=index,
                    status=status)
    assert status.item() == a2av.ERR_INVALID_ARGS and bool((y == 0).all())


def test_two_streams_at_once():
    """Calls share nothing: two streams' products and conversions side by side."""
    sets = [operands([300, 40], 256, 640, seed=s) for s in (1, 2)]
    want = [(moe.gmm_fp8(*s[0], *s[1], s[2]), moe.gmm_fp8_dx(*s[4], *s[1], s[2])) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(8):
        for i, (s, stream) in enumerate(zip(sets, streams)):
            got[i].append((moe.gmm_fp8(*s[0], *s[1], s[2], stream=stream),
                           moe.gmm_fp8_dx(*s[4], *s[1], s[2], stream=stream)))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for pair in g:
            assert torch.equal(pair[0], w[0]) and torch.equal(pair[1], w[1])
