"""Every kernel of the grouped products, over reductions long enough for its
inner loop, with whole numbers: their FP32 sums are exact, so each result equals
the float64 one rounded once and no lost or doubled term can hide."""
import pytest
import torch

from all_movement_amd import moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def whole(gen, *shape, dt):
    return torch.randint(-2, 3, shape, generator=gen, device=DEV).to(dt)


def check(counts, N, K, dt, tokens=None, sides=("fwd", "dx", "dw")):
    assert 4 * max(N, K, *counts) < 2 ** 24  # the sums are exact
    gen = torch.Generator(device=DEV).manual_seed(N * 3 + K)
    E, rows = len(counts), sum(counts)
    print("whole numbers", counts[:4], N, K, dt, tokens, sides, flush=True)
    x, w, dy = (whole(gen, *s, dt=dt) for s in ((tokens or rows, K), (E, N, K), (rows, N)))
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    index, xr = None, x
    if tokens:
        index = torch.randint(0, tokens, (rows,), generator=gen, device=DEV, dtype=torch.int32)
        xr = x[index.long()]
    first = [sum(counts[:e]) for e in range(E)]
    if "fwd" in sides:
        y = moe.gmm(x, w, c, index=index, check=True)
        for e, (a, m) in enumerate(zip(first, counts)):
            want = xr[a:a + m].double() @ w[e].double().t()
            assert torch.equal(y[a:a + m], want.float().to(dt)), f"expert {e}"
    if "dx" in sides:
        dx = moe.gmm_dx(dy, w, c, check=True)
        for e, (a, m) in enumerate(zip(first, counts)):
            want = dy[a:a + m].double() @ w[e].double()
            assert torch.equal(dx[a:a + m], want.float().to(dt)), f"expert {e}"
    if "dw" in sides:
        for odt in (dt, torch.float32):
            dw = moe.gmm_dw(dy, x, c, index=index, out_dtype=odt, check=True)
            for e, (a, m) in enumerate(zip(first, counts)):
                want = dy[a:a + m].double().t() @ xr[a:a + m].double()
                assert torch.equal(dw[e], want.float().to(odt)), f"expert {e}"


SOME = [30 + 3 * i for i in range(24)]  # 64 rows per expert


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,N,K,tokens", [
    ([5, 0, 9], 72, 1040, 7),          # few rows per expert
    ([30, 12], 72, 1048, None),
    (SOME, 2176, 512, 300),            # 128 x 128 tiles, two stages, forward
    (SOME, 512, 2176, None),           # and dx
    ([100, 0, 60], 264, 1600, 90),     # four stages
    ([520, 300], 16640, 136, None),    # 256 x 256 tiles, whole and cut ones
    ([520, 300], 16640, 640, 200),
    ([520, 300], 1032, 16640, 400),
    ([1100, 0, 3], 2048, 16640, None),
    ([700, 90], 1000, 8456, None),
    ([5000], 4096, 264, 999),
])
def test_aligned_rows(dt, counts, N, K, tokens):
    check(counts, N, K, dt, tokens)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,N,K,tokens,sides", [
    ([90, 0, 70], 131, 1003, 77, ("fwd", "dx", "dw")),      # 64 x 64 tiles
    ([2048], 4199, 395, 1000, ("fwd",)),                   # 128 x 128 tiles
    ([2048], 395, 4199, None, ("dx",)),
    ([300 + i for i in range(8)], 1101, 1093, 500, ("dw",)),
    ([90, 50], 3, 700, None, ("fwd", "dx", "dw")),         # rows of fewer than 8
    ([90, 50], 700, 5, 44, ("fwd", "dx", "dw")),
])
def test_unaligned_rows(dt, counts, N, K, tokens, sides):
    check(counts, N, K, dt, tokens, sides)


def far_rows(t, stride):
    wide = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype, device=DEV)
    return wide.as_strided(t.shape, (stride, 1)).copy_(t)


def test_rows_too_far_apart_for_32_bit_offsets():
    """256 rows of a stride that pass 4 GiB, with rows enough for a tile kernel."""
    gen = torch.Generator(device=DEV).manual_seed(8)
    dt, counts = torch.bfloat16, [43, 47]
    x, w, dy = (whole(gen, *s, dt=dt) for s in ((90, 320), (2, 72, 320), (90, 72)))
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    xf, dyf = far_rows(x, 2 ** 24), far_rows(dy, 2 ** 24)
    assert torch.equal(moe.gmm(xf, w, c, check=True), moe.gmm(x, w, c))
    assert torch.equal(moe.gmm_dx(dyf, w, c, check=True), moe.gmm_dx(dy, w, c))
    assert torch.equal(moe.gmm_dw(dyf, xf, c, check=True), moe.gmm_dw(dy, x, c))


def test_gathered_rows_past_4_gib():
    gen = torch.Generator(device=DEV).manual_seed(9)
    dt, counts, tokens = torch.bfloat16, [100, 60], 600
    x, w, dy = (whole(gen, *s, dt=dt) for s in ((tokens, 320), (2, 72, 320), (160, 72)))
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    index = torch.randint(0, tokens, (160,), generator=gen, device=DEV, dtype=torch.int32)
    index[:8] = tokens - 1
    xf = far_rows(x, 2 ** 22)
    assert torch.equal(moe.gmm(xf, w, c, index=index, check=True), moe.gmm(x, w, c, index=index))
    assert torch.equal(moe.gmm_dw(dy, xf, c, index=index, check=True),
                       moe.gmm_dw(dy, x, c, index=index))


def values(codes, scales):
    """float64 values of packed codes and scale bytes, on their device."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    table = torch.cat([table, -table])
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    step = torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    return table[c] * step


@pytest.mark.parametrize("counts,N,K,tokens", [
    ([5, 0, 9], 72, 2560, 7), ([30, 12], 72, 1056, None),               # few rows per expert
    (SOME, 2176, 1024, 300), (SOME, 2176, 2560, None),                  # two stages
    ([100, 0, 60], 264, 1536, 90), ([100, 0, 60], 264, 2560, None),     # four
    ([520, 300], 16640, 1024, None), ([520, 300], 16640, 1536, 300),    # whole 256 x 256 tiles
    ([520, 300], 16640, 2560, None), ([300, 200], 264, 5120, 77),
    ([90, 0, 70], 136, 1120, 50), ([300, 200], 264, 2880, None)])       # other scale groups
def test_4_bit_rows(counts, N, K, tokens):
    """Codes of every value with scales of 1/2, 1 and 2: products are sixteenths."""
    gen = torch.Generator(device=DEV).manual_seed(N + K)
    E, rows, B = len(counts), sum(counts), K // 32
    assert K % 32 == 0 and 16 * 144 * K < 2 ** 24  # the sums are exact
    print("4 bits", counts[:4], N, K, tokens, flush=True)

    def rand(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device=DEV, dtype=torch.uint8)
    xc, xs = rand(0, 256, tokens or rows, 16 * B), rand(126, 129, tokens or rows, B)
    wc, ws = rand(0, 256, E, N, 16 * B), rand(126, 129, E, N, B)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    index, x = None, values(xc, xs)
    if tokens:
        index = torch.randint(0, tokens, (rows,), generator=gen, device=DEV, dtype=torch.int32)
        x = x[index.long()]
    y = moe.gmm_mx4(xc, xs, wc, ws, c, index=index, dtype=torch.float32, check=True)
    at = 0
    for e, m in enumerate(counts):
        want = x[at:at + m] @ values(wc[e], ws[e]).t()
        assert torch.equal(y[at:at + m], want.float()), f"expert {e}"
        at += m


# Few workgroups of the streaming kernel: few experts or few columns, with 16 and
# with 32 rows to a tile, and many tiles of one expert.
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,N,K,tokens", [
    ([20, 20, 20, 20, 0, 31, 9, 40], 1024, 1048, None), ([18, 22, 0, 24], 2040, 264, 60),
    ([600], 256, 4096, 99), ([500], 250, 1024, None), ([40], 2048, 1032, None),
    ([7, 0, 3], 131, 1003, 9), ([300], 61, 397, 30), ([90, 0, 33], 64, 2048, 70)])
def test_streamed_rows(dt, counts, N, K, tokens):
    check(counts, N, K, dt, tokens, ("fwd",))


@pytest.mark.parametrize("counts,N,K,tokens", [
    ([20, 20, 20, 20, 0, 31, 9, 40], 2048, 1024, None), ([24, 0, 22, 18], 4096, 2560, 50),
    ([40, 50, 0, 60, 30, 40, 50, 44], 2048, 1056, 77), ([2000], 256, 2560, 300),
    ([1500], 256, 1056, None), ([33], 2048, 2880, None)])
def test_streamed_4_bit_rows(counts, N, K, tokens):
    test_4_bit_rows(counts, N, K, tokens)
