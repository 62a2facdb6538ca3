"""8-bit block-scaled floating point against a plain 64-bit implementation.

Quantisation is exact by definition: values are compared for equality.

Products: a block's 128 code products are exact and added in fp32, each
addition losing at most one unit (2^-23) of the block's sum of magnitudes; the
two scales' product is rounded once, and each block's addition to the running
sum once, together at most K/128 + 2 units of the magnitudes; the bias's
addition is one more.  Then one rounding to the output type, half a step."""
import threading

import pytest
import torch

import bmm_reducescatter_alltoall_gb300 as bra

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -23
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
MOST = {E4: 448.0, E5: 57344.0}


def randn(*s, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(s, generator=g, device="cuda")


def spread(s, M, K, rows):
    """A value to each element from one to each block of `rows` x 128."""
    return s.repeat_interleave(rows, -2).repeat_interleave(128, -1)[..., :M, :K]


def quantized(x, fmt, rows):
    """Values (float64) and scales by the definition: of the format's own 2^7 magnitudes the
    nearest, a tie to the even code."""
    M, K = x.shape[-2:]
    v = torch.nn.functional.pad(x.double(), (0, -K % 128, 0, -M % rows))
    b = v.unflatten(-1, (-1, 128)).unflatten(-3, (-1, rows)).abs()
    a = b.amax((-3, -1))
    ok = torch.isfinite(a)
    s = torch.full_like(a, 2.0 ** -126)
    for e in range(-125, 121):
        s = torch.where(a > s * MOST[fmt], torch.full_like(s, 2.0 ** e), s)
    grid = torch.arange(128, dtype=torch.uint8).view(fmt).double().cuda()
    grid = grid[torch.isfinite(grid)]                        # rising with the code
    se = spread(s, M, K, rows)
    u = torch.where(torch.isfinite(x.double()), x.double().abs(), 0.0) / se
    hi = torch.searchsorted(grid, u.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    down, up = u - grid[lo], grid[hi] - u
    code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    q = grid[code] * torch.where(torch.signbit(x.double()), -1.0, 1.0) * se
    okay = spread(ok.double(), M, K, rows) > 0
    return torch.where(okay, q, float("nan")), torch.where(ok, s, float("nan"))


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=1e300), torch.nan_to_num(b, nan=1e300))


def check_values(x, fmt=E4, counts=None, rows=None):
    q = bra.fp8_quantize(x, counts, fmt)
    want, scales = quantized(x, fmt, 1 if x.dim() == 2 else 128)
    n = x.shape[0] if rows is None else rows
    got = bra.fp8_dequantize(q, torch.float32, counts).double()
    # an fp32 holds each value but those that round up to 256 * 2^120 = 2^128: infinity there
    assert same(got[:n], want[:n].float().double())
    assert same(q.scales[:n, ..., :scales.shape[-1]].double(), scales[:n])
    return q


ALL = [torch.float16, torch.bfloat16, torch.float32]
SIZES = [(1, 1), (1, 128), (3, 127), (130, 129), (5, 16), (33, 255), (40, 256), (9, 1000), (3, 2048),
         (2, 5003), (129, 2064)]


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("rows,K", SIZES)
def test_quantized_rows(rows, K, dt, fmt):
    check_values((randn(rows, K) * torch.exp2(torch.randint(-8, 9, (rows, 1), device="cuda"))).to(dt),
                 fmt)


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (3, 130, 96), (2, 128, 128), (1, 257, 300), (5, 40, 1000)])
def test_quantized_weights(E, N, K, dt, fmt):
    x = randn(E, N, K) * torch.exp2(torch.randint(-8, 9, (E, N, 1), device="cuda"))
    check_values(x.to(dt), fmt)


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_every_16_bit_value(dt, fmt):
    """Each of the 2^16 values alone in its block, then next to a large one, then to a tiny one."""
    bits = torch.arange(-(1 << 15), 1 << 15, device="cuda").to(torch.int16).view(dt)
    for other in (0.0, 448.0, 1.0, 1.76, torch.finfo(dt).tiny, torch.finfo(dt).max):
        x = torch.zeros((1 << 16, 20), dtype=dt, device="cuda")
        x[:, 0], x[:, 17] = bits, other
        check_values(x, fmt)


@pytest.mark.parametrize("fmt", [E4, E5])
def test_ties_and_borders_of_fp32(fmt):
    """Halfway values and their neighbours at several scales; the largest values a scale takes."""
    grid = torch.arange(128, dtype=torch.uint8).view(fmt).double()
    grid = grid[torch.isfinite(grid)]
    ties = ((grid[1:] + grid[:-1]) / 2).float()
    around = torch.cat([ties, torch.nextafter(ties, ties * 2), torch.nextafter(ties, ties * 0)])
    most = torch.tensor(MOST[fmt], dtype=torch.float32)
    for e in (-110, -7, 0, 90):
        x = torch.zeros((around.numel(), 128), device="cuda")
        x[:, 3], x[:, 77], x[:, 127] = around.cuda(), -around.cuda(), most
        check_values(x * 2.0 ** e, fmt)
        edge = torch.stack([most, torch.nextafter(most, most * 2), torch.nextafter(most, most * 0)])
        check_values((edge * 2.0 ** e).cuda()[:, None], fmt)


def test_special_blocks():
    for dt in ALL:
        x = torch.zeros((7, 300), dtype=dt, device="cuda")
        x[0, 5], x[1, 140], x[2, 299] = float("nan"), float("inf"), float("-inf")
        x[3] = -0.0
        x[4] = torch.finfo(dt).smallest_normal / 64                      # subnormals
        x[5] = torch.finfo(dt).max
        x[6, ::2] = torch.finfo(dt).min
        x[:3, 10] = 1.0
        for fmt in (E4, E5):
            check_values(x, fmt)
            check_values(x[None].contiguous(), fmt)


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("K,pad", [(64, 8), (100, 3), (128, 1), (2051, 5)])
def test_pitched_and_unaligned_rows(K, pad, dt):
    buf = torch.full((50, K + pad), float("nan"), dtype=dt, device="cuda")
    buf[:, 1:K + 1] = randn(50, K).to(dt)
    q, z = bra.fp8_quantize(buf[:, 1:K + 1]), bra.fp8_quantize(buf[:, 1:K + 1].contiguous())
    assert torch.equal(q.codes.view(torch.uint8), z.codes.view(torch.uint8))
    assert torch.equal(q.scales, z.scales) and torch.isfinite(q.scales).all()
    assert not q.codes.view(torch.uint8)[:, K:].any() and not q.scales[:, -(-K // 128):].any()


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("K", [1, 7, 15, 17, 127, 129, 1021, 2046, 2047, 2049, 2055, 4099])
def test_any_offset(K, dt):
    """Rows and weights that begin at any element of memory that holds NaN before and after them,
    and back to memory of which nothing else is written."""
    R = 5
    data = randn(R, K).to(dt)
    want = bra.fp8_quantize(torch.nn.functional.pad(data, (0, -K % 8))[:, :K].contiguous(), format=E5)
    for off in range(0, 9):
        room = torch.full((off + R * K + 17,), float("nan"), dtype=dt, device="cuda")
        x = room[off:off + R * K].view(R, K)
        x.copy_(data)
        q = bra.fp8_quantize(x, format=E5)
        assert same(bra.fp8_dequantize(q, torch.float32).double(), quantized(data, E5, 1)[0])
        w = bra.fp8_quantize(x.view(1, R, K))
        assert same(bra.fp8_dequantize(w, torch.float32)[0].double(), quantized(data, E4, 128)[0])
        assert torch.equal(q.codes.view(torch.uint8), want.codes.view(torch.uint8))
        for t, values in ((q, quantized(data, E5, 1)[0]), (w, quantized(data, E4, 128)[0])):
            room = torch.full((off + R * K + 17,), 7.0, dtype=dt, device="cuda")
            y = room[off:off + R * K].view(t.shape)
            bra.fp8_dequantize(t, dt, out=y)
            assert torch.equal(y.view(R, K), values.to(dt))
            assert (room[:off] == 7.0).all() and (room[off + R * K:] == 7.0).all()


def test_rows_past_the_counts_are_left_alone():
    x = randn(70, 160).bfloat16()
    for counts in ([0, 1, 0, 5, 57, 0], [63], [1] * 63, [0, 0]):
        c, n = torch.tensor(counts, device="cuda"), sum(counts)
        out = bra.fp8_quantize(randn(70, 160, seed=1).bfloat16())
        old = bra.fp8_dequantize(out, torch.float32)
        bra.fp8_quantize(x, c, out=out)
        y = torch.full((70, 160), 7.0, device="cuda")
        bra.fp8_dequantize(out, torch.float32, c, out=y)
        assert (y[n:] == 7.0).all()
        got = bra.fp8_dequantize(out, torch.float32)
        assert torch.equal(got[n:], old[n:]) and torch.equal(got[:n], y[:n])
        assert same(got[:n].double(), quantized(x[:n], E4, 1)[0] if n else got[:0].double())


def test_dequantized_types():
    """Powers of two as scales: one rounding.  Any other scale: the product in fp32 first."""
    w = randn(3, 130, 97).half()
    q = bra.fp8_quantize(w)
    want = quantized(w, E4, 128)[0]
    for dt in ALL:
        assert torch.equal(bra.fp8_dequantize(q, dt), want.to(dt))
    s = torch.rand(q.scales.shape, device="cuda")
    z = bra.Fp8Tensor(q.codes, s, q.shape)
    codes = q.codes[:, :, :97].float()
    for dt in ALL:
        assert torch.equal(bra.fp8_dequantize(z, dt), (codes * spread(s, 130, 97, 128)).to(dt))
    assert bra.fp8_dequantize(bra.fp8_quantize(w[0][:0]), torch.float32).shape == (0, 97)


# ------------------------------------------------------------------------------------------------
# products
# ------------------------------------------------------------------------------------------------

def case(counts, K, N, seed=0, dt=torch.bfloat16, extra=0):
    R, E = sum(counts) + extra, len(counts)
    x = (randn(R, K, seed=seed) * torch.exp2(torch.randint(-3, 4, (R, 1), device="cuda"))).to(dt)
    x[:, ::37] *= 16
    w = (randn(E, N, K, seed=seed + 1) * K ** -0.5).to(dt)
    b = randn(E, N, seed=seed + 2).to(torch.float16 if dt == torch.float16 else torch.float32)
    return x, w, b, torch.tensor(counts, dtype=torch.int64, device="cuda")


def values(q):
    """The exact values of an Fp8Tensor in 64 bits."""
    M, K = q.shape[-2:]
    return q.codes[..., :K].float().double() * spread(q.scales.double(), M, K,
                                                      1 if len(q.shape) == 2 else 128)


def reference(xq, wq, b, counts, grad=False):
    xd, wd = values(xq), values(wq)
    if not grad:
        wd = wd.transpose(1, 2)
    y = torch.zeros((sum(counts), wd.shape[2]), dtype=torch.float64, device="cuda")
    mag, a = torch.zeros_like(y), 0
    for e, n in enumerate(counts):
        y[a:a + n] = xd[a:a + n] @ wd[e]
        mag[a:a + n] = xd[a:a + n].abs() @ wd[e].abs()
        if b is not None:
            y[a:a + n] += b[e].double()
            mag[a:a + n] += b[e].double().abs()
        a += n
    return y, mag


def assert_close(got, ref, mag, K):
    tol = HALF[got.dtype] * ref.abs() + (K / 128 + 132) * UNIT * mag + TINY[got.dtype]
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][:4].tolist(),
                           ref[bad][:4].tolist())


RAGGED = [[0, 1, 0, 5, 64, 0], [1], [127, 128, 129, 0, 257], [700, 3, 0, 300], [2] * 70]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts", RAGGED, ids=str)
@pytest.mark.parametrize("K,N", [(64, 128), (32, 8), (256, 256), (300, 200), (77, 131), (1, 1),
                                 (2048, 392), (4500, 130)])
def test_products_over_group_sizes(counts, K, N, dt):
    x, w, b, c = case(counts, K, N, dt=dt)
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    assert_close(bra.fp8_grouped_matmul(xq, wq, c, bias=b, dtype=dt), *reference(xq, wq, b, counts),
                 K)
    dq = bra.fp8_quantize(randn(x.shape[0], N, seed=5).to(dt), c, E5)
    assert_close(bra.fp8_grouped_matmul_grad(dq, wq, c, dtype=dt),
                 *reference(dq, wq, None, counts, True), N)
    assert bra.fault_status() == 0


@pytest.mark.parametrize("counts,K,N,tiles", [
    ([3, 0, 5], 8200, 300, "32x128 tiles, sums over 8 CTAs"),
    ([3, 0, 5], 1024, 2056, "32x128 tiles, sums over 2 CTAs"),
    ([3, 0, 5], 640, 300, "32x128 tiles"), ([1] * 40, 2048, 1030, "32x128 tiles"),
    ([200, 1, 90], 4224, 300, "128x128 tiles, sums over 8 CTAs"),
    ([200, 1, 90], 2050, 520, "128x128 tiles, sums over 4 CTAs"),
    ([700, 0, 513], 300, 300, "128x128 tiles"),
    ([700, 0, 513, 1027], 640, 8200, "256x256 tiles by CTA pairs"),
    ([4100, 3000], 130, 3333, "128x128 tiles"),
    ([4100, 3000], 1000, 1333, "256x256 tiles by CTA pairs")], ids=str)
def test_tiles(counts, K, N, tiles, monkeypatch, capfd):
    """Which kernel takes a call, by its log; the results of each."""
    monkeypatch.setenv("BRA_LOG", "1")
    x, w, b, c = case(counts, K, N)
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    capfd.readouterr()
    y = bra.fp8_grouped_matmul(xq, wq, c, bias=b)
    assert capfd.readouterr().err.strip().endswith(f"-> {tiles}")
    assert_close(y, *reference(xq, wq, b, counts), K)
    del x, w
    w2 = bra.fp8_quantize((randn(len(counts), K, N, seed=9) * K ** -0.5).bfloat16())
    dq = bra.fp8_quantize(randn(sum(counts), K, seed=7).bfloat16(), c, E5)
    capfd.readouterr()
    dx = bra.fp8_grouped_matmul_grad(dq, w2, c)
    assert capfd.readouterr().err.strip().endswith(f"-> {tiles}")
    assert_close(dx, *reference(dq, w2, None, counts, True), K)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts", [[3, 0, 5], [1], [32], [40], [0, 129, 0, 33], [100, 1, 300], [0, 0]],
                         ids=str)
@pytest.mark.parametrize("long,short", [(1025, 72), (2047, 129), (3333, 8), (4224, 300), (8200, 41)])
def test_few_tiles_and_a_long_contraction(counts, long, short, dt):
    """Tiles whose contraction several CTAs share; rows past the counts stay as they are."""
    x, w, b, c = case(counts, long, short, dt=dt, extra=3)
    n = sum(counts)
    xq, wq = bra.fp8_quantize(x), bra.fp8_quantize(w)
    for off in (0, 1):
        room = torch.full((off + (n + 3) * short,), 7.0, dtype=dt, device="cuda")
        y = room[off:].view(n + 3, short)
        bra.fp8_grouped_matmul(xq, wq, c, bias=b, out=y)
        part = bra.Fp8Tensor(xq.codes[:n], xq.scales[:n], (n, long))
        assert_close(y[:n], *reference(part, wq, b, counts), long)
        assert (y[n:] == 7.0).all() and (room[:off] == 7.0).all()
        first = y.clone()
        bra.fp8_grouped_matmul(xq, wq, c, bias=b, out=y)
        assert torch.equal(first, y)
    w2 = bra.fp8_quantize(randn(len(counts), long, short, seed=4).to(dt))
    dq = bra.fp8_quantize(x, format=E5)
    dx = torch.full((n + 3, short), 7.0, dtype=dt, device="cuda")
    bra.fp8_grouped_matmul_grad(dq, w2, c, out=dx)
    part = bra.Fp8Tensor(dq.codes[:n], dq.scales[:n], (n, long))
    assert_close(dx[:n], *reference(part, w2, None, counts, True), long)
    assert (dx[n:] == 7.0).all()
    assert bra.fault_status() == 0


@pytest.mark.parametrize("xf", [E4, E5])
@pytest.mark.parametrize("wf", [E4, E5])
@pytest.mark.parametrize("counts", [[6, 0, 3], [300, 41, 500, 0]], ids=str)
def test_formats(counts, xf, wf):
    x, w, b, c = case(counts, 320, 264)
    xq, wq = bra.fp8_quantize(x, c, xf), bra.fp8_quantize(w, format=wf)
    assert_close(bra.fp8_grouped_matmul(xq, wq, c, bias=b), *reference(xq, wq, b, counts), 320)
    dq = bra.fp8_quantize(randn(x.shape[0], 264).bfloat16(), c, xf)
    assert_close(bra.fp8_grouped_matmul_grad(dq, wq, c), *reference(dq, wq, None, counts, True), 264)


# rows that take a pair's tiles of 256 x 256 (see the tile rule), ragged ends and odd widths
LARGE = [([700, 0, 513, 1027], 640, 8200), ([300] * 10 + [1, 0, 777], 1100, 2056),
         ([4100], 260, 3333), ([256] * 8, 128, 2560)]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,K,N", LARGE, ids=str)
def test_large_tiles(counts, K, N, dt):
    x, w, b, c = case(counts, K, N, dt=dt)
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    assert_close(bra.fp8_grouped_matmul(xq, wq, c, bias=b, dtype=dt), *reference(xq, wq, b, counts),
                 K)
    del x, w
    w2 = (randn(len(counts), K, N, seed=9) * N ** -0.5).to(dt)           # dx has the N columns here
    w2q, dq = bra.fp8_quantize(w2), bra.fp8_quantize(randn(sum(counts), K, seed=7).to(dt), c, E5)
    assert_close(bra.fp8_grouped_matmul_grad(dq, w2q, c, dtype=dt),
                 *reference(dq, w2q, None, counts, True), K)
    assert bra.fault_status() == 0


def test_products_of_exact_values_are_exact():
    """Whole numbers, block scales that cancel: bit for bit, over every block of the contraction."""
    for counts in ([130, 7, 200], [6, 0, 3], [2000, 100, 2000]):
        g = torch.Generator(device="cuda").manual_seed(1)
        K, N, E = 1056, 2056, len(counts)
        pick = lambda *s: torch.tensor([0., 1, -1, 2, -3, 8, 0, 0], device="cuda")[        # noqa: E731
            torch.randint(0, 8, s, generator=g, device="cuda")]
        x, w = pick(sum(counts), K), pick(E, N, K)
        x[:, ::128], w[:, :, ::128] = 8, 8                    # every block's largest is 8
        p = torch.exp2(torch.randint(-20, 21, (-(-K // 128),), generator=g, device="cuda").float())
        p = p.repeat_interleave(128)[:K]
        c = torch.tensor(counts, device="cuda")
        y = bra.fp8_grouped_matmul(bra.fp8_quantize(x * p, c), bra.fp8_quantize(w / p), c,
                                   dtype=torch.float16)
        a, want = 0, torch.zeros_like(y)
        for e, n in enumerate(counts):
            want[a:a + n] = (x[a:a + n].double() @ w[e].t().double()).half()
            a += n
        assert torch.equal(y, want)


@pytest.mark.parametrize("counts", [[6, 0, 3], [900, 1000, 500]], ids=str)
def test_checkpoint_scales(counts):
    """Scales that are no powers of two, on both sides, and some of zero."""
    x, w, b, c = case(counts, 700, 2200)
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    xq = bra.Fp8Tensor(xq.codes, xq.scales * (0.5 + torch.rand_like(xq.scales)), xq.shape)
    s = wq.scales * (0.5 + torch.rand_like(wq.scales))
    s[0, 0, 2] = 0.0
    wq = bra.Fp8Tensor(wq.codes, s, wq.shape)
    assert_close(bra.fp8_grouped_matmul(xq, wq, c, bias=b), *reference(xq, wq, b, counts), 700)
    dq = bra.fp8_quantize(randn(x.shape[0], 2200).bfloat16(), c)
    assert_close(bra.fp8_grouped_matmul_grad(dq, wq, c), *reference(dq, wq, None, counts, True), 2200)


@pytest.mark.parametrize("counts", [[5, 3, 150, 400], [500, 600, 700, 800]], ids=str)
def test_a_row_without_a_value_stays_alone(counts):
    x, w, b, c = case(counts, 320, 2056)
    x[5, 100] = float("nan")
    x[200, 0] = float("inf")
    y = bra.fp8_grouped_matmul(bra.fp8_quantize(x, c), bra.fp8_quantize(w), c, bias=b)
    nan = torch.isnan(y)
    assert nan[5].all() and nan[200].all() and int(nan.sum()) == 2 * 2056
    w[1, 130, 300] = float("nan")                       # its block: columns 128 .. 255 of expert 1
    y = bra.fp8_grouped_matmul(bra.fp8_quantize(x, c), bra.fp8_quantize(w), c, bias=b)
    a = counts[0]
    nan = torch.isnan(y)
    assert nan[a:a + counts[1], 128:256].all()
    nan[a:a + counts[1], 128:256] = False
    nan[5] = nan[200] = False
    assert not nan.any()


def test_scales_whose_product_passes_the_largest_float():
    x = torch.zeros((4, 128), device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 1e38, 1.0, 1e-30
    w = torch.zeros((1, 16, 128), device="cuda")
    w[0, 0, 0], w[0, 1, 1] = 1e38, 1e38
    c = torch.tensor([4], device="cuda")
    y = bra.fp8_grouped_matmul(bra.fp8_quantize(x, c), bra.fp8_quantize(w), c)
    assert torch.isinf(y[0, 0]) and not torch.isnan(y).any()
    assert (y[:, 1:] == 0).all() and (y[3] == 0).all()
    assert torch.isfinite(y[1, 0]) and abs(float(y[1, 0]) / 1e38 - 1) < 0.1


@pytest.mark.parametrize("rows", [4, 60, 400])
def test_negative_scales_whose_product_passes_the_largest_float(rows):
    """A checkpoint's scales have any sign: blocks whose sum is zero stay zero."""
    c = torch.tensor([rows], device="cuda")
    x = bra.fp8_quantize(torch.ones((rows, 256), device="cuda"), c)
    w = torch.ones((1, 300, 256), device="cuda")
    w[:, :, :128:2] = -1.0                                # the first block's sum is zero
    w = bra.fp8_quantize(w)
    x = bra.Fp8Tensor(x.codes, x.scales.clone(), x.shape)
    w = bra.Fp8Tensor(w.codes, w.scales.clone(), w.shape)
    x.scales[:, 0], w.scales[:, :, 0] = 1e30, -1e30
    y = bra.fp8_grouped_matmul(x, w, c)
    want = 128 * float(x.codes[0, 0].float() * w.codes[0, 0, 1].float() * x.scales[0, 1] *
                       w.scales[0, 0, 1])
    assert (y.float() == want).all()


@pytest.mark.parametrize("counts,N", [([3, 0, 61], 72), ([1300, 0, 1200], 2053)], ids=str)
def test_rows_past_the_groups_and_row_pitch(counts, N):
    n = sum(counts)
    x, w, b, c = case(counts, 128, N, extra=9)
    x[n:] = float("nan")
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    for shift in (0, 1, 3):
        buf = torch.full((n + 9, N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        bra.fp8_grouped_matmul(xq, wq, c, bias=b, out=buf[:, shift:N + shift])
        z = bra.Fp8Tensor(xq.codes[:n], xq.scales[:n], (n, 128))
        assert_close(buf[:n, shift:N + shift], *reference(z, wq, b, counts), 128)
        assert (buf[n:] == 7.0).all() and (buf[:, N + shift:] == 7.0).all()
        assert (buf[:, :shift] == 7.0).all()


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,gap", [(200, 8), (1288, 16), (2053, 3), (1001, 7)])
@pytest.mark.parametrize("counts", [[300, 33, 31, 500], [1300, 0, 1201, 64, 95]], ids=str)
def test_whole_boxes_between_gaps(counts, N, gap, dt):
    """Rows at a 16-byte pitch of any length, stored in boxes: whole ones, parts of groups, and
    nothing between the rows or behind them."""
    n = sum(counts)
    x, w, b, c = case(counts, 200, N, dt=dt, extra=40)
    xq, wq = bra.fp8_quantize(x), bra.fp8_quantize(w)
    z = bra.Fp8Tensor(xq.codes[:n], xq.scales[:n], (n, 200))
    buf = torch.full((n + 40, N + gap), 7.0, dtype=dt, device="cuda")
    bra.fp8_grouped_matmul(xq, wq, c, bias=b, out=buf[:, :N])
    assert_close(buf[:n, :N], *reference(z, wq, b, counts), 200)
    assert (buf[n:] == 7.0).all() and (buf[:, N:] == 7.0).all()
    w2 = bra.fp8_quantize(randn(len(counts), 200, N, seed=3).to(dt))
    dx = torch.full((n + 40, N + gap), 7.0, dtype=dt, device="cuda")
    bra.fp8_grouped_matmul_grad(xq, w2, c, out=dx[:, :N])
    assert_close(dx[:n, :N], *reference(z, w2, None, counts, True), 200)
    assert (dx[n:] == 7.0).all() and (dx[:, N:] == 7.0).all()


@pytest.mark.parametrize("K,N", [(4096, 64), (64, 4104)])
def test_matrices_that_pass_32_bit_offsets(K, N):
    """Rows (of x, or of y) whose byte offsets pass 2^32, in the last two groups."""
    R = (1 << 32) // max(K, N) + 300
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    x[-200:] = randn(200, K)
    w = (randn(2, N, K, seed=1) * K ** -0.5).bfloat16()
    c = torch.tensor([R - 150, 150], device="cuda")
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    y = bra.fp8_grouped_matmul(xq, wq, c)
    assert not y[0].any() and not y[-300:-200].any()
    for e, a, z in ((0, R - 200, R - 150), (1, R - 150, R)):
        part = bra.Fp8Tensor(xq.codes[a:z], xq.scales[a:z], (z - a, K))
        we = bra.Fp8Tensor(wq.codes[e:e + 1], wq.scales[e:e + 1], (1, N, K))
        assert same(values(part), quantized(x[a:z], E4, 1)[0])
        assert_close(y[a:z], *reference(part, we, None, [z - a]), K)


def test_weights_that_pass_32_bit_offsets():
    E, N, K = 5, 1040, 1 << 20
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[-1, -3:] = randn(3, K)
    wq = bra.fp8_quantize(w)
    assert same(wq.codes[-1, -3:].float().double() *
                wq.scales[-1, -1].double().repeat_interleave(128), quantized(
                    torch.nn.functional.pad(w[-1:, 1024:], (0, 0, 0, 112)), E4, 128)[0][0, 13:16])
    del w
    c = torch.tensor([1, 0, 0, 1, 2], device="cuda")
    xq = bra.fp8_quantize(randn(4, K).bfloat16(), c)
    y = bra.fp8_grouped_matmul(xq, wq, c)
    last = bra.Fp8Tensor(wq.codes[-1:, 1024:], wq.scales[-1:, -1:].contiguous(), (1, 16, K))
    part = bra.Fp8Tensor(xq.codes[2:], xq.scales[2:], (2, K))
    assert_close(y[2:, 1024:], *reference(part, last, None, [2]), K)
    assert not y[:2].any() and not y[2:, :1037].any()
    dq = bra.fp8_quantize(randn(4, N).bfloat16(), c)
    dx = bra.fp8_grouped_matmul_grad(dq, wq, c)
    tail = bra.Fp8Tensor(dq.codes[2:, 1024:], dq.scales[2:, 8:].contiguous(), (2, 16))
    assert_close(dx[2:], *reference(tail, last, None, [2], True), N)
    assert not dx[:2].any()


def test_no_rows_and_counts_of_nothing():
    x, w, b, c = case([140], 96, 40)
    wq = bra.fp8_quantize(w)
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    assert bra.fp8_grouped_matmul(bra.fp8_quantize(x[:0]), wq, none).shape == (0, 40)
    y = torch.full((140, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    bra.fp8_grouped_matmul(bra.fp8_quantize(x), wq, none, bias=b, out=y)
    assert (y == 7.0).all()


def test_refused_counts_write_nothing():
    x, w, b, _ = case([20, 0, 0], 64, 72)
    wq, whole = bra.fp8_quantize(w), bra.fp8_quantize(x)
    dq = bra.fp8_quantize(randn(20, 72).bfloat16())
    for counts in ([4, -1, 3], [10, 10, 10], [1 << 62, 1 << 62, 0]):
        c = torch.tensor(counts, device="cuda")
        st = torch.zeros(4, dtype=torch.int32, device="cuda")
        q = bra.Fp8Tensor(torch.full((20, 64), 7, dtype=torch.uint8, device="cuda").view(E4),
                          torch.full((20, 4), 7.0, device="cuda"), (20, 64))
        bra.fp8_quantize(x, c, out=q, status=st[0:1])
        v = torch.full((20, 64), 7.0, device="cuda")
        bra.fp8_dequantize(whole, torch.float32, c, out=v, status=st[1:2])
        y = torch.full((20, 72), 7.0, dtype=torch.bfloat16, device="cuda")
        bra.fp8_grouped_matmul(whole, wq, c, out=y, status=st[2:3])
        dx = torch.full((20, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        bra.fp8_grouped_matmul_grad(dq, wq, c, out=dx, status=st[3:4])
        assert st.tolist() == [bra.ERR_INVALID] * 4
        assert (q.codes.view(torch.uint8) == 7).all() and (q.scales == 7).all()
        assert (v == 7).all() and (y == 7).all() and (dx == 7).all()


def test_counts_change_between_runs_of_a_graph():
    x, w, b, c = case([10, 20, 30], 128, 136)
    wq = bra.fp8_quantize(w)
    q = bra.fp8_quantize_plan(x, c)
    m = bra.fp8_grouped_matmul_plan(q.result, wq, c, bias=b)
    dq = bra.fp8_quantize(randn(60, 136).bfloat16())
    d = bra.fp8_grouped_matmul_grad_plan(dq, wq, c)
    for p in (q, m, d):
        p.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in (q, m, d):
            p.run()
    for counts in ([60, 0, 0], [0, 1, 59], [20, 20, 20]):
        c.copy_(torch.tensor(counts))
        graph.replay()
        assert_close(m.result, *reference(q.result, wq, b, counts), 128)
        assert_close(d.result, *reference(dq, wq, None, counts, True), 136)
    assert bra.fault_status() == 0


def test_calls_on_two_streams_and_from_two_threads():
    x, w, b, c = case([300, 400, 500], 512, 1000)
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    want = bra.fp8_grouped_matmul(xq, wq, c, bias=b)
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i] = bra.fp8_grouped_matmul(bra.fp8_quantize(x, c, stream=s), wq, c, bias=b, stream=s)
        s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(g, want) for g in got)


def test_results_do_not_change_from_run_to_run():
    x, w, b, c = case([1000, 30, 2000], 600, 2100)
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    y = bra.fp8_grouped_matmul(xq, wq, c, bias=b)
    for _ in range(5):
        assert torch.equal(y, bra.fp8_grouped_matmul(xq, wq, c, bias=b))


def test_gradient_against_differences():
    """y is linear in a row's values: a difference of one code's value changes y by dx's part."""
    x, w, _, c = case([3, 2], 130, 24)
    xq, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    dy = torch.zeros((5, 24), device="cuda")
    dy[torch.arange(5), torch.arange(5) * 4] = 1.0
    dx = bra.fp8_grouped_matmul_grad(bra.fp8_quantize(dy, c), wq, c)
    y0 = reference(xq, wq, None, [3, 2])[0]
    for k in (0, 5, 129):
        step = torch.zeros((5, 130), dtype=torch.float64, device="cuda")
        step[:, k] = 1.0
        z = bra.Fp8Tensor(xq.codes, xq.scales, xq.shape)
        v = values(z) + step
        d = torch.cat([v[:3] @ values(wq)[0].t(), v[3:] @ values(wq)[1].t()]) - y0
        want = d[torch.arange(5), torch.arange(5) * 4]
        assert torch.allclose(dx[:, k].double(), want, rtol=2.0 ** -8, atol=1e-9)


def test_refused_arguments():
    x, w, b, c = case([20, 4], 64, 72)
    q, wq = bra.fp8_quantize(x, c), bra.fp8_quantize(w)
    for bad in (x.double(), x.to(torch.int32), [1]):
        with pytest.raises(TypeError):
            bra.fp8_quantize(bad)
    with pytest.raises(TypeError):
        bra.fp8_quantize(x, format=torch.uint8)
    for bad in (x.cpu(), x.t(), x[0], x[:, :0], w[:, ::2], w[:0]):
        with pytest.raises(ValueError):
            bra.fp8_quantize(bad)
    with pytest.raises(ValueError):
        bra.fp8_quantize(w, c)
    with pytest.raises(ValueError):
        bra.fp8_dequantize(wq, torch.float32, c)
    with pytest.raises(TypeError):
        bra.fp8_dequantize(q, torch.float64)
    with pytest.raises(TypeError):
        bra.fp8_grouped_matmul(x, wq, c)
    with pytest.raises(TypeError):
        bra.fp8_grouped_matmul(q, wq, c, dtype=torch.float32)
    with pytest.raises(TypeError):
        bra.fp8_grouped_matmul(q, wq, c, bias=b.half())
    with pytest.raises(ValueError):
        bra.fp8_grouped_matmul(q, wq, c[:1])
    with pytest.raises(ValueError):
        bra.fp8_grouped_matmul(q, bra.fp8_quantize(w[:, :, :32].contiguous()), c)
    with pytest.raises(ValueError):
        bra.fp8_grouped_matmul_grad(q, wq, c)
    room = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")        # y over the rows' codes
    z = bra.Fp8Tensor(room[:24 * 64].view(E4).view(24, 64), q.scales, q.shape)
    with pytest.raises(bra.BraError):
        bra.fp8_grouped_matmul(z, wq, c, out=room[1024:1024 + 24 * 144].view(torch.bfloat16).view(24, 72))
    short = [bra.Fp8Tensor(q.codes[:-1], q.scales, q.shape),
             bra.Fp8Tensor(q.codes, q.scales[:-1], q.shape),
             bra.Fp8Tensor(q.codes, q.scales, (24, 65)), bra.Fp8Tensor(q.codes, q.scales, (25, 64)),
             bra.Fp8Tensor(q.codes.view(torch.uint8).cpu().view(E4), q.scales, q.shape),
             bra.Fp8Tensor(q.codes, q.scales, (64,))]
    for bad in short:
        with pytest.raises(ValueError):
            bra.fp8_dequantize(bad, torch.float32)
    for bad in (bra.Fp8Tensor(q.codes.view(torch.uint8), q.scales, q.shape),
                bra.Fp8Tensor(q.codes, q.scales.double(), q.shape)):
        with pytest.raises(TypeError):
            bra.fp8_dequantize(bad, torch.float32)
