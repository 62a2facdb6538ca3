"""4-bit microscaled floating point against a plain 64-bit implementation.

Quantisation is exact by definition: every value is compared for equality.
Products sum K exact products of dequantized values in fp32, 64 to a
tensor-core step: at most K/64 + 64 additions each lose one fp32 unit (2^-23 of
the magnitude sum), then one rounding to the output type."""
import numpy as np
import pytest
import torch

import bmm_reducescatter_alltoall_gb300 as bra

pytestmark = pytest.mark.gpu

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def quantized(x: torch.Tensor) -> np.ndarray:
    """The dequantized values (float64) by the definition."""
    v = x.double().cpu().numpy()
    K = v.shape[-1]
    v = np.concatenate([v, np.zeros(v.shape[:-1] + (-K % 32,))], -1)
    b = v.reshape(v.shape[:-1] + (-1, 32))
    a = np.abs(b).max(-1, keepdims=True)
    ok = np.isfinite(a)
    s = np.where(ok & (a > 0), np.frexp(np.where(ok, a, 1.0))[1] - 1 - 2, -127)
    unit = np.ldexp(1.0, np.maximum(s, -127))
    u = np.where(ok, np.abs(b), 0.0) / unit
    d = np.abs(u[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    # of two nearest neighbours the one with the even index; past 6: 6
    idx = np.where(near.sum(-1) == 2, np.where(near[..., ::2].any(-1),
                                               2 * near[..., ::2].argmax(-1), 0), near.argmax(-1))
    q = GRID[idx] * np.where(np.signbit(b), -1.0, 1.0) * unit
    q = np.where(ok, q, np.nan)
    return q.reshape(v.shape)[..., :K]


def check_values(x, counts=None, rows=None):
    q = bra.mxfp4_quantize(x, counts)
    got = bra.mxfp4_dequantize(q, torch.float32).double().cpu().numpy()
    want = quantized(x)
    n = want.shape[0] if rows is None else rows
    assert np.array_equal(got[:n], want[:n], equal_nan=True)
    return q


def randn(*s, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(s, generator=g, device="cuda")


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (130, 33), (5, 64), (257, 255),
                                    (40, 256), (9, 1000), (300, 1024), (2, 5000), (129, 2048)])
def test_quantized_values(rows, K, dt):
    check_values((randn(rows, K) * torch.exp2(torch.randint(-8, 9, (rows, 1), device="cuda"))).to(dt))


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_every_16_bit_value(dt):
    """Each of the 2^16 values alone in its block, then next to a large one, then to a tiny one."""
    bits = torch.arange(-(1 << 15), 1 << 15, device="cuda").to(torch.int16).view(dt)
    for other in (0.0, 6.0, 1.0, torch.finfo(dt).tiny, torch.finfo(dt).max):
        x = torch.full((1 << 16, 32), 0.0, dtype=dt, device="cuda")
        x[:, 0], x[:, 17] = bits, other
        check_values(x)


def test_ties_go_to_the_even_code():
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.75], device="cuda")
    for scale in (2.0 ** -100, 2.0 ** -7, 1.0, 2.0 ** 90):
        x = torch.zeros((9, 32), device="cuda")
        x[:, 3], x[:, 4], x[:, 30] = ties, -ties, 4.0
        check_values((x * scale).bfloat16())


def test_special_blocks():
    x = torch.zeros((6, 96), dtype=torch.bfloat16, device="cuda")
    x[0, 5], x[1, 40], x[2, 95] = float("nan"), float("inf"), float("-inf")
    x[3] = -0.0
    x[4] = torch.finfo(torch.bfloat16).smallest_normal / 64          # subnormals
    x[5] = torch.finfo(torch.bfloat16).max
    x[:3, 10] = 1.0
    check_values(x)


@pytest.mark.parametrize("K,pad", [(64, 8), (100, 3), (32, 1)])
def test_pitched_and_unaligned_rows(K, pad):
    buf = torch.full((50, K + pad), float("nan"), dtype=torch.float16, device="cuda")
    buf[:, 1:K + 1] = randn(50, K).half()
    q = bra.mxfp4_quantize(buf[:, 1:K + 1])
    z = bra.mxfp4_quantize(buf[:, 1:K + 1].contiguous())
    assert torch.equal(q.codes, z.codes)
    a, b = (bra.mxfp4_dequantize(t, torch.float32) for t in (q, z))
    assert torch.equal(a, b) and torch.isfinite(a).all()


@pytest.mark.parametrize("counts", [[0, 1, 0, 5, 64, 0], [127, 128, 129, 0, 257], [1] * 200], ids=str)
def test_grouped_rows_keep_their_values(counts):
    for extra in (0, 7):
        x = randn(sum(counts) + extra, 160).bfloat16()
        check_values(x, torch.tensor(counts, device="cuda"), rows=sum(counts))


def test_weights_and_dequantized_types():
    w = randn(3, 130, 96).half()
    q = bra.mxfp4_quantize(w)
    want = torch.from_numpy(quantized(w)).cuda()
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        assert torch.equal(bra.mxfp4_dequantize(q, dt), want.to(dt))
    with pytest.raises(TypeError):
        bra.mxfp4_dequantize(q, torch.float64)


def case(counts, K, N, seed=0, dt=torch.bfloat16, extra=0):
    R, E = sum(counts) + extra, len(counts)
    x = (randn(R, K, seed=seed) * torch.exp2(torch.randint(-3, 4, (R, 1), device="cuda"))).to(dt)
    w = (randn(E, N, K, seed=seed + 1) * K ** -0.5).to(dt)
    b = randn(E, N, seed=seed + 2).to(torch.float16 if dt == torch.float16 else torch.float32)
    return x, w, b, torch.tensor(counts, dtype=torch.int64, device="cuda")


def reference(x, w, b, counts):
    xd, wd = (torch.from_numpy(quantized(t)).cuda() for t in (x, w))
    y = torch.zeros((sum(counts), w.shape[1]), dtype=torch.float64, device="cuda")
    mag, a = torch.zeros_like(y), 0
    for e, n in enumerate(counts):
        y[a:a + n] = xd[a:a + n] @ wd[e].t()
        mag[a:a + n] = xd[a:a + n].abs() @ wd[e].abs().t()
        if b is not None:
            y[a:a + n] += b[e].double()
            mag[a:a + n] += b[e].double().abs()
        a += n
    return y, mag


def assert_close(got, ref, mag, K):
    tol = HALF[got.dtype] * ref.abs() + (K / 64 + 64) * 2.0 ** -23 * mag + 2.0 ** -24
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][:4].tolist(),
                           ref[bad][:4].tolist())


RAGGED = [[0, 1, 0, 5, 64, 0], [1], [127, 128, 129, 0, 257], [700, 3, 0, 300], [2] * 70]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts", RAGGED, ids=str)
@pytest.mark.parametrize("K,N", [(64, 128), (32, 8), (256, 256), (300, 200), (77, 131),
                                 (2048, 392)])
def test_products_over_group_sizes(counts, K, N, dt):
    x, w, b, c = case(counts, K, N, dt=dt)
    y = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w), c, bias=b,
                                 dtype=dt)
    assert_close(y, *reference(x, w, b, counts), K)


def test_products_of_exact_values_are_exact():
    """Whole numbers that 4 bits hold, with sums that fp16 holds: bit for bit, over both scales'
    positions in every 256 elements."""
    for counts in ([130, 7, 200], [6, 0, 3]):
        g = torch.Generator(device="cuda").manual_seed(1)
        K, N = 544, 264
        pick = lambda *s: torch.tensor([0., 1, -1, 2, -3, 0.5, 0, 0], device="cuda")[      # noqa: E731
            torch.randint(0, 8, s, generator=g, device="cuda")]
        x, w = pick(sum(counts), K), pick(len(counts), N, K)
        # a power of two for each block of 32 that cancels in the product
        p = torch.exp2(torch.randint(-20, 21, (K // 32,), generator=g, device="cuda").float())
        p = p.repeat_interleave(32)
        c = torch.tensor(counts, device="cuda")
        y = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize((x * p).bfloat16(), c),
                                     bra.mxfp4_quantize((w / p).bfloat16()), c,
                                     dtype=torch.float16)
        a, want = 0, torch.zeros_like(y)
        for e, n in enumerate(counts):
            want[a:a + n] = (x[a:a + n].double() @ w[e].t().double()).half()
            a += n
        assert torch.equal(y, want)


def test_a_row_without_a_value_stays_alone():
    counts = [5, 3, 150, 400]
    x, w, b, c = case(counts, 320, 264)
    x[5, 100] = float("nan")
    x[200, 0] = float("inf")
    y = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w), c, bias=b)
    nan = torch.isnan(y)
    assert nan[5].all() and nan[200].all() and int(nan.sum()) == 2 * 264


def test_rows_past_the_groups_and_row_pitch():
    counts, N = [3, 0, 61], 72
    x, w, b, c = case(counts, 128, N, extra=9)
    x[64:] = float("nan")
    buf = torch.full((73, N + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w), c, bias=b,
                             out=buf[:, :N])
    assert_close(buf[:64, :N], *reference(x[:64], w, b, counts), 128)
    assert (buf[64:] == 7.0).all() and (buf[:, N:] == 7.0).all()


def test_one_expert_without_counts_and_no_rows():
    x, w, b, c = case([140], 96, 40)
    a = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x), bra.mxfp4_quantize(w), c, bias=b)
    z = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w), c, bias=b)
    assert torch.equal(a, z)
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    q = bra.mxfp4_quantize(x[:0], none)
    assert bra.mxfp4_grouped_matmul(q, bra.mxfp4_quantize(w), none).shape == (0, 40)
    assert bra.mxfp4_dequantize(bra.mxfp4_quantize(x[:0]), torch.float32).shape == (0, 96)


@pytest.mark.parametrize("K,N", [(4096, 64), (64, 4104)])
def test_matrices_that_pass_32_bit_offsets(K, N):
    """Rows (of x, or of y) whose element offsets pass 2^32, in the last two groups."""
    R = (1 << 32) // max(K, N) + 300
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    x[-200:] = randn(200, K)
    w = (randn(2, N, K, seed=1) * K ** -0.5).bfloat16()
    c = torch.tensor([R - 150, 150], device="cuda")
    q = bra.mxfp4_quantize(x, c)
    y = bra.mxfp4_grouped_matmul(q, bra.mxfp4_quantize(w), c)
    last = bra.mxfp4_dequantize(q, torch.bfloat16)[-201:]
    assert not last[0].any() and np.array_equal(last[1:].double().cpu().numpy(), quantized(x[-200:]))
    assert not y[0].any() and not y[-300:-200].any()
    for e, a, z in ((0, R - 200, R - 150), (1, R - 150, R)):
        assert_close(y[a:z], *reference(x[a:z], w[e:e + 1], None, [z - a]), K)


def test_refused_counts_write_nothing():
    x, w, b, _ = case([20, 0, 0], 64, 72)
    wq = bra.mxfp4_quantize(w)
    for counts in ([4, -1, 3], [10, 10, 10], [1 << 62, 1 << 62, 0]):
        c = torch.tensor(counts, device="cuda")
        st = torch.zeros(3, dtype=torch.int32, device="cuda")
        codes = torch.full((20, 32), 7, dtype=torch.uint8, device="cuda")
        scales = torch.full((20 * 1024,), 7, dtype=torch.uint8, device="cuda")
        q = bra.MxTensor(codes, scales, (20, 64), c)
        bra.mxfp4_quantize(x, c, out=q, status=st[0:1])
        v = torch.full((20, 64), 7.0, device="cuda")
        bra.mxfp4_dequantize(q, torch.float32, out=v, status=st[1:2])
        y = torch.full((20, 72), 7.0, dtype=torch.bfloat16, device="cuda")
        bra.mxfp4_grouped_matmul(q, wq, c, out=y, status=st[2:3])
        assert st.tolist() == [bra.ERR_INVALID] * 3
        assert (codes == 7).all() and (scales == 7).all() and (v == 7).all() and (y == 7).all()


def test_counts_change_between_runs_of_a_graph():
    x, w, b, c = case([10, 20, 30], 128, 136)
    wq = bra.mxfp4_quantize(w)
    q = bra.mxfp4_quantize_plan(x, c)
    m = bra.mxfp4_grouped_matmul_plan(q.result, wq, c, bias=b)
    q.run(), m.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.run(), m.run()
    for counts in ([60, 0, 0], [0, 1, 59], [20, 20, 20]):
        c.copy_(torch.tensor(counts))
        graph.replay()
        assert_close(m.result, *reference(x, w, b, counts), 128)
    assert bra.fault_status() == 0


def test_refused_arguments():
    x, w, b, c = case([20, 4], 64, 72)
    q, wq = bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w)
    with pytest.raises(TypeError):
        bra.mxfp4_quantize(x.float())
    with pytest.raises(ValueError):
        bra.mxfp4_quantize(x.cpu())
    with pytest.raises(ValueError):
        bra.mxfp4_quantize(x.t())
    with pytest.raises(ValueError):
        bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x), wq, c)          # scales not grouped
    with pytest.raises(ValueError):
        bra.mxfp4_grouped_matmul(q, wq, c.clone())                      # by other counts
    with pytest.raises(TypeError):
        bra.mxfp4_grouped_matmul(x, wq, c)
    with pytest.raises(TypeError):
        bra.mxfp4_grouped_matmul(q, wq, c, dtype=torch.float32)
    with pytest.raises(TypeError):
        bra.mxfp4_grouped_matmul(q, wq, c, bias=b.half())
    with pytest.raises(ValueError):
        bra.mxfp4_grouped_matmul(q, bra.mxfp4_quantize(w[:, :, :32].contiguous()), c)


@pytest.mark.parametrize("R,N", [(384, 13312), (1152, 8192), (16512, 4096)])
def test_one_expert_without_counts_in_256_row_tiles(R, N):
    """An odd number of 128-row blocks in tiles of 256 rows: the second half of the last tile has
    no rows, and no scales in the buffer either."""
    x, w, b, c = case([R], 288, N)
    assert bra.mxfp4_quantize(x).scales.numel() == bra.mxfp4_quantize(x, c).scales.numel()
    a = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x), bra.mxfp4_quantize(w), c, bias=b)
    z = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w), c, bias=b)
    assert torch.equal(a, z)
    for at in (slice(0, 40), slice(R - 40, R)):
        assert_close(a[at], *reference(x[at], w, b, [40]), 288)
    assert bra.fault_status() == 0


def test_buffers_and_counts_that_do_not_fit_are_refused():
    """The kernels read what an MxTensor says it holds: its buffers have to hold it, and rows have to
    be grouped by all of the product's counts, not by the first of them."""
    x, w, b, c = case([20, 4, 30, 2], 320, 264)
    q, wq = bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w)

    def with_(t, codes=None, scales=None, shape=None, counts=None):
        return bra.MxTensor(t.codes if codes is None else codes, t.scales if scales is None else scales,
                            t.shape if shape is None else shape, t.counts if counts is None else counts)
    part = bra.mxfp4_quantize(x, c[:2])
    assert part.counts.data_ptr() == c.data_ptr()
    with pytest.raises(ValueError):
        bra.mxfp4_grouped_matmul(part, wq, c)
    short = [with_(q, codes=q.codes[:-1]), with_(q, scales=q.scales[:-1]),
             with_(q, shape=(57, 320)), with_(q, shape=(56, 353))]
    wrong = [with_(q, codes=q.codes.float()), with_(q, scales=q.scales.int()),
             with_(q, codes=None, scales=[1])]
    other = [with_(q, codes=q.codes.cpu()), with_(q, codes=q.codes[:, ::2]),
             with_(q, scales=q.scales[::2])]
    for bad, error in [(t, ValueError) for t in short + other] + [(t, TypeError) for t in wrong]:
        with pytest.raises(error):
            bra.mxfp4_dequantize(bad, torch.float32)
        with pytest.raises(error):
            bra.mxfp4_quantize(torch.zeros(bad.shape, dtype=x.dtype, device="cuda"), c, out=bad)
        if bad.shape[1] == 320:
            with pytest.raises(error):
                bra.mxfp4_grouped_matmul(bad, wq, c)
    for bad in (with_(wq, codes=wq.codes[:3]), with_(wq, scales=wq.scales[:-1]),
                with_(wq, shape=(4, 385, 320))):
        with pytest.raises(ValueError):
            bra.mxfp4_grouped_matmul(q, bad, c)
    # larger buffers serve, as they did
    big = bra.MxTensor(torch.empty(70 * 160, dtype=torch.uint8, device="cuda"),
                       torch.empty(8 * 2048, dtype=torch.uint8, device="cuda"), (56, 320), c)
    bra.mxfp4_quantize(x, c, out=big)
    assert torch.equal(bra.mxfp4_grouped_matmul(big, wq, c), bra.mxfp4_grouped_matmul(q, wq, c))
