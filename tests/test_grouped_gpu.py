"""Products grouped by expert against a plain 64-bit implementation.

Tolerance, per element: the kernels sum K products in fp32, 16 to a tensor-core
step, so that at most K/16 + 16 additions each lose one fp32 unit (2^-23 of
the magnitude sum) before one rounding to the output type (half a unit in the
last place: 2^-11 of the value for fp16, 2^-8 for bf16, both with their
subnormal spacing).
"""
import numpy as np
import pytest
import torch

import bmm_reducescatter_alltoall_gb300 as bra

pytestmark = pytest.mark.gpu

HALF = {torch.float16: (2.0 ** -11, 2.0 ** -24), torch.bfloat16: (2.0 ** -8, 2.0 ** -133)}


def assert_close(got, ref, mag, terms, what=""):
    unit, tiny = HALF.get(got.dtype, (2.0 ** -23, 0.0))
    tol = unit * ref.abs() + (terms / 16 + 16) * 2.0 ** -23 * mag + tiny
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(),
                           got[bad][:4].tolist(), ref[bad][:4].tolist())


def groups_of(counts):
    at = np.concatenate([[0], np.cumsum(counts)])
    return [(e, int(at[e]), int(at[e + 1])) for e in range(len(counts))]


def make(counts, K, N, dt, wt=False, seed=0, extra=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")       # noqa: E731
    R, E = sum(counts) + extra, len(counts)
    x = rnd(R, K).to(dt)
    w = (rnd(E, N, K) if wt else rnd(E, K, N)).mul_(K ** -0.5).to(dt)
    b = rnd(E, N).to(torch.float16 if dt == torch.float16 else torch.float32)
    dy = rnd(R, N).to(dt)
    return x, w, b, dy, torch.tensor(counts, dtype=torch.int64, device="cuda")


def forward_ref(x, w, b, counts, wt):
    E = len(counts)
    N = w.shape[1] if wt else w.shape[2]
    y = torch.zeros((sum(counts), N), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for e, r0, r1 in groups_of(counts):
        we = (w[e].t() if wt else w[e]).double()
        y[r0:r1] = x[r0:r1].double() @ we
        mag[r0:r1] = x[r0:r1].double().abs() @ we.abs()
        if b is not None:
            y[r0:r1] += b[e].double()
            mag[r0:r1] += b[e].double().abs()
    return y, mag


def check_forward(counts, K, N, dt, wt, bias, seed=0, **kw):
    x, w, b, _, c = make(counts, K, N, dt, wt, seed)
    b = b if bias else None
    y = bra.grouped_matmul(x, w, c, bias=b, transpose_weight=wt, **kw)
    ref, mag = forward_ref(x, w, b, counts, wt)
    assert_close(y, ref, mag, K)


def check_grad(counts, K, N, dt, wt, seed=0):
    x, w, b, dy, c = make(counts, K, N, dt, wt, seed)
    got = bra.grouped_matmul_grad(dy, x, w, c, bias=b, transpose_weight=wt)
    again = bra.grouped_matmul_grad(dy, x, w, c, bias=b, transpose_weight=wt)
    for k in got:
        assert torch.equal(got[k], again[k]), k
    for e, r0, r1 in groups_of(counts):
        we = (w[e].t() if wt else w[e]).double()
        d, xe = dy[r0:r1].double(), x[r0:r1].double()
        assert_close(got["dx"][r0:r1], d @ we.t(), d.abs() @ we.abs().t(), N, ("dx", e))
        dw = got["dweight"][e].t() if wt else got["dweight"][e]
        assert_close(dw, xe.t() @ d, xe.abs().t() @ d.abs(), r1 - r0, ("dweight", e))
        # every row is one addition: up to r1 - r0 of them in a chain
        assert_close(got["dbias"][e], d.sum(0), d.abs().sum(0), 16 * (r1 - r0), ("dbias", e))


RAGGED = [
    [0, 1, 0, 5, 64, 0],                     # empty and single-row experts
    [1],
    [127, 128, 129, 0, 257],                 # around the tiles' edges
    [700, 3, 0, 300],
    [2] * 70,                                # many small experts
]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts", RAGGED, ids=str)
@pytest.mark.parametrize("K,N,wt", [(64, 64, False), (136, 200, True), (512, 776, False),
                                    (8, 8, True), (2048, 264, True)])
def test_forward_over_group_sizes(counts, K, N, wt, dt):
    check_forward(counts, K, N, dt, wt, bias=True)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("K,N", [(1, 1), (7, 3), (65, 129), (1026, 775), (250, 254)])
@pytest.mark.parametrize("wt", [False, True])
def test_forward_of_odd_sizes(K, N, wt, dt):
    check_forward([3, 0, 130, 1], K, N, dt, wt, bias=True)


@pytest.mark.parametrize("counts", [[40] * 4, [600, 520, 700], [0, 0, 3000, 1]], ids=str)
def test_forward_without_bias_on_larger_groups(counts):
    check_forward(counts, 320, 1032, torch.bfloat16, False, bias=False)
    check_forward(counts, 320, 1032, torch.float16, True, bias=False)


def test_forward_of_512_groups():
    counts = [(7 * e) % 5 for e in range(512)]
    check_forward(counts, 96, 72, torch.bfloat16, False, bias=True)
    with pytest.raises(bra.BraError) as err:
        check_forward([1] * 513, 96, 72, torch.bfloat16, False, bias=True)
    assert err.value.code == bra.ERR_INVALID


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts", RAGGED, ids=str)
@pytest.mark.parametrize("K,N,wt", [(64, 64, False), (136, 200, True), (264, 512, False),
                                    (33, 71, False), (33, 71, True), (390, 135, True)])
def test_gradients_over_group_sizes(counts, K, N, wt, dt):
    check_grad(counts, K, N, dt, wt)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,K,N,wt", [
    ([1, 0, 2], 4096, 64, False), ([1], 2048, 200, True), ([5, 90], 1032, 264, False),
    ([3], 4090, 33, True), ([300], 2000, 130, False),
], ids=str)
def test_forward_with_the_contraction_split(counts, K, N, wt, dt):
    """Few tiles, long sums: a cluster shares each tile."""
    check_forward(counts, K, N, dt, wt, bias=True)
    check_forward(counts, K, N, dt, wt, bias=False)
    check_grad(counts, K, N, dt, wt)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,K,N,wt", [
    ([3000], 64, 64, False), ([2049, 0, 1, 4000], 101, 64, True), ([700, 900], 200, 136, False),
    ([513, 511], 129, 257, True), ([0, 9000, 0], 8, 8, False), ([1024], 40, 33, False),
], ids=str)
def test_gradients_with_the_rows_split(counts, K, N, wt, dt):
    """Few tiles, many rows: a cluster shares each tile of the weight's gradient."""
    check_grad(counts, K, N, dt, wt)
    check_forward(counts, K, N, dt, wt, bias=True)


@pytest.mark.parametrize("sizes", [[1], [15], [16], [17], [63], [64], [65], [0], [128]], ids=str)
def test_weight_gradient_at_the_ends_of_a_row_block(sizes):
    for K, N in ((64, 72), (264, 264)):
        check_grad(sizes + [40], K, N, torch.float16, False)


def test_gradients_are_those_of_differences():
    """y is linear in x and in the weight: with small whole numbers every sum is exact, and the
    difference of two outputs against dy equals the gradient against the step, exactly."""
    counts, K, N = [5, 0, 70, 1, 200], 40, 56
    g = torch.Generator(device="cuda").manual_seed(3)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").half()   # noqa: E731
    x, w, dy = ints(sum(counts), K), ints(len(counts), K, N), ints(sum(counts), N)
    b = ints(len(counts), N)
    sx, sw, sb = ints(*x.shape), ints(*w.shape), ints(*b.shape)
    c = torch.tensor(counts, device="cuda")
    f = lambda x, w, b: bra.grouped_matmul(x, w, c, bias=b).double()               # noqa: E731
    grad = bra.grouped_matmul_grad(dy, x, w, c, bias=b)
    y = f(x, w, b)
    dot = lambda a, b: float((a.double() * b.double()).sum())                       # noqa: E731
    assert dot(dy, f(x + sx, w, b) - y) == dot(grad["dx"], sx)
    assert dot(dy, f(x, w + sw, b) - y) == dot(grad["dweight"], sw)
    assert dot(dy, f(x, w, b + sb) - y) == dot(grad["dbias"], sb)


@pytest.mark.parametrize("K,N", [(128, 264), (70, 33)])
def test_rows_past_the_groups_are_neither_used_nor_written(K, N):
    counts, extra = [3, 0, 61], 9
    for dt in (torch.float16, torch.bfloat16):
        x, w, b, dy, c = make(counts, K, N, dt, extra=extra)
        R0 = sum(counts)
        x[R0:], dy[R0:] = float("nan"), float("inf")
        y = torch.full((R0 + extra, N), 7.0, dtype=dt, device="cuda")
        bra.grouped_matmul(x, w, c, bias=b, out=y)
        ref, mag = forward_ref(x[:R0], w, b, counts, False)
        assert_close(y[:R0], ref, mag, K)
        assert (y[R0:] == 7.0).all()
        dx = torch.full((R0 + extra, K), 7.0, dtype=dt, device="cuda")
        got = bra.grouped_matmul_grad(dy, x, w, c, bias=b, dx=dx)
        assert (dx[R0:] == 7.0).all()
        for n in ("dweight", "dbias"):
            assert torch.isfinite(got[n]).all(), n
        assert torch.isfinite(dx[:R0]).all()


def test_infinities_stay_within_their_group():
    """A row of infinities next to another group's last rows reaches its own group alone."""
    counts, K, N = [5, 3, 70], 264, 272
    x, w, b, dy, c = make(counts, K, N, torch.bfloat16)
    x[5], dy[5] = float("inf"), float("nan")
    y = bra.grouped_matmul(x, w, c, bias=b)
    fin = torch.isfinite(y).all(1)
    assert not fin[5] and fin[:5].all() and fin[6:].all()
    got = bra.grouped_matmul_grad(dy, x, w, c, bias=b)
    for n in ("dweight", "dbias"):
        assert torch.isfinite(got[n][0]).all() and torch.isfinite(got[n][2]).all(), n
        assert not torch.isfinite(got[n][1]).any(), n


@pytest.mark.parametrize("pad", [8, 3])
def test_pitched_rows(pad):
    counts, K, N = [30, 0, 200], 136, 264
    x, w, b, dy, c = make(counts, K, N, torch.bfloat16)
    R = sum(counts)
    xb = torch.full((R, K + pad), float("nan"), dtype=x.dtype, device="cuda")
    db = torch.full((R, N + pad), float("nan"), dtype=x.dtype, device="cuda")
    yb = torch.full((R, N + pad), 7.0, dtype=x.dtype, device="cuda")
    xb[:, :K], db[:, :N] = x, dy
    bra.grouped_matmul(xb[:, :K], w, c, bias=b, out=yb[:, :N])
    assert torch.equal(yb[:, :N], bra.grouped_matmul(x, w, c, bias=b))
    assert (yb[:, N:] == 7.0).all()
    a = bra.grouped_matmul_grad(db[:, :N], xb[:, :K], w, c, bias=b)
    z = bra.grouped_matmul_grad(dy, x, w, c, bias=b)
    for n in a:
        assert torch.equal(a[n], z[n]), n


def test_pointers_without_16_byte_alignment():
    counts, K, N = [30, 1, 100], 64, 72
    x, w, b, dy, c = make(counts, K, N, torch.float16)
    shift = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    y = shift(torch.zeros(sum(counts), N, dtype=torch.float16, device="cuda"))
    assert y.data_ptr() % 16 == 2
    bra.grouped_matmul(shift(x), shift(w), c, bias=b, out=y)
    assert torch.equal(y, bra.grouped_matmul(x, w, c, bias=b))
    a = bra.grouped_matmul_grad(shift(dy), shift(x), shift(w), c, bias=b, dx=shift(x),
                                dweight=shift(w))
    z = bra.grouped_matmul_grad(dy, x, w, c, bias=b)
    for n in a:
        assert torch.equal(a[n], z[n]), n


@pytest.mark.parametrize("counts", [[4, -1, 3], [10, 10, 10], [1 << 40, 0, 0],
                                    [1 << 62, 1 << 62, 0], [-(1 << 63), 5, 5]], ids=str)
def test_refused_counts_write_nothing(counts):
    K, N, R = 64, 72, 20
    x, w, b, dy, _ = make([R, 0, 0], K, N, torch.float16)
    c = torch.tensor(counts, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((R, N), 7.0, dtype=torch.float16, device="cuda")
    bra.grouped_matmul(x, w, c, bias=b, out=y, status=status)
    assert int(status) == bra.ERR_INVALID and (y == 7.0).all()
    dw, db = torch.full_like(w, 7.0), torch.full_like(b, 7.0)
    dx = torch.full_like(x, 7.0)
    status.zero_()
    bra.grouped_matmul_grad(dy, x, w, c, dx=dx, dweight=dw, dbias=db, status=status)
    assert int(status) == bra.ERR_INVALID
    assert (dx == 7.0).all() and (dw == 7.0).all() and (db == 7.0).all()
    bra.grouped_matmul(x, w, torch.tensor([R, 0, 0], device="cuda"), out=y, status=status)
    assert int(status) == 0


def test_no_rows_at_all():
    for extra in (0, 5):
        x, w, b, dy, c = make([0, 0], 64, 72, torch.bfloat16, extra=extra)
        y = torch.full((extra, 72), 7.0, dtype=x.dtype, device="cuda")
        bra.grouped_matmul(x, w, c, bias=b, out=y)
        got = bra.grouped_matmul_grad(dy, x, w, c, bias=b)
        assert (y == 7.0).all()
        assert not got["dweight"].any() and not got["dbias"].any()


def test_counts_change_between_runs_of_a_plan_and_a_graph():
    K, N = 128, 136
    x, w, b, _, c = make([10, 20, 30], K, N, torch.bfloat16)
    plan = bra.grouped_matmul_plan(x, w, c, bias=b)
    plan.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for counts in ([60, 0, 0], [0, 1, 59], [20, 20, 20]):
        c.copy_(torch.tensor(counts))
        graph.replay()
        ref, mag = forward_ref(x, w, b, counts, False)
        assert_close(plan.result, ref, mag, K)


def test_another_stream_and_concurrent_calls():
    K, N = 256, 520
    cases = [make([50 * (i + 1), 7, 0], K, N, torch.float16, seed=i) for i in range(4)]
    want = [bra.grouped_matmul(x, w, c, bias=b) for x, w, b, _, c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [bra.grouped_matmul(x, w, c, bias=b, stream=s)
           for (x, w, b, _, c), s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, z in zip(got, want):
        assert torch.equal(a, z)
    assert bra.fault_status() == 0


def test_a_matrix_that_passes_32_bit_offsets():
    """Rows whose element offsets pass 2^32, in the last group."""
    K, N = 4096, 64
    R = (1 << 32) // K + 300
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    x[-200:] = torch.randn((200, K), device="cuda")
    w = (torch.randn((2, K, N), device="cuda") / 64).bfloat16()
    counts = [R - 150, 150]
    c = torch.tensor(counts, device="cuda")
    y = bra.grouped_matmul(x, w, c)
    dw = bra.grouped_matmul_grad(torch.ones_like(y), x, w, c, want=("dweight",))["dweight"]
    assert not y[:-200].any()
    for e, a, z in ((0, R - 200, R - 150), (1, R - 150, R)):
        xe = x[a:z].double()
        assert_close(y[a:z], xe @ w[e].double(), xe.abs() @ w[e].double().abs(), K)
        ref = xe.sum(0)[:, None].expand(K, N)
        assert_close(dw[e], ref, xe.abs().sum(0)[:, None].expand(K, N), 256)


def test_refused_arguments():
    x, w, b, dy, c = make([4, 4], 64, 72, torch.float16)
    with pytest.raises(TypeError):
        bra.grouped_matmul(x.bfloat16(), w, c)
    with pytest.raises(TypeError):
        bra.grouped_matmul(x.float(), w.float(), c)
    with pytest.raises(ValueError):
        bra.grouped_matmul(x.cpu(), w, c)
    with pytest.raises(ValueError):
        bra.grouped_matmul(x[:, :32], w, c)
    with pytest.raises(ValueError):
        bra.grouped_matmul(x.t().contiguous().t(), w, c)
    with pytest.raises(ValueError):
        bra.grouped_matmul(x, w, c[:1])
    with pytest.raises(TypeError):
        bra.grouped_matmul(x, w, c.int())
    with pytest.raises(TypeError):
        bra.grouped_matmul(x, w, c, bias=b.float())
    with pytest.raises(ValueError):
        bra.grouped_matmul_grad(dy, x, w, c, want=("dz",))
    with pytest.raises(ValueError):
        bra.grouped_matmul_grad(dy, x, w, c, want=("dbias",))
    with pytest.raises(bra.BraError) as err:
        buf = torch.zeros((8, 136), dtype=torch.float16, device="cuda")
        bra.grouped_matmul(buf[:, :64], w, c, out=buf[:, 60:132])     # overlaps x
    assert err.value.code == bra.ERR_INVALID
    odd = torch.zeros((8, 65), dtype=torch.float16, device="cuda")
    wo = torch.zeros((2, 65, 72), dtype=torch.float16, device="cuda")
    with pytest.raises(bra.BraError) as err:
        bra.grouped_matmul(odd, wo, c, workspace=None)                # needs a copy
    assert err.value.code == bra.ERR_UNSUPPORTED
    with pytest.raises(bra.BraError) as err:
        bra.grouped_matmul(odd, wo, c,
                           workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert err.value.code == bra.ERR_INVALID
