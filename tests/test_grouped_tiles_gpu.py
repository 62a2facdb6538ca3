"""The grouped products' kernels at the sizes that take them: each case names the
tiles that its calls have to report, so that a changed rule cannot leave a kernel
untested.  Tolerances as in test_grouped_gpu.py and test_mxfp4_gpu.py; sums of
small whole numbers are exact in fp32, and compared for equality."""
import re

import pytest
import torch

import bmm_reducescatter_alltoall_gb300 as bra
import test_mxfp4_gpu as mx
from test_grouped_gpu import assert_close, check_forward, check_grad, forward_ref, groups_of, make

pytestmark = pytest.mark.gpu

PAIR = "256x256 tiles by CTA pairs"
WIDE, NARROW, COLUMN = "128x256 tiles", "128x128 tiles", "128x64 tiles"
OVER = "128x128 tiles, sums over %d CTAs"
# uneven groups of more than 1024 rows on average: ends of every kind of a row block, empty ones
LARGE = [1500, 1037, 2049, 1100, 0, 2000]
MIXED = [3000, 5, 0, 1, 64, 63, 5000, 1037]


@pytest.fixture
def took(monkeypatch, capfd):
    """took(): the tiles of each call since the last one, by operator."""
    monkeypatch.setenv("BRA_LOG", "1")
    capfd.readouterr()

    def read():
        lines = re.findall(r"\[bra\] (\S+(?: d\w+)?) rows=.* -> (.*)", capfd.readouterr().err)
        out = {}
        for name, tiles in lines:
            out.setdefault(name.split()[-1], set()).add(tiles)
        return {k: v.pop() if len(v) == 1 else v for k, v in out.items()}
    return read


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("counts,K,N,tiles", [
    (LARGE, 2056, 1288, PAIR), (MIXED, 1290, 1550, PAIR), (MIXED, 1291, 1551, PAIR),
    ([1100, 0, 2500, 1], 1030, 2051, PAIR), (LARGE, 1290, 1550, WIDE), (LARGE, 521, 779, NARROW),
    ([256, 512, 0, 1024], 1032, 2056, WIDE), ([2500, 1700], 264, 264, NARROW),
    ([3, 0, 5, 1] * 8, 264, 2056, WIDE), ([2, 1, 0, 1], 264, 2055, COLUMN),
    ([2, 1, 0, 1, 3], 520, 1288, COLUMN), ([1] * 16, 520, 1288, NARROW),
    ([5, 90], 2056, 264, OVER % 8),
], ids=str)
def test_forward(counts, K, N, tiles, bias, dt, took):
    for wt in (False, True):
        check_forward(counts, K, N, dt, wt, bias, seed=K + wt)
        assert took() == {"grouped_matmul": tiles}
    assert bra.fault_status() == 0


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("wt", [False, True])
@pytest.mark.parametrize("counts,K,N,dx,dw", [
    (LARGE, 520, 776, PAIR, PAIR), (LARGE, 521, 779, PAIR, PAIR), (MIXED, 1290, 1550, PAIR, PAIR),
    (MIXED, 1032, 2056, PAIR, PAIR), ([2500, 1700], 1291, 1551, PAIR, PAIR),
    ([2500, 1700], 1032, 2056, NARROW, PAIR), ([256, 512, 0, 1024], 1290, 1550, PAIR, WIDE),
    ([256, 512, 0, 1024], 2051, 1285, WIDE, WIDE), ([2500, 1700], 264, 264, NARROW, OVER % 8),
], ids=str)
def test_gradients(counts, K, N, dx, dw, wt, dt, took):
    check_grad(counts, K, N, dt, wt, seed=N)
    got = took()
    assert got.pop("dx") == dx and got.pop("dweight") == dw and not got
    assert bra.fault_status() == 0


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_exact_sums_on_cta_pairs(dt, took):
    """Small whole numbers: every sum is exact, forward and back, each rounded once."""
    for K, N, wt in ((2056, 1288, False), (2051, 1285, True)):
        g = torch.Generator(device="cuda").manual_seed(K)
        ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(dt)   # noqa: E731
        E, R = len(LARGE), sum(LARGE)
        x, dy = ints(R, K), ints(R, N)
        w = ints(E, N, K) if wt else ints(E, K, N)
        c = torch.tensor(LARGE, device="cuda")
        y = bra.grouped_matmul(x, w, c, transpose_weight=wt)
        d = bra.grouped_matmul_grad(dy, x, w, c, want=("dx", "dweight"), transpose_weight=wt)
        assert took() == {"grouped_matmul": PAIR, "dx": PAIR, "dweight": PAIR}
        assert torch.equal(y, forward_ref(x, w, None, LARGE, wt)[0].to(dt))
        for e, a, z in groups_of(LARGE):
            we = (w[e].t() if wt else w[e]).double()
            assert torch.equal(d["dx"][a:z], (dy[a:z].double() @ we.t()).to(dt)), e
            dw = x[a:z].double().t() @ dy[a:z].double()
            assert torch.equal(d["dweight"][e], (dw.t() if wt else dw).to(dt)), e


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_pairs_leave_other_rows_alone(dt, took):
    """Rows of infinities and NaN at a group's ends reach their own group alone, rows past the
    groups nothing; those of the outputs past the groups, and between pitched rows, are kept."""
    counts, K, N, extra, pad = [1301, 0, 1047, 2300, 1529], 1288, 1032, 300, 5
    x, w, b, dy, c = make(counts, K, N, dt, extra=extra)
    R0 = sum(counts)
    x[R0:], dy[R0:] = float("nan"), float("inf")
    bad = slice(1301, 1301 + 1047)                            # the third group
    x[1301], dy[1301] = float("inf"), float("nan")
    x[1301 + 1046], dy[1301 + 1046] = float("nan"), float("-inf")
    y = torch.full((R0 + extra, N + pad), 7.0, dtype=dt, device="cuda")
    bra.grouped_matmul(x, w, c, bias=b, out=y[:, :N])
    assert (y[R0:] == 7.0).all() and (y[:, N:] == 7.0).all()
    dx = torch.full((R0 + extra, K), 7.0, dtype=dt, device="cuda")
    got = bra.grouped_matmul_grad(dy, x, w, c, bias=b, dx=dx)
    assert took() == {"grouped_matmul": PAIR, "dx": PAIR, "dweight": PAIR}
    assert (dx[R0:] == 7.0).all()
    ends = torch.zeros(R0, dtype=torch.bool, device="cuda")
    ends[[bad.start, bad.stop - 1]] = True
    for t in (y[:R0, :N], dx[:R0]):
        assert torch.equal(torch.isfinite(t).all(1), ~ends)
    fine = [0, 1, 3, 4]
    for n in ("dweight", "dbias"):
        assert torch.isfinite(got[n][fine]).all() and not torch.isfinite(got[n][2]).any(), n
    assert not got["dweight"][1].any() and not got["dbias"][1].any()
    ref, mag = forward_ref(x[:R0], w, b, counts, False)
    assert_close(y[:R0, :N][~ends], ref[~ends], mag[~ends], K)
    for e, a, z in groups_of(counts):
        if e != 2:
            xe, d = x[a:z].double(), dy[a:z].double()
            assert_close(got["dweight"][e], xe.t() @ d, xe.abs().t() @ d.abs(), z - a)


MX_COUNTS = [700, 3, 0, 300, 900, 1297]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,K,N,tiles", [
    (MX_COUNTS, 300, 1411, PAIR), (MX_COUNTS, 32, 1288, PAIR), (MX_COUNTS, 1029, 1550, PAIR),
    ([1280, 129, 383], 1024, 2824, PAIR), ([256] * 16, 264, 1288, PAIR),
    (MX_COUNTS, 300, 1032, "128x128 tiles"), ([100] * 20, 544, 2056, "128x128 tiles"),
], ids=str)
def test_4_bit_products(counts, K, N, tiles, dt, took):
    for bias in (True, False):
        x, w, b, c = mx.case(counts, K, N, dt=dt, seed=N)
        b = b if bias else None
        y = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w), c, bias=b,
                                     dtype=dt)
        assert took() == {"mxfp4_grouped_matmul": tiles}
        mx.assert_close(y, *mx.reference(x, w, b, counts), K)
    assert bra.fault_status() == 0


@pytest.mark.parametrize("K,N", [(544, 1411), (2056, 1288), (256, 1551)])
def test_exact_4_bit_sums_on_cta_pairs(K, N, took):
    """Multiples of a quarter that fp32 sums exactly; a power of two for each block of 32 that
    cancels in the product: every scale is in its place."""
    g = torch.Generator(device="cuda").manual_seed(K)
    pick = lambda *s: torch.tensor([0., 1, -1, 2, -3, 0.5, 0, 0], device="cuda")[          # noqa: E731
        torch.randint(0, 8, s, generator=g, device="cuda")]
    x, w = pick(sum(MX_COUNTS), K), pick(len(MX_COUNTS), N, K)
    blocks = -(-K // 32)
    p = torch.exp2(torch.randint(-20, 21, (blocks,), generator=g, device="cuda").float())
    p = p.repeat_interleave(32)[:K]
    rows = torch.exp2(torch.randint(-4, 5, (len(x), 1), generator=g, device="cuda").float())
    cols = torch.exp2(torch.randint(-4, 5, (len(MX_COUNTS), N, 1), generator=g, device="cuda").float())
    c = torch.tensor(MX_COUNTS, device="cuda")
    y = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize((x * p * rows).bfloat16(), c),
                                 bra.mxfp4_quantize((w / p * cols).bfloat16()), c,
                                 dtype=torch.float16)
    assert took() == {"mxfp4_grouped_matmul": PAIR}
    for e, a, z in groups_of(MX_COUNTS):
        want = (x[a:z].double() @ w[e].t().double()) * rows[a:z].double() * cols[e].double().t()
        assert torch.equal(y[a:z], want.half()), e


def test_a_row_without_a_value_stays_alone_on_cta_pairs(took):
    x, w, b, c = mx.case(MX_COUNTS, 320, 1411)
    lost = [0, 699, 700, 702, 703, 1002, 1100, 3199]
    x[lost, 100] = float("nan")
    x[1100, 0] = float("inf")
    y = bra.mxfp4_grouped_matmul(bra.mxfp4_quantize(x, c), bra.mxfp4_quantize(w), c, bias=b)
    assert took() == {"mxfp4_grouped_matmul": PAIR}
    nan = torch.isnan(y)
    assert nan[lost].all() and int(nan.sum()) == len(lost) * 1411


def test_a_group_whose_sum_takes_longer_than_a_wait(took):
    """The weight gradient of 1.1e9 rows in one of 80 experts: each of a tile's 17 million row blocks
    arrives in time, their sum takes over four seconds (0.27 us a block)."""
    R, E, K = 1100000000, 80, 16
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 7, 500000000, R - 3, R - 1], device="cuda")
    x[at] = torch.arange(1, 6, device="cuda")[:, None].expand(5, K).bfloat16()
    c = torch.zeros(E, dtype=torch.int64, device="cuda")
    c[3], c[4] = R - 2, 2
    w = torch.empty((E, K, K), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = bra.grouped_matmul_grad(x, x, w, c, want=("dweight",), status=status)["dweight"]
    assert took() == {"dweight": NARROW}
    assert int(status) == 0 and bra.fault_status() == 0
    assert (dw[3] == 1 + 4 + 9 + 16).all() and (dw[4] == 25).all()
    assert not dw[:3].any() and not dw[5:].any()
