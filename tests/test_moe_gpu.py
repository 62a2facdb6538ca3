"""The router and the row permutation against plain 64-bit implementations.

Whole numbers (experts, counts, slots, tokens) have to be equal.  A weight is
exp(l - m) over a sum of such: the difference is rounded once (its exponential
then errs by |l - m| units), the exponential and the quotient by a few units of
2^-23, the sum by one for each of its E/32 + 5 levels.  Row sums of k products
err by one fp32 unit (2^-23 of the magnitude sum) an addition, and are rounded
once to the row type; dot products of H by H/256 + 16 units."""
import math
import threading

import numpy as np
import pytest
import torch

import bmm_reducescatter_alltoall_gb300 as bra

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -23
HALF = {torch.float16: (2.0 ** -11, 2.0 ** -24), torch.bfloat16: (2.0 ** -8, 2.0 ** -133),
        torch.float32: (2.0 ** -24, 2.0 ** -149)}
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def route_ref(logits, k, renorm):
    """ids, weights, counts, slots, tokens by the definition, in float64."""
    l = np.nan_to_num(logits.double().cpu().numpy(), nan=-np.inf, posinf=3.4028234663852886e38,
                      neginf=-np.inf)
    T, E = l.shape
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(l, order, 1)
    has = top > -np.inf
    m = np.where(has[:, :1], top[:, :1], 0.0)
    with np.errstate(under="ignore"):
        p = np.where(l > -np.inf, np.exp(np.maximum(l - m, -800)), 0.0)
        c = np.where(has, np.exp(np.maximum(top - m, -800)), 0.0)
    s = (c if renorm else p).sum(1, keepdims=True)
    w = c / np.where(s > 0, s, 1.0)
    p = p / np.where(p.sum(1, keepdims=True) > 0, p.sum(1, keepdims=True), 1.0)
    ids = np.where(has, order, -1)
    flat = np.where(has, order, E).reshape(-1)
    perm = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=E + 1)[:E]
    slots = np.empty(T * k, dtype=np.int64)
    slots[perm] = np.arange(T * k)
    slots = np.where(has, slots.reshape(T, k), -1)
    tokens = np.where(np.arange(T * k) < counts.sum(), perm // k, -1)
    far = np.where(l > -np.inf, np.minimum(m - l, 110.0), 0.0).max(1, keepdims=True)
    return ids, w, counts, slots, tokens, p, far


def check_route(logits, k, renorm, dw=None):
    T, E = logits.shape
    r = bra.moe_route(logits, k, renormalize=renorm)
    ids, w, counts, slots, tokens, p, far = route_ref(logits, k, renorm)
    for name, want in (("ids", ids), ("counts", counts), ("slots", slots), ("tokens", tokens)):
        assert np.array_equal(r[name].cpu().numpy(), want), name
    got = r["weights"].double().cpu().numpy()
    scale = (E / 32 + 24 + 2 * far) * UNIT
    assert (np.abs(got - w) <= scale * w + 2.0 ** -125).all()
    if dw is None:
        return r
    dl = bra.moe_route_grad(dw, logits, r["ids"], r["weights"], renormalize=renorm)
    g = np.where(ids >= 0, dw.double().cpu().numpy(), 0.0)
    at = np.where(ids >= 0, ids, 0)
    s, mag = (w * g).sum(1, keepdims=True), np.abs(w * g).sum(1, keepdims=True)
    gi, chosen = np.zeros((T, E)), np.zeros((T, E))
    np.add.at(gi, (np.arange(T)[:, None], at), g)
    np.add.at(chosen, (np.arange(T)[:, None], at), np.where(ids >= 0, w, 0.0))
    pi = chosen if renorm else p
    want = pi * (gi - s)
    unit, tiny = HALF[logits.dtype]
    tol = unit * np.abs(want) + 4 * scale * pi * (np.abs(gi) + mag) + tiny + 2.0 ** -120
    err = np.abs(dl.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()
    return r


def logits_of(T, E, dt, seed=0, ties=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn((T, E), generator=g, device="cuda") * 2
    if ties:
        l = torch.round(l)                                  # many equal logits
    return l.to(dt)


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 2, 2), (31, 5, 3), (64, 64, 8), (65, 64, 8), (300, 33, 4),
          (1000, 128, 8), (70, 512, 16), (2500, 200, 6), (129, 512, 1), (5000, 16, 16)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("renorm", [True, False])
def test_route_and_its_gradient(T, E, k, renorm, dt):
    dw = torch.randn((T, k), device="cuda")
    check_route(logits_of(T, E, dt), k, renorm, dw)
    check_route(logits_of(T, E, dt, ties=True), k, renorm, dw)


@pytest.mark.parametrize("T", [5, 700])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dt", DTYPES)
def test_masks(T, renorm, dt):
    """Closed experts, whole closed rows, rows with fewer open experts than choices, the type's
    lowest value, NaN and infinities."""
    E, k = 40, 6
    l = logits_of(T, E, dt)
    inf = float("inf")
    l[:, 7] = -inf
    l[0] = -inf
    l[1] = float("nan")
    l[2] = -inf
    l[2, 39], l[2, 3], l[2, 4] = 1.0, float("nan"), -5.0
    l[3] = torch.finfo(dt).min
    l[4, 10:] = torch.finfo(dt).min
    l[4, 5] = float("nan")
    if T > 9:
        l[5, 9] = inf
        l[6, 9] = l[6, 30] = inf
        l[7] = 0.0
        l[7, ::2] = -0.0
        l[8] = torch.finfo(dt).max
    r = check_route(l, k, renorm, torch.randn((T, k), device="cuda"))
    assert (r["ids"][0] == -1).all() and (r["weights"][0] == 0).all()
    assert (r["slots"][1] == -1).all() and int(r["counts"][7]) == 0


def test_no_open_expert_and_no_token():
    r = bra.moe_route(torch.full((70, 8), -math.inf, device="cuda"), 2)
    assert not r["counts"].any() and (r["tokens"] == -1).all() and (r["slots"] == -1).all()
    for name in ("weights",):
        assert not r[name].any()
    r = bra.moe_route(torch.zeros((0, 8), device="cuda"), 2)
    assert r["counts"].tolist() == [0] * 8 and r["tokens"].numel() == 0
    assert bra.moe_route_grad(r["weights"], torch.zeros((0, 8), device="cuda"), r["ids"],
                              r["weights"]).shape == (0, 8)


@pytest.mark.parametrize("T", [40, 131073, 150001])
def test_many_tokens(T):
    check_route(logits_of(T, 24, torch.bfloat16), 3, True)
    # everyone to the same two experts
    l = torch.zeros((T, 24), device="cuda")
    l[:, 20], l[:, 3] = 5.0, 4.0
    r = check_route(l, 2, False)
    assert r["counts"].tolist() == [T if e in (3, 20) else 0 for e in range(24)]


@pytest.mark.parametrize("T,E", [(155648, 16), (155649, 40), (400003, 40), (1300001, 9)])
def test_more_chunks_than_processors(T, E):
    """From 152 * 1024 tokens on there are several chunks to an SM, of even and odd numbers of
    words, and the counts of all chunks are summed in between (32 experts a block)."""
    check_route(logits_of(T, E, torch.float16, seed=T), 2, True)
    l = torch.full((T, E), float("-inf"), device="cuda")
    l[T - 1, E - 1] = l[7, 0] = l[T // 2, 0] = 1.0
    r = bra.moe_route(l, 2)
    assert r["counts"].tolist() == [2] + [0] * (E - 2) + [1]
    assert r["tokens"][:3].tolist() == [7, T // 2, T - 1] and (r["tokens"][3:] == -1).all()
    assert [r["slots"][t, 0].item() for t in (7, T // 2, T - 1)] == [0, 1, 2]
    assert (r["slots"] >= 0).sum().item() == 3


def test_the_gradient_is_that_of_differences():
    """Central differences of the weights in fp32: with steps of 2^-7 the third derivative's term
    is below 2^-14 * |g| and the rounding of a weight 2^-22 / 2^-7."""
    T, E, k, h = 6, 12, 3, 2.0 ** -7
    l = logits_of(T, E, torch.float32, seed=5) / 2
    g = torch.randn((T, k), device="cuda")
    for renorm in (True, False):
        r = bra.moe_route(l, k, renormalize=renorm)
        dl = bra.moe_route_grad(g, l, r["ids"], r["weights"], renormalize=renorm)
        for e in range(E):
            up, dn = l.clone(), l.clone()
            up[:, e] += h
            dn[:, e] -= h
            a, b = (bra.moe_route(t, k, renormalize=renorm) for t in (up, dn))
            same = ((a["ids"] == r["ids"]) & (b["ids"] == r["ids"])).all(1)
            num = ((a["weights"].double() - b["weights"]) * g).sum(1) / (2 * h)
            tol = (2.0 ** -14 + k * 2.0 ** -15) * g.abs().sum(1)
            assert ((num - dl[:, e].double()).abs() <= tol)[same].all(), e
            assert same.float().mean() > 0.5


def test_route_in_a_graph_and_on_streams():
    l = logits_of(900, 32, torch.float32)
    plan = bra.moe_route_plan(l, 4)
    plan.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for seed in (1, 2):
        l.copy_(logits_of(900, 32, torch.float32, seed=seed))
        graph.replay()
        want = bra.moe_route(l, 4, stream=torch.cuda.current_stream())
        for n in want:
            assert torch.equal(plan.result[n], want[n]), n


# ------------------------------------------------------------------ permutation

def routed(T, E, k, closed=0.0, seed=0):
    l = logits_of(T, E, torch.float32, seed=seed)
    if closed:
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        l[torch.rand((T, E), generator=g, device="cuda") < closed] = -math.inf
    return bra.moe_route(l, k)


def close(got, ref, mag, terms):
    unit, tiny = HALF[got.dtype]
    tol = unit * ref.abs() + terms * UNIT * mag + tiny
    assert ((got.double() - ref).abs() <= tol).all()


def check_permute(T, E, k, H, dt, closed=0.0, seed=0):
    r = routed(T, E, k, closed, seed)
    slots, w, tok = r["slots"].long(), r["weights"], r["tokens"].long()
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    rnd = lambda n: torch.randn((n, H), generator=g, device="cuda").to(dt)       # noqa: E731
    x, ys, dxs, dy = rnd(T), rnd(T * k), rnd(T * k), rnd(T)
    has, at = slots >= 0, slots.clamp(min=0)
    xs = bra.moe_dispatch(x, r["tokens"])
    want = torch.where((tok >= 0)[:, None], x[tok.clamp(min=0)], torch.zeros((), dtype=dt, device="cuda"))
    assert torch.equal(xs, want)
    pick = lambda rows: rows[at].double() * has[:, :, None]                       # noqa: E731
    y = bra.moe_combine(ys, r["slots"], w)
    terms = pick(ys) * w.double()[:, :, None]
    close(y, terms.sum(1), terms.abs().sum(1), k + 1)
    dx = bra.moe_dispatch_grad(dxs, r["slots"])
    close(dx, pick(dxs).sum(1), pick(dxs).abs().sum(1), k + 1)
    out = bra.moe_combine_grad(dy, ys, r["slots"], w, r["tokens"])
    prod = pick(ys) * dy.double()[:, None]
    close(out["dweights"], prod.sum(2), prod.abs().sum(2), H / 256 + 16)
    dys = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
    dys[slots[has]] = (w.double()[:, :, None] * dy.double()[:, None])[has]
    close(out["dys"], dys, dys.abs(), 1)
    assert not out["dys"][tok < 0].any() and not out["dweights"][~has].any()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("H", [1, 7, 8, 64, 250, 264, 1000, 1024, 1031, 4096])
def test_permutation_over_widths(H, dt):
    check_permute(50, 9, 3, H, dt)
    check_permute(37, 40, 8, H, dt, closed=0.9)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 16, 16), (2, 64, 6), (515, 30, 5), (4000, 64, 16)])
@pytest.mark.parametrize("H", [40, 1025, 2048])
def test_permutation_over_tokens(T, E, k, H):
    check_permute(T, E, k, H, torch.bfloat16, closed=0.3)


@pytest.mark.parametrize("dt,H", [(torch.bfloat16, 4096), (torch.float32, 2050),
                                  (torch.float16, 4001)])
def test_dispatch_of_many_long_rows(dt, H):
    """Token rows past L2, whose rows are listed first: tokens in any order, some with more rows
    than a list holds, some without, entries out of range."""
    T = 8000
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn((T, H), generator=g, device="cuda").to(dt)
    assert x.numel() * x.element_size() >= 48 << 20
    tokens = torch.randint(-1, T, (2 * T + 777,), generator=g, device="cuda", dtype=torch.int32)
    tokens[100:140] = 17                                  # 40 rows of one token
    tokens[5000:5003] = torch.tensor([T, -5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    want = torch.where(((tokens >= 0) & (tokens < T))[:, None], x[tokens.long().clamp(0, T - 1)],
                       torch.zeros((), dtype=dt, device="cuda"))
    plan = bra.moe_dispatch_plan(x, tokens)
    for _ in range(2):
        plan.result.fill_(7.0)
        assert torch.equal(plan.run(), want)


def test_entries_out_of_range_are_left_out():
    x = torch.randn((4, 64), device="cuda")
    tokens = torch.tensor([0, 4, -7, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    xs = bra.moe_dispatch(x, tokens)
    assert torch.equal(xs[0], x[0]) and torch.equal(xs[3], x[3]) and not xs[[1, 2, 4]].any()
    slots = torch.tensor([[0, 5], [-3, 4]], dtype=torch.int32, device="cuda")
    w = torch.ones((2, 2), device="cuda")
    ys = torch.randn((5, 64), device="cuda")
    y = bra.moe_combine(ys, slots, w)
    assert torch.equal(y[0], ys[0]) and torch.equal(y[1], ys[4])
    out = bra.moe_combine_grad(torch.ones((2, 64), device="cuda"), ys, slots, w)
    assert float(out["dweights"][0, 1]) == 0 and float(out["dweights"][1, 0]) == 0


def test_masked_rows_may_hold_anything():
    """A row that no slot names is not read: NaN in it reaches nothing."""
    r = routed(20, 8, 4, closed=0.6)
    R = 80
    used = int(r["counts"].sum())
    assert used < R
    ys = torch.randn((R, 96), device="cuda").half()
    ys[used:] = float("nan")
    assert torch.isfinite(bra.moe_combine(ys, r["slots"], r["weights"])).all()
    out = bra.moe_combine_grad(torch.ones((20, 96), device="cuda").half(), ys, r["slots"],
                               r["weights"], r["tokens"])
    assert torch.isfinite(out["dys"]).all() and torch.isfinite(out["dweights"]).all()


def test_unused_rows_are_kept_without_tokens():
    r = routed(20, 8, 4, closed=0.6)
    ys = torch.randn((80, 96), device="cuda")
    dys = torch.full((80, 96), 7.0, device="cuda")
    bra.moe_combine_grad(torch.ones((20, 96), device="cuda"), ys, r["slots"], r["weights"], dys=dys)
    assert (dys[r["tokens"] < 0] == 7.0).all()


def test_permutation_of_a_matrix_that_passes_32_bit_offsets():
    H, k = 4096, 2
    T = (1 << 31) // H // k + 40                              # R * H passes 2^31 elements
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[-30:] = torch.randn((30, H), device="cuda")
    l = torch.zeros((T, 4), device="cuda")
    r = bra.moe_route(l, k)                                   # everyone to experts 0 and 1
    xs = bra.moe_dispatch(x, r["tokens"])
    assert torch.equal(xs[T - 30:T], x[-30:]) and torch.equal(xs[-30:], x[-30:])
    y = bra.moe_combine(xs, r["slots"], r["weights"])
    assert torch.equal(y, x)
    out = bra.moe_combine_grad(x, xs, r["slots"], r["weights"], r["tokens"])
    assert torch.equal(out["dys"][-30:], (x[-30:].float() / 2).bfloat16())
    ref = x[-30:].double().square().sum(1)
    close(out["dweights"][-30:, 1], ref, ref, H / 256 + 16)


def test_the_gradients_of_the_moves_are_their_adjoints():
    """<dispatch(x), d> = <x, dispatch_grad(d)> and the same of combine, exactly, on small whole
    numbers and weights of a half."""
    r = routed(100, 16, 4, closed=0.5)
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = lambda n: torch.randint(-3, 4, (n, 72), generator=g, device="cuda").float()  # noqa: E731
    x, ys, d, dy = ints(100), ints(400), ints(400), ints(100)
    dot = lambda a, b: float((a.double() * b.double()).sum())                           # noqa: E731
    assert dot(bra.moe_dispatch(x, r["tokens"]), d) == dot(x, bra.moe_dispatch_grad(d, r["slots"])) \
        + dot(bra.moe_dispatch(x, r["tokens"])[r["tokens"] < 0], d[r["tokens"] < 0])
    w = torch.full((100, 4), 0.5, device="cuda")
    y = bra.moe_combine(ys, r["slots"], w)
    out = bra.moe_combine_grad(dy, ys, r["slots"], w, r["tokens"])
    assert dot(y, dy) == dot(ys, out["dys"]) == dot(w, out["dweights"])


def test_refused_arguments():
    l = torch.zeros((4, 8), device="cuda")
    for bad in (0, 9, 17):
        with pytest.raises((bra.BraError, RuntimeError)):
            bra.moe_route(l, bad)
    with pytest.raises(bra.BraError) as err:
        bra.moe_route(torch.zeros((4, 513), device="cuda"), 2)
    assert err.value.code == bra.ERR_INVALID
    with pytest.raises(TypeError):
        bra.moe_route(l.double(), 2)
    with pytest.raises(ValueError):
        bra.moe_route(l.t(), 2)
    with pytest.raises(ValueError):
        bra.moe_route(l.cpu(), 2)
    with pytest.raises(bra.BraError) as err:
        bra.moe_route(torch.zeros((400, 8), device="cuda"), 2, workspace=None)
    assert err.value.code == bra.ERR_NULLPTR
    r = bra.moe_route(l, 2)
    x = torch.zeros((4, 64), device="cuda")
    ys = torch.zeros((8, 64), device="cuda")
    with pytest.raises(TypeError):
        bra.moe_dispatch(x, r["tokens"].long())
    with pytest.raises(bra.BraError) as err:                          # needs lists
        bra.moe_dispatch(torch.empty((8192, 4096), device="cuda"),
                         torch.zeros(16384, dtype=torch.int32, device="cuda"), workspace=None)
    assert err.value.code == bra.ERR_NULLPTR
    with pytest.raises(TypeError):
        bra.moe_combine(ys, r["slots"], r["weights"].half())
    with pytest.raises(ValueError):
        bra.moe_combine(ys, r["slots"], r["weights"][:3])
    with pytest.raises(ValueError):
        bra.moe_combine_grad(x[:3], ys, r["slots"], r["weights"])
    with pytest.raises(bra.BraError) as err:
        bra.moe_combine(ys, r["slots"], r["weights"], out=ys[2:6])
    assert err.value.code == bra.ERR_INVALID


def test_routes_of_different_sizes_from_two_threads():
    """Calls whose shared memory differs, from host threads at once: neither is refused, both are
    right.  (512 experts: 62 KB for 150000 tokens, 42 KB for 200000.)"""
    sizes = [(150000, 512), (200000, 512), (150000, 400), (160000, 300)]
    plans = [bra.moe_route_plan(logits_of(T, E, torch.bfloat16, seed=E + T), 1) for T, E in sizes]
    want = []
    for p in plans:
        p.run()
        want.append({n: t.clone() for n, t in p.result.items()})
    torch.cuda.synchronize()
    streams, failed = [torch.cuda.Stream() for _ in plans], []

    def loop(plan, stream):
        try:
            for _ in range(400):
                plan.run(stream)
        except Exception as e:                                # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=loop, args=a) for a in zip(plans, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[:2]
    for p, w in zip(plans, want):
        for n in w:
            assert torch.equal(p.result[n], w[n]), n


@pytest.mark.parametrize("T,dt,H", [(2, torch.float32, 64), (2, torch.bfloat16, 1031),
                                    (0, torch.float16, 264)])
def test_combine_gradient_of_rows_whose_token_is_out_of_range(T, dt, H):
    """Tokens outside [0, T) count as -1: their rows get zeros."""
    slots = torch.tensor([[0, 5], [-3, 4]], dtype=torch.int32, device="cuda")[:T]
    w = torch.ones((T, 2), device="cuda")
    ys = torch.randn((7, H), device="cuda").to(dt)
    dy = torch.randn((T, H), device="cuda").to(dt)
    tokens = torch.tensor([0, T, -5, 2 ** 31 - 1, 1, 0, -1], dtype=torch.int32, device="cuda")
    if T == 0:
        tokens[[0, 4, 5]] = -1
    dys = torch.full_like(ys, float("nan"))
    bra.moe_combine_grad(dy, ys, slots, w, tokens, dys=dys)
    assert not dys[[1, 2, 3, 6]].any()
    if T:
        assert all(torch.equal(dys[r], dy[t]) for r, t in ((0, 0), (5, 0), (4, 1)))
    else:
        assert not dys.any()


@pytest.mark.parametrize("E,k", [(12, 3), (300, 16)])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradients_that_are_not_finite_leave_closed_experts_at_zero(E, k, renorm):
    l = logits_of(6, E, torch.float32, seed=E)
    l[:, ::3] = -math.inf
    l[4] = -math.inf
    l[4, 5] = 1.0
    dw = torch.randn((6, k), device="cuda")
    r = bra.moe_route(l, k, renormalize=renorm)
    want = bra.moe_route_grad(dw, l, r["ids"], r["weights"], renormalize=renorm)
    dw[0, 1], dw[1, 0], dw[2] = math.inf, math.nan, -math.inf
    dw[4, 1:] = math.nan                                      # choices that are missing
    dl = bra.moe_route_grad(dw, l, r["ids"], r["weights"], renormalize=renorm)
    assert not dl[l == -math.inf].any()
    assert torch.equal(dl[3:], want[3:])
    assert not torch.isfinite(dl[:3]).all(1).any()
