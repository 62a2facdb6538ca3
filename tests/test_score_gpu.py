"""The router by scores against a plain 64-bit implementation.

Whole numbers (experts, counts, slots, tokens) have to be equal: the choice is the one in 64 bits.
A sigmoid weight errs by a few units of 2^-23 (exponential 2, sum, quotient), a softmax weight as
in the router without scores: by 2 |l - m| + E/32 + 24 units; renormalising adds the sum's 16
units, the scale one."""
import math

import numpy as np
import pytest
import torch

import bmm_reducescatter_alltoall_gb300 as bra

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -23
HALF = {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
        torch.float32: (2.0 ** -24, 2.0 ** -150)}
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def reference(logits, k, renorm, score, bias, groups, top, best, scale):
    l = np.nan_to_num(logits.double().cpu().numpy(), nan=-np.inf, posinf=3.4028234663852886e38,
                      neginf=-np.inf)
    T, E = l.shape
    shut = l == -np.inf
    m = np.where(shut.all(1, keepdims=True), 0.0, l.max(1, keepdims=True))
    with np.errstate(over="ignore", under="ignore"):
        if score == "sigmoid":
            p = np.where(shut, 0.0, 1.0 / (1.0 + np.exp(-l)))
        else:
            p = np.where(shut, 0.0, np.exp(l - m))
            p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    if bias is None:
        rank = l
    else:
        b = bias.double().cpu().numpy()
        rank = np.where(shut | np.isnan(b), -np.inf, p + np.where(np.isnan(b), 0.0, b))
    if top < groups:
        of = l if bias is None and best == 1 else np.where(shut, -np.inf, p) if bias is None else rank
        s = -np.sort(-of.reshape(T, groups, -1), axis=2)[:, :, :best]
        v = np.where(s > -np.inf, s, 0.0).sum(2)
        v = np.where(s[:, :, 0] > -np.inf, v, -np.inf)
        order = np.argsort(-v, axis=1, kind="stable")[:, :top]
        kept = np.zeros((T, groups), dtype=bool)
        np.put_along_axis(kept, order, True, 1)
        rank = np.where(np.repeat(kept, E // groups, 1), rank, -np.inf)
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    has = np.take_along_axis(rank, ids, 1) > -np.inf
    w = np.where(has, np.take_along_axis(p, ids, 1), 0.0)
    at = np.take_along_axis(l, ids, 1)
    if renorm and score == "sigmoid":
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    elif renorm:
        peak = np.where(has, at, -np.inf).max(1, keepdims=True)
        with np.errstate(under="ignore", invalid="ignore"):
            w = np.where(has, np.exp(at - np.where(np.isfinite(peak), peak, 0.0)), 0.0)
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    flat = np.where(has, ids, E).reshape(-1)
    perm = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=E + 1)[:E]
    slots = np.empty(T * k, dtype=np.int64)
    slots[perm] = np.arange(T * k)
    far = np.where(shut, 0.0, np.minimum(m - l, 110.0)).max(1, keepdims=True)
    if score == "sigmoid":
        far = np.zeros_like(far)
    return {"ids": np.where(has, ids, -1), "counts": counts,
            "slots": np.where(has, slots.reshape(T, k), -1),
            "tokens": np.where(np.arange(T * k) < counts.sum(), perm // k, -1)}, w, p, at, has, far


def check(logits, k, renorm=True, score="sigmoid", bias=None, groups=1, top=1, best=2, scale=1.0,
          dw=None):
    T, E = logits.shape
    r = bra.moe_route(logits, k, renormalize=renorm, score=score, bias=bias, groups=groups,
                      top_groups=top, group_best=best, scale=scale)
    whole, w, p, at, has, far = reference(logits, k, renorm, score, bias, groups, top, best, scale)
    for name, want in whole.items():
        got = r[name].cpu().numpy()
        assert np.array_equal(got, want), (name, np.argwhere(got != want)[:4].tolist())
    unit = (E / 32 + 44 + 2 * far) * UNIT
    err = np.abs(r["weights"].double().cpu().numpy() - w * scale)
    # sigmoid scores below fp32's range of exp(-l) count as 0
    tiny = 2.0 ** -120 if not renorm or score == "softmax" else 1e-17
    assert (err <= abs(scale) * (unit * w + tiny)).all(), err.max()
    if dw is None:
        return r
    dl = bra.moe_route_grad(dw, logits, r["ids"], r["weights"], renormalize=renorm, score=score,
                            scale=scale)
    g = np.where(has, dw.double().cpu().numpy(), 0.0)
    mean, mag = (w * g).sum(1, keepdims=True), np.abs(w * g).sum(1, keepdims=True)
    want, size = np.zeros((T, E)), np.zeros((T, E))
    rows, safe = np.arange(T)[:, None], np.where(has, whole["ids"], 0)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            rest = 1.0 / (1.0 + np.exp(np.where(has, at, 0.0)))
        if not renorm:
            mean, mag = 0.0, 0.0
        np.add.at(want, (rows, safe), np.where(has, w * (g - mean) * rest, 0.0))
        np.add.at(size, (rows, safe), np.where(has, w * (np.abs(g) + mag) * rest, 0.0))
    elif renorm:
        np.add.at(want, (rows, safe), w * (g - mean))
        np.add.at(size, (rows, safe), w * (np.abs(g) + mag))
    else:
        gi = np.zeros((T, E))
        np.add.at(gi, (rows, safe), g)
        want, size = p * (gi - mean), p * (np.abs(gi) + mag)
    half, least = HALF[logits.dtype]
    tol = abs(scale) * (half * np.abs(want) + 4 * unit * size + 2.0 ** -115 +
                        (1e-17 * np.abs(g).max() if g.size else 0)) + least
    err = np.abs(dl.double().cpu().numpy() - want * scale)
    assert (err <= tol).all(), (err - tol).max()
    return r


def logits_of(T, E, dt, seed=0, ties=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn((T, E), generator=g, device="cuda") * 2
    return (torch.round(l) if ties else l).to(dt)


def bias_of(E, seed=1, step=0.001):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-60, 61, (E,), generator=g, device="cuda") * step


# tokens, experts, choices, groups, groups kept: every layout of lanes, groups that fill no lane,
# numbers of groups that are no powers of two, experts that are no multiple of four
SHAPES = [(1, 1, 1, 1, 1), (3, 2, 2, 2, 1), (5, 6, 2, 3, 2), (70, 16, 16, 4, 2), (64, 64, 8, 8, 4),
          (65, 256, 8, 8, 4), (300, 160, 6, 8, 3), (129, 60, 4, 12, 5), (33, 510, 16, 3, 2),
          (200, 510, 5, 17, 4), (100, 512, 16, 32, 7), (40, 512, 8, 1, 1), (1000, 128, 8, 16, 16),
          (2500, 35, 3, 5, 1), (500, 500, 9, 4, 3), (77, 300, 4, 2, 1)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,E,k,G,top", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_routes_and_gradients(T, E, k, G, top, score, dt):
    dw = torch.randn((T, k), device="cuda")
    for seed, (renorm, best, biased, scale) in enumerate([
            (True, 2, True, 2.5), (False, 1, True, 1.0), (True, 1, False, 0.5), (False, 2, False, -3.0)]):
        for ties in (False, True):
            check(logits_of(T, E, dt, seed, ties), k, renorm, score, bias_of(E) if biased else None, G,
                  top, best, scale, dw)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,top,best", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_masks(score, G, top, best, dt):
    """Closed experts, rows and groups, fewer open experts than choices, the lowest value, NaN and
    infinities, saturated scores, with and without a bias."""
    T, E, k, inf = 40, 40, 6, math.inf
    l = logits_of(T, E, dt)
    l[:, 7] = -inf
    l[0], l[1], l[2] = -inf, float("nan"), -inf
    l[2, 39], l[2, 3], l[2, 4] = 1.0, float("nan"), -5.0
    l[3] = torch.finfo(dt).min
    l[4, 10:] = torch.finfo(dt).min
    l[4, 5] = float("nan")
    l[5, 9] = inf
    l[6, 9] = l[6, 30] = inf
    l[7] = 0.0
    l[7, ::2] = -0.0
    l[8] = torch.finfo(dt).max
    l[9] = torch.arange(40, device="cuda").to(dt) + 10.0       # sigmoid: 1 in 32 bits, from 37 in 64
    l[10] = -l[9]
    l[11] = 60.0
    l[12, 5:] = -inf
    for bias in (None, bias_of(E), torch.zeros(E, device="cuda")):
        for renorm in (True, False):
            r = check(l, k, renorm, score, bias, G, top, best, 1.5, torch.randn((T, k), device="cuda"))
            assert (r["ids"][0] == -1).all() and not r["weights"][0].any()
            assert int(r["counts"][7]) == 0


def test_biases_that_are_not_finite():
    l = logits_of(50, 24, torch.float32)
    b = bias_of(24)
    b[3], b[10], b[20], b[5] = -math.inf, float("nan"), 1e38, -1e38
    for best in (1, 2):
        r = check(l, 4, True, "sigmoid", b, 4, 2, best)
        assert (r["ids"][:, 0] == 20).all() and not ((r["ids"] == 3) | (r["ids"] == 10)).any()
    b[21] = math.inf
    r = bra.moe_route(l, 4, score="sigmoid", bias=b)
    assert (r["ids"][:, 0] == 21).all() and (r["ids"][:, 1] == 20).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_borders_are_decided_in_64_bits(score, dt):
    """Biases that put neighbours a few 2^-24 or 2^-40 apart, among them and across groups."""
    T, E, k = 400, 64, 6
    l = logits_of(T, E, dt, ties=True)
    l = torch.where(l == 0, l, l * 4)                        # saturates: 1 - 2^-17 and closer
    for step in (2.0 ** -24, 2.0 ** -26, 2.0 ** -40, 0.0):
        b = torch.arange(E, device="cuda").flip(0) * step
        for best in (1, 2):
            check(l, k, True, score, b, 8, 3, best)
            check(l, k, False, score, b)
        check(l, k, True, score, None, 8, 3, 2)


@pytest.mark.parametrize("E", [16, 64, 200, 512])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_better_one_behind_ties(E, dt):
    """The last chosen and the first ones left out are a tie; one behind them is better by less
    than 32 bits hold."""
    for ties in (2, 3, 9):
        l = torch.full((3, E), -3.0, dtype=dt, device="cuda")
        l[:, 0] = 5.0
        l[:, 1:ties + 2] = 1.0
        b = torch.zeros(E, device="cuda")
        b[1:ties + 1] = 0.25
        b[ties + 1] = torch.nextafter(torch.tensor(0.25), torch.tensor(1.0))
        for k in (2, min(3, ties)):
            r = check(l, k, True, "sigmoid", b)
            assert (r["ids"][:, 1] == ties + 1).all()
            check(l, k, False, "softmax", b)
    if dt == torch.float32:                               # without a bias: logits one unit apart
        l = torch.full((3, E), -3.0, device="cuda")
        l[:, 2:8] = 1.0
        l[:, 9] = torch.nextafter(torch.tensor(1.0), torch.tensor(2.0))
        assert (check(l, 1, True, "sigmoid")["ids"] == 9).all()
        assert (check(l, 2, True, "softmax", scale=2.0)["ids"][:, 0] == 9).all()


@pytest.mark.parametrize("offset", [0.0, 100.0, -1000.0, 1e6])
@pytest.mark.parametrize("E,G,top", [(64, 8, 3), (510, 3, 1), (256, 16, 5)])
def test_groups_of_scores_of_large_logits(E, G, top, offset):
    """Group sums of softmax scores whose logits are large: their last bits count."""
    l = logits_of(4000, E, torch.float32) * 0.1 + offset
    check(l, 4, True, "softmax", None, G, top, 2)


@pytest.mark.parametrize("T", [64, 5000, 131073, 170000])
def test_many_tokens(T):
    """One chunk, several, and as many as are summed by a launch of their own."""
    E, k = 24, 3
    check(logits_of(T, E, torch.bfloat16), k, True, "sigmoid", bias_of(E), 4, 2, 2, 2.5,
          torch.randn((T, k), device="cuda"))


def test_the_plain_route_by_scores():
    """softmax without bias and groups is moe_route; all groups kept are none."""
    l, dw = logits_of(700, 40, torch.float32), torch.randn((700, 4), device="cuda")
    for renorm in (True, False):
        a = bra.moe_route(l, 4, renormalize=renorm)
        b = bra.moe_route(l, 4, renormalize=renorm, groups=8, top_groups=8)
        c = bra.moe_route(l, 4, renormalize=renorm, scale=2.0)
        for n in ("ids", "counts", "slots", "tokens"):
            assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n])
        assert torch.allclose(a["weights"] * 2, c["weights"], rtol=1e-5, atol=0)
        assert torch.allclose(a["weights"], b["weights"], rtol=1e-5, atol=0)
        d = [bra.moe_route_grad(dw, l, r["ids"], r["weights"], renormalize=renorm, scale=s)
             for r, s in ((a, 1.0), (c, 2.0))]
        assert torch.allclose(d[0] * 2, d[1], rtol=1e-4, atol=1e-6)


def test_gradient_against_differences():
    T, E, k = 30, 32, 4
    l = logits_of(T, E, torch.float32).double()
    b, dw = bias_of(E, step=0.01), torch.randn((T, k), device="cuda")
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            r = bra.moe_route(l.float(), k, renormalize=renorm, score=score, bias=b, groups=4,
                              top_groups=2, scale=2.5)
            ids = r["ids"].long()

            def loss(z):
                p = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
                w = p.gather(1, ids)
                return ((w / w.sum(1, keepdim=True) if renorm else w) * 2.5 * dw.double()).sum(1)
            dl = bra.moe_route_grad(dw, l.float(), r["ids"], r["weights"], renormalize=renorm,
                                    score=score, scale=2.5).double()
            for i in range(E):
                h = torch.zeros_like(l)
                h[:, i] = 1e-5
                d = (loss(l + h) - loss(l - h)) / 2e-5
                assert torch.allclose(dl[:, i], d, rtol=1e-4, atol=1e-5)


def test_a_graph_follows_logits_and_bias():
    l, b = logits_of(900, 64, torch.bfloat16), bias_of(64)
    plan = bra.moe_route_plan(l, 6, score="sigmoid", bias=b, groups=8, top_groups=4)
    want = bra.moe_route_plan(l, 6, score="sigmoid", bias=b, groups=8, top_groups=4)
    plan.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for seed in range(3):
        l.copy_(logits_of(900, 64, torch.bfloat16, seed + 5))
        b.copy_(bias_of(64, seed + 9))
        graph.replay()
        r = want.run()
        for n in r:
            assert torch.equal(plan.result[n], r[n]), n


def test_two_streams():
    l, b = logits_of(3000, 256, torch.float32), bias_of(256)
    kw = dict(score="sigmoid", bias=b, groups=8, top_groups=4)
    want = bra.moe_route(l, 8, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[bra.moe_route(l, 8, stream=s, **kw) for s in streams] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(r[n], want[n]) for pair in got for r in pair for n in want)


def test_refusals():
    l, b = logits_of(10, 24, torch.float32), bias_of(24)
    for bad in (dict(groups=5), dict(groups=0), dict(groups=33), dict(groups=4, top_groups=5),
                dict(groups=4, top_groups=0), dict(groups=4, top_groups=2, group_best=3),
                dict(scale=0.0), dict(scale=math.inf), dict(scale=math.nan), dict(scale=1e-38)):
        with pytest.raises(bra.BraError):
            bra.moe_route(l, 3, **bad)
    with pytest.raises(bra.BraError):
        bra.moe_route(l, 25, score="sigmoid")
    for bad in (dict(score="tanh"), dict(bias=b[:20]), dict(bias=b.cpu()), dict(groups=1 << 31)):
        with pytest.raises(ValueError):
            bra.moe_route(l, 3, **bad)
    with pytest.raises(TypeError):
        bra.moe_route(l, 3, bias=b.double())
    with pytest.raises(TypeError):
        bra.moe_route(l.double(), 3, score="sigmoid")
    r = bra.moe_route(l, 3, score="sigmoid")
    for bad in (dict(score="tanh"), ):
        with pytest.raises(ValueError):
            bra.moe_route_grad(r["weights"], l, r["ids"], r["weights"], **bad)
    with pytest.raises(bra.BraError):
        bra.moe_route_grad(r["weights"], l, r["ids"], r["weights"], scale=0.0)
    with pytest.raises(bra.BraError):                        # one buffer as two outputs
        bra.moe_route(l, 3, score="sigmoid", ids=r["slots"], slots=r["slots"])
    wide = torch.zeros(54, device="cuda")                    # weights over the bias
    with pytest.raises(bra.BraError):
        bra.moe_route(l, 3, score="sigmoid", bias=wide[:24], weights=wide[20:50].view(10, 3))
