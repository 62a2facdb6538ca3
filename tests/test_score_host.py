"""Host-side tests of the router by scores (no GPU needed, no kernel launched)."""
import ctypes
import math
import pathlib
import re

import pytest

import bmm_reducescatter_alltoall_gb300 as bra
from bmm_reducescatter_alltoall_gb300._build import CSRC, code_text

NULLPTR, INVALID = bra.ERR_NULLPTR, bra.ERR_INVALID
# stand-in addresses, never dereferenced by a refused call
L, B, I, W, C, S, K, WS = (0x10000000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module")
def lib():
    return bra.library()


def args(**kw):
    a = bra.ScoreArgs()
    base = dict(tokens=100, experts=64, choices=4, dtype=bra.BF16, renormalize=1, score=1, groups=8,
                top_groups=4, group_best=2, scale=2.5)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def test_struct_layout():
    assert ctypes.sizeof(bra.ScoreArgs) == 56 and bra.ScoreArgs.scale.offset == 48


def test_workspace_is_the_plain_routers(lib):
    for T in (0, 1, 64, 65, 5000, 1 << 20):
        r = bra.RouteArgs()
        r.tokens, r.experts, r.choices, r.dtype = T, 64, 4, bra.BF16
        assert lib.moe_route_scored_workspace_size(args(tokens=T)) == \
            lib.moe_route_workspace_size(ctypes.byref(r))


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(tokens=1 << 31), dict(tokens=1 << 30), dict(experts=0), dict(experts=520),
    dict(choices=0), dict(choices=17), dict(experts=8, choices=9), dict(dtype=bra.INT8), dict(score=2),
    dict(score=-1), dict(groups=0), dict(groups=-8), dict(groups=7), dict(groups=64), dict(top_groups=0),
    dict(top_groups=9), dict(group_best=0), dict(group_best=3), dict(scale=0.0), dict(scale=math.nan),
    dict(scale=math.inf), dict(scale=2.0 ** -101), dict(scale=-(2.0 ** 101)), dict(reserved=1),
], ids=str)
def test_refused_sizes(lib, change):
    assert lib.moe_route_scored_workspace_size(args(**change)) == -INVALID
    assert lib.moe_route_scored(L, B, I, W, C, S, K, WS, 1 << 40, args(**change), None) == INVALID
    assert lib.moe_route_scored_grad(W, L, I, S, K, args(**change), None) == INVALID


def test_refused_pointers(lib):
    ok = [L, B, I, W, C, S, K, WS]
    run = lambda p, n=1 << 20: lib.moe_route_scored(*p, n, args(), None)        # noqa: E731
    for i in range(8):
        bad = list(ok)
        if i != 1:
            bad[i] = None
            assert run(bad) == NULLPTR, i
        bad[i] = ok[i] + 1
        assert run(bad) == INVALID, i
        if i != 1:
            bad[i] = B                               # an output (or the logits' row) over the bias
            assert i == 0 or run(bad) == INVALID, i
    assert run(ok, 0) == INVALID
    assert lib.moe_route_scored(*ok, 0, None, None) == NULLPTR
    assert lib.moe_route_scored_workspace_size(None) == -NULLPTR
    good = [W, L, I, S, K]
    for i in range(5):
        bad = list(good)
        bad[i] = None
        assert lib.moe_route_scored_grad(*bad, args(), None) == NULLPTR, i
        bad[i] = good[i] + 1
        assert lib.moe_route_scored_grad(*bad, args(), None) == INVALID, i
        bad[i] = K
        assert i == 4 or lib.moe_route_scored_grad(*bad, args(), None) == INVALID, i
    assert lib.moe_route_scored_grad(W, None, I, S, K, args(score=0, renormalize=0), None) == NULLPTR


def layout(E, groups):
    """The lanes of a token as the source's rule lays them out."""
    g = 1 << (groups - 1).bit_length()
    for i in range(6):
        lanes_all, most = (4 << i if i < 4 else 32), (8 if i < 4 else 16 if i == 4 else 32)
        if lanes_all < g:
            continue
        lanes = lanes_all // g
        per = -(-(-(-(E // groups) // lanes)) // 4) * 4
        if per <= most or i == 5:
            return lanes_all, most, lanes, per


def test_every_expert_has_a_lane():
    text = code_text((pathlib.Path(CSRC) / "moe_score.cu").read_bytes()).decode()
    assert re.search(r"per = \(\(size \+ lanes - 1\) / lanes \+ 3\) / 4 \* 4", text)
    for groups in range(1, bra.MAX_EXPERT_GROUPS + 1):
        for E in range(groups, bra.MAX_GROUPS + 1, groups):
            width, most, lanes, per = layout(E, groups)
            assert per <= most and width <= 32 and E <= width * most
            size, seen = E // groups, []
            for lane in range(width):
                g, off = lane // lanes, (lane % lanes) * per
                if g < groups:
                    seen += [g * size + i for i in range(off, min(off + per, size))]
            assert seen == list(range(E)), (E, groups)


def test_kernels_of_the_router_read_with_loads_that_see_writes():
    for name in ("route.cuh", "moe_score.cu"):
        text = code_text((pathlib.Path(CSRC) / name).read_bytes()).decode()
        assert not re.search(r"__ldg\b|__restrict__|ld\.global[\w.]*\.nc\b", text), name
