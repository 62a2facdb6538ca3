"""Host-side tests of include/bra_moe.h (no GPU needed, no kernel launched):
exports, workspace sizes, and calls that must be refused before any launch."""
import ctypes
import os
import pathlib
import re

import pytest

import bmm_reducescatter_alltoall_gb300 as bra

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bra_moe.h")
NULLPTR, INVALID, UNSUPPORTED = bra.ERR_NULLPTR, bra.ERR_INVALID, bra.ERR_UNSUPPORTED

# stand-in addresses, never dereferenced by a refused call
X, W, B, C, Y, G, S = (0x10000000 * (i + 1) for i in range(7))


@pytest.fixture(scope="module")
def lib():
    return bra.library()


def test_every_declared_symbol_is_exported(lib):
    names = re.findall(r"^BRA_API\s+[\w\s\*]+?\b(\w+)\s*\(", pathlib.Path(HEADER).read_text(),
                       flags=re.M)
    assert "grouped_matmul" in names
    for name in names:
        assert hasattr(lib, name), name


def test_limits_match_the_header():
    text = pathlib.Path(HEADER).read_text()
    assert int(re.search(r"#define BRA_MAX_GROUPS (\d+)", text).group(1)) == bra.MAX_GROUPS


def args(**kw):
    a = bra.GroupedArgs()
    base = dict(rows=16, groups=4, in_=64, out=72, dtype=bra.FP16)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


def test_grouped_struct_layout():
    assert ctypes.sizeof(bra.GroupedArgs) == 80
    assert bra.GroupedArgs.workspace.offset == 56 and bra.GroupedArgs.status.offset == 72


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(rows=(1 << 31) - 65535), INVALID), (dict(groups=0), INVALID),
    (dict(groups=513), INVALID), (dict(in_=0), INVALID), (dict(out=0), INVALID),
    (dict(out=(1 << 24) + 1), INVALID), (dict(dtype=bra.FP32), INVALID),
    (dict(x_pitch=63), INVALID), (dict(y_pitch=71), INVALID), (dict(status=S + 1), INVALID),
    (dict(workspace=S + 128, workspace_bytes=1 << 20), INVALID),
    (dict(workspace_bytes=5), INVALID), (dict(in_=65), UNSUPPORTED),
    (dict(in_=65, workspace=S, workspace_bytes=256), INVALID),
], ids=str)
def test_grouped_matmul_refuses(lib, change, code):
    assert lib.grouped_matmul(X, W, B, C, Y, ctypes.byref(args(**change)), None) == code
    if "in_" not in change or change["in_"] == 0:
        assert lib.grouped_matmul_grad(Y, X, W, C, G, None, None, ctypes.byref(args(**change)),
                                       None) == code


def test_grouped_matmul_refuses_pointers(lib):
    a = ctypes.byref(args())
    call = lib.grouped_matmul
    for ptrs in ((None, W, B, C, Y), (X, None, B, C, Y), (X, W, B, None, Y), (X, W, B, C, None)):
        assert call(*ptrs, a, None) == NULLPTR
    assert call(X, W, B, C, Y, None, None) == NULLPTR
    for ptrs in ((X + 1, W, B, C, Y), (X, W + 1, B, C, Y), (X, W, B + 1, C, Y),
                 (X, W, B, C + 4, Y), (X, W, B, C, Y + 1)):
        assert call(*ptrs, a, None) == INVALID
    for y in (X, X + 64, W + 100, B, C):
        assert call(X, W, B, C, y, a, None) == INVALID
    bf = ctypes.byref(args(dtype=bra.BF16))
    assert call(X, W, B + 2, C, Y, bf, None) == INVALID


def test_grouped_matmul_grad_refuses_pointers(lib):
    a = ctypes.byref(args())
    call = lib.grouped_matmul_grad
    assert call(Y, X, W, C, None, None, None, a, None) == NULLPTR
    assert call(None, X, W, C, G, None, None, a, None) == NULLPTR
    assert call(Y, X, None, C, G, None, None, a, None) == NULLPTR
    assert call(Y, None, W, C, None, G, None, a, None) == NULLPTR
    assert call(Y, X, W, C, Y + 64, None, None, a, None) == INVALID      # dx over dy
    assert call(Y, X, W, C, G, G + 64, None, a, None) == INVALID         # dx over dweight
    assert call(Y, X, W, C, None, None, W + 64, a, None) == INVALID      # dbias over weight


def test_pitches_past_64_bits_are_refused(lib):
    """Rows times pitch is an address range: it has to stay in 64 bits."""
    rows, wide = (1 << 31) - (1 << 16), 1 << 36
    for change in (dict(x_pitch=wide), dict(y_pitch=wide)):
        a = ctypes.byref(args(rows=rows, **change))
        assert lib.grouped_matmul(X, W, None, C, Y, a, None) == INVALID
        assert lib.grouped_matmul_grad(Y, X, W, C, G, None, None, a, None) == INVALID
        assert lib.grouped_matmul_workspace_size(X, W, a) == -INVALID
    m = ctypes.byref(mx(rows=rows, rows_per_group=0, x_pitch=wide))
    assert lib.mxfp4_quantize(X, C, W, B, m, None) == INVALID
    assert lib.grouped_matmul_workspace_size(X + 2, W, ctypes.byref(args(x_pitch=wide))) == 16 * 64 * 2


def test_workspace_over_an_input_is_refused(lib):
    """The copies would overwrite what they are made from."""
    def a(at, size):
        return ctypes.byref(args(in_=65, transpose_weight=1, workspace=at, workspace_bytes=size))
    size = lib.grouped_matmul_workspace_size(X, W, a(S, 1 << 20))
    for at in (X, W, B, C, X - size + 256):
        assert lib.grouped_matmul(X, W, B, C, Y, a(at, size), None) == INVALID
    size = lib.grouped_matmul_grad_workspace_size(Y, X, W, 1, 0, a(S, 1 << 20))
    for at in (X, W, C, Y, W - size + 256):                              # dx alone: the weight's copy
        assert lib.grouped_matmul_grad(Y, X, W, C, G, None, None, a(at, size), None) == INVALID


def test_workspace_sizes(lib):
    size = lambda x, w, **kw: lib.grouped_matmul_workspace_size(         # noqa: E731
        x, w, ctypes.byref(args(**kw)))
    assert size(X, W) == 0
    assert size(X + 2, W) == 16 * 64 * 2
    assert size(X, W + 2) == 4 * 64 * 128 * 2
    assert size(X, W, in_=65) == 16 * 128 * 2                            # the weight's rows are N long
    assert size(X, W, in_=65, transpose_weight=1) == 16 * 128 * 2 + 4 * 72 * 128 * 2
    assert size(X, W, x_pitch=67) == 16 * 64 * 2
    assert size(X, W, x_pitch=80) == 0
    assert size(X + 2, W, rows=0) == 0
    assert size(X, W, dtype=7) == -INVALID
    grad = lambda want, **kw: lib.grouped_matmul_grad_workspace_size(    # noqa: E731
        Y, X, W, *want, ctypes.byref(args(**kw)))
    assert grad((1, 1)) == 0
    assert grad((0, 0), out=75) == 0
    assert grad((0, 1), out=75) == 16 * 128 * 2                          # dy
    assert grad((1, 0), out=75) == 16 * 128 * 2 + 4 * 64 * 128 * 2       # dy and the weight
    assert grad((0, 1), in_=65) == 16 * 128 * 2                          # x


def mx(**kw):
    a = bra.MxArgs()
    base = dict(rows=16, k=64, groups=4, rows_per_group=4, dtype=bra.FP16)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


def test_mx_struct_layout():
    assert ctypes.sizeof(bra.MxArgs) == 56 and bra.MxArgs.status.offset == 48


def test_mx_buffer_sizes(lib):
    code = lambda **kw: lib.mxfp4_code_bytes(ctypes.byref(mx(**kw)))     # noqa: E731
    scale = lambda **kw: lib.mxfp4_scale_bytes(ctypes.byref(mx(**kw)))   # noqa: E731
    assert code() == 16 * 32 and code(k=65) == 16 * 48 and code(k=1) == 16 * 16
    assert scale() == 4 * 1024                                  # four groups, one block each
    assert scale(k=257) == 4 * 2048
    assert scale(rows=1000, groups=4, rows_per_group=250) == 8 * 1024
    assert scale(rows=1000, groups=4, rows_per_group=0) == (7 + 4) * 1024
    assert scale(rows=2, groups=4, rows_per_group=0) == 2 * 1024
    assert code(rows=15) == -INVALID and scale(k=0) == -INVALID


@pytest.mark.parametrize("change,code", [
    (dict(rows=15), INVALID), (dict(rows=-4), INVALID), (dict(k=0), INVALID),
    (dict(groups=513, rows=513 * 4), INVALID), (dict(dtype=bra.INT8), INVALID),
    (dict(dtype=bra.FP32), INVALID), (dict(x_pitch=63), INVALID), (dict(reserved=1), INVALID),
    (dict(status=S + 2), INVALID),
], ids=str)
def test_mx_quantize_refuses(lib, change, code):
    assert lib.mxfp4_quantize(X, None, W, B, ctypes.byref(mx(**change)), None) == code
    if change != dict(dtype=bra.FP32):
        assert lib.mxfp4_dequantize(W, B, None, X, ctypes.byref(mx(**change)), None) == code


def test_mx_refuses_pointers(lib):
    a = ctypes.byref(mx())
    for ptrs in ((None, None, W, B), (X, None, None, B), (X, None, W, None)):
        assert lib.mxfp4_quantize(*ptrs, a, None) == NULLPTR
    assert lib.mxfp4_quantize(X, None, W, B, ctypes.byref(mx(rows_per_group=0)), None) == NULLPTR
    for ptrs in ((X + 1, None, W, B), (X, None, W + 8, B), (X, None, W, B + 8), (X, None, X, B),
                 (X, None, W, X), (X, None, W, W)):
        assert lib.mxfp4_quantize(*ptrs, a, None) == INVALID
    g = ctypes.byref(args())
    call = lib.mxfp4_grouped_matmul
    ok = [X, X + 0x1000000, W, W + 0x1000000, B, C, Y]
    for i in (0, 1, 2, 3, 5, 6):
        bad = list(ok)
        bad[i] = None
        assert call(*bad, g, None) == NULLPTR, i
        bad[i] = ok[i] + 1
        assert call(*bad, g, None) == INVALID, i
    for i in range(6):
        assert call(*ok[:6], ok[i], g, None) == INVALID, i          # y over an input
    for change in (dict(transpose_weight=1), dict(x_pitch=64), dict(dtype=bra.FP32)):
        assert call(*ok, ctypes.byref(args(**change)), None) == INVALID


def route(**kw):
    a = bra.RouteArgs()
    base = dict(tokens=100, experts=16, choices=4, dtype=bra.FP32)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


def permute(**kw):
    a = bra.PermuteArgs()
    base = dict(tokens=16, rows=64, choices=4, width=72, dtype=bra.FP16)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


def test_route_limits_and_workspace(lib):
    text = pathlib.Path(HEADER).read_text()
    assert int(re.search(r"#define BRA_MAX_CHOICES (\d+)", text).group(1)) == bra.MAX_CHOICES
    assert ctypes.sizeof(bra.RouteArgs) == 32 and ctypes.sizeof(bra.PermuteArgs) == 40
    size = lambda **kw: lib.moe_route_workspace_size(ctypes.byref(route(**kw)))   # noqa: E731
    assert size(tokens=0) == 0 and size(tokens=64) == 0
    assert size(tokens=65) == 256                        # three chunks of 32 tokens, 16 experts
    assert size(tokens=65536, experts=128) == (147 * 128 * 4 + 255) // 256 * 256
    assert size(experts=513) == -INVALID


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(tokens=1 << 31), dict(tokens=1 << 30, choices=2), dict(experts=0),
    dict(experts=513), dict(choices=0), dict(choices=17), dict(experts=3), dict(dtype=bra.INT8),
], ids=str)
def test_route_refuses_sizes(lib, change):
    a = ctypes.byref(route(**change))
    assert lib.moe_route(X, W, B, C, Y, G, S, 1 << 40, a, None) == INVALID
    assert lib.moe_route_grad(B, X, W, C, G, a, None) == INVALID


def test_route_refuses_pointers(lib):
    a = ctypes.byref(route())
    ok = [X, W, B, C, Y, G, S]
    for i in range(7):
        bad = list(ok)
        bad[i] = None
        assert lib.moe_route(*bad, 1 << 20, a, None) == NULLPTR, i
        bad[i] = ok[i] + 2
        assert lib.moe_route(*bad, 1 << 20, a, None) == INVALID, i
    assert lib.moe_route(*ok, 128, a, None) == INVALID                  # workspace too small
    assert lib.moe_route(X, X, B, C, Y, G, S, 1 << 20, a, None) == INVALID
    assert lib.moe_route(X, W, B, C, Y, Y + 64, S, 1 << 20, a, None) == INVALID
    g = [B, X, W, C, G]
    for i in (0, 2, 3, 4):
        bad = list(g)
        bad[i] = None
        assert lib.moe_route_grad(*bad, a, None) == NULLPTR, i
    assert lib.moe_route_grad(B, None, W, C, G, a, None) == NULLPTR     # needed: not renormalised
    assert lib.moe_route_grad(B, X, W, C, X, a, None) == INVALID
    assert lib.moe_route(X, W, B, C, Y, G, S, 1 << 20, None, None) == NULLPTR


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(rows=1 << 31), dict(choices=0), dict(choices=17), dict(width=0),
    dict(width=(1 << 24) + 1), dict(dtype=bra.INT8), dict(reserved=1),
], ids=str)
def test_permute_refuses_sizes(lib, change):
    a = ctypes.byref(permute(**change))
    assert lib.moe_dispatch(X, W, Y, None, 0, a, None) == INVALID
    assert lib.moe_dispatch_grad(X, W, Y, a, None) == INVALID
    assert lib.moe_combine(X, W, B, Y, a, None) == INVALID
    assert lib.moe_combine_grad(X, W, B, C, None, Y, G, a, None) == INVALID


def test_permute_refuses_pointers(lib):
    a = ctypes.byref(permute())
    dispatch = lambda x, tokens, xs, a, s: lib.moe_dispatch(x, tokens, xs, None, 0, a, s)  # noqa: E731
    calls = [(dispatch, [X, W, Y]), (lib.moe_dispatch_grad, [X, W, Y]),
             (lib.moe_combine, [X, W, B, Y]), (lib.moe_combine_grad, [X, W, B, C, S, Y, G])]
    for fn, ok in calls:
        for i in range(len(ok)):
            bad = list(ok)
            bad[i] = None
            if not (fn is lib.moe_combine_grad and i == 4):             # its tokens may be left out
                assert fn(*bad, a, None) == NULLPTR, (fn, i)
            bad[i] = ok[i] + 1
            assert fn(*bad, a, None) == INVALID, (fn, i)
        bad = list(ok)
        bad[-1] = ok[0]
        assert fn(*bad, a, None) == INVALID                             # an output over an input
        assert fn(*ok, None, None) == NULLPTR


def test_dispatch_workspace(lib):
    size = lambda **kw: lib.moe_dispatch_workspace_size(ctypes.byref(permute(**kw)))      # noqa: E731
    big = dict(tokens=16384, rows=131072, width=4096)
    assert size() == 0 and size(tokens=16384, rows=16384, width=4096) == 0
    assert size(**big) == 16384 * 17 * 4
    assert size(tokens=-1) == -INVALID
    a = ctypes.byref(permute(**big))
    x, t, y, w = 1 << 34, 1 << 35, 1 << 36, 1 << 37
    assert lib.moe_dispatch(x, t, y, None, 0, a, None) == NULLPTR
    assert lib.moe_dispatch(x, t, y, w, 16384 * 17 * 4 - 1, a, None) == INVALID
    assert lib.moe_dispatch(x, t, y, w + 128, 1 << 30, a, None) == INVALID
    assert lib.moe_dispatch(x, t, y, y + 256, 1 << 30, a, None) == INVALID


def test_scale_blocks_hold_every_grouping(lib):
    """The product's map of the rows' scales ends where mxfp4_scale_bytes ends, so no tile may ask
    for a block in between the rows' last one and the map's end: with one group, which may have
    been quantized without counts, the two sizes are the same; with several, some grouping needs
    every block."""
    def blocks(R, E, each):
        return lib.mxfp4_scale_bytes(ctypes.byref(mx(rows=R, groups=E, rows_per_group=each))) // 1024
    for R in list(range(1, 1300)) + [16512, 16513, (1 << 31) - (1 << 16)]:
        assert blocks(R, 1, 0) == blocks(R, 1, R) == -(-R // 128), R
    for E in (2, 3, 8, 512):
        for R in (1, 2, 127, 128, 129, 255, 256, 257, 383, 384, 385, 1000, 4096, 70000):
            few = min(E, R)
            counts = [1] * (few - 1) + [R - few + 1]         # one row here, the rest there
            most = max(sum(-(-n // 128) for n in counts),
                       sum(-(-n // 128) for n in [129] * ((R - 1) // 129) + [R - (R - 1) // 129 * 129])
                       if -(-R // 129) <= E else 0)
            assert most <= blocks(R, E, 0) <= (R + 127 * few) // 128, (R, E)


def test_workspace_of_another_device_is_refused():
    torch = pytest.importorskip("torch")

    class Scratch:
        is_cuda, device = True, torch.device("cuda", 1)
        is_contiguous = staticmethod(lambda: True)
        numel = staticmethod(lambda: 4096)
        element_size = staticmethod(lambda: 1)
        data_ptr = staticmethod(lambda: S)

    a = bra.GroupedArgs()
    with pytest.raises(ValueError):
        bra.moe._take_workspace(Scratch(), 256, torch.device("cuda", 0), a)
    assert not a.workspace
    bra.moe._take_workspace(Scratch(), 256, torch.device("cuda", 1), a)
    assert a.workspace == S and a.workspace_bytes == 4096
    for bad in (5, [1, 2]):
        with pytest.raises(TypeError):
            bra.moe._take_workspace(bad, 256, torch.device("cuda", 0), a)
