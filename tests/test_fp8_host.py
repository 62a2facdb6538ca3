"""Host-side tests of the 8-bit block-scaled operators (no GPU needed, no kernel launched): buffer
sizes, calls that must be refused before any launch, and the rules of their sources."""
import ctypes
import os
import re

import pytest

import bmm_reducescatter_alltoall_gb300 as bra
from bmm_reducescatter_alltoall_gb300._build import CSRC, KERNEL_SOURCES, code_text

NULLPTR, INVALID, UNSUPPORTED = bra.ERR_NULLPTR, bra.ERR_INVALID, bra.ERR_UNSUPPORTED

# stand-in addresses, never dereferenced by a refused call
X, XS, W, WS, B, C, Y = (0x10000000 * (i + 1) for i in range(7))


@pytest.fixture(scope="module")
def lib():
    return bra.library()


def fill(a, base, kw):
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def conv(**kw):
    return fill(bra.Fp8Args(), dict(rows=16, k=200, groups=4, dtype=bra.FP16), kw)


def prod(**kw):
    return fill(bra.Fp8ProductArgs(), dict(rows=16, groups=4, in_=200, out=72, dtype=bra.FP16), kw)


def test_struct_layouts():
    assert ctypes.sizeof(bra.Fp8Args) == 56 and bra.Fp8Args.status.offset == 48
    assert ctypes.sizeof(bra.Fp8ProductArgs) == 64 and bra.Fp8ProductArgs.y_pitch.offset == 48


def test_buffer_sizes(lib):
    code, scale = lib.fp8_code_bytes, lib.fp8_scale_bytes
    assert code(conv()) == 16 * 208 and code(conv(k=1)) == 16 * 16 and code(conv(k=16)) == 16 * 16
    assert scale(conv()) == 16 * 4 * 4 and scale(conv(k=513)) == 16 * 8 * 4
    w = dict(rows=4 * 130, rows_per_group=130)
    assert code(conv(**w)) == 520 * 208 and scale(conv(**w)) == 4 * 2 * 2 * 4
    assert code(conv(rows=0)) == 0 and scale(conv(rows=0)) == 0
    assert code(conv(k=0)) == -INVALID and scale(conv(rows=15, rows_per_group=4)) == -INVALID
    assert code(None) == -NULLPTR


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(rows=(1 << 31) - 65535), dict(k=0), dict(k=(1 << 24) + 1), dict(groups=0),
    dict(groups=513), dict(rows_per_group=3), dict(rows_per_group=-4), dict(dtype=bra.INT8),
    dict(format=2), dict(format=-1), dict(x_pitch=199), dict(x_pitch=(1 << 36) + 1), dict(status=Y + 2),
    dict(rows=(1 << 31) - (1 << 16), x_pitch=1 << 36),
], ids=str)
def test_conversions_refuse_sizes(lib, change):
    assert lib.fp8_quantize(X, None, W, WS, conv(**change), None) == INVALID
    assert lib.fp8_dequantize(W, WS, None, X, conv(**change), None) == INVALID


def test_conversions_refuse_pointers(lib):
    ok = [X, C, W, WS]
    for i in (0, 2, 3):
        bad = list(ok)
        bad[i] = None
        assert lib.fp8_quantize(*bad, conv(), None) == NULLPTR, i
    for i, by in ((0, 1), (1, 4), (2, 8), (3, 8)):
        bad = list(ok)
        bad[i] += by
        assert lib.fp8_quantize(*bad, conv(), None) == INVALID, i
        assert lib.fp8_dequantize(bad[2], bad[3], bad[1], bad[0], conv(), None) == INVALID, i
    assert lib.fp8_quantize(X + 2, None, W, WS, conv(dtype=bra.FP32), None) == INVALID
    for bad in ((X, C, X, WS), (X, C, W, X + 16), (X, C, W, W), (X, C, C, WS), (X, C, W, C)):
        assert lib.fp8_quantize(*bad, conv(), None) == INVALID
    for y in (W, WS, C):
        assert lib.fp8_dequantize(W, WS, C, y, conv(), None) == INVALID
    assert lib.fp8_quantize(X, C, W, WS, conv(rows=64, rows_per_group=16), None) == INVALID
    assert lib.fp8_dequantize(W, WS, None, X, conv(x_pitch=200), None) == INVALID
    assert lib.fp8_quantize(X, None, W, WS, None, None) == NULLPTR
    assert lib.fp8_quantize(None, None, None, None, conv(rows=0), None) == 0


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(rows=(1 << 31) - 65535), dict(groups=0), dict(groups=513), dict(in_=0),
    dict(out=0), dict(out=(1 << 24) + 1), dict(dtype=bra.FP32), dict(x_format=2), dict(w_format=-1),
    dict(reserved=1), dict(y_pitch=71), dict(y_pitch=(1 << 36) + 1), dict(status=Y + 1),
    dict(rows=(1 << 31) - (1 << 16), y_pitch=1 << 36),
], ids=str)
def test_products_refuse_sizes(lib, change):
    assert lib.fp8_grouped_matmul(X, XS, W, WS, B, C, Y, prod(**change), None) == INVALID
    assert lib.fp8_grouped_matmul_grad(X, XS, W, WS, C, Y, prod(**change), None) == INVALID


def test_products_refuse_pointers(lib):
    ok = [X, XS, W, WS, B, C, Y]
    forward = lambda p: lib.fp8_grouped_matmul(*p, prod(), None)                       # noqa: E731
    back = lambda p: lib.fp8_grouped_matmul_grad(*p[:4], *p[5:], prod(y_pitch=200), None)  # noqa: E731
    for i in range(7):
        bad = list(ok)
        bad[i] = None
        if i != 4:
            assert forward(bad) == NULLPTR and back(bad) == NULLPTR, i
        bad[i] = ok[i] + 1
        assert forward(bad) == INVALID, i
        if i != 4:
            assert back(bad) == INVALID, i
        if i != 6:
            over = ok[:6] + [ok[i]]
            assert forward(over) == INVALID and (i == 4 or back(over) == INVALID), i
    assert lib.fp8_grouped_matmul(X + 8, XS, W, WS, B, C, Y, prod(), None) == INVALID
    assert lib.fp8_grouped_matmul(X, XS + 4, W, WS, B, C, Y, prod(), None) == INVALID
    assert lib.fp8_grouped_matmul(X, XS, W, WS, B + 2, C, Y, prod(dtype=bra.BF16), None) == INVALID
    assert lib.fp8_grouped_matmul(*ok, None, None) == NULLPTR
    assert lib.fp8_grouped_matmul(None, None, W, WS, None, C, None, prod(rows=0), None) == 0


def launched_by(word):
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            with open(os.path.join(CSRC, name), "rb") as f:
                text = re.sub(r'"\s*"', "", code_text(f.read()).decode())
            if word in text:
                yield name, text


def test_overlapped_kernels_read_with_loads_that_see_writes():
    """Kernels launched through launch_clusters may begin while their inputs are still written."""
    found = dict(launched_by("launch_clusters"))
    assert {"fp8_quant.cu", "fp8_tc.cu"} <= set(found)
    for name, text in found.items():
        assert not re.search(r"__ldg\b|__restrict__|__restrict\b|ld\.global[\w.]*\.nc\b", text), name
        for body in re.split(r"__global__", text)[1:]:
            assert "grid_wait();" in body, (name, body[:80])


def test_kernels_name_their_sources():
    for kernel, source in KERNEL_SOURCES.items():
        with open(os.path.join(CSRC, source)) as f:
            assert re.search(r"\b%s\b" % kernel, f.read()), kernel


def test_register_split_fits_the_launch():
    """A split whose sum passes the launch's registers would wait for ever."""
    (_, text), = launched_by("setmaxnreg")
    get = lambda n: int(re.search(n + r" = (\d+)", text).group(1))          # noqa: E731
    launch, role, epi = get("LAUNCH_REGS"), get("ROLE_REGS"), get("EPI_REGS")
    assert 128 * role + 256 * epi <= 384 * launch <= 65536
    assert role % 8 == 0 and epi % 8 == 0 and 24 <= role and epi <= 256
