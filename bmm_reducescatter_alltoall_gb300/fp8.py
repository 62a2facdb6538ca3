"""8-bit floating point with a scale to each block of 128: conversions and the
products grouped by expert.

Bindings of include/bra_moe.h in the manner of moe.py: each function has a
`_plan` form that checks its tensors once, and the one-shot form is that plan
run once.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import bmm_reducescatter_alltoall_gb300 as _bra

from .moe import _bias_dtype, _counts, _dense, _on, _ptr, _row_dtype, _rows, _same_device, _status

__all__ = ["E4M3", "E5M2", "Fp8Args", "Fp8ProductArgs", "Fp8Tensor", "fp8_quantize",
           "fp8_quantize_plan", "fp8_dequantize", "fp8_dequantize_plan", "fp8_grouped_matmul",
           "fp8_grouped_matmul_plan", "fp8_grouped_matmul_grad", "fp8_grouped_matmul_grad_plan"]

E4M3, E5M2 = 0, 1


class Fp8Args(ctypes.Structure):
    """bra_fp8_args of the C header."""
    _fields_ = [("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("rows_per_group", ctypes.c_int64), ("x_pitch", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("format", ctypes.c_int32),
                ("status", ctypes.c_void_p)]


class Fp8ProductArgs(ctypes.Structure):
    """bra_fp8_product_args of the C header."""
    _fields_ = [("rows", ctypes.c_int64), ("groups", ctypes.c_int64), ("in_", ctypes.c_int64),
                ("out", ctypes.c_int64), ("dtype", ctypes.c_int32), ("x_format", ctypes.c_int32),
                ("w_format", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("y_pitch", ctypes.c_int64), ("status", ctypes.c_void_p)]


def declare(lib) -> None:
    """Argument types of the library's functions (called once when it is loaded)."""
    vp, i64, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    ap, pp = ctypes.POINTER(Fp8Args), ctypes.POINTER(Fp8ProductArgs)
    for fn in (lib.fp8_code_bytes, lib.fp8_scale_bytes):
        fn.argtypes, fn.restype = [ap], i64
    for fn in (lib.fp8_quantize, lib.fp8_dequantize):
        fn.argtypes, fn.restype = [vp, vp, vp, vp, ap, vp], c_int
    lib.fp8_grouped_matmul.argtypes = [vp, vp, vp, vp, vp, vp, vp, pp, vp]
    lib.fp8_grouped_matmul_grad.argtypes = [vp, vp, vp, vp, vp, vp, pp, vp]
    lib.fp8_grouped_matmul.restype = lib.fp8_grouped_matmul_grad.restype = c_int


def _format(dt) -> int:
    torch = _bra._torch()
    codes = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
    if dt not in codes:
        raise TypeError(f"8-bit codes are float8_e4m3fn or float8_e5m2, got {dt}")
    return codes[dt]


class Fp8Tensor:
    """Rows or weights in 8-bit block-scaled floating point (fp8_quantize, or
    a checkpoint's).

    shape: (R, K), or (E, N, K) for weights.  codes: float8_e4m3fn or
    float8_e5m2, rows of K codes at a pitch of ceil(K / 16) * 16.  scales:
    float32; of rows (R, S), S = ceil(K / 128) rounded up to a multiple of 4;
    of weights (E, ceil(N / 128), ceil(K / 128)).  A value is its code times
    its block's scale, which may be any float."""

    def __init__(self, codes, scales, shape):
        self.codes, self.scales, self.shape = codes, scales, tuple(shape)
        self._checked = None             # the parts that _holds has found to fit

    def _parts(self):
        return self.codes, self.scales, self.shape

    @property
    def device(self):
        return self.codes.device

    @property
    def format(self):
        return self.codes.dtype

    def _args(self, format) -> Fp8Args:
        a = Fp8Args()
        a.k = self.shape[-1]
        a.groups = 1
        a.rows = self.shape[0]
        if len(self.shape) == 3:
            a.groups, a.rows_per_group = self.shape[0], self.shape[1]
            a.rows = a.groups * a.rows_per_group
        a.format = _format(format)
        return a

    def _needs(self, format):
        """Bytes of the codes and of the scales."""
        a, lib = self._args(format), _bra.library()
        needs = lib.fp8_code_bytes(ctypes.byref(a)), lib.fp8_scale_bytes(ctypes.byref(a))
        if min(needs) < 0:
            raise _bra.BraError(-min(needs), f"8-bit tensor of shape {self.shape}")
        return needs


def _holds(t: Fp8Tensor, what: str) -> None:
    """Checks that the buffers of an Fp8Tensor hold what it says: once for the same tensors, which
    have to keep their storage, as those of a Plan."""
    if t._checked is not None and all(a is b for a, b in zip(t._checked, t._parts())):
        return
    torch = _bra._torch()
    if len(t.shape) not in (2, 3):
        raise ValueError(f"{what} must hold rows (R, K) or weights (E, N, K), got {t.shape}")
    _bra._dev_tensor(t.codes, f"{what}'s codes")
    _bra._dev_tensor(t.scales, f"{what}'s scales", torch.float32)
    needs = t._needs(t.codes.dtype)
    for part, buf, need in zip(("codes", "scales"), (t.codes, t.scales), needs):
        n = buf.numel() * buf.element_size()
        if n < need:
            raise ValueError(f"{what}'s {part} have {n} bytes, {t.shape} takes {need}")
    if t.codes.device != t.scales.device:
        raise ValueError(f"{what}'s codes and scales must be on one device")
    t._checked = t._parts()


def fp8_quantize_plan(x, counts=None, format=None, out: Optional[Fp8Tensor] = None, status=None):
    """fp8_quantize prepared once (see Plan); plan.run() returns the Fp8Tensor."""
    torch = _bra._torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    code = _row_dtype(x.dtype, "fp8_quantize")
    if x.dim() == 3:
        _bra._dev_tensor(x, "x")
        pitch = 0
        if counts is not None:
            raise ValueError("counts are for rows (R, K); weights are quantized whole")
        if x.shape[0] < 1 or x.shape[1] < 1:
            raise ValueError(f"weights must have matrices and rows, got shape {tuple(x.shape)}")
    else:
        pitch = _rows(x, "x")
    if x.shape[-1] == 0:
        raise ValueError("x has rows of no elements")
    if counts is not None:
        _counts(counts)
    if format is None:
        format = out.format if out is not None else torch.float8_e4m3fn
    shape = tuple(x.shape)
    if out is None:
        probe = Fp8Tensor(None, None, shape)
        cb, sb = probe._needs(format)
        new = lambda n, dt: torch.empty(n, dtype=dt, device=x.device)      # noqa: E731
        blocks = lambda n: -(-n // 128)                                    # noqa: E731
        rows = shape[:1] if x.dim() == 2 else (shape[0], blocks(shape[1]))
        per = -(-blocks(shape[-1]) // 4) * 4 if x.dim() == 2 else blocks(shape[-1])
        out = Fp8Tensor(new(cb, torch.uint8).view(format).view(shape[:-1] + (-(-shape[-1] // 16) * 16,)),
                        new(sb // 4, torch.float32).view(rows + (per,)), shape)
        out._checked = out._parts()
    else:
        if out.shape != shape or out.format != format:
            raise ValueError(f"out holds {out.shape} in {out.format}, expected {shape} in {format}")
        _holds(out, "out")
    _same_device(x, out.codes, out.scales, counts, status)
    a = out._args(format)
    if counts is not None:
        a.groups = counts.numel()
    a.x_pitch, a.dtype, a.status = pitch, code, _status(status)
    args = (_ptr(x), _ptr(counts), _ptr(out.codes), _ptr(out.scales), ctypes.byref(a))
    return _bra.Plan(_bra.library().fp8_quantize, args, "fp8_quantize", out, (x, counts, a, status))


def fp8_quantize(x, counts=None, format=None, out: Optional[Fp8Tensor] = None, status=None,
                 stream=None) -> Fp8Tensor:
    """x (fp16, bf16 or fp32) in 8-bit floating point with a scale to each block.

    Rows (R, K), of any pitch: a scale to each 128 elements of a row; with
    `counts` (CUDA int64) rows past their sum are left out.  Weights (E, N,
    K): a scale to each 128 x 128.  format: torch.float8_e4m3fn (default) or
    float8_e5m2.  The scale is the smallest power of two (2^-126 at least) at
    which the block's values stay within the format; codes are the nearest,
    ties to even.  A block with a NaN or an infinity becomes NaN."""
    with _on(stream):
        return fp8_quantize_plan(x, counts, format, out, status).run()


def fp8_dequantize_plan(q: Fp8Tensor, dtype, counts=None, out=None, status=None):
    """fp8_dequantize prepared once (see Plan); plan.run() returns out."""
    torch = _bra._torch()
    if not isinstance(q, Fp8Tensor):
        raise TypeError("q must be an Fp8Tensor")
    code = _row_dtype(dtype, "fp8_dequantize")
    _holds(q, "q")
    if counts is not None:
        _counts(counts)
        if len(q.shape) != 2:
            raise ValueError("counts are for rows (R, K)")
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    _dense(out, "out", dtype, q.shape)
    _same_device(q.codes, out, counts, status)
    a = q._args(q.format)
    if counts is not None:
        a.groups = counts.numel()
    a.dtype, a.status = code, _status(status)
    args = (_ptr(q.codes), _ptr(q.scales), _ptr(counts), _ptr(out), ctypes.byref(a))
    return _bra.Plan(_bra.library().fp8_dequantize, args, "fp8_dequantize", out,
                     (q, counts, a, status))


def fp8_dequantize(q: Fp8Tensor, dtype, counts=None, out=None, status=None, stream=None):
    """The values of an Fp8Tensor as fp16, bf16 or fp32: code times scale in
    fp32, rounded to dtype.  With `counts` rows past their sum are not written."""
    with _on(stream):
        return fp8_dequantize_plan(q, dtype, counts, out, status).run()


def _product_plan(rows: Fp8Tensor, weight: Fp8Tensor, counts, bias, out, dtype, status, grad: bool):
    torch = _bra._torch()
    name, what = ("fp8_grouped_matmul_grad", "dy") if grad else ("fp8_grouped_matmul", "x")
    if not isinstance(rows, Fp8Tensor) or not isinstance(weight, Fp8Tensor):
        raise TypeError(f"{what} and weight must be Fp8Tensors (fp8_quantize)")
    if len(rows.shape) != 2 or len(weight.shape) != 3:
        raise ValueError(f"{what} must hold rows and weight matrices (E, N, K)")
    E, N, K = weight.shape
    takes, gives = (N, K) if grad else (K, N)
    R = rows.shape[0]
    if rows.shape[1] != takes:
        raise ValueError(f"{what} has rows of {rows.shape[1]}, weight takes {takes}")
    _counts(counts, E)
    _holds(rows, what)
    _holds(weight, "weight")
    dt = dtype if dtype is not None else out.dtype if out is not None else torch.bfloat16
    code = _bra._fused_dtype(dt)
    if bias is not None:
        _dense(bias, "bias", _bias_dtype(dt), (E, gives))
    if out is None:
        out = torch.empty((R, gives), dtype=dt, device=rows.device)
    pitch = _rows(out, "out", dt, (R, gives))
    _same_device(rows.codes, weight.codes, counts, bias, out, status)
    a = Fp8ProductArgs()
    a.rows, a.groups, a.in_, a.out, a.dtype = R, E, K, N, code
    a.x_format, a.w_format = _format(rows.format), _format(weight.format)
    a.y_pitch, a.status = pitch, _status(status)
    args = (_ptr(rows.codes), _ptr(rows.scales), _ptr(weight.codes), _ptr(weight.scales)) + \
        (() if grad else (_ptr(bias),)) + (_ptr(counts), _ptr(out), ctypes.byref(a))
    return _bra.Plan(getattr(_bra.library(), name), args, name, out,
                     (rows, weight, counts, bias, a, status))


def fp8_grouped_matmul_plan(x: Fp8Tensor, weight: Fp8Tensor, counts, bias=None, out=None, dtype=None,
                            status=None):
    """fp8_grouped_matmul prepared once (see Plan); plan.run() returns out."""
    return _product_plan(x, weight, counts, bias, out, dtype, status, False)


def fp8_grouped_matmul(x: Fp8Tensor, weight: Fp8Tensor, counts, bias=None, out=None, dtype=None,
                       status=None, stream=None):
    """grouped_matmul on 8-bit operands: y[r] = x[r] @ weight[e].T + bias[e].

    x: rows (R, K); weight: (E, N, K), quantized or a checkpoint's, in any of
    the two formats each.  A block's code products are summed in fp32, times
    both scales, in fp32; one rounding to dtype (bf16 by default, or fp16).
    counts, bias, out, status as grouped_matmul."""
    with _on(stream):
        return fp8_grouped_matmul_plan(x, weight, counts, bias, out, dtype, status).run()


def fp8_grouped_matmul_grad_plan(dy: Fp8Tensor, weight: Fp8Tensor, counts, out=None, dtype=None,
                                 status=None):
    """fp8_grouped_matmul_grad prepared once (see Plan); plan.run() returns out."""
    return _product_plan(dy, weight, counts, None, out, dtype, status, True)


def fp8_grouped_matmul_grad(dy: Fp8Tensor, weight: Fp8Tensor, counts, out=None, dtype=None,
                            status=None, stream=None):
    """Gradient of fp8_grouped_matmul's rows: dx[r] = dy[r] @ weight[e].

    dy: the output's gradient, rows (R, N) quantized along N; weight as there.
    The weight's own gradient contracts over the rows, across their scales:
    grouped_matmul_grad(..., want=("dweight",)) on 16-bit operands."""
    with _on(stream):
        return fp8_grouped_matmul_grad_plan(dy, weight, counts, out, dtype, status).run()
