"""Ragged expert operators: products grouped by expert with their gradients,
the same on 4-bit weights, the router, and the moves of token rows.

Bindings of include/bra_moe.h in the manner of the package's other calls: each
function has a `_plan` form that checks its tensors once and returns a Plan,
and the one-shot form is that plan run once.  Rows are sorted by expert and
`counts` (CUDA int64, one per expert) says how many each has.

Streams: a one-shot call given a `stream` allocates what it allocates (outputs
and scratch memory) for that stream.  A plan's buffers belong to the stream
that was current when it was made; run on another one, the two have to be
ordered, as with any tensor.  Ordering the inputs is the caller's part.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import bmm_reducescatter_alltoall_gb300 as _bra

__all__ = ["GroupedArgs", "MAX_GROUPS", "grouped_matmul", "grouped_matmul_plan",
           "grouped_matmul_grad", "grouped_matmul_grad_plan", "MxArgs", "MxTensor",
           "mxfp4_quantize", "mxfp4_quantize_plan", "mxfp4_dequantize", "mxfp4_dequantize_plan",
           "mxfp4_grouped_matmul", "mxfp4_grouped_matmul_plan", "MAX_CHOICES", "RouteArgs",
           "PermuteArgs", "ScoreArgs", "MAX_EXPERT_GROUPS", "moe_route", "moe_route_plan", "moe_route_grad", "moe_route_grad_plan",
           "moe_dispatch", "moe_dispatch_plan", "moe_dispatch_grad", "moe_dispatch_grad_plan",
           "moe_combine", "moe_combine_plan", "moe_combine_grad", "moe_combine_grad_plan"]

MAX_GROUPS = 512
MAX_CHOICES = 16
MAX_EXPERT_GROUPS = 32


class GroupedArgs(ctypes.Structure):
    """bra_grouped_args of the C header."""
    _fields_ = [("rows", ctypes.c_int64), ("groups", ctypes.c_int64), ("in_", ctypes.c_int64),
                ("out", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("transpose_weight", ctypes.c_int32), ("x_pitch", ctypes.c_int64),
                ("y_pitch", ctypes.c_int64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64), ("status", ctypes.c_void_p)]


class MxArgs(ctypes.Structure):
    """bra_mx_args of the C header."""
    _fields_ = [("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("rows_per_group", ctypes.c_int64), ("x_pitch", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("status", ctypes.c_void_p)]


class RouteArgs(ctypes.Structure):
    """bra_route_args of the C header."""
    _fields_ = [("tokens", ctypes.c_int64), ("experts", ctypes.c_int64),
                ("choices", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("renormalize", ctypes.c_int32)]


class ScoreArgs(ctypes.Structure):
    """bra_score_args of the C header."""
    _fields_ = [("tokens", ctypes.c_int64), ("experts", ctypes.c_int64),
                ("choices", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class PermuteArgs(ctypes.Structure):
    """bra_permute_args of the C header."""
    _fields_ = [("tokens", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("choices", ctypes.c_int64), ("width", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def declare(lib) -> None:
    """Argument types of the library's functions (called once when it is loaded)."""
    vp, i64, i32, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    gp = ctypes.POINTER(GroupedArgs)
    lib.grouped_matmul.argtypes = [vp, vp, vp, vp, vp, gp, vp]
    lib.grouped_matmul.restype = c_int
    lib.grouped_matmul_grad.argtypes = [vp, vp, vp, vp, vp, vp, vp, gp, vp]
    lib.grouped_matmul_grad.restype = c_int
    lib.grouped_matmul_workspace_size.argtypes = [vp, vp, gp]
    lib.grouped_matmul_workspace_size.restype = i64
    lib.grouped_matmul_grad_workspace_size.argtypes = [vp, vp, vp, c_int, c_int, gp]
    lib.grouped_matmul_grad_workspace_size.restype = i64
    mp = ctypes.POINTER(MxArgs)
    for fn in (lib.mxfp4_code_bytes, lib.mxfp4_scale_bytes):
        fn.argtypes, fn.restype = [mp], i64
    for fn in (lib.mxfp4_quantize, lib.mxfp4_dequantize):
        fn.argtypes, fn.restype = [vp, vp, vp, vp, mp, vp], c_int
    lib.mxfp4_grouped_matmul.argtypes = [vp, vp, vp, vp, vp, vp, vp, gp, vp]
    lib.mxfp4_grouped_matmul.restype = c_int
    rp, pp = ctypes.POINTER(RouteArgs), ctypes.POINTER(PermuteArgs)
    lib.moe_route.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, rp, vp]
    lib.moe_route_workspace_size.argtypes = [rp]
    lib.moe_route_workspace_size.restype = i64
    lib.moe_route_grad.argtypes = [vp, vp, vp, vp, vp, rp, vp]
    sp = ctypes.POINTER(ScoreArgs)
    lib.moe_route_scored.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, sp, vp]
    lib.moe_route_scored_workspace_size.argtypes = [sp]
    lib.moe_route_scored_workspace_size.restype = i64
    lib.moe_route_scored_grad.argtypes = [vp, vp, vp, vp, vp, sp, vp]
    lib.moe_dispatch.argtypes = [vp, vp, vp, vp, i64, pp, vp]
    lib.moe_dispatch_workspace_size.argtypes = [pp]
    lib.moe_dispatch_workspace_size.restype = i64
    lib.moe_dispatch_grad.argtypes = [vp, vp, vp, pp, vp]
    lib.moe_combine.argtypes = [vp, vp, vp, vp, pp, vp]
    lib.moe_combine_grad.argtypes = [vp, vp, vp, vp, vp, vp, vp, pp, vp]
    for fn in (lib.moe_route, lib.moe_route_grad, lib.moe_route_scored, lib.moe_route_scored_grad,
               lib.moe_dispatch, lib.moe_dispatch_grad,
               lib.moe_combine, lib.moe_combine_grad):
        fn.restype = c_int


def _on(stream):
    """A context in which `stream` (torch's, a raw handle or None) is current."""
    if stream is None:
        return contextlib.nullcontext()
    torch = _bra._torch()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _rows(t, what: str, dtype=None, shape=None) -> int:
    """Row pitch of a 2-D CUDA tensor whose rows are contiguous (0 = dense)."""
    torch = _bra._torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (got {t.device})")
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D (got shape {tuple(t.shape)})")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype} (got {t.dtype})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return 0
    r, n = t.shape
    # strides of unit dimensions address nothing
    pitch = t.stride(0) if r > 1 else n
    if (n > 1 and t.stride(1) != 1) or pitch < n:
        raise ValueError(f"{what} must have contiguous rows (got strides {t.stride()})")
    return 0 if pitch == n else pitch


def _dense(t, what: str, dtype, shape):
    _bra._dev_tensor(t, what, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _counts(counts, groups: Optional[int] = None):
    torch = _bra._torch()
    _bra._dev_tensor(counts, "counts", torch.int64)
    if counts.dim() != 1 or (groups is not None and counts.numel() != groups):
        raise ValueError(f"counts must be ({groups if groups is not None else 'E'},), got "
                         f"{tuple(counts.shape)}")
    return counts


def _status(status) -> Optional[int]:
    if status is None:
        return None
    torch = _bra._torch()
    _bra._dev_tensor(status, "status", torch.int32)
    if status.numel() < 1:
        raise ValueError("status must have at least one element")
    return status.data_ptr()


def _same_device(first, *others) -> None:
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError(f"every tensor must be on {first.device} (got {t.device})")


def _take_workspace(workspace, need: int, device, args):
    """Resolves `workspace` ("auto", None or a tensor) against `need` bytes."""
    torch = _bra._torch()
    if need < 0:
        raise _bra.BraError(-need, "workspace size")
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be a CUDA tensor, None or "auto"')
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if workspace is not None:
        if not hasattr(workspace, "data_ptr"):
            raise TypeError('workspace must be a CUDA tensor, None or "auto"')
        if not (workspace.is_cuda and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous CUDA tensor")
        if workspace.device != device:
            raise ValueError(f"workspace must be on {device} (got {workspace.device})")
        if workspace.numel():
            args.workspace = workspace.data_ptr()
            args.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _weight_dims(weight, transpose_weight: bool):
    torch = _bra._torch()
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor")
    if weight.dim() != 3:
        raise ValueError(f"weight must be 3-D (got shape {tuple(weight.shape)})")
    E, a, b = weight.shape
    return (E, b, a) if transpose_weight else (E, a, b)


def _bias_dtype(dt):
    torch = _bra._torch()
    return torch.float16 if dt == torch.float16 else torch.float32


def _grouped_args(R, E, K, N, dt, transpose_weight, xp, yp, status) -> GroupedArgs:
    a = GroupedArgs()
    a.rows, a.groups, a.in_, a.out = R, E, K, N
    a.dtype = _bra._fused_dtype(dt)
    a.transpose_weight = 1 if transpose_weight else 0
    a.x_pitch, a.y_pitch = xp, yp
    a.status = _status(status)
    return a


def grouped_matmul_plan(x, weight, counts, bias=None, out=None, transpose_weight: bool = False,
                        workspace="auto", status=None):
    """grouped_matmul prepared once (see Plan); plan.run() returns out."""
    torch = _bra._torch()
    E, K, N = _weight_dims(weight, transpose_weight)
    dt = weight.dtype
    _bra._fused_dtype(dt)
    _dense(weight, "weight", dt, weight.shape)
    xp = _rows(x, "x", dt)
    if x.shape[1] != K:
        raise ValueError(f"x has rows of {x.shape[1]}, weight takes {K}")
    R = x.shape[0]
    _counts(counts, E)
    if bias is not None:
        _dense(bias, "bias", _bias_dtype(dt), (E, N))
    if out is None:
        out = torch.empty((R, N), dtype=dt, device=x.device)
    yp = _rows(out, "out", dt, (R, N))
    _same_device(x, weight, counts, bias, out, status)
    a = _grouped_args(R, E, K, N, dt, transpose_weight, xp, yp, status)
    lib = _bra.library()
    need = lib.grouped_matmul_workspace_size(_ptr(x), _ptr(weight), ctypes.byref(a))
    workspace = _take_workspace(workspace, need, x.device, a)
    args = (_ptr(x), _ptr(weight), _ptr(bias), _ptr(counts), _ptr(out), ctypes.byref(a))
    return _bra.Plan(lib.grouped_matmul, args, "grouped_matmul", out,
                     (x, weight, bias, counts, a, workspace, status))


def grouped_matmul(x, weight, counts, bias=None, out=None, transpose_weight: bool = False,
                   workspace="auto", status=None, stream=None):
    """y[r] = x[r] @ weight[e] + bias[e] for the rows r of each expert e.

    x: CUDA (R, K), rows sorted by expert (a row-pitched view is read in
    place).  weight: (E, K, N), or (E, N, K) with transpose_weight; fp16 or
    bf16, as x.  counts: CUDA int64 (E,), rows of each expert, on the device;
    their sum may be below R: the rows after it are not written.  bias: None
    or (E, N), fp16 for fp16 and fp32 for bf16.  workspace: scratch memory
    for operands whose rows lack a 16-byte pitch ("auto": from torch's
    allocator, only when needed).  status: optional CUDA int32, ERR_INVALID
    when the counts were refused (nothing is written then).  Returns out
    (R, N), allocated when None.  Asynchronous on `stream`."""
    with _on(stream):
        return grouped_matmul_plan(x, weight, counts, bias, out, transpose_weight, workspace,
                                   status).run()


def grouped_matmul_grad_plan(dy, x, weight, counts, bias=None, dx=None, dweight=None, dbias=None,
                             want=("dx", "dweight", "dbias"), transpose_weight: bool = False,
                             workspace="auto", status=None):
    """grouped_matmul_grad prepared once (see Plan); plan.run() returns its dict."""
    torch = _bra._torch()
    unknown = set(want) - {"dx", "dweight", "dbias"}
    if unknown:
        raise ValueError(f"want takes dx, dweight and dbias (got {sorted(unknown)})")
    E, K, N = _weight_dims(weight, transpose_weight)
    dt = weight.dtype
    _bra._fused_dtype(dt)
    _dense(weight, "weight", dt, weight.shape)
    yp = _rows(dy, "dy", dt)
    R = dy.shape[0]
    if dy.shape[1] != N:
        raise ValueError(f"dy has rows of {dy.shape[1]}, weight gives {N}")
    xp = _rows(x, "x", dt, (R, K))
    _counts(counts, E)
    bdt = _bias_dtype(dt)
    if bias is not None:
        _dense(bias, "bias", bdt, (E, N))
    new = lambda shape, d: torch.empty(shape, dtype=d, device=dy.device)   # noqa: E731
    if "dx" in want:
        dx = _dense(new((R, K), dt) if dx is None else dx, "dx", dt, (R, K))
    elif dx is not None:
        raise ValueError("dx was given and is not wanted")
    if "dweight" in want:
        dweight = _dense(new(tuple(weight.shape), dt) if dweight is None else dweight, "dweight",
                         dt, weight.shape)
    elif dweight is not None:
        raise ValueError("dweight was given and is not wanted")
    if "dbias" in want and (bias is not None or dbias is not None):
        dbias = _dense(new((E, N), bdt) if dbias is None else dbias, "dbias", bdt, (E, N))
    elif dbias is not None:
        raise ValueError("dbias was given and is not wanted")
    if dx is None and dweight is None and dbias is None:
        raise ValueError("no gradient is wanted")
    _same_device(dy, x, weight, counts, bias, dx, dweight, dbias, status)
    a = _grouped_args(R, E, K, N, dt, transpose_weight, xp, yp, status)
    lib = _bra.library()
    need = lib.grouped_matmul_grad_workspace_size(_ptr(dy), _ptr(x), _ptr(weight), dx is not None,
                                                  dweight is not None, ctypes.byref(a))
    workspace = _take_workspace(workspace, need, dy.device, a)
    args = (_ptr(dy), _ptr(x), _ptr(weight), _ptr(counts), _ptr(dx), _ptr(dweight), _ptr(dbias),
            ctypes.byref(a))
    result = {"dx": dx, "dweight": dweight, "dbias": dbias}
    return _bra.Plan(lib.grouped_matmul_grad, args, "grouped_matmul_grad", result,
                     (dy, x, weight, bias, counts, a, workspace, status))


def grouped_matmul_grad(dy, x, weight, counts, bias=None, dx=None, dweight=None, dbias=None,
                        want=("dx", "dweight", "dbias"), transpose_weight: bool = False,
                        workspace="auto", status=None, stream=None) -> dict:
    """Gradients of grouped_matmul for the output's gradient dy (R, N).

    Returns {'dx': (R, K), 'dweight': the weight's shape, 'dbias': (E, N)},
    with None for what `want` leaves out and for dbias when there is no bias
    (neither `bias` nor an output `dbias` given).  Experts without rows get
    zero; rows of dx after the counts' sum are not written.  Results do not
    change from run to run."""
    with _on(stream):
        return grouped_matmul_grad_plan(dy, x, weight, counts, bias, dx, dweight, dbias, want,
                                        transpose_weight, workspace, status).run()


class MxTensor:
    """Rows in 4-bit microscaled floating point (mxfp4_quantize).

    shape: (R, K), or (E, N, K) for weights.  codes: uint8, two codes to a
    byte, rows padded to 32 elements.  scales: uint8, one to 32 elements, in
    the tensor core's order (include/bra_moe.h).  counts: the tensor of row
    counts the rows were grouped with, or None: then each matrix of N rows is
    a group."""

    def __init__(self, codes, scales, shape, counts):
        self.codes, self.scales, self.shape, self.counts = codes, scales, tuple(shape), counts
        self._checked = None             # the parts that _holds has found to fit

    def _parts(self):
        return self.codes, self.scales, self.shape, self.counts

    @property
    def device(self):
        return self.codes.device

    def _args(self) -> MxArgs:
        a = MxArgs()
        a.k = self.shape[-1]
        if self.counts is not None:
            a.rows, a.groups = self.shape[0], self.counts.numel()
        else:
            a.groups = self.shape[0] if len(self.shape) == 3 else 1
            a.rows_per_group = self.shape[-2]
            a.rows = a.groups * a.rows_per_group
            if a.rows == 0:
                a.rows_per_group = 0
        return a


def _holds(t: MxTensor, what: str) -> None:
    """Checks that the buffers of an MxTensor hold what it says: once for the same tensors (8 us),
    which have to keep their storage, as those of a Plan."""
    if t._checked is not None and all(a is b for a, b in zip(t._checked, t._parts())):
        return
    torch = _bra._torch()
    if len(t.shape) != 2 and (len(t.shape) != 3 or t.counts is not None):
        raise ValueError(f"{what} must hold rows (R, K) or matrices (E, N, K), got {t.shape}")
    if t.counts is not None:
        _counts(t.counts)
    a, lib, byte = t._args(), _bra.library(), torch.uint8
    ref = ctypes.byref(a)
    needs = lib.mxfp4_code_bytes(ref), lib.mxfp4_scale_bytes(ref)
    if min(needs) < 0:
        raise _bra.BraError(-min(needs), what)
    for part, buf, need in zip(("codes", "scales"), (t.codes, t.scales), needs):
        if not isinstance(buf, torch.Tensor) or buf.dtype is not byte or not buf.is_cuda or \
                not buf.is_contiguous():
            _bra._dev_tensor(buf, f"{what}'s {part}", byte)              # says which
        if buf.numel() < need:
            raise ValueError(f"{what}'s {part} have {buf.numel()} bytes, {t.shape} takes {need}")
    if t.codes.device != t.scales.device or t.counts is not None and t.counts.device != t.codes.device:
        raise ValueError(f"{what}'s buffers and counts must be on one device")
    t._checked = t._parts()


def mxfp4_quantize_plan(x, counts=None, out: Optional[MxTensor] = None, status=None):
    """mxfp4_quantize prepared once (see Plan); plan.run() returns the MxTensor."""
    torch = _bra._torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    code = _bra._fused_dtype(x.dtype)
    if x.dim() == 3 and counts is None:
        _bra._dev_tensor(x, "x")
        pitch = 0
    else:
        pitch = _rows(x, "x")
    if x.numel() == 0 and x.shape[-1] == 0:
        raise ValueError("x has rows of no elements")
    if counts is not None:
        _counts(counts)
    shape = tuple(x.shape)
    probe = MxTensor(x, None, shape, counts)._args()
    lib = _bra.library()
    cb = lib.mxfp4_code_bytes(ctypes.byref(probe))
    sb = lib.mxfp4_scale_bytes(ctypes.byref(probe))
    if cb < 0 or sb < 0:
        raise _bra.BraError(-min(cb, sb), "mxfp4_quantize")
    if out is None:
        new = lambda n: torch.empty(n, dtype=torch.uint8, device=x.device)   # noqa: E731
        out = MxTensor(new(cb).view(shape[:-1] + (-(-shape[-1] // 32) * 16,)), new(sb), shape,
                       counts)
        out._checked = out._parts()
    elif out.shape != shape or out.counts is not counts:
        raise ValueError(f"out holds {out.shape} and its own counts, expected {shape} with counts")
    else:
        _holds(out, "out")
    _same_device(x, out.codes, out.scales, counts, status)
    a = probe
    a.x_pitch, a.dtype, a.status = pitch, code, _status(status)
    args = (_ptr(x), _ptr(counts), _ptr(out.codes), _ptr(out.scales), ctypes.byref(a))
    return _bra.Plan(lib.mxfp4_quantize, args, "mxfp4_quantize", out, (x, counts, a, status))


def mxfp4_quantize(x, counts=None, out: Optional[MxTensor] = None, status=None,
                   stream=None) -> MxTensor:
    """x (fp16 or bf16) in 4-bit microscaled floating point (MXFP4).

    Each 32 elements of a row share the scale 2^s, s = floor(log2 max|x|) - 2;
    values are the nearest multiples by {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to
    the even code.  x: (R, K) rows of any pitch, grouped by `counts` (CUDA
    int64) if given, or (E, N, K) weights.  A block with a NaN or an infinity
    becomes NaN."""
    with _on(stream):
        return mxfp4_quantize_plan(x, counts, out, status).run()


def mxfp4_dequantize_plan(q: MxTensor, dtype, out=None, status=None):
    """mxfp4_dequantize prepared once (see Plan); plan.run() returns out."""
    torch = _bra._torch()
    codes = {torch.float16: _bra.FP16, torch.bfloat16: _bra.BF16, torch.float32: _bra.FP32}
    if dtype not in codes:
        raise TypeError(f"mxfp4_dequantize gives float16, bfloat16 or float32, got {dtype}")
    _holds(q, "q")
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    _dense(out, "out", dtype, q.shape)
    _same_device(q.codes, out, status)
    a = q._args()
    a.dtype, a.status = codes[dtype], _status(status)
    args = (_ptr(q.codes), _ptr(q.scales), _ptr(q.counts), _ptr(out), ctypes.byref(a))
    return _bra.Plan(_bra.library().mxfp4_dequantize, args, "mxfp4_dequantize", out,
                     (q, a, status))


def mxfp4_dequantize(q: MxTensor, dtype, out=None, status=None, stream=None):
    """The values of an MxTensor as fp16, bf16 or fp32 (one rounding)."""
    with _on(stream):
        return mxfp4_dequantize_plan(q, dtype, out, status).run()


def mxfp4_grouped_matmul_plan(x: MxTensor, weight: MxTensor, counts, bias=None, out=None,
                              dtype=None, status=None):
    """mxfp4_grouped_matmul prepared once (see Plan); plan.run() returns out."""
    torch = _bra._torch()
    if not isinstance(x, MxTensor) or not isinstance(weight, MxTensor):
        raise TypeError("x and weight must be MxTensors (mxfp4_quantize)")
    if len(x.shape) != 2 or len(weight.shape) != 3 or weight.counts is not None:
        raise ValueError("x must hold rows (R, K) and weight matrices (E, N, K)")
    (R, K), (E, N, Kw) = x.shape, weight.shape
    if K != Kw:
        raise ValueError(f"x has rows of {K}, weight takes {Kw}")
    _counts(counts, E)
    _holds(x, "x")
    _holds(weight, "weight")
    if x.counts is None and E != 1 or x.counts is not None and \
            (x.counts.data_ptr() != counts.data_ptr() or x.counts.numel() != E):
        raise ValueError("x has to be quantized with these counts: its scales are grouped by them")
    dt = dtype if dtype is not None else out.dtype if out is not None else torch.bfloat16
    code = _bra._fused_dtype(dt)
    if bias is not None:
        _dense(bias, "bias", _bias_dtype(dt), (E, N))
    if out is None:
        out = torch.empty((R, N), dtype=dt, device=x.device)
    yp = _rows(out, "out", dt, (R, N))
    _same_device(x.codes, weight.codes, counts, bias, out, status)
    a = GroupedArgs()
    a.rows, a.groups, a.in_, a.out = R, E, K, N
    a.dtype, a.y_pitch, a.status = code, yp, _status(status)
    args = (_ptr(x.codes), _ptr(x.scales), _ptr(weight.codes), _ptr(weight.scales), _ptr(bias),
            _ptr(counts), _ptr(out), ctypes.byref(a))
    return _bra.Plan(_bra.library().mxfp4_grouped_matmul, args, "mxfp4_grouped_matmul", out,
                     (x, weight, counts, bias, a, status))


def mxfp4_grouped_matmul(x: MxTensor, weight: MxTensor, counts, bias=None, out=None, dtype=None,
                         status=None, stream=None):
    """grouped_matmul on 4-bit operands: y[r] = x[r] @ weight[e].T + bias[e].

    x: rows quantized with these `counts` (with one expert, also without).
    weight: (E, N, K) quantized.  Products and sums of the dequantized values
    in fp32, one rounding to dtype (bf16 by default, or fp16).  The rest as
    grouped_matmul."""
    with _on(stream):
        return mxfp4_grouped_matmul_plan(x, weight, counts, bias, out, dtype, status).run()


def _row_dtype(dt, what: str) -> int:
    torch = _bra._torch()
    codes = {torch.float16: _bra.FP16, torch.bfloat16: _bra.BF16, torch.float32: _bra.FP32}
    if dt not in codes:
        raise TypeError(f"{what} takes float16, bfloat16 or float32, got {dt}")
    return codes[dt]


def _matrix(t, what: str, dtype=None, shape=None):
    """A dense 2-D CUDA tensor."""
    _bra._dev_tensor(t, what, dtype)
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D (got shape {tuple(t.shape)})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


SCORES = {"softmax": 0, "sigmoid": 1}


def _route_args(logits, k: int, renormalize: bool, score: str = "softmax", bias=None,
                groups: int = 1, top_groups=None, group_best: int = 2, scale: float = 1.0):
    """RouteArgs, or ScoreArgs where a call asks for more than they say."""
    if score not in SCORES:
        raise ValueError(f"score is one of {sorted(SCORES)}, got {score!r}")
    groups, group_best, scale = int(groups), int(group_best), float(scale)
    top = groups if top_groups is None else int(top_groups)
    plain = score == "softmax" and bias is None and scale == 1.0 and groups == top == 1
    a = RouteArgs() if plain else ScoreArgs()
    a.tokens, a.experts = logits.shape
    a.choices = int(k)
    a.dtype = _row_dtype(logits.dtype, "moe_route")
    a.renormalize = 1 if renormalize else 0
    if not plain:
        if abs(max(groups, top, group_best, key=abs)) >= 1 << 31:
            raise ValueError("groups, top_groups and group_best are 32-bit numbers")
        a.score, a.groups, a.top_groups, a.group_best = SCORES[score], groups, top, group_best
        a.scale = scale
    return a


def moe_route_plan(logits, k: int, renormalize: bool = True, ids=None, weights=None, counts=None,
                   slots=None, tokens=None, workspace="auto", *, score: str = "softmax", bias=None,
                   groups: int = 1, top_groups=None, group_best: int = 2, scale: float = 1.0):
    """moe_route prepared once (see Plan); plan.run() returns its dict."""
    torch = _bra._torch()
    _matrix(logits, "logits")
    a = _route_args(logits, k, renormalize, score, bias, groups, top_groups, group_best, scale)
    T, E = logits.shape
    if bias is not None:
        _dense(bias, "bias", torch.float32, (E,))
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=logits.device)   # noqa: E731
    i32 = torch.int32
    ids = _dense(new((T, k), i32) if ids is None else ids, "ids", i32, (T, k))
    weights = _dense(new((T, k), torch.float32) if weights is None else weights, "weights",
                     torch.float32, (T, k))
    counts = _counts(new((E,), torch.int64) if counts is None else counts, E)
    slots = _dense(new((T, k), i32) if slots is None else slots, "slots", i32, (T, k))
    tokens = _dense(new((T * k,), i32) if tokens is None else tokens, "tokens", i32, (T * k,))
    _same_device(logits, ids, weights, counts, slots, tokens, bias)
    lib = _bra.library()
    plain = isinstance(a, RouteArgs)
    need = (lib.moe_route_workspace_size if plain else lib.moe_route_scored_workspace_size)(
        ctypes.byref(a))
    box = GroupedArgs()                                   # holds the workspace's address
    workspace = _take_workspace(workspace, need, logits.device, box)
    result = {"ids": ids, "weights": weights, "counts": counts, "slots": slots, "tokens": tokens}
    args = (_ptr(logits),) + (() if plain else (_ptr(bias),)) + (
        _ptr(ids), _ptr(weights), _ptr(counts), _ptr(slots), _ptr(tokens), box.workspace,
        box.workspace_bytes, ctypes.byref(a))
    name = "moe_route" if plain else "moe_route_scored"
    return _bra.Plan(getattr(lib, name), args, name, result, (logits, bias, a, workspace))


def moe_route(logits, k: int, renormalize: bool = True, ids=None, weights=None, counts=None,
              slots=None, tokens=None, workspace="auto", stream=None, *, score: str = "softmax",
              bias=None, groups: int = 1, top_groups=None, group_best: int = 2,
              scale: float = 1.0) -> dict:
    """Each token's k experts, and the order that sorts the pairs by expert.

    logits: CUDA (T, E), fp16, bf16 or fp32; -inf or NaN closes an expert to
    a token.  Returns {'ids' (T, k) int32, 'weights' (T, k) fp32, 'counts'
    (E,) int64, 'slots' (T, k) int32, 'tokens' (T*k,) int32}: the chosen
    experts, largest logit first (ties: the lowest index), their softmax
    weights (renormalised over the chosen by default), rows of each expert,
    the row of each pair when sorted by expert, and the token of each row.  A
    token with fewer than k open experts has -1, weight 0 and slot -1 for the
    rest; rows past the last pair have token -1.

    score: "softmax", or "sigmoid" of each logit.  bias: CUDA (E,) fp32, added
    to the scores for the choice (largest sum first), not to the weights.
    groups, top_groups: choose from the experts of the top_groups best of
    `groups` groups of consecutive experts (None: all), a group ranked by its
    best expert (group_best=1) or the sum of its two best (2).  scale: a
    factor of the weights.  The choice is what scores, sums and ranks in 64
    bits give, ties to the lowest group and index."""
    with _on(stream):
        return moe_route_plan(logits, k, renormalize, ids, weights, counts, slots, tokens,
                              workspace, score=score, bias=bias, groups=groups,
                              top_groups=top_groups, group_best=group_best, scale=scale).run()


def moe_route_grad_plan(dweights, logits, ids, weights, renormalize: bool = True, out=None, *,
                        score: str = "softmax", scale: float = 1.0):
    """moe_route_grad prepared once (see Plan); plan.run() returns out."""
    torch = _bra._torch()
    _matrix(logits, "logits")
    _matrix(ids, "ids", torch.int32)
    T, k = ids.shape
    a = _route_args(logits, k, renormalize, score, scale=scale)
    if logits.shape[0] != T:
        raise ValueError(f"logits have {logits.shape[0]} tokens, ids {T}")
    _matrix(dweights, "dweights", torch.float32, (T, k))
    _matrix(weights, "weights", torch.float32, (T, k))
    if out is None:
        out = torch.empty_like(logits)
    _matrix(out, "out", logits.dtype, logits.shape)
    _same_device(logits, dweights, ids, weights, out)
    args = (_ptr(dweights), _ptr(logits), _ptr(ids), _ptr(weights), _ptr(out), ctypes.byref(a))
    name = "moe_route_grad" if isinstance(a, RouteArgs) else "moe_route_scored_grad"
    return _bra.Plan(getattr(_bra.library(), name), args, name, out,
                     (dweights, logits, ids, weights, a))


def moe_route_grad(dweights, logits, ids, weights, renormalize: bool = True, out=None,
                   stream=None, *, score: str = "softmax", scale: float = 1.0):
    """Gradient of the logits for the gradient of moe_route's weights, of the
    same score, renormalize and scale (the choice itself is constant)."""
    with _on(stream):
        return moe_route_grad_plan(dweights, logits, ids, weights, renormalize, out, score=score,
                                   scale=scale).run()


def _permute_args(T: int, R: int, k: int, rows, what: str) -> PermuteArgs:
    a = PermuteArgs()
    a.tokens, a.rows, a.choices, a.width = T, R, k, rows.shape[1]
    a.dtype = _row_dtype(rows.dtype, what)
    return a


def moe_dispatch_plan(x, tokens, out=None, workspace="auto"):
    """moe_dispatch prepared once (see Plan); plan.run() returns out."""
    torch = _bra._torch()
    _matrix(x, "x")
    _bra._dev_tensor(tokens, "tokens", torch.int32)
    R = tokens.numel()
    if out is None:
        out = torch.empty((R, x.shape[1]), dtype=x.dtype, device=x.device)
    _matrix(out, "out", x.dtype, (R, x.shape[1]))
    _same_device(x, tokens, out)
    a = _permute_args(x.shape[0], R, 1, x, "moe_dispatch")
    lib = _bra.library()
    box = GroupedArgs()                                   # holds the workspace's address
    workspace = _take_workspace(workspace, lib.moe_dispatch_workspace_size(ctypes.byref(a)),
                                x.device, box)
    args = (_ptr(x), _ptr(tokens), _ptr(out), box.workspace, box.workspace_bytes, ctypes.byref(a))
    return _bra.Plan(lib.moe_dispatch, args, "moe_dispatch", out, (x, tokens, a, workspace))


def moe_dispatch(x, tokens, out=None, workspace="auto", stream=None):
    """Token rows in expert order: out[r] = x[tokens[r]], zeros for -1.

    workspace: scratch memory for the lists of each token's rows, used when
    there are many ("auto": from torch's allocator)."""
    with _on(stream):
        return moe_dispatch_plan(x, tokens, out, workspace).run()


def _to_tokens_plan(rows, slots, weights, out, name: str, what: str):
    torch = _bra._torch()
    _matrix(rows, what)
    _matrix(slots, "slots", torch.int32)
    T, k = slots.shape
    if weights is not None:
        _matrix(weights, "weights", torch.float32, (T, k))
    if out is None:
        out = torch.empty((T, rows.shape[1]), dtype=rows.dtype, device=rows.device)
    _matrix(out, "out", rows.dtype, (T, rows.shape[1]))
    _same_device(rows, slots, weights, out)
    a = _permute_args(T, rows.shape[0], k, rows, name)
    args = (_ptr(rows), _ptr(slots)) + (() if weights is None else (_ptr(weights),)) + \
        (_ptr(out), ctypes.byref(a))
    return _bra.Plan(getattr(_bra.library(), name), args, name, out, (rows, slots, weights, a))


def moe_dispatch_grad_plan(dxs, slots, out=None):
    """moe_dispatch_grad prepared once (see Plan); plan.run() returns out."""
    return _to_tokens_plan(dxs, slots, None, out, "moe_dispatch_grad", "dxs")


def moe_dispatch_grad(dxs, slots, out=None, stream=None):
    """Gradient of moe_dispatch: out[t] = sum of dxs[slots[t, j]] over j."""
    with _on(stream):
        return moe_dispatch_grad_plan(dxs, slots, out).run()


def moe_combine_plan(ys, slots, weights, out=None):
    """moe_combine prepared once (see Plan); plan.run() returns out."""
    if weights is None:
        raise TypeError("weights must be a torch.Tensor")
    return _to_tokens_plan(ys, slots, weights, out, "moe_combine", "ys")


def moe_combine(ys, slots, weights, out=None, stream=None):
    """Expert rows back to tokens: out[t] = sum of weights[t, j] * ys[slots[t, j]]
    over j (fp32, one rounding); slots of -1 are left out."""
    with _on(stream):
        return moe_combine_plan(ys, slots, weights, out).run()


def moe_combine_grad_plan(dy, ys, slots, weights, tokens=None, dys=None, dweights=None):
    """moe_combine_grad prepared once (see Plan); plan.run() returns its dict."""
    torch = _bra._torch()
    _matrix(dy, "dy")
    _matrix(ys, "ys", dy.dtype)
    _matrix(slots, "slots", torch.int32)
    T, k = slots.shape
    R, H = ys.shape
    if tuple(dy.shape) != (T, H):
        raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {(T, H)}")
    _matrix(weights, "weights", torch.float32, (T, k))
    if tokens is not None:
        _dense(tokens, "tokens", torch.int32, (R,))
    dys = _matrix(torch.empty_like(ys) if dys is None else dys, "dys", ys.dtype, (R, H))
    dweights = _matrix(torch.empty_like(weights) if dweights is None else dweights, "dweights",
                       torch.float32, (T, k))
    _same_device(dy, ys, slots, weights, tokens, dys, dweights)
    a = _permute_args(T, R, k, ys, "moe_combine_grad")
    args = (_ptr(dy), _ptr(ys), _ptr(slots), _ptr(weights), _ptr(tokens), _ptr(dys),
            _ptr(dweights), ctypes.byref(a))
    return _bra.Plan(_bra.library().moe_combine_grad, args, "moe_combine_grad",
                     {"dys": dys, "dweights": dweights}, (dy, ys, slots, weights, tokens, a))


def moe_combine_grad(dy, ys, slots, weights, tokens=None, dys=None, dweights=None,
                     stream=None) -> dict:
    """Gradients of moe_combine: {'dys': (R, H), 'dweights': (T, k) fp32}.

    tokens (of moe_route): rows without a token get zeros; without it those
    rows of dys are not written."""
    with _on(stream):
        return moe_combine_grad_plan(dy, ys, slots, weights, tokens, dys, dweights).run()
