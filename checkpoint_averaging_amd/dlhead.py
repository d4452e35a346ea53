"""ctypes binding of the output head's calls (C ABI in include/dlhead.h).

Argument marshalling only, as in ``dlmerge``: function names mirror the C
functions, torch tensors become device pointers with their leading dimension
and type, the stream defaults to torch's current stream, and a negative
status becomes a DLError.  A matrix argument is a 2-D tensor whose last
dimension is contiguous (rows may be strided: its leading dimension is the
row stride), a contiguous 1-D tensor, or, for tests that need exact pointers,
an integer device address with its ``ld`` and dtype.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .dlmerge import DL_BF16, DL_F32, Array, _check, _ws, raw_lib

DL_E4M3 = 2
DL_SCALE_NONE = 0
DL_SCALE_ROW = 1
DL_SCALE_BLOCK32 = 2
DL_MAX_NORM_COLS = 32768
DL_MAX_VECTORS = 32
DL_MAX_TOP = 32

SYMBOLS = ("dl_rmsnorm", "dl_rmsnorm_workspace_bytes", "dl_rmsnorm_backward",
           "dl_w4_bytes", "dl_w4_quantize", "dl_w4_matvec",
           "dl_logprobs_workspace_bytes", "dl_logprobs", "dl_logprobs_backward")

_lib = raw_lib()
_p, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
_lib.dl_rmsnorm.argtypes = [_p, _i64, _p, _i64, _i32, _p, _f32, _i64, _i64, _p, _i64, _p, _i64,
                            _i32, _p, _i32, _p, _p]
_lib.dl_rmsnorm_workspace_bytes.argtypes = [_i64, _i64, ctypes.POINTER(_i64)]
_lib.dl_rmsnorm_backward.argtypes = [_p, _i64, _p, _i64, _p, _i64, _i32, _p, _p, _i64, _i64, _p,
                                     _i64, _p, _p, _i64, _p]
_lib.dl_w4_bytes.argtypes = [_i64, _i64, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
_lib.dl_w4_quantize.argtypes = [_p, _i64, _i32, _i64, _i64, _p, _p, _p, _i64, _p]
_lib.dl_w4_matvec.argtypes = [_p, _p, _i64, _i64, _p, _i64, _i32, _p, _i32, _i32, _p, _i64, _i32,
                              _p]
_lib.dl_logprobs_workspace_bytes.argtypes = [_i64, _i64, _i32, ctypes.POINTER(_i64)]
_lib.dl_logprobs.argtypes = [_p, _i64, _i32, _i64, _i64, _p, _p, _p, _p, _i32, _p, _p, _p, _i64,
                             _p]
_lib.dl_logprobs_backward.argtypes = [_p, _i64, _i32, _i64, _i64, _p, _p, _p, _p, _p, _p, _i64, _p]
for _name in SYMBOLS:
    getattr(_lib, _name).restype = _i32

_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_DTYPES = {torch.float32: DL_F32, torch.bfloat16: DL_BF16, torch.float8_e4m3fn: DL_E4M3}


def _stream(stream) -> Optional[int]:
    """The stream's handle; by default the current one of the current device
    (asked for directly: a torch.cuda.Stream object costs 3 us a call)."""
    if stream is None:
        if not torch.cuda.is_initialized():
            return None
        return _raw_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _matrix(a: Array, rows: int, cols: int, ld: Optional[int], name: str
            ) -> Tuple[Optional[int], int]:
    """(address, leading dimension) of a rows x cols matrix argument."""
    if not isinstance(a, torch.Tensor):
        return (None if a is None else int(a)), int(cols if ld is None else ld)
    if not a.is_cuda:
        raise TypeError(f"{name}: device tensor required")
    shape, stride = a.shape, a.stride()
    if len(shape) == 2:
        if rows > 0 and (shape[0] < rows or shape[1] < cols):
            raise ValueError(f"{name}: {tuple(shape)} does not hold {rows} x {cols}")
        if stride[1] != 1 and shape[1] > 1:
            raise TypeError(f"{name}: rows must be contiguous")
        if shape[0] == 1:
            ld = max(cols, stride[0]) if ld is None else ld
        elif ld is None:
            ld = stride[0]
        elif ld != stride[0]:
            raise ValueError(f"{name}: ld {ld} is not its row stride {stride[0]}")
    else:
        if len(shape) != 1 or (stride[0] != 1 and shape[0] > 1):
            raise TypeError(f"{name}: 2-D tensor, or contiguous 1-D tensor, required")
        ld = cols if ld is None else ld
        if rows > 0 and shape[0] < (rows - 1) * ld + cols:
            raise ValueError(f"{name}: {shape[0]} elements do not hold {rows} x {cols}")
    return a.data_ptr(), ld


def _dtype_of(a: Array, dtype: Optional[int], name: str) -> int:
    if isinstance(a, torch.Tensor):
        got = _DTYPES.get(a.dtype)
        if got is None or (dtype is not None and int(dtype) != got):
            raise TypeError(f"{name}: {a.dtype} is not the type asked for")
        return got
    if dtype is None:
        raise TypeError(f"{name}: its type is required with a raw address")
    return int(dtype)


def _same_type(a: Array, dtype: int, name: str) -> None:
    if isinstance(a, torch.Tensor) and _DTYPES.get(a.dtype) != dtype:
        raise TypeError(f"{name}: {a.dtype} differs from the call's type")


def _vector(a: Array, n: int, dtype: torch.dtype, name: str) -> Optional[int]:
    """Address of a contiguous array of at least n elements of dtype."""
    if a is None:
        return None
    if not isinstance(a, torch.Tensor):
        return int(a)
    if a.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not (a.is_cuda and a.is_contiguous()):
        raise TypeError(f"{name}: contiguous device tensor required")
    if a.numel() < n:
        raise ValueError(f"{name}: {a.numel()} elements, {n} needed")
    return a.data_ptr()


def _scales(a: Array, kind: int, rows: int, cols: int, name: str) -> Optional[int]:
    if kind == DL_SCALE_ROW:
        return _vector(a, rows, torch.float32, name)
    return _vector(a, rows * ((cols + 31) // 32), torch.uint8, name)


def _workspace(workspace: Array, workspace_bytes: Optional[int]) -> Tuple[Optional[int], int]:
    return (None, 0) if workspace is None else _ws(workspace, workspace_bytes)


def dl_rmsnorm(x: Array, rows: int, cols: int, weight: Array, y: Array, eps: float = 1e-5,
               residual: Array = None, sum_: Array = None, scales: Array = None,
               scale_kind: int = DL_SCALE_NONE, inv_rms: Array = None,
               ldx: Optional[int] = None, ldres: Optional[int] = None,
               ldsum: Optional[int] = None, ldy: Optional[int] = None,
               dtype: Optional[int] = None, y_dtype: Optional[int] = None, stream=None) -> None:
    dtype = _dtype_of(x, dtype, "x")
    y_dtype = _dtype_of(y, y_dtype, "y")
    _same_type(residual, dtype, "residual")
    _same_type(sum_, dtype, "sum")
    xa, ldx = _matrix(x, rows, cols, ldx, "x")
    ra, ldres = _matrix(residual, rows, cols, ldres, "residual")
    sa, ldsum = _matrix(sum_, rows, cols, ldsum, "sum")
    ya, ldy = _matrix(y, rows, cols, ldy, "y")
    _check(_lib.dl_rmsnorm(xa, ldx, ra, ldres, dtype, _vector(weight, cols, torch.float32,
                                                              "weight"),
                           eps, rows, cols, sa, ldsum, ya, ldy, y_dtype,
                           _scales(scales, scale_kind, rows, cols, "scales"), scale_kind,
                           _vector(inv_rms, rows, torch.float32, "inv_rms"), _stream(stream)),
           "dl_rmsnorm")


def dl_rmsnorm_workspace_bytes(rows: int, cols: int) -> int:
    b = _i64()
    _check(_lib.dl_rmsnorm_workspace_bytes(int(rows), int(cols), ctypes.byref(b)),
           "dl_rmsnorm_workspace_bytes")
    return b.value


def dl_rmsnorm_backward(dy: Array, sum_: Array, rows: int, cols: int, weight: Array,
                        inv_rms: Array, dx: Array, dsum: Array = None, dweight: Array = None,
                        workspace: Array = None, workspace_bytes: Optional[int] = None,
                        lddy: Optional[int] = None, lddsum: Optional[int] = None,
                        ldsum: Optional[int] = None, lddx: Optional[int] = None,
                        dtype: Optional[int] = None, stream=None) -> None:
    dtype = _dtype_of(dy, dtype, "dy")
    for a, name in ((sum_, "sum"), (dx, "dx"), (dsum, "dsum")):
        _same_type(a, dtype, name)
    ya, lddy = _matrix(dy, rows, cols, lddy, "dy")
    da, lddsum = _matrix(dsum, rows, cols, lddsum, "dsum")
    sa, ldsum = _matrix(sum_, rows, cols, ldsum, "sum")
    xa, lddx = _matrix(dx, rows, cols, lddx, "dx")
    w, wb = _workspace(workspace, workspace_bytes)
    _check(_lib.dl_rmsnorm_backward(ya, lddy, da, lddsum, sa, ldsum, dtype,
                                    _vector(weight, cols, torch.float32, "weight"),
                                    _vector(inv_rms, rows, torch.float32, "inv_rms"), rows, cols,
                                    xa, lddx, _vector(dweight, cols, torch.float32, "dweight"),
                                    w, wb, _stream(stream)),
           "dl_rmsnorm_backward")


def dl_w4_bytes(rows: int, cols: int) -> Tuple[int, int]:
    """(bytes of the codes, bytes of the scales) of a rows x cols matrix in 4 bits."""
    pb, sb = _i64(), _i64()
    _check(_lib.dl_w4_bytes(int(rows), int(cols), ctypes.byref(pb), ctypes.byref(sb)),
           "dl_w4_bytes")
    return pb.value, sb.value


def _w4(packed: Array, scales: Array, rows: int, cols: int):
    kb = (cols + 31) // 32
    return (_vector(packed, rows * kb * 16, torch.uint8, "packed"),
            _vector(scales, rows * kb, torch.uint8, "scales"))


def dl_w4_quantize(w: Array, rows: int, cols: int, packed: Array, scales: Array,
                   values: Array = None, ldw: Optional[int] = None,
                   ldvalues: Optional[int] = None, dtype: Optional[int] = None,
                   stream=None) -> None:
    dtype = _dtype_of(w, dtype, "w")
    _same_type(values, dtype, "values")
    wa, ldw = _matrix(w, rows, cols, ldw, "w")
    va, ldvalues = _matrix(values, rows, cols, ldvalues, "values")
    pa, sa = _w4(packed, scales, rows, cols)
    _check(_lib.dl_w4_quantize(wa, ldw, dtype, rows, cols, pa, sa, va, ldvalues,
                               _stream(stream)),
           "dl_w4_quantize")


def dl_w4_matvec(packed: Array, scales: Array, rows: int, cols: int, x: Array, count: int,
                 y: Array, x_scales: Array = None, x_scale_kind: int = DL_SCALE_NONE,
                 ldx: Optional[int] = None, ldy: Optional[int] = None,
                 x_dtype: Optional[int] = None, y_dtype: Optional[int] = None,
                 stream=None) -> None:
    x_dtype = _dtype_of(x, x_dtype, "x")
    y_dtype = _dtype_of(y, y_dtype, "y")
    xa, ldx = _matrix(x, count, cols, ldx, "x")
    ya, ldy = _matrix(y, count, rows, ldy, "y")
    pa, sa = _w4(packed, scales, rows, cols)
    _check(_lib.dl_w4_matvec(pa, sa, rows, cols, xa, ldx, x_dtype,
                             _scales(x_scales, x_scale_kind, count, cols, "x_scales"),
                             x_scale_kind, count, ya, ldy, y_dtype, _stream(stream)),
           "dl_w4_matvec")


def dl_logprobs_workspace_bytes(rows: int, vocab: int, top_k: int = 0) -> int:
    b = _i64()
    _check(_lib.dl_logprobs_workspace_bytes(int(rows), int(vocab), int(top_k), ctypes.byref(b)),
           "dl_logprobs_workspace_bytes")
    return b.value


def dl_logprobs(logits: Array, rows: int, vocab: int, targets: Array = None,
                logprobs: Array = None, entropy: Array = None, stats: Array = None,
                top_k: int = 0, top_ids: Array = None, top_logprobs: Array = None,
                workspace: Array = None, workspace_bytes: Optional[int] = None,
                ldl: Optional[int] = None, dtype: Optional[int] = None, stream=None) -> None:
    dtype = _dtype_of(logits, dtype, "logits")
    la, ldl = _matrix(logits, rows, vocab, ldl, "logits")
    w, wb = _workspace(workspace, workspace_bytes)
    f32, i64 = torch.float32, torch.int64
    _check(_lib.dl_logprobs(la, ldl, dtype, rows, vocab, _vector(targets, rows, i64, "targets"),
                            _vector(logprobs, rows, f32, "logprobs"),
                            _vector(entropy, rows, f32, "entropy"),
                            _vector(stats, 2 * rows, f32, "stats"), top_k,
                            _vector(top_ids, rows * top_k, i64, "top_ids"),
                            _vector(top_logprobs, rows * top_k, f32, "top_logprobs"), w, wb,
                            _stream(stream)),
           "dl_logprobs")


def dl_logprobs_backward(logits: Array, rows: int, vocab: int, targets: Array, stats: Array,
                         dlogprobs: Array, dlogits: Array, entropy: Array = None,
                         dentropy: Array = None, ldl: Optional[int] = None,
                         lddl: Optional[int] = None, dtype: Optional[int] = None,
                         stream=None) -> None:
    dtype = _dtype_of(logits, dtype, "logits")
    _same_type(dlogits, dtype, "dlogits")
    la, ldl = _matrix(logits, rows, vocab, ldl, "logits")
    da, lddl = _matrix(dlogits, rows, vocab, lddl, "dlogits")
    f32 = torch.float32
    _check(_lib.dl_logprobs_backward(la, ldl, dtype, rows, vocab,
                                     _vector(targets, rows, torch.int64, "targets"),
                                     _vector(stats, 2 * rows, f32, "stats"),
                                     _vector(entropy, rows, f32, "entropy"),
                                     _vector(dlogprobs, rows, f32, "dlogprobs"),
                                     _vector(dentropy, rows, f32, "dentropy"), da, lddl,
                                     _stream(stream)),
           "dl_logprobs_backward")
