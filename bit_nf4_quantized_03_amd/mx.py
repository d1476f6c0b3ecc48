"""Python binding of the microscaled formats, RMSNorm and the microscaled
products (include/qlora_mx.h).

As in the package itself, the functions carry the names of the C entry points
and only marshal arguments: torch supplies device memory and the current
stream of the tensors' device. They are re-exported by the package.
"""
from __future__ import annotations

import ctypes
import dataclasses
from ctypes import byref
from typing import Optional, Tuple

import torch

from . import QLORA_BF16, QLORA_F32, QloraError, lib, qlora_last_error

try:
    from . import _fastcall as _fast   # whole calls with new outputs; None where the call is not that simple
except ImportError:
    _fast = None   # not built, or for another torch: every call has its whole path here too, at 5 to 8 us more host time

__all__ = [
    "MXMatrix", "QLORA_MX_FP4", "QLORA_MX_FP8", "MX_EXPORTED_SYMBOLS", "qlora_mx_scale_pitch",
    "qlora_mx_storage_bytes", "qlora_mx_quantize", "qlora_mx_dequantize", "qlora_rmsnorm_fwd",
    "qlora_rmsnorm_mx", "qlora_rmsnorm_bwd", "qlora_rmsnorm_bwd_workspace_bytes", "qlora_mx_linear",
    "qlora_mx_linear_grouped",
]

MX_EXPORTED_SYMBOLS = (
    "qlora_mx_scale_pitch", "qlora_mx_storage_bytes", "qlora_mx_quantize", "qlora_mx_dequantize",
    "qlora_rmsnorm_fwd", "qlora_rmsnorm_mx", "qlora_rmsnorm_bwd", "qlora_rmsnorm_bwd_workspace_bytes",
    "qlora_mx_linear", "qlora_mx_linear_grouped",
)

QLORA_MX_FP4 = 0   # sign, 2 exponent bits, 1 mantissa bit; two to a byte
QLORA_MX_FP8 = 1   # sign, 4 exponent bits, 3 mantissa bits
_TYPES = (QLORA_MX_FP4, QLORA_MX_FP8)
_MAX_COLS = 1 << 22


class _MX(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("type", ctypes.c_int32)]


def _declare():
    i64, sz, vp, i32, f64, ci = (ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int32, ctypes.c_double,
                                 ctypes.c_int)
    mp = ctypes.POINTER(_MX)
    sigs = {
        "qlora_mx_scale_pitch": (i64, [i64]),
        "qlora_mx_storage_bytes": (sz, [i64, i64, ci]),
        "qlora_mx_quantize": (ci, [vp, ci, i64, i64, mp, vp]),
        "qlora_mx_dequantize": (ci, [mp, vp, ci, vp]),
        "qlora_rmsnorm_fwd": (ci, [vp, vp, vp, ci, i64, i64, f64, vp, vp, vp, vp]),
        "qlora_rmsnorm_mx": (ci, [vp, vp, vp, ci, i64, i64, f64, mp, vp, vp]),
        "qlora_rmsnorm_bwd_workspace_bytes": (sz, [i64, i64]),
        "qlora_rmsnorm_bwd": (ci, [vp, vp, vp, ci, vp, vp, i64, i64, vp, vp, vp, sz, vp]),
        "qlora_mx_linear": (ci, [mp, mp, vp, vp]),
        "qlora_mx_linear_grouped": (ci, [mp, mp, vp, i32, vp, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args


_declare()

_DTYPES = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}
_DTYPES_OR_NONE = (None, torch.float32, torch.bfloat16)


# a torch without GPU support lacks them; no call gets as far there
_stream, _current = (getattr(torch._C, name, None) for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))


def _fast_on(t):
    """(device index, stream) for a whole call on the current device when ``t``
    lies there, else None."""
    if _fast is not None and isinstance(t, torch.Tensor) and t.is_cuda:
        index = t.get_device()
        if index == _current():
            return index, _stream(index)
    return None


def _entry(name: str):
    """The entry point as a call (device index, *arguments) on that device's
    current stream, with the device current (the library launches on the current
    one)."""
    fn = getattr(lib, name)

    def call(index, *args):
        if index == _current():
            status = fn(*args, _stream(index))
        else:
            with torch.cuda.device(index):
                status = fn(*args, _stream(index))
        if status != 0:
            raise QloraError(name, status, qlora_last_error())
    return call


_quantize, _dequantize = _entry("qlora_mx_quantize"), _entry("qlora_mx_dequantize")
_rmsnorm_fwd, _rmsnorm_mx, _rmsnorm_bwd = (_entry("qlora_rmsnorm_" + x) for x in ("fwd", "mx", "bwd"))
_linear, _linear_grouped = _entry("qlora_mx_linear"), _entry("qlora_mx_linear_grouped")


def _dtype(name, dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    return _DTYPES[dtype]


def _tensor(name, t, dtype, shape, index=None):
    """``t`` must be a contiguous CUDA tensor of this dtype (None: any) and
    shape, on device ``index`` (None: any): the C ABI takes bare pointers.
    Returns its address."""
    if isinstance(t, torch.Tensor) and t.is_cuda and (dtype is None or t.dtype is dtype) and t.shape == shape and \
            t.is_contiguous() and (index is None or t.get_device() == index):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


# torch.empty by another name: 1.3 us a call instead of 1.7
def _empty(rows, cols, dtype, device):
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _empty_1d(n, dtype, device):
    return torch.empty_strided((n,), (1,), dtype=dtype, device=device)


def _rows_cols(name, t, dtype=None):
    """Shape of a contiguous 2-D CUDA tensor with at least one row and column."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and (dtype is None or t.dtype is dtype) and \
            t.is_contiguous():
        rows, cols = t.shape
        if rows and cols:
            return rows, cols
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dim() != 2 or t.numel() == 0:
        raise ValueError(f"{name} must be 2-D with at least one row and one column, got {tuple(t.shape)}")
    _tensor(name, t, dtype, t.shape)   # raises


def qlora_mx_scale_pitch(cols: int) -> int:
    """Bytes between the scales of two rows of a matrix with ``cols`` columns (0 if cols is invalid)."""
    return int(lib.qlora_mx_scale_pitch(cols))


def qlora_mx_storage_bytes(rows: int, cols: int, mx: int) -> int:
    return int(lib.qlora_mx_storage_bytes(rows, cols, mx))


@dataclasses.dataclass
class MXMatrix:
    """Microscaled matrix [rows, cols] in device tensors: ``codes`` uint8
    [rows, cols / 2] (4-bit elements) or [rows, cols] (8-bit), ``scales`` uint8
    [rows, qlora_mx_scale_pitch(cols)], ``mx`` the element type."""
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor
    mx: int = QLORA_MX_FP4

    @staticmethod
    def empty(rows: int, cols: int, device, mx: int = QLORA_MX_FP4) -> "MXMatrix":
        if mx not in _TYPES:
            raise ValueError(f"mx must be QLORA_MX_FP4 or QLORA_MX_FP8, got {mx}")
        if rows < 1 or cols < 32 or cols % 32 or cols > _MAX_COLS:
            raise ValueError(f"{rows} x {cols}: needs rows >= 1 and cols a multiple of 32 up to 2^22")
        return MXMatrix(rows, cols, _empty(rows, cols // 2 if mx == QLORA_MX_FP4 else cols, torch.uint8, device),
                        _empty(rows, -(-cols // 512) * 16, torch.uint8, device), mx)

    @property
    def device(self):
        return self.codes.device

    def c_struct(self, name: str = "matrix", index=None) -> _MX:
        """The C struct, after checking the buffers against rows and cols (on device ``index`` when given)."""
        rows, cols, mx, codes, scales = self.rows, self.cols, self.mx, self.codes, self.scales
        if mx not in _TYPES:
            raise ValueError(f"{name}.mx must be QLORA_MX_FP4 or QLORA_MX_FP8, got {mx}")
        shape, pitch = (rows, cols if mx else cols // 2), (rows, -(-cols // 512) * 16)
        if index is None:
            index = codes.get_device() if isinstance(codes, torch.Tensor) else -1
        if not (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) and codes.is_cuda and codes.dtype is torch.uint8 and codes.shape == shape and codes.is_contiguous() and
                scales.is_cuda and scales.dtype is torch.uint8 and scales.shape == pitch and scales.is_contiguous() and
                codes.get_device() == scales.get_device() == index):
            _tensor(f"{name}.codes", codes, torch.uint8, shape, index)
            _tensor(f"{name}.scales", scales, torch.uint8, pitch, index)
        return _MX(rows, cols, codes.data_ptr(), scales.data_ptr(), mx)


def qlora_mx_quantize(X, mx: Optional[int] = None, out: Optional[MXMatrix] = None) -> MXMatrix:
    """Quantize a 2-D fp32 or bf16 CUDA tensor (columns a multiple of 32) to
    microscaled floats of type ``mx`` (``out.mx`` when ``out`` is given, else
    4 bits)."""
    if out is None and (at := _fast_on(X)):
        new = _fast.quantize(*at, X, QLORA_MX_FP4 if mx is None else mx)
        if new is not None:
            return MXMatrix(*X.shape, *new, QLORA_MX_FP4 if mx is None else mx)
    rows, cols = _rows_cols("X", X)
    dt = _dtype("X", X.dtype)
    if out is None:
        out = MXMatrix.empty(rows, cols, X.device, QLORA_MX_FP4 if mx is None else mx)
    elif mx is not None and mx != out.mx:
        raise ValueError(f"mx {mx} differs from out.mx {out.mx}")
    index = X.get_device()
    _quantize(index, X.data_ptr(), dt, rows, cols, byref(out.c_struct("out", index)))
    return out


def qlora_mx_dequantize(q: MXMatrix, dtype=None, out=None):
    """The values of ``q`` as a [rows, cols] tensor of ``dtype`` (float32 or bfloat16)."""
    if out is None and dtype in _DTYPES_OR_NONE and (at := _fast_on(q.codes)):
        new = _fast.dequantize(*at, q.codes, q.scales, q.rows, q.cols, q.mx, dtype is torch.bfloat16)
        if new is not None:
            return new
    st = q.c_struct("q")
    dtype = torch.float32 if dtype is None else dtype
    dt = _dtype("dtype", dtype)
    index = q.codes.get_device()
    if out is None:
        out = _empty(q.rows, q.cols, dtype, q.codes.device)
        at = out.data_ptr()
    else:
        at = _tensor("out", out, dtype, (q.rows, q.cols), index)
    _dequantize(index, byref(st), at, dt)
    return out


def _at(t):
    return None if t is None else t.data_ptr()


def _norm_inputs(X, weight, residual, h):
    """(rows, cols, device index, addresses and weight type as the entry points take them, h)"""
    rows, cols = _rows_cols("X", X, torch.bfloat16)
    index = X.get_device()
    w = _tensor("weight", weight, None, (cols,), index)
    dt = _dtype("weight", weight.dtype)
    if residual is None:
        if h is not None:
            raise ValueError("h is only written with a residual")
        return rows, cols, index, (X.data_ptr(), None, w, dt, rows, cols), None
    r = _tensor("residual", residual, torch.bfloat16, (rows, cols), index)
    if h is None:
        h = torch.empty_like(X)
    else:
        _tensor("h", h, torch.bfloat16, (rows, cols), index)
    return rows, cols, index, (X.data_ptr(), r, w, dt, rows, cols), h


def qlora_rmsnorm_fwd(X, weight, eps: float = 1e-6, residual=None, out=None, h=None, rstd=None):
    """(Y, H, rstd): Y = H * rstd * weight in bf16 with H = bf16(X + residual),
    rstd = 1 / sqrt(mean(H^2) + eps) fp32 [rows]. Without a residual H is X
    itself, or None where ``out`` is X and has taken its place. ``h`` may be X or
    ``residual`` (in place)."""
    if out is None and h is None and rstd is None and (at := _fast_on(X)):
        new = _fast.norm_fwd(*at, X, weight, eps, residual)
        if new is not None:
            return new
    rows, cols, index, args, h = _norm_inputs(X, weight, residual, h)
    if out is None:
        out = torch.empty_like(X)
    else:
        _tensor("out", out, torch.bfloat16, (rows, cols), index)
    if rstd is None:
        rstd = _empty_1d(rows, torch.float32, X.device)
    else:
        _tensor("rstd", rstd, torch.float32, (rows,), index)
    _rmsnorm_fwd(index, *args, float(eps), out.data_ptr(), _at(h), rstd.data_ptr())
    if h is None and out.data_ptr() != X.data_ptr():
        h = X
    return out, h, rstd


def qlora_rmsnorm_mx(X, weight, eps: float = 1e-6, residual=None, mx: Optional[int] = None,
                     out: Optional[MXMatrix] = None, h=None) -> Tuple[MXMatrix, torch.Tensor]:
    """(Y, H) of qlora_rmsnorm_fwd with Y in microscaled floats of type ``mx``
    (``out.mx`` when ``out`` is given, else 8 bits)."""
    if out is None and h is None and (at := _fast_on(X)):
        new = _fast.norm_mx(*at, X, weight, eps, residual, QLORA_MX_FP8 if mx is None else mx)
        if new is not None:
            return MXMatrix(*X.shape, new[0], new[1], QLORA_MX_FP8 if mx is None else mx), new[2]
    rows, cols, index, args, h = _norm_inputs(X, weight, residual, h)
    if out is None:
        out = MXMatrix.empty(rows, cols, X.device, QLORA_MX_FP8 if mx is None else mx)
    elif mx is not None and mx != out.mx:
        raise ValueError(f"mx {mx} differs from out.mx {out.mx}")
    _rmsnorm_mx(index, *args, float(eps), byref(out.c_struct("out", index)), _at(h))
    return out, X if h is None else h


def qlora_rmsnorm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib.qlora_rmsnorm_bwd_workspace_bytes(rows, cols))


def qlora_rmsnorm_bwd(dY, H, weight, rstd, dH=None, ws=None, outs: Optional[Tuple] = None):
    """(dX, dW) of qlora_rmsnorm_fwd from its H and rstd. dX (bf16) is the
    gradient of X and of the residual; ``dH`` is the gradient that reaches H
    through the residual stream; dW is fp32 [cols]."""
    if ws is None and outs is None and (at := _fast_on(H)):
        new = _fast.norm_bwd(*at, dY, H, weight, rstd, dH)
        if new is not None:
            return new
    rows, cols = _rows_cols("H", H, torch.bfloat16)
    index = H.get_device()
    dy = _tensor("dY", dY, torch.bfloat16, (rows, cols), index)
    w = _tensor("weight", weight, None, (cols,), index)
    dt = _dtype("weight", weight.dtype)
    rs = _tensor("rstd", rstd, torch.float32, (rows,), index)
    dh = None if dH is None else _tensor("dH", dH, torch.bfloat16, (rows, cols), index)
    if outs is None:
        dX, dW = torch.empty_like(dY), _empty_1d(cols, torch.float32, H.device)
    else:
        dX, dW = outs
        _tensor("dX", dX, torch.bfloat16, (rows, cols), index)
        _tensor("dW", dW, torch.float32, (cols,), index)
    if ws is None:
        size = lib.qlora_rmsnorm_bwd_workspace_bytes(rows, cols)
        ws = _empty_1d(size, torch.uint8, H.device) if size else None
    else:
        _tensor("ws", ws, None, ws.shape, index)
        size = ws.numel() * ws.element_size()
    _rmsnorm_bwd(index, dy, H.data_ptr(), w, dt, rs, dh, rows, cols, dX.data_ptr(), dW.data_ptr(), _at(ws), size)
    return dX, dW


def qlora_mx_linear(X: MXMatrix, W: MXMatrix, out=None):
    """Y = X W^T in bf16: X [M, K] in 8- or 4-bit, W [N, K] in 4-bit microscaled floats."""
    if out is None and (at := _fast_on(X.codes)):
        new = _fast.linear(*at, X.codes, X.scales, X.rows, X.cols, X.mx, W.codes, W.scales, W.rows, W.cols, W.mx)
        if new is not None:
            return new
    sx = X.c_struct("X")
    index = X.codes.get_device()
    sw = W.c_struct("W", index)
    if out is None:
        out = _empty(X.rows, W.rows, torch.bfloat16, X.codes.device)
        at = out.data_ptr()
    else:
        at = _tensor("out", out, torch.bfloat16, (X.rows, W.rows), index)
    _linear(index, byref(sx), byref(sw), at)
    return out


def qlora_mx_linear_grouped(X: MXMatrix, W: MXMatrix, offsets, out=None):
    """Y[i] = X[i] W_e^T for offsets[e] <= i < offsets[e + 1]: X [M, K] with its
    rows sorted by expert, W [experts * N, K] the experts' weights one below the
    other, offsets int32 [experts + 1] on the device. Rows that no expert has
    are left as they were (zero in a new Y)."""
    sx = X.c_struct("X")
    index = X.codes.get_device()
    sw = W.c_struct("W", index)
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be a tensor [experts + 1]")
    off = _tensor("offsets", offsets, torch.int32, offsets.shape, index)
    experts = offsets.shape[0] - 1
    if W.rows % experts:
        raise ValueError(f"W has {W.rows} rows, not a multiple of {experts} experts")
    shape = (X.rows, W.rows // experts)
    if out is None:
        out = torch.zeros(shape, dtype=torch.bfloat16, device=X.codes.device)
        at = out.data_ptr()
    else:
        at = _tensor("out", out, torch.bfloat16, shape, index)
    _linear_grouped(index, byref(sx), byref(sw), off, experts, at)
    return out
