"""ctypes binding of the root-mean-square norm (include/rms.h) in libgdn.so.

Argument marshalling only.  ``rms_forward`` and ``rms_backward`` are the raw calls on
caller-provided tensors; ``forward`` and ``backward`` allocate the outputs.
"""
from __future__ import annotations

import ctypes

import torch

from . import gdn
from .decode import DTYPE_CODES, _allocating_on, _hand_over, _stream

_lib = gdn._lib

# Every symbol include/rms.h declares.
EXPORTS = ["rms_backward_workspace_bytes", "rms_forward", "rms_backward"]

E4M3 = 3
Y_CODES = {**DTYPE_CODES, torch.float8_e4m3fn: E4M3}


class RmsParams(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("D", ctypes.c_int64), ("x_s", ctypes.c_int64), ("res_s", ctypes.c_int64),
        ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("group", ctypes.c_int32),
        ("eps", ctypes.c_float), ("reserved0", ctypes.c_int32),
    ]


_P, _vp = ctypes.POINTER(RmsParams), ctypes.c_void_p
_lib.rms_backward_workspace_bytes.argtypes = [_P]
_lib.rms_backward_workspace_bytes.restype = ctypes.c_size_t
_lib.rms_forward.argtypes = [_P] + [_vp] * 8
_lib.rms_forward.restype = ctypes.c_int
_lib.rms_backward.argtypes = [_P] + [_vp] * 8 + [ctypes.c_size_t, _vp]
_lib.rms_backward.restype = ctypes.c_int


def make_params(rows, D, x_dtype=gdn.DTYPE_F32, w_dtype=gdn.DTYPE_F32, y_dtype=gdn.DTYPE_F32, group=0, eps=1e-6, x_s=None,
                res_s=None) -> RmsParams:
    return RmsParams(rows, D, D if x_s is None else x_s, D if res_s is None else res_s, int(x_dtype), int(w_dtype), int(y_dtype),
                     int(group), float(eps), 0)


def _code(t, codes, what):
    code = codes.get(t)
    if code is None:
        raise TypeError(f"{what}: unsupported type {t}")
    return code


def _row_stride(t, what):
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be [rows, D] with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def params_for(x, weight=None, eps=1e-6, y_dtype=None, group=0, residual=None) -> RmsParams:
    """Parameters for these tensors: x [rows, D] (backward: h), residual (backward: dy) of the
    same shape and type, both with any row stride, weight [D].  y_dtype: a torch dtype (default x's);
    torch.float8_e4m3fn makes codes with one scale a row (group 0) or per `group` columns."""
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual must have x's shape and type")
    if weight is not None and (tuple(weight.shape) != (x.shape[1],) or not weight.is_contiguous()):
        raise ValueError("weight must be contiguous [D]")
    xc = _code(x.dtype, DTYPE_CODES, "x")
    return make_params(x.shape[0], x.shape[1], xc, gdn.DTYPE_F32 if weight is None else _code(weight.dtype, DTYPE_CODES, "weight"),
                       xc if y_dtype is None else _code(y_dtype, Y_CODES, "y"), group, eps, _row_stride(x, "x"),
                       None if residual is None else _row_stride(residual, "residual"))


def backward_workspace_bytes(p: RmsParams) -> int:
    return int(_lib.rms_backward_workspace_bytes(ctypes.byref(p)))


def workspace(p: RmsParams, device):
    """A workspace for rms_backward's dweight with these parameters."""
    return torch.empty(max(backward_workspace_bytes(p), 16), dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def rms_forward(p: RmsParams, x, residual, weight, h, y, scales, rstd, stream=None):
    """Raw C-ABI call; residual, weight, h, scales and rstd may be None."""
    st = _lib.rms_forward(ctypes.byref(p), x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(h), y.data_ptr(), _ptr(scales), _ptr(rstd),
                          _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, "rms_forward")


def rms_backward(p: RmsParams, h, weight, rstd, dy, dh, dx, dweight, workspace, stream=None):
    """Raw C-ABI call; weight, dh, dweight (and then the workspace) may be None."""
    st = _lib.rms_backward(ctypes.byref(p), h.data_ptr(), _ptr(weight), rstd.data_ptr(), dy.data_ptr(), _ptr(dh), dx.data_ptr(), _ptr(dweight),
                           _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
                           _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, "rms_backward")


def forward(x, weight=None, residual=None, eps=1e-6, y_dtype=None, group=0, stream=None):
    """Allocate and run rms_forward on x [rows, D].  Returns (y, h, rstd), or (y, scales, h, rstd)
    where y holds e4m3 codes.  Without a residual h is x itself."""
    p = params_for(x, weight, eps, y_dtype, group, residual)
    rows, D, dev = x.shape[0], x.shape[1], x.device
    with _allocating_on(stream):
        h = None if residual is None else torch.empty((rows, D), dtype=x.dtype, device=dev)
        y = torch.empty((rows, D), dtype=x.dtype if y_dtype is None else y_dtype, device=dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        scales = torch.empty((rows, D // group) if group else (rows,), dtype=torch.float32, device=dev) if p.y_dtype == E4M3 else None
        rms_forward(p, x, residual, weight, h, y, scales, rstd, stream)
    _hand_over(stream, h, y, rstd, scales)
    h = x if residual is None else h
    return (y, h, rstd) if scales is None else (y, scales, h, rstd)


def backward(h, rstd, dy, weight=None, dh=None, stream=None):
    """Allocate and run rms_backward.  h, dy [rows, D] may have any row stride; dh, of h's type, and
    rstd (fp32, a number a row) are dense.  Returns (dx, dweight); dweight is None without a weight."""
    p = params_for(h, weight, residual=dy)
    if rstd.dtype != torch.float32 or (dh is not None and dh.dtype != h.dtype):
        raise TypeError("rstd must be float32, and dh of h's type")
    if rstd.numel() != h.shape[0] or not rstd.is_contiguous() or (dh is not None and (dh.shape != h.shape or not dh.is_contiguous())):
        raise ValueError("rstd must be contiguous [rows], and dh contiguous of h's shape")
    with _allocating_on(stream):
        dx = torch.empty(tuple(h.shape), dtype=h.dtype, device=h.device)
        dw = ws = None
        if weight is not None:
            dw, ws = torch.empty(h.shape[1], dtype=torch.float32, device=h.device), workspace(p, h.device)
        rms_backward(p, h, weight, rstd, dy, dh, dx, dw, ws, stream)
    _hand_over(stream, dx, dw)
    return dx, dw
