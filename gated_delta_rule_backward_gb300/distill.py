"""ctypes binding of distillation from a teacher's top logits (include/distill.h) in libgdn.so.

Argument marshalling only.  ``distill_forward`` and ``distill_backward`` are the raw calls on caller-provided
tensors; ``forward`` and ``backward`` allocate the outputs.
"""
from __future__ import annotations

import ctypes

import torch

from . import gdn
from .decode import _allocating_on, _code, _hand_over, _index, _on_device, _stream

_lib = gdn._lib

# Every symbol include/distill.h declares.
EXPORTS = ["distill_forward", "distill_backward"]


class DistillParams(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int64), ("V", ctypes.c_int64), ("K", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("d_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("teacher_dtype", ctypes.c_int32), ("temperature", ctypes.c_float), ("reserved0", ctypes.c_int32),
    ]


_P, _vp = ctypes.POINTER(DistillParams), ctypes.c_void_p
_lib.distill_forward.argtypes = [_P] + [_vp] * 8
_lib.distill_forward.restype = ctypes.c_int
_lib.distill_backward.argtypes = [_P] + [_vp] * 7
_lib.distill_backward.restype = ctypes.c_int


def make_params(N, V, K, dtype=gdn.DTYPE_F32, teacher_dtype=gdn.DTYPE_F32, temperature=1.0, row_stride=None, d_stride=None) -> DistillParams:
    return DistillParams(N, V, K, V if row_stride is None else row_stride, V if d_stride is None else d_stride, int(dtype), int(teacher_dtype),
                         float(temperature), 0)


def _row_stride(t, what):
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be [N, V] with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def params_for(logits, indices, teacher, temperature=1.0, dlogits=None) -> DistillParams:
    """Parameters for logits [N, V] (any row stride), indices int32 and teacher [N, K] dense; dlogits (default: dense) of
    logits' shape and type, with any row stride."""
    N, V = logits.shape if logits.dim() == 2 else (0, 0)
    stride = _row_stride(logits, "logits")
    if indices.dim() != 2 or indices.shape != teacher.shape or indices.shape[0] != N or (teacher.numel() and not teacher.is_contiguous()):
        raise ValueError("indices and teacher must be contiguous [N, K]")
    _index(indices, "indices")
    if dlogits is not None and (dlogits.shape != logits.shape or dlogits.dtype != logits.dtype):
        raise ValueError("dlogits must have logits' shape and type")
    return make_params(N, V, indices.shape[1], _code(logits, "logits"), _code(teacher, "teacher"), temperature, stride,
                       None if dlogits is None else _row_stride(dlogits, "dlogits"))


def _ptr(t):
    return None if t is None else t.data_ptr()


def distill_forward(p: DistillParams, logits, indices, teacher, loss, lse, dloss=None, dlogits=None, stream=None):
    """Raw C-ABI call; with dloss and dlogits the gradient comes in the same call."""
    _on_device(logits, indices, teacher, loss, lse, dloss, dlogits)
    st = _lib.distill_forward(ctypes.byref(p), logits.data_ptr(), indices.data_ptr(), teacher.data_ptr(), loss.data_ptr(), lse.data_ptr(),
                              _ptr(dloss), _ptr(dlogits), _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, "distill_forward")


def distill_backward(p: DistillParams, logits, indices, teacher, lse, dloss, dlogits, stream=None):
    """Raw C-ABI call."""
    _on_device(logits, indices, teacher, lse, dloss, dlogits)
    st = _lib.distill_backward(ctypes.byref(p), logits.data_ptr(), indices.data_ptr(), teacher.data_ptr(), lse.data_ptr(), dloss.data_ptr(),
                               dlogits.data_ptr(), _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, "distill_backward")


def _rows(t, N, what):
    if t.dtype != torch.float32:
        raise TypeError(f"{what} must be float32")
    if t.numel() != N or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous [N]")


def forward(logits, indices, teacher, temperature=1.0, dloss=None, in_place=False, stream=None):
    """Allocate and run distill_forward.  Returns (loss, lse), and dlogits as a third where dloss [N] is given;
    in_place: the gradient replaces the logits."""
    p = params_for(logits, indices, teacher, temperature, logits if in_place else None)
    if dloss is not None:
        _rows(dloss, p.N, "dloss")
    elif in_place:
        raise ValueError("in_place needs dloss")
    with _allocating_on(stream):
        loss, lse = (torch.empty(p.N, dtype=torch.float32, device=logits.device) for _ in range(2))
        dlogits = None if dloss is None else logits if in_place else torch.empty(tuple(logits.shape), dtype=logits.dtype, device=logits.device)
        distill_forward(p, logits, indices, teacher, loss, lse, dloss, dlogits, stream)
    _hand_over(stream, loss, lse, None if in_place else dlogits)
    return (loss, lse) if dloss is None else (loss, lse, dlogits)


def backward(logits, indices, teacher, lse, dloss, temperature=1.0, in_place=False, stream=None):
    """Allocate and run distill_backward.  Returns dlogits; in_place: the gradient replaces the logits."""
    p = params_for(logits, indices, teacher, temperature, logits if in_place else None)
    _rows(lse, p.N, "lse")
    _rows(dloss, p.N, "dloss")
    with _allocating_on(stream):
        dlogits = logits if in_place else torch.empty(tuple(logits.shape), dtype=logits.dtype, device=logits.device)
        distill_backward(p, logits, indices, teacher, lse, dloss, dlogits, stream)
    _hand_over(stream, None if in_place else dlogits)
    return dlogits
