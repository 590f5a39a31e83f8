"""ctypes binding of a beam search's selection (include/beam.h) in libgdn.so.

Argument marshalling only.  ``beam_select`` is the raw call on caller-provided tensors;
``select`` allocates the outputs and the workspace.
"""
from __future__ import annotations

import ctypes

import torch

from . import gdn
from .decode import DTYPE_CODES, _allocating_on, _hand_over, _stream

_lib = gdn._lib

# Every symbol include/beam.h declares.
EXPORTS = ["beam_workspace_bytes", "beam_select"]


class BeamParams(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("V", ctypes.c_int64), ("row_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("n_out", ctypes.c_int32), ("pad_token", ctypes.c_int32), ("reserved0", ctypes.c_int32),
    ]


_P, _vp = ctypes.POINTER(BeamParams), ctypes.c_void_p
_lib.beam_workspace_bytes.argtypes = [_P]
_lib.beam_workspace_bytes.restype = ctypes.c_size_t
_lib.beam_select.argtypes = [_P] + [_vp] * 9 + [ctypes.c_size_t, _vp]
_lib.beam_select.restype = ctypes.c_int


def make_params(N, K, V, dtype=gdn.DTYPE_F32, n_out=None, pad_token=0, row_stride=None) -> BeamParams:
    return BeamParams(N, K, V, V if row_stride is None else row_stride, int(dtype), K if n_out is None else n_out, pad_token, 0)


def params_for(logits, scores, n_out=None, pad_token=0) -> BeamParams:
    """Parameters for logits [N K, V] (any row stride) and scores [N, K] fp32; n_out defaults to K."""
    code = DTYPE_CODES.get(logits.dtype)
    if code is None or scores.dtype != torch.float32:
        raise TypeError("logits must be float32, bfloat16 or float16, and scores float32")
    if logits.dim() != 2 or scores.dim() != 2 or logits.shape[0] != scores.numel() or (scores.numel() and not scores.is_contiguous()) or \
            (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [N K, V] with contiguous rows, and scores contiguous [N, K]")
    N, K = scores.shape
    V = logits.shape[1]
    return make_params(N, K, V, code, n_out, pad_token, logits.stride(0) if logits.shape[0] > 1 else V)


def workspace_bytes(p: BeamParams) -> int:
    return int(_lib.beam_workspace_bytes(ctypes.byref(p)))


def workspace(p: BeamParams, device):
    """A workspace for beam_select with these parameters (scratch: no call needs it zeroed)."""
    return torch.empty(max(workspace_bytes(p), 16), dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def beam_select(p: BeamParams, logits, scores, done, slots, scores_out, parent, token, src_slots, workspace, stream=None):
    """Raw C-ABI call; done (uint8 or bool), slots and src_slots may be None."""
    st = _lib.beam_select(ctypes.byref(p), logits.data_ptr(), scores.data_ptr(), _ptr(done), _ptr(slots), scores_out.data_ptr(),
                          parent.data_ptr(), token.data_ptr(), _ptr(src_slots), workspace.data_ptr(),
                          workspace.numel() * workspace.element_size(), _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, "beam_select")


def select(logits, scores, done=None, slots=None, n_out=None, pad_token=0, stream=None):
    """Allocate and run beam_select.  Returns (scores, parent, token), each [N, n_out], and the
    parents' slots as a fourth where slots [N, K] int32 is given."""
    p = params_for(logits, scores, n_out, pad_token)
    for t, types in ((done, (torch.uint8, torch.bool)), (slots, (torch.int32,))):
        if t is not None and (t.shape != scores.shape or t.dtype not in types or not t.is_contiguous()):
            raise ValueError("done (uint8 or bool) and slots (int32) must be contiguous [N, K]")
    N, dev = scores.shape[0], logits.device
    i32 = lambda: torch.empty((N, p.n_out), dtype=torch.int32, device=dev)
    with _allocating_on(stream):
        out = [torch.empty((N, p.n_out), dtype=torch.float32, device=dev), i32(), i32()]
        src = i32() if slots is not None else None
        beam_select(p, logits, scores, done, slots, *out, src, workspace(p, dev), stream)
    _hand_over(stream, *out, src)
    return tuple(out) if src is None else (*out, src)
