"""ctypes binding of linear attention with a decay for each head (include/la.h) in libgdn.so.

Argument marshalling only.  ``la_forward`` and ``la_backward`` are the raw calls on caller-provided tensors;
``forward`` and ``backward`` allocate the outputs and the workspace.  The states of several layers, and their moves
between slots, are ``decode``'s.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import gdn
from .decode import _allocating_on, _code, _hand_over, _index, _on_device, _rows, _stream

_lib = gdn._lib

# Every symbol include/la.h declares.
EXPORTS = ["la_form", "la_workspace_bytes", "la_backward_workspace_bytes", "la_forward", "la_backward", "la_selftest_wait_timeout"]

FORMS = {0: "token", 1: "chunked"}


class LaParams(ctypes.Structure):
    _fields_ = [
        ("n_seq", ctypes.c_int64), ("T", ctypes.c_int64), ("n_tok", ctypes.c_int64),
        ("H_k", ctypes.c_int64), ("H_v", ctypes.c_int64), ("S_k", ctypes.c_int64), ("S_v", ctypes.c_int64),
        ("n_slots", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
        ("q_s", ctypes.c_int64 * 2), ("k_s", ctypes.c_int64 * 2), ("v_s", ctypes.c_int64 * 2), ("g_s", ctypes.c_int64 * 2),
        ("in_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
    ]


_P, _vp = ctypes.POINTER(LaParams), ctypes.c_void_p
_lib.la_form.argtypes = [_P]
_lib.la_form.restype = ctypes.c_int
for _name in ("la_workspace_bytes", "la_backward_workspace_bytes"):
    getattr(_lib, _name).argtypes = [_P]
    getattr(_lib, _name).restype = ctypes.c_size_t
for _name in ("la_forward", "la_selftest_wait_timeout"):
    getattr(_lib, _name).argtypes = [_P] + [_vp] * 10 + [ctypes.c_size_t, _vp]
    getattr(_lib, _name).restype = ctypes.c_int
_lib.la_backward.argtypes = [_P] + [_vp] * 15 + [ctypes.c_size_t, _vp]
_lib.la_backward.restype = ctypes.c_int


def make_params(n_seq, T, H_k, H_v, S, S_v=None, n_tok=None, n_slots=None, slot_stride=None, scale=None, q_s=None, k_s=None, v_s=None,
                g_s=None, in_dtype=gdn.DTYPE_F32, gate_dtype=gdn.DTYPE_F32, y_dtype=gdn.DTYPE_F32) -> LaParams:
    """Parameter struct; S is the key head size, S_v the value head size (default S); strides
    default to the contiguous [n_tok, H, S] layouts, the pool to n_seq dense slots."""
    SV = S if S_v is None else int(S_v)
    p = LaParams()
    p.n_seq, p.T, p.n_tok = n_seq, T, n_seq * T if n_tok is None else n_tok
    p.H_k, p.H_v, p.S_k, p.S_v = H_k, H_v, S, SV
    p.n_slots = n_seq if n_slots is None else n_slots
    p.slot_stride = H_v * SV * S if slot_stride is None else slot_stride
    p.q_s[:] = q_s or (H_k * S, S)
    p.k_s[:] = k_s or (H_k * S, S)
    p.v_s[:] = v_s or (H_v * SV, SV)
    p.g_s[:] = g_s or (H_v, 1)
    p.in_dtype, p.gate_dtype, p.y_dtype = int(in_dtype), int(gate_dtype), int(y_dtype)
    p.scale = (1.0 / math.sqrt(S)) if scale is None else float(scale)
    return p


def params_for(q, k, v, g, pool, n_seq, T=None, y_dtype=None, scale=None) -> LaParams:
    """Parameters for these tensors: q, k [n_tok,H_k,S_k], v [n_tok,H_v,S_v] (row views of a packed buffer are fine),
    g [n_tok,H_v] of any strides (an expanded [H_v] is one decay a head), pool [n_slots,H_v,S_v,S_k] fp32 (dense slots, any
    distance between them).  T: the tokens of the longest sequence (default n_tok / n_seq; needed with cu_tokens, and best the
    true maximum: it decides the form and the workspace).  y_dtype: a torch dtype (default float32)."""
    n_tok, H_k, S = q.shape
    H_v, SV = v.shape[1], v.shape[2]
    if k.shape != q.shape or v.shape[0] != n_tok:
        raise ValueError("q, k and v must hold the same tokens")
    if tuple(g.shape) != (n_tok, H_v):
        raise ValueError("g must be [tokens, H_v]")
    if pool.dtype != torch.float32 or tuple(pool.shape[1:]) != (H_v, SV, S) or (pool.numel() and not pool[0].is_contiguous()):
        raise ValueError("the pool must be float32 [n_slots, H_v, S_v, S_k] with dense slots")
    dt = _code(q, "q")
    if _code(k, "k") != dt or _code(v, "v") != dt:
        raise TypeError("q, k, v must share one type")
    return make_params(n_seq, (n_tok // n_seq if n_seq else 0) if T is None else T, H_k, H_v, S, S_v=SV, n_tok=n_tok, n_slots=pool.shape[0],
                       slot_stride=pool.stride(0) if pool.shape[0] > 1 else H_v * SV * S, scale=scale, q_s=_rows(q, "q"), k_s=_rows(k, "k"),
                       v_s=_rows(v, "v"), g_s=(g.stride(0), g.stride(1)), in_dtype=dt, gate_dtype=_code(g, "g"),
                       y_dtype=gdn.DTYPE_F32 if y_dtype is None else _code(y_dtype, "y"))


def form(p: LaParams) -> str:
    """"token" or "chunked": the form these sizes run."""
    f = int(_lib.la_form(ctypes.byref(p)))
    if f < 0:
        raise ValueError("linear attention: unsupported sizes or types")
    return FORMS[f]


def workspace_bytes(p: LaParams) -> int:
    return int(_lib.la_workspace_bytes(ctypes.byref(p)))


def backward_workspace_bytes(p: LaParams) -> int:
    return int(_lib.la_backward_workspace_bytes(ctypes.byref(p)))


def workspace(p: LaParams, device):
    """A workspace for la_forward with these parameters (scratch: no call needs it zeroed)."""
    return torch.empty(max(workspace_bytes(p), 16), dtype=torch.uint8, device=device)


def backward_workspace(p: LaParams, device):
    """A workspace for la_backward with these parameters."""
    return torch.empty(max(backward_workspace_bytes(p), 16), dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _sequences(p, cu_tokens, *slots):
    if any(s.numel() != p.n_seq for s in slots) or (cu_tokens is not None and cu_tokens.numel() != p.n_seq + 1):
        raise ValueError("slots must have n_seq entries, cu_tokens n_seq + 1")
    return None if cu_tokens is None else _index(cu_tokens, "cu_tokens")


def _forward(name, p, q, k, v, g, cu_tokens, pool, slot_in, slot_out, y, workspace, stream):
    cu = _sequences(p, cu_tokens, slot_in, slot_out)
    slots = _index(slot_in, "slot_in"), _index(slot_out, "slot_out")
    _on_device(q, k, v, g, cu_tokens, pool, slot_in, slot_out, y, workspace)
    st = getattr(_lib, name)(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), cu, pool.data_ptr(),
                             *slots, y.data_ptr(), _ptr(workspace),
                             0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, name)


def la_forward(p: LaParams, q, k, v, g, cu_tokens, pool, slot_in, slot_out, y, workspace, stream=None):
    """Raw C-ABI call on caller-provided tensors; cu_tokens and the workspace (where it needs no bytes) may be None."""
    _forward("la_forward", p, q, k, v, g, cu_tokens, pool, slot_in, slot_out, y, workspace, stream)


def selftest_wait_timeout(p: LaParams, q, k, v, g, cu_tokens, pool, slot_in, slot_out, y, workspace, stream=None):
    """la_forward's chunked form with a hand-over withheld: its bounded waits run out, and the next device_status says so."""
    _forward("la_selftest_wait_timeout", p, q, k, v, g, cu_tokens, pool, slot_in, slot_out, y, workspace, stream)


def la_backward(p: LaParams, q, k, v, g, cu_tokens, pool, slot_in, dy, dstate_T, dq, dk, dv, dg, dstate_0, workspace, stream=None):
    """Raw C-ABI call; cu_tokens, dstate_T and dstate_0 may be None."""
    cu = _sequences(p, cu_tokens, slot_in)
    slots = _index(slot_in, "slot_in")
    _on_device(q, k, v, g, cu_tokens, pool, slot_in, dy, dstate_T, dq, dk, dv, dg, dstate_0, workspace)
    st = _lib.la_backward(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), cu, pool.data_ptr(),
                          slots, dy.data_ptr(), _ptr(dstate_T), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(),
                          _ptr(dstate_0), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, "la_backward")


def forward(q, k, v, g, pool, slot_in, slot_out=None, cu_tokens=None, T=None, scale=None, y_dtype=None, stream=None):
    """Allocate y and run la_forward (slot_out None: in place).  Returns y [n_tok,H_v,S_v]."""
    if cu_tokens is not None and T is None:
        raise ValueError("with cu_tokens, T (the tokens of the longest sequence) must be given")
    p = params_for(q, k, v, g, pool, slot_in.numel(), T=T, y_dtype=y_dtype, scale=scale)
    with _allocating_on(stream):
        y = torch.empty(v.shape, dtype=torch.float32 if y_dtype is None else y_dtype, device=v.device)
        ws = workspace(p, v.device) if workspace_bytes(p) else None
        la_forward(p, q, k, v, g, cu_tokens, pool, slot_in, slot_in if slot_out is None else slot_out, y, ws, stream)
    _hand_over(stream, y)
    return y


def backward(q, k, v, g, pool, slot_in, dy, dstate_T=None, cu_tokens=None, T=None, scale=None, stream=None):
    """Allocate and run la_backward.  dy [n_tok,H_v,S_v] dense, of q's type; dstate_T fp32 [n_seq,H_v,S_v,S_k] dense, or None.
    Returns (dq, dk, dv, dg, dstate_0); dg is fp32 [n_tok,H_v] (of an expanded g, the gradient is its sum over the tokens)."""
    if cu_tokens is not None and T is None:
        raise ValueError("with cu_tokens, T (the tokens of the longest sequence) must be given")
    n_seq = slot_in.numel()
    p = params_for(q, k, v, g, pool, n_seq, T=T, scale=scale)
    if dy.dtype != q.dtype or (dstate_T is not None and dstate_T.dtype != torch.float32):
        raise TypeError("dy must have q's type, and dstate_T float32")
    states = (n_seq, *pool.shape[1:])
    if dy.shape != v.shape or not dy.is_contiguous() or (dstate_T is not None and (tuple(dstate_T.shape) != states or not dstate_T.is_contiguous())):
        raise ValueError("dy must be contiguous of v's shape, and dstate_T contiguous [n_seq, H_v, S_v, S_k]")
    with _allocating_on(stream):
        new = lambda shape, dtype: torch.empty(tuple(shape), dtype=dtype, device=q.device)
        out = [new(q.shape, q.dtype), new(k.shape, q.dtype), new(v.shape, q.dtype), new(g.shape, torch.float32), new(states, torch.float32)]
        la_backward(p, q, k, v, g, cu_tokens, pool, slot_in, dy, dstate_T, *out, backward_workspace(p, q.device), stream)
    _hand_over(stream, *out)
    return tuple(out)
