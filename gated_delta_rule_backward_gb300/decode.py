"""ctypes binding of the gated delta rule's serving form (include/gdn_decode.h) in libgdn.so:
the recurrence over a pool of states, and the moves of states between its slots.

Argument marshalling only.  The raw calls (``gdn_decode``, ``gdn_states_move``) take
caller-provided tensors on the current CUDA device and raise ``gdn.GdnError`` on a non-OK
status; ``decode`` allocates the output.  A decoding loop keeps ``params_for``'s answer while
its shapes and strides stay.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import gdn

_lib = gdn._lib

# Every symbol include/gdn_decode.h declares.
EXPORTS = ["gdn_decode_supported", "gdn_decode", "gdn_states_move"]

DTYPE_CODES = {torch.float32: gdn.DTYPE_F32, torch.bfloat16: gdn.DTYPE_BF16, torch.float16: gdn.DTYPE_F16}


class DecodeParams(ctypes.Structure):
    _fields_ = [
        ("n_seq", ctypes.c_int64), ("T", ctypes.c_int64), ("n_tok", ctypes.c_int64),
        ("H_k", ctypes.c_int64), ("H_v", ctypes.c_int64), ("S_k", ctypes.c_int64), ("S_v", ctypes.c_int64),
        ("n_slots", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
        ("q_s", ctypes.c_int64 * 2), ("k_s", ctypes.c_int64 * 2), ("v_s", ctypes.c_int64 * 2),
        ("gate", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved0", ctypes.c_int32),
    ]


_P = ctypes.POINTER(DecodeParams)
_vp, _i64 = ctypes.c_void_p, ctypes.c_int64
_lib.gdn_decode_supported.argtypes = [_P]
_lib.gdn_decode_supported.restype = ctypes.c_int
_lib.gdn_decode.argtypes = [_P] + [_vp] * 11
_lib.gdn_decode.restype = ctypes.c_int
_lib.gdn_states_move.argtypes = [_vp] + [_i64] * 5 + [_vp] * 2 + [_i64] * 2 + [_vp]
_lib.gdn_states_move.restype = ctypes.c_int


def make_params(n_seq, T, H_k, H_v, S, kda=False, S_v=None, n_tok=None, n_slots=None, slot_stride=None, scale=None,
                q_s=None, k_s=None, v_s=None, in_dtype=gdn.DTYPE_F32, gate_dtype=gdn.DTYPE_F32,
                y_dtype=gdn.DTYPE_F32) -> DecodeParams:
    """Parameter struct; S is the key head size, S_v the value head size (default S); strides
    default to the contiguous [n_tok, H, S] layouts, the pool to n_seq dense slots."""
    SV = S if S_v is None else int(S_v)
    p = DecodeParams()
    p.n_seq, p.T, p.n_tok = n_seq, T, n_seq * T if n_tok is None else n_tok
    p.H_k, p.H_v, p.S_k, p.S_v = H_k, H_v, S, SV
    p.n_slots = n_seq if n_slots is None else n_slots
    p.slot_stride = H_v * SV * S if slot_stride is None else slot_stride
    p.q_s[:] = q_s or (H_k * S, S)
    p.k_s[:] = k_s or (H_k * S, S)
    p.v_s[:] = v_s or (H_v * SV, SV)
    p.gate = gdn.GATE_KDA if kda else gdn.GATE_SCALAR
    p.in_dtype, p.gate_dtype, p.y_dtype = int(in_dtype), int(gate_dtype), int(y_dtype)
    p.scale = (1.0 / math.sqrt(S)) if scale is None else float(scale)
    return p


def _code(t, what):
    code = DTYPE_CODES.get(t if isinstance(t, torch.dtype) else t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32, bfloat16 or float16")
    return code


def _rows(t, what):
    """Element strides {token, head} of a [n_tok, H, S] view."""
    if t.dim() != 3 or (t.numel() and t.stride(2) != 1):
        raise ValueError(f"{what} must be [tokens, heads, head size] with contiguous heads")
    return (t.stride(0), t.stride(1)) if t.numel() else (t.shape[1] * t.shape[2], t.shape[2])


def params_for(q, k, v, g, beta, pool, n_seq, y_dtype=None, scale=None) -> DecodeParams:
    """Parameters for these tensors: q, k [n_tok,H_k,S_k], v [n_tok,H_v,S_v] (row views of a
    packed buffer are fine), g [n_tok,H_v] or [n_tok,H_v,S_k], beta [n_tok,H_v], pool
    [n_slots,H_v,S_v,S_k] fp32 (dense slots, any distance between them).  y_dtype: a torch
    dtype (default float32).  Calls without cu_tokens take n_tok / n_seq tokens a sequence."""
    n_tok, H_k, S = q.shape
    H_v, SV = v.shape[1], v.shape[2]
    kda = g.dim() == 3
    if k.shape != q.shape or v.shape[0] != n_tok:
        raise ValueError("q, k and v must hold the same tokens")
    if tuple(g.shape) != ((n_tok, H_v, S) if kda else (n_tok, H_v)) or tuple(beta.shape) != (n_tok, H_v):
        raise ValueError("g must be [tokens, H_v] or [tokens, H_v, S_k], and beta [tokens, H_v]")
    if pool.dtype != torch.float32 or tuple(pool.shape[1:]) != (H_v, SV, S) or \
            (pool.numel() and not pool[0].is_contiguous()):
        raise ValueError("the pool must be float32 [n_slots, H_v, S_v, S_k] with dense slots")
    if g.numel() and not (g.is_contiguous() and beta.is_contiguous()):
        raise ValueError("g and beta must be contiguous")
    dt, gt = _code(q, "q"), _code(g, "g")
    if _code(k, "k") != dt or _code(v, "v") != dt or _code(beta, "beta") != gt:
        raise TypeError("q, k, v must share one type, and g, beta one type")
    return make_params(n_seq, n_tok // n_seq if n_seq else 0, H_k, H_v, S, kda, S_v=SV, n_tok=n_tok, n_slots=pool.shape[0],
                       slot_stride=pool.stride(0) if pool.shape[0] > 1 else H_v * SV * S, scale=scale,
                       q_s=_rows(q, "q"), k_s=_rows(k, "k"), v_s=_rows(v, "v"), in_dtype=dt, gate_dtype=gt,
                       y_dtype=gdn.DTYPE_F32 if y_dtype is None else _code(y_dtype, "y"))


def supported(p: DecodeParams) -> int:
    """0 (GDN_OK) when the sizes and types are supported, else the status gdn_decode would return."""
    return int(_lib.gdn_decode_supported(ctypes.byref(p)))


def _stream(stream):
    """A stream's handle as a number (default: the current device's current stream)."""
    if stream is not None:
        return stream.cuda_stream
    # the handle itself: torch.cuda.current_stream() makes an object around it, 3 us a call
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _allocating_on(stream):
    """What an allocating call makes comes from the pool of the stream that uses it: memory of the current stream's may
    still be in use there, and a workspace that goes back to it could be handed out while `stream` works in it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _hand_over(stream, *tensors):
    """Outputs made on `stream` are also the current stream's: freed ones are not used again before its work on them
    is done.  (That the current stream waits for `stream` first is the caller's part.)"""
    if stream is not None:
        here = torch.cuda.current_stream()
        for t in tensors:
            if t is not None:
                t.record_stream(here)


def _index(t, what):
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise TypeError(f"{what} must be contiguous int32")
    return t.data_ptr()


def _on_device(*tensors):
    """Refuses tensors that are not on the current device, whose addresses its kernels must not touch."""
    at = tensors[0].get_device()
    for t in tensors:  # a loop: any() would take half as long again
        if t is not None and t.get_device() != at:
            at = -1
    if at < 0 or at != torch._C._cuda_getDevice():
        raise ValueError("every tensor must be on the current CUDA device")


def gdn_decode(p: DecodeParams, q, k, v, g, beta, cu_tokens, pool, slot_in, slot_out, y, stream=None):
    """Raw C-ABI call on caller-provided tensors; cu_tokens may be None."""
    if slot_in.numel() != p.n_seq or slot_out.numel() != p.n_seq or (cu_tokens is not None and cu_tokens.numel() != p.n_seq + 1):
        raise ValueError("slot_in and slot_out must have n_seq entries, cu_tokens n_seq + 1")
    st = _lib.gdn_decode(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                         None if cu_tokens is None else _index(cu_tokens, "cu_tokens"), pool.data_ptr(),
                         _index(slot_in, "slot_in"), _index(slot_out, "slot_out"), y.data_ptr(), _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, "gdn_decode")


def decode(q, k, v, g, beta, pool, slot_in, slot_out=None, cu_tokens=None, scale=None, y_dtype=None, stream=None):
    """Allocate y and run gdn_decode (slot_out None: in place).  Returns y [n_tok,H_v,S_v]."""
    p = params_for(q, k, v, g, beta, pool, slot_in.numel(), y_dtype=y_dtype, scale=scale)
    with _allocating_on(stream):
        y = torch.empty(v.shape, dtype=torch.float32 if y_dtype is None else y_dtype, device=v.device)
        gdn_decode(p, q, k, v, g, beta, cu_tokens, pool, slot_in, slot_in if slot_out is None else slot_out, y, stream)
    _hand_over(stream, y)
    return y


def gdn_states_move(pool, src, dst, group=1, stream=None):
    """Slot dst[i] = what slot src[i] held (zeros for -1), in every layer, the moves of each
    consecutive `group` simultaneous.  pool: [n_layers, n_slots, ...] of any type, every
    (layer, slot) dense; src, dst: int32 device tensors of one length."""
    shape, strides, es = pool.shape, pool.stride(), pool.element_size()
    n = src.numel()
    if len(shape) < 2 or dst.numel() != n:
        raise ValueError("pool must be [n_layers, n_slots, ...], and src and dst of one length")
    state = 1  # a slot's elements, dense from the last dimension on
    for size, step in zip(shape[:1:-1], strides[:1:-1]):
        if size != 1 and step != state and pool.numel():
            raise ValueError("each layer's slots must be dense")
        state *= size
    L, S = shape[0], shape[1]
    st = _lib.gdn_states_move(pool.data_ptr(), L, strides[0] * es if L > 1 else 0, S, strides[1] * es if S > 1 else state * es,
                              state * es, _index(src, "src"), _index(dst, "dst"), n, group, _stream(stream))
    if st != gdn.GDN_OK:
        raise gdn.GdnError(st, "gdn_states_move")
