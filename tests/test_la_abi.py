"""Linear attention's C ABI (include/la.h) on the CPU: exports, sizes and argument validation.
Every call below fails its checks before any device work is enqueued."""
import ctypes
import os
import re

import pytest

from gated_delta_rule_backward_gb300 import gdn, la

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4
BASE, MB = 0x7F0000000000, 1 << 26  # fake, aligned device addresses (never dereferenced)


def test_header_symbols_exported():
    hdr = open(os.path.join(ROOT, "include", "la.h")).read()
    declared = set(re.findall(r"^\w[\w\s\*]*?\b(la_\w+)\(", hdr, flags=re.M))
    assert declared == set(la.EXPORTS)
    for name in declared:
        assert hasattr(gdn.library(), name), name
    assert ctypes.sizeof(la.LaParams) == 9 * 8 + 8 * 8 + 16


F = ("q", "k", "v", "g", "cu", "pool", "slot_in", "slot_out", "y", "ws")
B = ("q", "k", "v", "g", "cu", "pool", "slot_in", "dy", "dstate_T", "dq", "dk", "dv", "dg", "dstate_0", "ws")


def _call(fn, names, p, ws_bytes, ptrs):
    a = {n: BASE + i * MB for i, n in enumerate(names)}
    a.update(cu=None)
    a.update(ptrs)
    return fn(ctypes.byref(p), *[a[n] for n in names], ws_bytes, None)


def _fwd(p, ws_bytes=None, **ptrs):
    return _call(gdn.library().la_forward, F, p, la.workspace_bytes(p) if ws_bytes is None else ws_bytes, ptrs)


def _bwd(p, ws_bytes=None, **ptrs):
    return _call(gdn.library().la_backward, B, p, la.backward_workspace_bytes(p) if ws_bytes is None else ws_bytes, ptrs)


@pytest.mark.parametrize("change,code", [
    (dict(n_seq=-1), INVALID), (dict(T=-1), INVALID), (dict(H_k=0), INVALID), (dict(H_k=3), INVALID), (dict(in_dtype=3), INVALID),
    (dict(gate_dtype=-1), INVALID), (dict(y_dtype=7), INVALID), (dict(q_s=(-1, 64)), INVALID), (dict(g_s=(0, -4)), INVALID), (dict(slot_stride=64), INVALID),
    (dict(slot_stride=4 * 64 * 64 + 2), INVALID), (dict(S=48), UNSUPPORTED), (dict(S=512), UNSUPPORTED), (dict(S_v=24), UNSUPPORTED),
    (dict(S_v=272), UNSUPPORTED), (dict(H_k=70000, H_v=70000), UNSUPPORTED), (dict(n_tok=1 << 31), UNSUPPORTED), (dict(n_seq=1 << 28, n_tok=0, T=0), UNSUPPORTED),
])
def test_sizes_refused(change, code):
    p = la.make_params(**{**dict(n_seq=2, T=3, H_k=2, H_v=4, S=64), **change})
    assert _fwd(p, 1 << 30) == code and _bwd(p, 1 << 30) == code
    assert la.workspace_bytes(p) == 0 and la.backward_workspace_bytes(p) == 0 and gdn.library().la_form(ctypes.byref(p)) == -1


def test_head_sizes_of_the_backward_pass():
    p = la.make_params(2, 3, 2, 4, 64, S_v=48)
    assert gdn.library().la_form(ctypes.byref(p)) >= 0 and la.backward_workspace_bytes(p) == 0 and _bwd(p, 1 << 30) == UNSUPPORTED


def test_forward_validation():
    p = la.make_params(2, 3, 2, 4, 64)
    for n in ("q", "k", "v", "g", "pool", "slot_in", "slot_out", "y"):
        assert _fwd(p, **{n: None}) == INVALID, n
    for n in ("q", "k", "v", "g", "cu", "slot_in", "slot_out", "y"):
        assert _fwd(p, **{n: BASE + 20 * MB + 2}) == INVALID, n      # off its element
    assert _fwd(p, pool=BASE + 20 * MB + 8) == INVALID
    assert _fwd(p, y=BASE + 2 * MB + 64) == ALIAS and _fwd(p, pool=BASE) == ALIAS and _fwd(p, y=BASE + 5 * MB) == ALIAS
    assert _fwd(la.make_params(2, 3, 2, 4, 64, n_tok=7)) == INVALID   # without cu_tokens
    assert _fwd(la.make_params(0, 3, 2, 4, 64)) == OK


def test_backward_validation():
    p = la.make_params(2, 3, 2, 4, 64)
    assert la.backward_workspace_bytes(p) > 0
    for n in ("q", "k", "v", "g", "pool", "slot_in", "dy", "dq", "dk", "dv", "dg"):
        assert _bwd(p, **{n: None}) == INVALID, n
    for n in ("dstate_T", "dstate_0", "ws"):
        assert _bwd(p, **{n: BASE + 20 * MB + 8}) == INVALID, n
    assert _bwd(p, ws_bytes=la.backward_workspace_bytes(p) - 1) == WORKSPACE and _bwd(p, ws=None) == WORKSPACE
    assert _bwd(p, dq=BASE) == ALIAS and _bwd(p, dk=BASE + 9 * MB) == ALIAS and _bwd(p, dstate_0=BASE + 8 * MB) == ALIAS and _bwd(p, ws=BASE + 11 * MB) == ALIAS
    assert _bwd(p, dv=BASE + 7 * MB) == ALIAS


def test_binding_refuses_tensors():
    torch = pytest.importorskip("torch")
    q, v, g, pool = torch.zeros(6, 2, 32), torch.zeros(6, 4, 32), torch.zeros(6, 4), torch.zeros(3, 4, 32, 32)
    ok = dict(q=q, k=q, v=v, g=g, pool=pool, n_seq=2)
    la.params_for(**ok)
    assert tuple(la.params_for(**{**ok, "g": torch.zeros(4).expand(6, 4)}).g_s) == (0, 1)
    for bad, err in ((dict(k=q[:5]), ValueError), (dict(v=v[:5]), ValueError), (dict(g=g[:, :3]), ValueError), (dict(g=torch.zeros(6, 4, 32)), ValueError),
                     (dict(pool=pool.half()), ValueError), (dict(pool=pool.transpose(2, 3)), ValueError), (dict(k=q.half()), TypeError),
                     (dict(q=q.double(), k=q.double()), TypeError), (dict(g=g.double()), TypeError), (dict(y_dtype=torch.int8), TypeError),
                     (dict(q=torch.zeros(6, 2, 64)[:, :, ::2], k=torch.zeros(6, 2, 64)[:, :, ::2]), ValueError)):
        with pytest.raises(err):
            la.params_for(**{**ok, **bad})
    slot = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        la.forward(q, q, v, g, pool, slot, cu_tokens=torch.zeros(3, dtype=torch.int32))    # T is needed
    for bad, err in ((dict(dy=v.half()), TypeError), (dict(dy=v[:5]), ValueError), (dict(dy=torch.zeros(6, 4, 64)[:, :, :32]), ValueError),
                     (dict(dy=v, dstate_T=torch.zeros(3, 4, 32, 32)), ValueError), (dict(dy=v, dstate_T=torch.zeros(2, 4, 32, 32).double()), TypeError),
                     (dict(dy=v, dstate_T=torch.zeros(2, 4, 32, 32).transpose(2, 3)), ValueError)):
        with pytest.raises(err):
            la.backward(q, q, v, g, pool, slot, **bad)
    p = la.params_for(**ok)
    with pytest.raises(ValueError):
        la.la_forward(p, q, q, v, g, None, pool, slot[:1], slot, v, None)
    with pytest.raises(TypeError):
        la.la_forward(p, q, q, v, g, None, pool, slot.long(), slot, v, None)
