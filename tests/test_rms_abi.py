"""The norm's C ABI (include/rms.h) on the CPU: exports, sizes and argument validation.
Every call below fails its checks before any device work is enqueued."""
import ctypes
import os
import re

import pytest

from gated_delta_rule_backward_gb300 import gdn, rms

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4
BASE, MB = 0x7F0000000000, 1 << 24  # fake, aligned device addresses (never dereferenced)


def test_header_symbols_exported():
    hdr = open(os.path.join(ROOT, "include", "rms.h")).read()
    declared = set(re.findall(r"^\w[\w\s\*]*?\b(rms_\w+)\(", hdr, flags=re.M))
    assert declared == set(rms.EXPORTS)
    for name in declared:
        assert hasattr(gdn.library(), name), name


def _fwd(p, **ptrs):
    names = ("x", "residual", "weight", "h", "y", "scales", "rstd")
    a = {n: BASE + i * MB for i, n in enumerate(names)}
    a.update(ptrs)
    return gdn.library().rms_forward(ctypes.byref(p), *[a[n] for n in names], None)


def _bwd(p, ws_bytes=None, **ptrs):
    names = ("h", "weight", "rstd", "dy", "dh", "dx", "dweight", "ws")
    a = {n: BASE + i * MB for i, n in enumerate(names)}
    a.update(ptrs)
    return gdn.library().rms_backward(ctypes.byref(p), *[a[n] for n in names], rms.backward_workspace_bytes(p) if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(D=0), INVALID), (dict(x_s=63), INVALID), (dict(res_s=0), INVALID), (dict(x_dtype=3), INVALID),
    (dict(w_dtype=3), INVALID), (dict(y_dtype=4), INVALID), (dict(y_dtype=3, group=8), UNSUPPORTED), (dict(y_dtype=3, group=256), UNSUPPORTED),
    (dict(y_dtype=3, group=128), INVALID), (dict(D=1 << 29), UNSUPPORTED),
])
def test_sizes_refused(change, code):
    p = rms.make_params(**{**dict(rows=4, D=64), **change})
    assert _fwd(p) == code and _bwd(p, 1 << 20) == code
    assert rms.backward_workspace_bytes(p) == 0


def test_forward_validation():
    p = rms.make_params(4, 64)
    assert _fwd(p, x=None) == INVALID and _fwd(p, y=None) == INVALID
    assert _fwd(rms.make_params(4, 64, y_dtype=rms.E4M3), scales=None) == INVALID
    for n in ("x", "residual", "weight", "h", "y", "scales", "rstd"):
        assert _fwd(p, **{n: BASE + 20 * MB + 2}) == INVALID, n      # off its element
    assert _fwd(p, y=BASE + 64) == ALIAS and _fwd(p, h=BASE + 64) == ALIAS and _fwd(p, rstd=BASE + 2 * MB) == ALIAS
    assert _fwd(p, y=BASE + 3 * MB) == ALIAS                          # y over h
    assert _fwd(rms.make_params(4, 64, x_s=128), h=BASE) == ALIAS     # in place only on dense rows
    assert _fwd(rms.make_params(0, 64)) == OK


def test_backward_validation():
    p = rms.make_params(1000, 64)
    assert rms.backward_workspace_bytes(p) > 0
    for n in ("h", "rstd", "dy", "dx"):
        assert _bwd(p, **{n: None}) == INVALID, n
    assert _bwd(p, ws_bytes=rms.backward_workspace_bytes(p) - 1) == WORKSPACE and _bwd(p, ws=None) == WORKSPACE
    assert _bwd(p, ws=BASE + 7 * MB + 4) == INVALID
    assert _bwd(p, dx=BASE) == ALIAS and _bwd(p, dweight=BASE + MB) == ALIAS and _bwd(p, dx=BASE + 7 * MB) == ALIAS


def test_binding_refuses_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(3, 64), torch.zeros(64)
    rms.params_for(x, w, y_dtype=torch.float8_e4m3fn, group=32)
    for bad, err in ((dict(x=x.double()), TypeError), (dict(x=torch.zeros(3, 128)[:, ::2]), ValueError), (dict(weight=w[:32]), ValueError),
                     (dict(weight=w.double()), TypeError), (dict(residual=x.half()), ValueError), (dict(y_dtype=torch.int8), TypeError)):
        with pytest.raises(err):
            rms.params_for(**{**dict(x=x, weight=w), **bad})
