"""Distillation's C ABI (include/distill.h) on the CPU: exports, sizes and argument validation.
Every call below fails its checks before any device work is enqueued."""
import ctypes
import os
import re

import pytest

from gated_delta_rule_backward_gb300 import distill, gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIAS = 0, 1, 2, 3
BASE, MB = 0x7F0000000000, 1 << 24  # fake, aligned device addresses (never dereferenced)


def test_header_symbols_exported():
    hdr = open(os.path.join(ROOT, "include", "distill.h")).read()
    declared = set(re.findall(r"^\w[\w\s\*]*?\b(distill_\w+)\(", hdr, flags=re.M))
    assert declared == set(distill.EXPORTS)
    for name in declared:
        assert hasattr(gdn.library(), name), name


F = ("logits", "indices", "teacher", "loss", "lse", "dloss", "dlogits")
B = ("logits", "indices", "teacher", "lse", "dloss", "dlogits")


def _call(name, names, p, ptrs):
    a = {n: BASE + i * MB for i, n in enumerate(names)}
    a.update(ptrs)
    return getattr(gdn.library(), name)(ctypes.byref(p), *[a[n] for n in names], None)


def _fwd(p, **ptrs):
    return _call("distill_forward", F, p, ptrs)


def _bwd(p, **ptrs):
    return _call("distill_backward", B, p, ptrs)


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), INVALID), (dict(V=0), INVALID), (dict(K=-1), INVALID), (dict(row_stride=99), INVALID), (dict(d_stride=99), INVALID), (dict(dtype=3), INVALID),
    (dict(teacher_dtype=-1), INVALID), (dict(temperature=0.0), INVALID), (dict(temperature=-1.0), INVALID), (dict(temperature=float("nan")), INVALID),
    (dict(temperature=float("inf")), INVALID), (dict(K=1025), UNSUPPORTED), (dict(V=(1 << 30) + 1), UNSUPPORTED), (dict(N=(1 << 27) + 1), UNSUPPORTED),
])
def test_sizes_refused(change, code):
    p = distill.make_params(**{**dict(N=4, V=100, K=8), **change})
    assert _fwd(p) == code and _bwd(p) == code


def test_pointers_refused():
    p = distill.make_params(4, 100, 8)
    for n in ("logits", "indices", "teacher", "loss", "lse", "dloss", "dlogits"):
        assert _fwd(p, **{n: None}) == INVALID, n          # one of dloss and dlogits without the other as well
        assert _fwd(p, **{n: BASE + 20 * MB + 2}) == INVALID, n
    for n in B:
        assert _bwd(p, **{n: None}) == INVALID, n
        assert _bwd(p, **{n: BASE + 20 * MB + 2}) == INVALID, n
    assert _fwd(distill.make_params(0, 100, 8)) == OK and _bwd(distill.make_params(0, 100, 8)) == OK


def test_aliases_refused():
    p = distill.make_params(4, 100, 8)
    assert _fwd(p, dlogits=BASE + 400) == ALIAS and _fwd(p, loss=BASE) == ALIAS and _fwd(p, lse=BASE + MB) == ALIAS and _fwd(p, lse=BASE + 3 * MB) == ALIAS
    assert _bwd(p, dlogits=BASE + 2 * MB) == ALIAS and _bwd(p, dlogits=BASE + 4) == ALIAS
    assert _fwd(distill.make_params(4, 100, 8, row_stride=128), dlogits=BASE) == ALIAS   # in place only with equal strides


def test_binding_refuses_tensors():
    torch = pytest.importorskip("torch")
    x, i, t = torch.zeros(6, 50), torch.zeros(6, 4, dtype=torch.int32), torch.zeros(6, 4)
    ok = dict(logits=x, indices=i, teacher=t)
    distill.params_for(**ok)
    assert distill.params_for(torch.zeros(6, 64)[:, :50], i, t).row_stride == 64
    for bad, err in ((dict(logits=x.double()), TypeError), (dict(logits=torch.zeros(6, 100)[:, ::2]), ValueError), (dict(logits=x[0]), ValueError),
                     (dict(indices=i.long()), TypeError), (dict(indices=i[:5]), ValueError), (dict(indices=i[:, :3]), ValueError),
                     (dict(teacher=t.double()), TypeError), (dict(teacher=torch.zeros(4, 6).t()), ValueError), (dict(indices=torch.zeros(4, 6, dtype=torch.int32).t()), TypeError),
                     (dict(dlogits=x.half()), ValueError), (dict(dlogits=x[:5]), ValueError)):
        with pytest.raises(err):
            distill.params_for(**{**ok, **bad})
    one = torch.zeros(6)
    for bad, err in ((dict(lse=one[:5]), ValueError), (dict(dloss=one.half()), TypeError), (dict(dloss=torch.zeros(12)[::2]), ValueError),
                     (dict(dloss=torch.zeros(1).expand(6)), ValueError)):
        with pytest.raises(err):
            distill.backward(x, i, t, **{**dict(lse=one, dloss=one), **bad})
    with pytest.raises(ValueError):
        distill.forward(x, i, t, in_place=True)
    with pytest.raises(TypeError):
        distill.forward(x, i, t, dloss=one.double())
