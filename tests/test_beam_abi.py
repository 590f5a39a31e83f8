"""The beam selection's C ABI (include/beam.h) on the CPU: exports, sizes and argument validation.
Every call below fails its checks before any device work is enqueued."""
import ctypes
import os
import re

import pytest

from gated_delta_rule_backward_gb300 import beam, gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4
BASE, MB = 0x7F0000000000, 1 << 24  # fake, aligned device addresses (never dereferenced)
NAMES = ("logits", "scores", "done", "slots", "scores_out", "parent", "token", "src_slots", "ws")


def test_header_symbols_exported():
    hdr = open(os.path.join(ROOT, "include", "beam.h")).read()
    declared = set(re.findall(r"^\w[\w\s\*]*?\b(beam_\w+)\(", hdr, flags=re.M))
    assert declared == set(beam.EXPORTS)
    for name in declared:
        assert hasattr(gdn.library(), name), name


def _call(p, ws_bytes=None, **ptrs):
    a = {n: BASE + i * MB for i, n in enumerate(NAMES)}
    a.update(ptrs)
    return gdn.library().beam_select(ctypes.byref(p), *[a[n] for n in NAMES], beam.workspace_bytes(p) if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(row_stride=99), INVALID), (dict(dtype=3), INVALID),
    (dict(n_out=0), INVALID), (dict(V=2, row_stride=2, n_out=9), INVALID), (dict(K=65), UNSUPPORTED), (dict(n_out=65), UNSUPPORTED),
    (dict(V=1 << 30, row_stride=1 << 30), UNSUPPORTED), (dict(N=1 << 28), UNSUPPORTED),
])
def test_sizes_refused(change, code):
    p = beam.make_params(**{**dict(N=2, K=4, V=100, n_out=4), **change})
    assert beam.workspace_bytes(p) == 0 and _call(p, 1 << 20) == code


def test_pointers_refused():
    p = beam.make_params(2, 4, 100)
    assert beam.workspace_bytes(p) > 0
    for n in ("logits", "scores", "scores_out", "parent", "token", "slots"):
        assert _call(p, **{n: None}) == INVALID, n
    for n in ("logits", "scores", "slots", "scores_out", "parent", "token", "src_slots", "ws"):
        assert _call(p, **{n: BASE + 20 * MB + 2}) == INVALID, n
    assert _call(p, ws=None) == WORKSPACE and _call(p, beam.workspace_bytes(p) - 1) == WORKSPACE
    assert _call(p, scores_out=BASE + MB) == ALIAS and _call(p, token=BASE + 5 * MB) == ALIAS and _call(p, ws=BASE) == ALIAS
    for pad in (-1, 100):
        assert _call(beam.make_params(2, 4, 100, pad_token=pad)) == INVALID
    assert _call(beam.make_params(0, 4, 100)) == OK


def test_binding_refuses_tensors():
    torch = pytest.importorskip("torch")
    x, s = torch.zeros(6, 50), torch.zeros(2, 3)
    beam.params_for(x, s)
    for args, err in (((x.double(), s), TypeError), ((x, s.half()), TypeError), ((x[:5], s), ValueError), ((x.t(), s), ValueError),
                      ((torch.zeros(6, 100)[:, ::2], s), ValueError), ((x, torch.zeros(3, 2).t()), ValueError)):
        with pytest.raises(err):
            beam.params_for(*args)
    for kw in (dict(done=torch.zeros(2, 2, dtype=torch.bool)), dict(done=s), dict(slots=torch.zeros(2, 3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            beam.select(x, s, **kw)
