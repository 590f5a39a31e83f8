"""The serving form's C ABI (include/gdn_decode.h) on the CPU: exports and argument
validation.  Every call below fails its checks before any device work is enqueued."""
import ctypes
import os
import re

import pytest

from gated_delta_rule_backward_gb300 import decode, gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIAS = 0, 1, 2, 3
BASE, MB = 0x7F0000000000, 1 << 24  # fake, aligned device addresses (never dereferenced)


def test_header_symbols_exported():
    hdr = open(os.path.join(ROOT, "include", "gdn_decode.h")).read()
    declared = set(re.findall(r"^\w[\w\s\*]*?\b(gdn_\w+)\(", hdr, flags=re.M))
    assert declared == set(decode.EXPORTS)
    for name in declared:
        assert hasattr(gdn.library(), name), name


def _call(p, **ptrs):
    names = ("q", "k", "v", "g", "beta", "cu", "pool", "slot_in", "slot_out", "y")
    a = {n: BASE + i * MB for i, n in enumerate(names)}
    a["cu"] = None
    a.update(ptrs)
    return gdn.library().gdn_decode(ctypes.byref(p), *[a[n] for n in names], None)


@pytest.mark.parametrize("change,code", [
    (dict(S=48), UNSUPPORTED), (dict(S=512), UNSUPPORTED), (dict(S=64, S_v=24), UNSUPPORTED), (dict(S=64, S_v=272), UNSUPPORTED),
    (dict(H_v=5), INVALID), (dict(n_seq=-1), INVALID), (dict(H_k=0, H_v=0), INVALID), (dict(n_slots=-1), INVALID),
    (dict(q_s=(-1, 64)), INVALID), (dict(in_dtype=3), INVALID), (dict(gate_dtype=-1), INVALID), (dict(y_dtype=7), INVALID),
    (dict(slot_stride=4 * 64 * 64 - 4), INVALID), (dict(slot_stride=4 * 64 * 64 + 2), INVALID),
    (dict(n_seq=1 << 40, n_tok=0), UNSUPPORTED), (dict(n_tok=5), INVALID),
])
def test_sizes_refused(change, code):
    kw = dict(n_seq=2, T=1, H_k=2, H_v=4, S=64)
    kw.update(change)
    p = decode.make_params(**kw)
    if "n_tok" not in change or change["n_tok"] == 0:
        assert decode.supported(p) == code
    assert _call(p) == code


def test_pointers_refused():
    p = decode.make_params(2, 1, 2, 4, 64)
    for name in ("q", "k", "v", "g", "beta", "pool", "slot_in", "slot_out", "y"):
        assert _call(p, **{name: None}) == INVALID, name
    assert _call(p, pool=BASE + 6 * MB + 8) == INVALID          # the pool off its 16 bytes
    assert _call(p, q=BASE + 2) == INVALID                      # an fp32 input off its element
    assert _call(p, cu=BASE + 5 * MB + 2) == INVALID
    assert _call(p, y=BASE + 16) == ALIAS                       # y over q
    assert _call(p, pool=BASE + 2 * MB) == ALIAS                # the pool over v
    assert _call(p, y=BASE + 6 * MB + 64) == ALIAS              # y inside the pool
    assert _call(p, slot_in=BASE + 6 * MB + 64) == ALIAS        # the slots inside the pool
    assert b"overlaps" in gdn.library().gdn_last_error()


def test_no_sequences_is_no_work():
    assert _call(decode.make_params(0, 1, 2, 4, 64)) == OK


def _move(pool=BASE, L=2, ls=1 << 20, n=4, ss=4096, sb=4096, src=BASE + MB, dst=BASE + MB + 64, m=4, group=1):
    return gdn.library().gdn_states_move(pool, L, ls, n, ss, sb, src, dst, m, group, None)


@pytest.mark.parametrize("change,code", [
    (dict(L=-1), INVALID), (dict(n=-1), INVALID), (dict(m=-1), INVALID), (dict(sb=-16), INVALID), (dict(group=0), INVALID),
    (dict(pool=None), INVALID), (dict(src=None), INVALID), (dict(dst=None), INVALID), (dict(pool=BASE + 8), INVALID),
    (dict(ls=(1 << 20) + 8), INVALID), (dict(ss=4104), INVALID), (dict(sb=4088), INVALID), (dict(src=BASE + MB + 2), INVALID),
    (dict(ss=4080), INVALID), (dict(ls=4 * 4096 - 16), INVALID), (dict(m=2000, group=1025), UNSUPPORTED),
    (dict(src=BASE + 64), ALIAS), (dict(dst=BASE + (1 << 20) + 128), ALIAS),
    (dict(L=0), OK), (dict(m=0), OK), (dict(sb=0), OK), (dict(n=0), OK),
])
def test_moves_refused(change, code):
    assert _move(**change) == code


def test_binding_refuses_tensors():
    torch = pytest.importorskip("torch")
    q, v = torch.zeros(3, 2, 32), torch.zeros(3, 4, 32)
    g, pool, slots = torch.zeros(3, 4), torch.zeros(3, 4, 32, 32), torch.zeros(3, dtype=torch.int32)
    decode.params_for(q, q, v, g, g, pool, 3)
    for bad, err in ((dict(q=q.double(), k=q.double(), v=v.double()), TypeError), (dict(k=q.half()), TypeError), (dict(beta=g.half()), TypeError),
                     (dict(k=q[:2]), ValueError), (dict(g=g[:, :2]), ValueError), (dict(pool=pool.half()), ValueError),
                     (dict(pool=pool.transpose(2, 3)), ValueError), (dict(q=torch.zeros(3, 2, 64)[..., ::2]), ValueError)):
        with pytest.raises(err):
            decode.params_for(**{**dict(q=q, k=q, v=v, g=g, beta=g, pool=pool, n_seq=3), **bad})
    p = decode.params_for(q, q, v, g, g, pool, 3)
    with pytest.raises(ValueError):
        decode.gdn_decode(p, q, q, v, g, g, None, pool, slots[:2], slots, v)
    with pytest.raises(TypeError):
        decode._index(slots.long(), "slot_in")
    with pytest.raises(ValueError):
        decode.gdn_states_move(pool[None], slots, slots[:2])
