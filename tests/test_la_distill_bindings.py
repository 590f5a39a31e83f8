"""The allocating calls of linear attention and distillation on the CPU, with the library's raw calls replaced by ones that record: what they
allocate and where (test_serving_bindings.py's way)."""
import pytest

torch = pytest.importorskip("torch")

from gated_delta_rule_backward_gb300 import distill, la  # noqa: E402
from test_serving_bindings import Stream, calls  # noqa: E402,F401


@pytest.fixture
def raw(calls, monkeypatch):  # noqa: F811
    for module, name in ((la, "la_forward"), (la, "la_backward"), (distill, "distill_forward"), (distill, "distill_backward")):
        monkeypatch.setattr(module, name, lambda *a, **kw: calls.append(("call", a[-1])))
    return calls


def every_call(stream):
    q, v, g, pool = torch.zeros(3, 2, 32), torch.zeros(3, 4, 32), torch.zeros(3, 4), torch.zeros(3, 4, 32, 32)
    slots = torch.zeros(3, dtype=torch.int32)
    la.forward(q, q, v, g, pool, slots, stream=stream)                        # token form: y, no workspace
    big = torch.zeros(4096, 1, 128, dtype=torch.bfloat16)
    la.forward(big, big, big, torch.zeros(4096, 1), torch.zeros(1, 1, 128, 128), slots[:1], stream=stream)   # segments: y and a workspace
    la.backward(q, q, v, g, pool, slots, v.clone(), stream=stream)            # five gradients and a workspace
    x, idx, t = torch.zeros(5, 100), torch.zeros(5, 4, dtype=torch.int32), torch.zeros(5, 4)
    rows = torch.ones(5)
    distill.forward(x, idx, t, stream=stream)                                 # loss and lse
    distill.forward(x, idx, t, dloss=rows, stream=stream)                     # and a gradient
    distill.forward(x, idx, t, dloss=rows, in_place=True, stream=stream)
    distill.backward(x, idx, t, rows, rows, stream=stream)
    distill.backward(x, idx, t, rows, rows, in_place=True, stream=stream)


def test_memory_comes_from_the_stream_that_uses_it(raw):
    side = Stream()
    every_call(side)
    made = [c for c in raw if isinstance(c[0], int)]
    assert len(made) == 17 and all(stream is side for _, stream in made)   # 15 outputs and two workspaces
    assert [c for c in raw if c[0] == "call"] == [("call", side)] * 8
    assert [c for c in raw if c[0] == "recorded"] == [("recorded", None)] * 15


def test_without_a_stream_the_current_one_is_left_alone(raw):
    every_call(None)
    assert len(raw) == 25 and all(stream is None and what != "recorded" for what, stream in raw)


def test_segments_need_a_workspace_only_where_they_pay():
    """One segment of a sequence and head keeps its state on chip."""
    p = lambda T, H, n=1, S=128: la.make_params(n, T, H, H, S, in_dtype=1, n_tok=n * T)
    assert la.form(p(4096, 8)) == "chunked" and la.workspace_bytes(p(4096, 8)) > 0
    assert la.workspace_bytes(p(512, 8)) == 0 and la.workspace_bytes(p(4096, 200)) == 0 and la.workspace_bytes(p(31, 8)) == 0
    for T in (1, 32, 100, 1000, 5000, 100000):
        for H in (1, 3, 16, 76, 77, 152):
            n, chunks = la.workspace_bytes(p(T, H)) // (4 * H * (128 * 128 + 1)), (T + 127) // 128
            assert n <= min(16, max(1, 152 // H), chunks) and n != 1
