"""The serving operators' allocating calls on the CPU, with the library's raw calls replaced by ones that record: what
they allocate and where, and which tensors they refuse."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from gated_delta_rule_backward_gb300 import beam, decode, rms  # noqa: E402


class Stream:
    cuda_stream = 1


@pytest.fixture
def calls(monkeypatch):
    """Allocations as (bytes, the stream that is current), raw calls as ("call", the stream they were given), outputs
    that another stream may use as ("recorded", that stream)."""
    log, now, empty = [], [None], torch.empty

    @contextlib.contextmanager
    def current(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    def recorded(*size, **kw):
        t = empty(*size, **kw)
        log.append((t.numel() * t.element_size(), now[0]))
        return t

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now[0])
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("recorded", s)))
    for module, name in ((rms, "rms_forward"), (rms, "rms_backward"), (beam, "beam_select"), (decode, "gdn_decode")):
        monkeypatch.setattr(module, name, lambda *a, **kw: log.append(("call", a[-1])))
    return log


def every_call(stream):
    x, w, rstd = torch.zeros(6, 64), torch.ones(64), torch.ones(6)
    rms.forward(x, w, x.clone(), stream=stream)
    rms.forward(x, w, y_dtype=torch.float8_e4m3fn, group=32, stream=stream)
    rms.backward(x, rstd, x.clone(), w, stream=stream)
    beam.select(torch.zeros(6, 50), torch.zeros(2, 3), slots=torch.zeros(2, 3, dtype=torch.int32), stream=stream)
    q, v, g, pool = torch.zeros(3, 2, 32), torch.zeros(3, 4, 32), torch.zeros(3, 4), torch.zeros(3, 4, 32, 32)
    decode.decode(q, q, v, g, g, pool, torch.zeros(3, dtype=torch.int32), stream=stream)


def test_memory_comes_from_the_stream_that_uses_it(calls):
    """Memory of another stream's pool may still be in use there, and what is freed goes back to it: a workspace
    given back to the current stream while `stream` still works in it could be handed out again at once."""
    side = Stream()
    every_call(side)
    made = [c for c in calls if isinstance(c[0], int)]
    assert len(made) == 15 and all(stream is side for _, stream in made)   # 13 outputs and two workspaces
    assert [c for c in calls if c[0] == "call"] == [("call", side)] * 5
    assert [c for c in calls if c[0] == "recorded"] == [("recorded", None)] * 13   # and for the caller's own stream


def test_without_a_stream_the_current_one_is_left_alone(calls):
    every_call(None)
    assert len(calls) == 20 and all(stream is None and what != "recorded" for what, stream in calls)


def test_norm_gradient_refuses_what_it_would_misread(calls):
    """dh is read as dense [rows, D] of h's type and rstd as dense fp32 [rows]; h and dy may have any row stride."""
    wide, w, rstd = torch.zeros(6, 128), torch.ones(64), torch.ones(6)
    h, dy, dense = wide[:, :64], wide[:, 64:], torch.zeros(6, 64)
    rms.backward(h, rstd, dy, w, dense)
    rms.backward(h, rstd[:, None], dy, w, dense)             # [rows, 1] holds the same numbers
    rms.backward(h[:1], rstd[:1], dy[:1], w, wide[:1, :64])  # one row is dense whatever its stride
    done = [c for c in calls if c[0] == "call"]
    assert len(done) == 3
    for bad, err in ((dict(dh=wide[:, :64]), ValueError), (dict(dh=torch.zeros(6, 1).expand(6, 64)), ValueError),
                     (dict(dh=torch.zeros(64, 6).t()), ValueError), (dict(dh=dense[:5]), ValueError), (dict(dh=torch.zeros(64, 6)), ValueError),
                     (dict(dh=dense.bfloat16()), TypeError), (dict(dh=dense.double()), TypeError),
                     (dict(rstd=torch.ones(5)), ValueError), (dict(rstd=torch.ones(12)[::2]), ValueError), (dict(rstd=torch.ones(1).expand(6)), ValueError),
                     (dict(rstd=rstd.bfloat16()), TypeError), (dict(rstd=rstd.double()), TypeError)):
        with pytest.raises(err):
            rms.backward(**{**dict(h=h, rstd=rstd, dy=dy, weight=w, dh=dense), **bad})
    with pytest.raises(TypeError):
        rms.backward(h.bfloat16(), rstd, dy.bfloat16(), w, dense)   # an fp32 dh beside bf16 rows
    assert [c for c in calls if c[0] == "call"] == done
