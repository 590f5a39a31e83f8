"""Linear attention's and distillation's raw calls refuse tensors of the host or of another device than the current one, on the CPU: the library's functions are replaced by one
that must not be reached."""
import types

import pytest

torch = pytest.importorskip("torch")

from gated_delta_rule_backward_gb300 import distill, la  # noqa: E402


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on CUDA device `where`."""
    where = 0

    def get_device(self):
        return self.where


def on(t, where):
    t = t.as_subclass(Elsewhere)
    t.where = where
    return t


@pytest.fixture
def reached(monkeypatch):
    log = []
    call = lambda *a: log.append(a) or 0
    names = ("la_forward", "la_backward", "distill_forward", "distill_backward")
    lib = types.SimpleNamespace(**{n: call for n in names})
    monkeypatch.setattr(la, "_lib", lib)
    monkeypatch.setattr(distill, "_lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    return log


def arguments():
    q, v, g, pool = torch.zeros(3, 2, 32), torch.zeros(3, 4, 32), torch.zeros(3, 4), torch.zeros(3, 4, 32, 32)
    i3, i4, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    x, idx, t, n = torch.zeros(5, 100), torch.zeros(5, 4, dtype=torch.int32), torch.zeros(5, 4), torch.ones(5)
    p, d = la.make_params(3, 1, 2, 4, 32), distill.make_params(5, 100, 4)
    return [(la.la_forward, p, [q, q, v, g, i4, pool, i3, i3, v, ws]),
            (la.la_backward, p, [q, q, v, g, i4, pool, i3, v, pool, q, q, v, g, pool, ws]),
            (distill.distill_forward, d, [x, idx, t, n, n, n, x]),
            (distill.distill_backward, d, [x, idx, t, n, n, x])]


def test_refused_elsewhere(reached):
    stream = types.SimpleNamespace(cuda_stream=0)
    for call, p, tensors in arguments():
        here = [on(t.clone(), 1) for t in tensors]
        for i in range(len(here)):
            for where in (0, -1):                       # another device, the host
                with pytest.raises(ValueError):
                    call(p, *here[:i], on(tensors[i].clone(), where), *here[i + 1:], stream=stream)
        assert not reached
        call(p, *here, stream=stream)
        assert len(reached) == 1
        reached.clear()


def test_refused_on_the_host(reached):
    for call, p, tensors in arguments():
        with pytest.raises(ValueError):
            call(p, *tensors)
    assert not reached
