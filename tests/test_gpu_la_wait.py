"""Linear attention's chunked form where a hand-over between its warps never comes (a flag that nothing sets): bounded waits run out, the kernels return, say so, and leave
tensor and shared memory as the next call needs them."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import la_plain as P  # noqa: E402
from gated_delta_rule_backward_gb300 import gdn, la  # noqa: E402
from test_gpu_la import i32  # noqa: E402

BF16 = torch.bfloat16


@pytest.mark.parametrize("shift", [0, 1])       # tiles by TMA, and element by element
@pytest.mark.parametrize("T", [200, 2000])      # one kernel, and segments before it
@pytest.mark.parametrize("S", [64, 128])
def test_a_wait_that_runs_out(S, T, shift):
    x = P.problem([T], 1, 2, S, dtype=BF16, slots=2, seed=T, shift=shift)
    p = la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], 1, y_dtype=BF16)
    assert la.form(p) == "chunked" and (la.workspace_bytes(p) > 0) == (T == 2000)
    ws, before = la.workspace(p, "cuda"), x["pool"].clone()
    y = [torch.zeros(T, 2, S, dtype=BF16, device="cuda") for _ in range(3)]
    call = lambda f, y: f(p, x["q"], x["k"], x["v"], x["g"], None, x["pool"], i32([0]), i32([1]), y, ws)
    call(la.la_forward, y[0])
    after = x["pool"].clone()
    assert gdn.device_status() == 0 and not torch.equal(after, before)
    x["pool"].copy_(before)
    call(la.selftest_wait_timeout, y[1])
    assert gdn.device_status() == 6 and b"linear attention: timed out)" in gdn.library().gdn_last_error()   # nothing left in flight
    assert torch.equal(x["pool"], before) and gdn.device_status() == 0
    call(la.la_forward, y[2])
    assert gdn.device_status() == 0 and torch.equal(y[2], y[0]) and torch.equal(x["pool"], after)


def test_the_token_form_has_no_waits():
    x = P.problem([4], 1, 2, 64, slots=2)
    p = la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], 1)
    with pytest.raises(gdn.GdnError):
        la.selftest_wait_timeout(p, x["q"], x["k"], x["v"], x["g"], None, x["pool"], i32([0]), i32([1]), torch.zeros(4, 2, 64, device="cuda"), None)
