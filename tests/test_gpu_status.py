"""The device status word where two kinds of report meet: neither hides the other."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import decode, gdn  # noqa: E402


def bad_move():
    pool, i32 = torch.zeros(1, 4, 16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    decode.gdn_states_move(pool, torch.tensor([4], **i32), torch.tensor([0], **i32))


@pytest.mark.parametrize("wait_first", [False, True])
def test_a_timeout_does_not_hide_a_bad_slot(wait_first):
    """The self-test's kernel waits on a flag that nothing sets, gives up after its limit and returns."""
    assert gdn.device_status() == 0
    for step in ((gdn.selftest_wait_timeout, bad_move) if wait_first else (bad_move, gdn.selftest_wait_timeout)):
        step()
    assert gdn.device_status() == 6 and b"gave up" in gdn.library().gdn_last_error()
    assert gdn.device_status() == 1 and b"gdn_states_move" in gdn.library().gdn_last_error()
    assert gdn.device_status() == 0
