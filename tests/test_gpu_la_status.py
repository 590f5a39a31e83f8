"""What linear attention's kernels report (include/la.h), in a process of its own: a captured call is the first that the process makes, and both forms' reports come at once."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

PROGRAM = """
import torch
from gated_delta_rule_backward_gb300 import gdn, la
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
assert gdn.device_status() == 0
pool, calls = torch.zeros(3, 2, 64, 64, device="cuda"), []
for T in (4, 200):                                     # the token form, the chunked form
    q, v = (torch.randn(T, H, 64, device="cuda").bfloat16() for H in (1, 2))
    calls.append((q, q.clone(), v, torch.zeros(T, 2, device="cuda"), pool, i32([0]), i32([T // 200])))
assert [la.form(la.params_for(*c[:5], 1)) for c in calls] == ["token", "chunked"]
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    y = [la.forward(*c) for c in calls]
graph.replay()
assert gdn.device_status() == 0 and all(torch.isfinite(t).all() for t in y)
bad = lambda n, slot: (calls[n][5].fill_(slot), graph.replay(), gdn.device_status(), gdn.device_status())[2:]
for n in (0, 1):
    assert bad(n, 3) == (1, 0) and b"la_forward" in gdn.library().gdn_last_error()
    assert bad(n, 0) == (0, 0)
calls[0][5].fill_(-2), calls[1][5].fill_(7)            # both
graph.replay()
assert gdn.device_status() == 1 and gdn.device_status() == 0
graph.replay()
gdn.selftest_wait_timeout()                            # a wait that gave up is told first, and hides neither
assert [gdn.device_status() for _ in range(3)] == [6, 1, 0]
print("reported")
"""


def test_reports_of_a_captured_call_that_is_the_first():
    out = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "reported" in out.stdout, out.stderr[-2000:]
