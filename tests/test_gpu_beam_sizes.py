"""The selection at the ends of its range: the longest row that it takes, and masks of the type's lowest value."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import beam  # noqa: E402


@pytest.mark.parametrize("shift", [0, 3])
def test_the_longest_row(shift):
    """2^31 - 1 logits, the best in the row's last elements.  All but three are equal, so that a sum of 4096 equal terms a lane
    may round the same way each time: 4096 2^-24 on the logarithm, and the scores' own 4 2^-24 |score|."""
    V = 2**31 - 1
    x = torch.zeros(V + shift, dtype=torch.bfloat16, device="cuda")[shift:].view(1, V)
    best = {V - 1: 30.0, V - 20000: 28.0, 123: 29.0}   # in three different segments
    for i, v in best.items():
        x[0, i] = v
    score, parent, token = beam.select(x, torch.full((1, 1), -2.0, device="cuda"), n_out=3)
    assert (parent == 0).all() and token.tolist() == [[V - 1, 123, V - 20000]]
    total = math.log((V - 3) + sum(math.exp(v) for v in best.values()))
    ref = np.array([-2.0 + v - total for v in (30.0, 29.0, 28.0)])
    assert (np.abs(score[0].double().cpu().numpy() - ref) <= 4096 * 2.0**-24 + 4 * 2.0**-24 * np.abs(ref)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_masks_of_the_lowest_value(dtype):
    """Tokens masked with the type's lowest number instead of -inf: they have no part in the sum, and fill up in the order of
    score and index what the allowed ones leave.  fp32 and bf16: the masked scores round to the mask's value itself."""
    N, K, V, low = 2, 3, 40001, torch.finfo(dtype).min
    x = torch.full((N * K, V), low, device="cuda", dtype=dtype)
    x[:, 777], x[:, 30000] = 1.0, 3.0            # two tokens allowed in every beam
    x[4] = low                                   # a beam with none: uniform
    s = torch.tensor([[-1.0, -5.0, -9.0], [-1.0, -40.0, -9.0]], device="cuda")
    score, parent, token = beam.select(x, s, n_out=6)
    a, b = 3.0 - math.log(math.exp(3.0) + math.exp(1.0)), 1.0 - math.log(math.exp(3.0) + math.exp(1.0))
    ref = [-1 + a, -1 + b, -5 + a, -5 + b, -9 + a, -9 + b]
    assert parent[0].tolist() == [0, 0, 1, 1, 2, 2] and token[0].tolist() == [30000, 777] * 3
    assert np.allclose(score[0].double().cpu(), ref, rtol=0, atol=2e-6 * 11)
    ref = [-1 + a, -1 + b, -9 + a, -9 + b] + [-40 - math.log(V)] * 2
    assert parent[1].tolist() == [0, 0, 2, 2, 1, 1] and token[1].tolist() == [30000, 777, 30000, 777, 0, 1]
    assert np.allclose(score[1].double().cpu(), ref, rtol=0, atol=2e-6 * 52)
    score, parent, token = beam.select(x[:3], s[:1], n_out=9)
    assert parent[0].tolist() == [0, 0, 1, 1, 2, 2, 0, 0, 0] and token[0, 6:].tolist() == [0, 1, 2]
    assert (score[0, 6:] <= low / 2).all() and torch.isfinite(score).all()
