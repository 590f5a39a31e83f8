"""Distillation's temperatures at fp32's limits, on the CPU: those whose reciprocal fp32 does not hold are refused before any device work."""
import pytest

from gated_delta_rule_backward_gb300 import distill
from test_distill_abi import INVALID, OK, _bwd, _fwd


@pytest.mark.parametrize("tau,ok", [(2.0 ** -126, True), (3.4e38, True), (2.0 ** -127, False), (1e-45, False), (2.0 ** -149, False)])
def test_smallest_and_largest(tau, ok):
    p = distill.make_params(0, 100, 8, temperature=tau)    # no rows: nothing is launched
    assert p.temperature > 0
    assert _fwd(p) == _bwd(p) == (OK if ok else INVALID)
