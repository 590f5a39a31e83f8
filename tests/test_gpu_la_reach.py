"""How far an infinity or NaN in one token's inputs reaches in linear attention's gradients (include/la.h), in both forms: where the formulas carry it, the chunk of 128
tokens for dv in the chunked form, and dg of every earlier token where it is in a dq or dk that dg's running sum passes."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import la_plain as P  # noqa: E402
from gated_delta_rule_backward_gb300 import gdn, la  # noqa: E402
from test_gpu_la import cu_of, i32  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("counts,S,dtype,at", [([300, 200], 64, BF16, 130), ([700, 90], 128, BF16, 300), ([20, 9], 32, F32, 7), ([30, 31], 64, BF16, 12)])
@pytest.mark.parametrize("name", ["v", "k", "q", "dy", "g"])
def test_gradients(name, counts, S, dtype, at, value):
    T, chunked = counts[0], max(counts) >= 32
    x = P.problem(counts, 1, 2, S, dtype=dtype, slots=2, seed=4)
    x["q"], x["k"], x["v"] = (x[n].clone() for n in ("q", "k", "v"))
    p = la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], 2, T=max(counts))
    assert la.form(p) == ("chunked" if chunked else "token")
    run = lambda: la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([0, 1]), x["dy"], x["dstate"], cu_of(counts), T=max(counts))
    want = run()
    if name == "g":
        x["g"] = x["g"].clone()
        x["g"][at, 0] = float("nan")
    else:
        x[name][at, 0, 3] = value
    dq, dk, dv, dg, first = run()
    for a, b in zip((dq, dk, dv, dg), want):          # the second sequence, to the bit
        assert torch.equal(a[T:], b[T:])
    assert torch.equal(first[1], want[4][1])
    if name != "q" and name != "k":                   # heads share those
        assert torch.equal(dv[:T, 1], want[2][:T, 1]) and torch.equal(dg[:T, 1], want[3][:T, 1]) and torch.equal(first[0, 1], want[4][0, 1])
    fine = lambda t: torch.isfinite(t[:T].float()).flatten(1).all(1).tolist()
    every, none = set(range(T)), set()
    upto, since = set(range(at + 1)), set(range(at, T))
    chunk = set(range(max(0, T - 128 * ((T - at - 1) // 128 + 1)), T - 128 * ((T - at - 1) // 128))) if chunked else none
    # the tokens that the formulas carry it to: dq, dk, dv, and dg with its running sum
    reach = {"v": (since, {at}, none, every), "k": (since, none, {at}, every), "q": (none, upto, upto, upto), "dy": ({at}, upto, upto, upto),
             "g": (since, upto - {at}, upto - {at}, every)}[name]
    for what, t, tokens in zip(("dq", "dk", "dv", "dg"), (dq, dk, dv[:, 0], dg[:, 0]), reach):
        t = t[:, None] if t.dim() == 1 else t
        bad = {n for n, ok in enumerate(fine(t)) if not ok}
        if what == "dv":
            assert tokens <= bad <= tokens | chunk, (what, sorted(bad)[:5], sorted(bad)[-5:])
        else:
            assert bad == tokens, (what, sorted(bad)[:5], sorted(bad)[-5:])
    assert gdn.device_status() == 0
