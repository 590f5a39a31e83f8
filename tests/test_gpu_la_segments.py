"""Linear attention's gradients (include/la.h) at the lengths and in as many segments as their stated exactness is for."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import la_plain as P  # noqa: E402
from gated_delta_rule_backward_gb300 import gdn, la  # noqa: E402
from test_gpu_la import cu_of, i32  # noqa: E402


@pytest.mark.parametrize("S,counts,segments", [(128, [1024], 8), (128, [4096], 8), (64, [4096], 8), (64, [1024, 700], 8), (128, [2300], 6)])
def test_decays_gradient(S, counts, segments):
    """test_gpu_la_chunk.py's bound on dg for bf16: where a segment begins, the sum jumps by a quarter of 1.1e-5 of its size at random, eight times at most: 7.8e-6; with the
    token form's own roundings, 4e-6 over 4096 tokens, 8.8e-6.  1e-5 of dg's norm."""
    N, H = len(counts), 2
    # as many segments as 608 CTAs of 64 rows allow, whole chunks, eight at most
    ctas, chunks = N * H * S // 64, -(-max(counts) // 128)
    per = -(-chunks // min(8, 608 // ctas, chunks))
    assert -(-chunks // per) == segments
    x = P.problem(counts, 1, H, S, dtype=torch.bfloat16, slots=N, seed=31)
    slots = list(range(N))
    got = la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32(slots), x["dy"], x["dstate"], cu_of(counts), T=max(counts))
    want = P.backward(x, counts, slots, S ** -0.5)
    off = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert off(got[3], want[3]) <= 1e-5
    for a, b in zip(got[:3], want):                     # of 16 bits: errors spread over half a unit, 2^-8 of a power of two that the value is not below
        assert off(a, b) <= 2.0 ** -8 / 3 ** 0.5
    assert off(got[4], want[4]) <= 3 * 2.0 ** -16
    assert gdn.device_status() == 0


@pytest.mark.parametrize("S,T,H", [(128, 1000, 6), (64, 1000, 4), (128, 2048, 2), (64, 4096, 4)])
def test_segments_are_as_exact_as_one_walk(S, T, H):
    """The same numbers as fp32 tensors go in one walk of the token form.  The segments' first states are sums in fp32 too, of keys whose weights are split without a rest, so that dg is off
    by no more than the walk's: errors of one size, drawn anew at eight places; half as much again."""
    x = P.problem([T], 1, H, S, dtype=torch.bfloat16, slots=1, seed=S + T)
    want = P.backward(x, [T], [0], S ** -0.5)[3]
    grads = lambda x: la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([0]), x["dy"], x["dstate"])[3]
    off = lambda a: float((a.double() - want).norm() / want.norm())
    wide = {n: t.float() for n, t in x.items()}
    assert la.form(la.params_for(wide["q"], wide["k"], wide["v"], wide["g"], wide["pool"], 1)) == "token"
    assert off(grads(x)) <= 1.5 * off(grads(wide))
    assert gdn.device_status() == 0
