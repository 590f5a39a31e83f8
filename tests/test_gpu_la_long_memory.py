"""Linear attention (include/la.h) token by token with decays that stay the same over thousands of tokens: what one decay is off by must not add up over the tokens remembered.

Tolerance, of norms.  A token rounds a state's element twice, by 2^-24 of it at most and at random: sqrt(2 T / 3) 2^-24 over T tokens.  A decay is a + b with what both leave out
below 2^-24 |g|, times the 1 / |g| tokens remembered: 2^-24; decays beyond half a token's memory 2^-23.  So a state is within (sqrt(T) + 4) 2^-24 of its norm, and
what is read from it, a dot of up to 64 products, within 8 2^-24 more.  dg is a running sum of T differences of two such dots each, whose errors are random too: (2 sqrt(T) + 16) 2^-24
of the terms, which are up to as many times dg as it takes them to cancel: for the inputs here four times its norm."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import la_plain as P  # noqa: E402
from gated_delta_rule_backward_gb300 import gdn, la  # noqa: E402
from test_gpu_la import cu_of, i32  # noqa: E402

U = 2.0 ** -24


def lasting(counts, H, S, dtype, seed=0, gate=torch.float32):
    """Every head forgets at its own rate: half a token to 4096 of them."""
    x = P.problem(counts, 1, H, S, dtype=dtype, slots=len(counts), seed=seed)
    keep = 1 - 2.0 ** -torch.linspace(1, 12, H, dtype=torch.float64) * (1 + 0.3 * torch.rand(H, dtype=torch.float64, generator=torch.Generator().manual_seed(seed)))
    x["g"] = keep.clamp(min=0.3).log().to(gate).cuda().expand(sum(counts), H)
    return x


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def rounding(t):
    return 0.0 if t.dtype == torch.float32 else torch.finfo(t.dtype).eps / 2 / 3 ** 0.5


@pytest.mark.parametrize("dtype,gate", [(torch.float32, torch.float32), (torch.float16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("S", [32, 64])
def test_token_form(S, dtype, gate):
    T = 2000
    x = lasting([T], 12, S, dtype, seed=S, gate=gate)
    p = la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], 1)
    assert la.form(p) == "token"
    sc = S ** -0.5
    grads = la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([0]), x["dy"], x["dstate"])
    want = P.backward(x, [T], [0], sc)
    y0, after, _ = P.forward(x, [T], [0], sc)
    y = la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([0]))
    state = (math.sqrt(T) + 4) * U
    for n in range(12):                        # head by head: those that remember longest are the ones it is about
        assert off(x["pool"][0, n], after[0, n]) <= state, n
        assert off(y[:, n], y0[:, n]) <= state + 8 * U, n
        assert off(grads[2][:, n], want[2][:, n]) <= state + 8 * U + rounding(grads[2]), n
        assert off(grads[4][0, n], want[4][0, n]) <= state + 4 * U, n
    for a, b in zip(grads[:2], want):
        assert off(a, b) <= state + 8 * U + rounding(a)
    assert off(grads[3], want[3]) <= 4 * (2 * math.sqrt(T) + 16) * U
    assert gdn.device_status() == 0


@pytest.mark.parametrize("counts,H,S", [([700] * 5, 64, 64), ([4096], 4, 64), ([1500, 1100], 6, 128)])
def test_decays_gradient_of_chunked_sizes(counts, H, S):
    """One segment and eight: test_gpu_la_segments.py's 1e-5 of dg's norm, whatever the decays."""
    x = lasting(counts, H, S, torch.bfloat16, seed=H)
    got = la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32(range(len(counts))), x["dy"], x["dstate"], cu_of(counts), T=max(counts))
    want = P.backward(x, counts, list(range(len(counts))), S ** -0.5)
    assert off(got[3], want[3]) <= 1e-5
    assert gdn.device_status() == 0


@pytest.mark.parametrize("N,H,S,T", [(20, 8, 64, 16384), (1, 16, 128, 32768)])     # one segment, and several
def test_states_of_long_prompts(N, H, S, T):
    """Decays that stay the same have a closed form.  The keys' weights and the state are two bf16 terms: 3 2^-18 of its norm at random; and the tensor cores' sums are cut off, as include/la.h
    says 2^-22 of the state a chunk that it remembers, counted at their weights."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    q, k, v = rnd(N * T, 1, S).bfloat16(), rnd(N * T, 1, S).bfloat16(), rnd(N * T, H, S).bfloat16()
    g = -1.1 * 2.0 ** -torch.linspace(8, 17, H, device="cuda")
    pool = rnd(N, H, S, S)
    before = pool.double()
    la.forward(q, k, v, g.expand(N * T, H), pool, i32(range(N)), y_dtype=torch.bfloat16)
    weights = torch.exp(g.double()[:, None] * torch.arange(T - 1, -1, -1, device="cuda").double())
    for n in (0, N - 1):
        at = slice(n * T, (n + 1) * T)
        want = torch.einsum("thj,ht,ti->hji", v[at].double(), weights, k[at, 0].double()) + torch.exp(g.double() * T)[:, None, None] * before[n]
        for h in range(H):
            assert off(pool[n, h], want[h]) <= 3 * 2.0 ** -18 + float(weights[h].sum()) / 128 * 2.0 ** -22, (n, h)
    assert gdn.device_status() == 0
