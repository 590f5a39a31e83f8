"""Linear attention's chunked form (include/la.h) on the GPU against the recurrence in 64 bits (la_plain.py).

Tolerance.  Relative to the sum A of the magnitudes that a result is made of: the state, the weighted scores and the
decayed keys are each split into two bf16 numbers (2^-16), of which a result meets two in turn at most and a third through
the state: 3 2^-16.  The tensor cores' fp32 sums over 128 terms in two passes round (or cut off) at most 256 + 44 times at
2^-23, a state and its decays 8 times more a chunk.  So |error| <= (3 2^-16 + (300 + 8 chunks) 2^-23) A.
Since the splits' errors have no common sign, they add as the terms themselves do where those have random signs: the
root mean square of the errors of an fp32 result is also within 3 2^-16 of the result's.
dg: a running sum of both dots' errors over the tokens that follow, T roundings more."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import la_plain as P  # noqa: E402
from gated_delta_rule_backward_gb300 import gdn, la  # noqa: E402
from test_gpu_la import check_backward, check_forward, cu_of, i32  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def eps_of(counts):
    return 3 * 2.0 ** -16 + (300 + 8 * (max(counts) + 127) // 128) * 2.0 ** -23


def forward(x, counts, slot_in, slot_out, **kw):
    p = la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], len(counts), T=max(counts))
    assert la.form(p) == "chunked"
    return check_forward(x, counts, slot_in, slot_out, eps=eps_of(counts), **kw)


def backward(x, counts, slot_in, **kw):
    return check_backward(x, counts, slot_in, eps=eps_of(counts), **kw)


@pytest.mark.parametrize("S", [64, 128])
@pytest.mark.parametrize("counts,H_k,H_v", [([32], 1, 1), ([128], 1, 2), ([129], 2, 2), ([127, 1, 0, 300], 2, 6), ([1000], 1, 1), ([40] * 7, 3, 3), ([260, 0, 511, 33], 5, 10),
                                            ([2100], 1, 1), ([700, 3, 1500], 1, 3), ([33] * 90, 2, 4), ([256, 256], 1, 4), ([1400], 16, 48), ([900, 1000], 8, 40)])
def test_forward(counts, H_k, H_v, S):
    N = len(counts)
    x = P.problem(counts, H_k, H_v, S, dtype=BF16, slots=2 * N, seed=S + sum(counts))
    slot_in, slot_out = [(n + 1) % N for n in range(N)], [N + n for n in range(N)]
    if N > 2:
        slot_in[2], slot_out[1] = -1, -1
    y = forward(x, counts, slot_in, slot_out, ragged=len(set(counts)) > 1)
    ref = P.forward(x, counts, slot_in, S ** -0.5)[0]
    assert float((y.double() - ref).square().mean().sqrt()) <= 3 * 2.0 ** -16 * float(ref.square().mean().sqrt())


@pytest.mark.parametrize("S", [64, 128])
@pytest.mark.parametrize("counts,H_k,H_v", [([32], 1, 1), ([129], 2, 2), ([127, 1, 0, 300], 2, 6), ([1000], 1, 1), ([40] * 7, 3, 3), ([700, 3, 900], 1, 3), ([800], 16, 48)])
def test_backward(counts, H_k, H_v, S):
    N = len(counts)
    x = P.problem(counts, H_k, H_v, S, dtype=BF16, seed=S + sum(counts))
    slot_in = [(n + 1) % N for n in range(N)]
    if N > 2:
        slot_in[2] = -1
    for with_state in (True, False):
        backward(x, counts, slot_in, with_state=with_state, ragged=len(set(counts)) > 1)


@pytest.mark.parametrize("y_dtype", [BF16, F16, F32])
def test_output_types_in_place_and_unaligned_rows(y_dtype):
    for shift in (0, 1, 4):
        counts = [300, 77]
        x = P.problem(counts, 1, 2, 128, dtype=BF16, slots=3, seed=shift, shift=shift)
        forward(x, counts, [2, 0], [2, 0], y_dtype=y_dtype)          # each sequence's state is replaced
        backward(x, counts, [2, 0])
    x = P.problem([1100], 1, 1, 128, dtype=BF16, slots=1, seed=9)    # the same with several segments
    forward(x, [1100], [0], [0])


@pytest.mark.parametrize("gate", [dict(constant=True), dict(gate=BF16), dict(gate=F16, constant=True), dict(strength=0.0), dict(strength=-3.0), dict(strength=-20.0),
                                  dict(strength=-200.0), dict(strength=0.01)])
def test_gates(gate):
    counts = [290, 150]
    x = P.problem(counts, 2, 4, 64, dtype=BF16, slots=4, seed=5, **gate)
    forward(x, counts, [0, 1], [2, 3])
    backward(x, counts, [0, 1])


def test_resets_and_mixed_decays():
    """Strong decays and resets among weak ones: a chunk's running sum is large, what matters are its small differences."""
    counts = [400]
    x = P.problem(counts, 1, 2, 128, dtype=BF16, slots=2, seed=6)
    g = torch.full((400, 2), -1e-3, device="cuda")
    g[::50] = -90.0
    g[7] = float("-inf")
    g[130:160, 1] = -40.0
    g[301, 0] = float("-inf")
    x["g"] = g
    forward(x, counts, [0], [1])
    backward(x, counts, [0])
    wide = torch.zeros(400, 6, device="cuda")
    wide[:, ::3] = g
    x["g"] = wide[:, ::3]
    forward(x, counts, [0], [1])


def test_token_by_token_goes_on_from_a_prompt():
    """A prompt in the chunked form, then single tokens in the token form, against one walk over all."""
    counts = [200, 200]
    x = P.problem(counts, 2, 4, 128, dtype=BF16, slots=4, seed=8)
    y0, after, _ = P.forward(x, counts, [0, 1], 128 ** -0.5)
    A_y, A_s, _ = P.forward(x, counts, [0, 1], 128 ** -0.5, absolute=True)
    rows = lambda lo, hi: torch.cat([torch.arange(lo, hi), torch.arange(200 + lo, 200 + hi)]).cuda()
    part = lambda r: [x[n][r] for n in ("q", "k", "v", "g")]
    r = rows(0, 190)
    y = torch.empty(400, 4, 128, device="cuda")
    y[r] = la.forward(*part(r), x["pool"], i32([0, 1]), i32([2, 3]))
    for t in range(190, 200):
        r = rows(t, t + 1)
        y[r] = la.forward(*part(r), x["pool"], i32([2, 3]))
    eps = eps_of(counts) + 88 * 2.0 ** -24
    P.within(y, y0, A_y, eps, "y")
    P.within(x["pool"][2:], after, A_s, eps, "state")
    assert gdn.device_status() == 0


def test_the_same_bits_again_on_another_stream_and_in_a_graph():
    counts = [500, 90]
    x = P.problem(counts, 1, 2, 128, dtype=BF16, slots=4, seed=4)
    s_in, s_out, cu = i32([0, 1]), i32([2, 3]), cu_of(counts)
    step = lambda stream=None: (la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], s_in, s_out, cu, T=500, stream=stream), x["pool"][2:].clone(),
                                *la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], s_in, x["dy"], x["dstate"], cu, T=500, stream=stream))
    direct = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(direct, other)) if i != 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    x["v"].copy_(torch.randn(x["v"].shape, device="cuda"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))
    assert not torch.equal(captured[0], direct[0]) and gdn.device_status() == 0


def test_rows_and_slots_that_are_not_the_calls_own_are_left_alone():
    x = P.problem([300], 1, 2, 64, dtype=BF16, slots=6, seed=7)
    cu = i32([20, 120, 260])
    p = la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], 2, T=140)
    y = torch.full((300, 2, 64), 7.0, device="cuda")
    before = x["pool"].clone()
    la.la_forward(p, x["q"], x["k"], x["v"], x["g"], cu, x["pool"], i32([0, 1]), i32([4, -1]), y, la.workspace(p, "cuda"))
    assert (y[:20] == 7).all() and (y[260:] == 7).all() and (y[20:260] != 7).any(-1).all()
    assert torch.equal(x["pool"][[0, 1, 2, 3, 5]], before[[0, 1, 2, 3, 5]]) and not torch.equal(x["pool"][4], before[4])
    out = [torch.full((300, h, 64), 7.0, device="cuda", dtype=BF16) for h in (1, 1, 2)] + [torch.full((300, 2), 7.0, device="cuda"), torch.empty(2, 2, 64, 64, device="cuda")]
    la.la_backward(p, x["q"], x["k"], x["v"], x["g"], cu, x["pool"], i32([0, 1]), x["dy"], None, *out, la.backward_workspace(p, "cuda"))
    for o in out[:4]:
        assert (o[:20] == 7).all() and (o[260:] == 7).all() and (o[20:260] != 7).any()
    # what only the device can see
    bad = i32([0, 120, 290])                                           # the second is longer than T
    y.fill_(7.0)
    la.la_forward(p, x["q"], x["k"], x["v"], x["g"], bad, x["pool"], i32([0, 1]), i32([2, 3]), y, la.workspace(p, "cuda"))
    assert gdn.device_status() == 1 and b"la_forward" in gdn.library().gdn_last_error()
    assert (y[120:] == 7).all() and torch.equal(x["pool"][3], before[3]) and not torch.equal(x["pool"][2], before[2])
    assert gdn.device_status() == 0


def test_lengths_that_change_between_replays():
    """A captured step serves whatever lengths its cu_tokens hold at replay, no sequence above T: several segments, one chunk, nothing."""
    x = P.problem([1500], 2, 4, 128, dtype=BF16, slots=6, seed=12)
    s_in, s_out, cu = i32([0, 1, 2]), i32([3, 4, 5]), i32([0, 1500, 1500, 1500])
    step = lambda: (la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], s_in, s_out, cu, T=1500), x["pool"][3:].clone(),
                    *la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], s_in, x["dy"], x["pool"][:3].contiguous(), cu, T=1500))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for lengths in ([1500, 0, 0], [1, 1499, 0], [0, 0, 0], [100, 700, 690], [0, 33, 1400]):
        cu.copy_(cu_of(lengths))
        n = sum(lengths)
        graph.replay()
        again = step()
        part = {k: v[:n] if k in ("q", "k", "v", "g", "dy") else v for k, v in x.items()}
        for k, (a, b) in enumerate(zip(captured, again)):
            rows = slice(None) if k in (1, 6) else slice(0, n)
            assert torch.equal(a[rows], b[rows]), (lengths, k)
        y0, after, _ = P.forward(part, lengths, [0, 1, 2], 128 ** -0.5)
        A_y, A_s, _ = P.forward(part, lengths, [0, 1, 2], 128 ** -0.5, absolute=True)
        P.within(captured[0][:n], y0, A_y, eps_of(lengths), "y")
        P.within(captured[1], after, A_s, eps_of(lengths), "state")
    assert gdn.device_status() == 0


def test_nothing_at_all():
    """Sequences without tokens copy their states, and hand dstate_T back, whatever T allows."""
    x = P.problem([0, 0], 1, 2, 64, dtype=BF16, slots=4, seed=2)
    cu = i32([0, 0, 0])
    y = la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([1, -1]), i32([2, 3]), cu, T=500)
    assert y.shape == (0, 2, 64) and torch.equal(x["pool"][2], x["pool"][1]) and (x["pool"][3] == 0).all()
    out = la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([1, -1]), x["dy"], x["dstate"], cu, T=500)
    assert torch.equal(out[4], x["dstate"]) and gdn.device_status() == 0


def test_heads_that_share_one_place():
    """Heads of q, k and v that lie at one address (strides of 0), and keys that are the queries."""
    x = P.problem([300], 2, 4, 128, dtype=BF16, slots=2, seed=3)
    x["q"], x["v"] = x["q"][:, :1].expand(300, 2, 128), x["v"][:, :1].expand(300, 4, 128)
    x["k"] = x["q"]
    forward(x, [300], [0], [1])
    backward(x, [300], [0])


def test_an_infinity_stays_with_its_chunk_and_sequence():
    counts = [300, 200]
    x = P.problem(counts, 1, 2, 64, dtype=BF16, slots=4, seed=4)
    want = la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([0, 1]), i32([2, 3]), cu_of(counts), T=300)
    state = x["pool"][3].clone()
    x["v"][200, 0, 3] = float("inf")      # the first sequence's second chunk
    got = la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([0, 1]), i32([2, 3]), cu_of(counts), T=300)
    assert torch.equal(got[:128], want[:128]) and torch.equal(got[300:], want[300:]) and torch.equal(x["pool"][3], state)
    assert not torch.isfinite(got[201:300, 0, 3]).any()


@pytest.mark.parametrize("S,counts", [(128, [640]), (64, [300, 130]), (128, [1100, 90])])
def test_decays_gradient_is_as_exact_as_fp32(S, counts):
    """dg is a running sum of small differences of q . dq and k . dk, which are therefore taken in fp32.  A segment's first state is the
    chunked form's, off by up to 3 2^-18 of its norm at random (two splits' halves and its own): at eight segments the sum jumps by sqrt(8) 1.1e-5 / 4
    of its own; the token form's roundings are below that.  1e-5 of dg's norm."""
    x = P.problem(counts, 1, 2, S, dtype=BF16, slots=2, seed=21)
    slots = list(range(len(counts)))
    got = la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32(slots), x["dy"], x["dstate"], cu_of(counts), T=max(counts))[3]
    want = P.backward(x, counts, slots, S ** -0.5)[3]
    assert float((got.double() - want).norm() / want.norm()) <= 1e-5
    assert gdn.device_status() == 0
