"""Linear attention (include/la.h) on the GPU, token form, against the recurrence in 64 bits (la_plain.py).

Tolerance.  Errors are relative to the sum A of the magnitudes that a result is made of (the same recurrence on absolute
values).  Per token a state's element meets exp (1 unit in the last place: 2^-23), a product and a contracted sum (2^-24
each): 4 2^-24; a dot over up to 256 columns adds 40 roundings in one order, the outer factors 4.  So the token form
is within (4 T + 48) 2^-24 A, proven, whatever the signs.  dg is a running sum of dots over up to 2 x 256
columns, twice T terms: its A is the sum of all their magnitudes, and it rounds T times more: the same bound with 8 T + 100."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import la_plain as P  # noqa: E402
from gated_delta_rule_backward_gb300 import decode, gdn, la  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(counts):
    return i32([sum(counts[:n]) for n in range(len(counts) + 1)])


def check_forward(x, counts, slot_in, slot_out, ragged=True, y_dtype=None, scale=None, eps=None):
    S = x["q"].shape[2]
    sc = S ** -0.5 if scale is None else scale
    y0, after, _ = P.forward(x, counts, slot_in, sc)
    A_y, A_s, _ = P.forward(x, counts, slot_in, sc, absolute=True)
    T = max(counts, default=0)
    eps = (4 * T + 48) * U if eps is None else eps
    before = x["pool"].clone()
    y = la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32(slot_in), i32(slot_out), cu_of(counts) if ragged else None, T=T if ragged else None,
                   y_dtype=y_dtype, scale=scale)
    assert gdn.device_status() == 0
    P.within(y, y0, A_y, eps, "y")
    written = [s for s in slot_out if s >= 0]
    for n, s in enumerate(slot_out):
        if s >= 0:
            P.within(x["pool"][s], after[n], A_s[n], eps, f"state {n}")
    for s in range(len(before)):
        if s not in written:
            assert torch.equal(x["pool"][s], before[s])
    return y


def check_backward(x, counts, slot_in, ragged=True, with_state=True, scale=None, eps=None):
    S = x["q"].shape[2]
    sc = S ** -0.5 if scale is None else scale
    T = max(counts, default=0)
    ref = P.backward(x, counts, slot_in, sc, with_state)
    mag = P.backward(x, counts, slot_in, sc, with_state, absolute=True)
    eps = (4 * T + 48) * U if eps is None else eps
    got = la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32(slot_in), x["dy"], x["dstate"] if with_state else None,
                      cu_of(counts) if ragged else None, T=T if ragged else None, scale=scale)
    assert gdn.device_status() == 0
    for name, a, b, m in zip(("dq", "dk", "dv", "dg", "dstate_0"), got, ref, mag):
        P.within(a, b, m, eps + (4 * T + 52) * U * (name == "dg"), name)
    return got


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("counts,H_k,H_v,S,SV", [
    ([1], 1, 1, 16, 16), ([1] * 5, 2, 6, 64, 64), ([3, 0, 1, 17], 2, 2, 32, 48), ([5, 2], 1, 3, 128, 128), ([2] * 40, 4, 8, 128, 128),
    ([1, 30], 1, 2, 256, 112), ([9, 4, 0], 3, 3, 256, 256), ([7] * 11, 4, 4, 64, 16), ([1] * 70, 2, 2, 16, 256)])
def test_forward(counts, H_k, H_v, S, SV, dtype):
    N = len(counts)
    x = P.problem(counts, H_k, H_v, S, SV, dtype, slots=2 * N + 1, seed=S + N, shift=3 if S == 32 else 0)
    slot_in = [(3 * n + 1) % N if N % 3 else n for n in range(N)]
    slot_in[-1] = -1 if N > 1 else slot_in[-1]
    slot_out = [N + n for n in range(N)]
    if N > 2:
        slot_out[1] = -1
    assert la.form(la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], N, T=max(counts))) == "token"
    check_forward(x, counts, slot_in, slot_out, y_dtype=dtype if dtype != F32 else None, ragged=len(set(counts)) > 1)


def test_in_place_forked_and_in_steps():
    counts = [4, 4]
    x = P.problem(counts, 2, 4, 64, slots=4, seed=3)
    start = x["pool"].clone()
    check_forward(x, counts, [1, 1], [2, 3], ragged=False)            # two sequences from one slot
    x["pool"].copy_(start)
    check_forward(x, counts, [0, 2], [0, 2], ragged=False)            # in place
    whole = x["pool"].clone()
    x["pool"].copy_(start)
    for t in range(4):                                                # token by token: the same states to the bit
        pick = lambda a: a[[t, 4 + t]]
        la.forward(pick(x["q"]), pick(x["k"]), pick(x["v"]), pick(x["g"]), x["pool"], i32([0, 2]))
    assert torch.equal(x["pool"], whole)


def test_gates():
    counts = [6, 9]
    for kw in (dict(constant=True), dict(gate=BF16), dict(gate=F16, constant=True), dict(strength=0.0), dict(strength=-200.0), dict(strength=0.5)):
        x = P.problem(counts, 2, 4, 32, slots=4, seed=5, **kw)
        check_forward(x, counts, [0, 1], [2, 3])
        check_backward(x, counts, [0, 1])
    x = P.problem(counts, 2, 4, 32, slots=4, seed=5)
    wide = torch.zeros(15, 12, device="cuda")
    wide[:, ::3] = x["g"]
    x["g"] = wide[:, ::3]                                             # any strides
    x["g"][7, 1] = float("-inf")                                      # a reset: what was before leaves nothing
    check_forward(x, counts, [0, 1], [2, 3])
    check_backward(x, counts, [0, 1])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("counts,H_k,H_v,S,SV", [([1], 1, 1, 16, 16), ([3, 0, 1, 17], 2, 2, 32, 64), ([5, 2], 1, 3, 128, 128), ([9, 4, 0], 2, 4, 256, 16),
                                                ([40], 2, 2, 64, 256), ([2] * 30, 4, 4, 64, 64)])
def test_backward(counts, H_k, H_v, S, SV, dtype):
    N = len(counts)
    x = P.problem(counts, H_k, H_v, S, SV, dtype, seed=S + N)
    slot_in = list(range(N))
    slot_in[0] = -1 if N > 1 else 0
    for with_state in (True, False):
        check_backward(x, counts, slot_in, with_state=with_state, ragged=len(set(counts)) > 1)


def test_gradient_against_differences():
    """Central differences of the 64-bit loss sum(y dy) + sum(M_T dM_T): step h leaves h^2 times a third derivative of the
    size of the loss's terms (1e-8 of their sum's magnitude, since the loss is at most exponential in g and bilinear in the rest)."""
    counts = [5, 3]
    x = P.problem(counts, 1, 2, 16, seed=11)
    got = la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32([0, 1]), x["dy"], x["dstate"], cu_of(counts), T=5)
    x = {n: t.double() for n, t in x.items()}

    def loss():
        y, after, _ = P.forward(x, counts, [0, 1], 0.25)
        return float((y * x["dy"]).sum() + (after * x["dstate"]).sum())

    gen = torch.Generator().manual_seed(0)
    h = 1e-5
    for name, grad in zip(("q", "k", "v", "g", "pool"), got):
        flat = x[name].contiguous()
        x[name] = flat
        for i in torch.randint(0, flat.numel(), (6,), generator=gen).tolist():
            old = float(flat.view(-1)[i])
            flat.view(-1)[i] = old + h
            up = loss()
            flat.view(-1)[i] = old - h
            down = loss()
            flat.view(-1)[i] = old
            numeric = (up - down) / (2 * h)
            assert abs(numeric - float(grad.reshape(-1)[i])) <= 2e-4 * (1 + abs(numeric)), (name, i)


def test_what_no_sequence_owns_is_left_alone():
    counts = [3, 2]
    x = P.problem([9], 2, 2, 32, slots=4, seed=7)
    cu = i32([2, 5, 7])                                               # rows 0, 1, 7 and 8 belong to nobody
    p = la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], 2, T=3)
    y = torch.full((9, 2, 32), 7.0, device="cuda")
    la.la_forward(p, x["q"], x["k"], x["v"], x["g"], cu, x["pool"], i32([0, 1]), i32([2, 3]), y, None)
    assert (y[[0, 1, 7, 8]] == 7).all() and (y[2:7] != 7).any(-1).all()
    out = [torch.full((9, 2, 32), 7.0, device="cuda") for _ in range(3)] + [torch.full((9, 2), 7.0, device="cuda"), torch.empty(2, 2, 32, 32, device="cuda")]
    la.la_backward(p, x["q"], x["k"], x["v"], x["g"], cu, x["pool"], i32([0, 1]), x["dy"], None, *out, la.backward_workspace(p, "cuda"))
    for o in out[:4]:
        assert (o[[0, 1, 7, 8]] == 7).all() and (o[2:7] != 7).any()


@pytest.mark.parametrize("cu,slots", [([0, 4, 2], [0, 1]), ([0, 4, 9], [0, 1]), ([-1, 2, 6], [0, 1]), ([0, 6, 6], [0, 1]), ([0, 3, 6], [0, 4]), ([0, 3, 6], [-2, 1])])
def test_bad_sequences_are_skipped_and_reported(cu, slots):
    """A range that falls, leaves the rows or is longer than T, a slot outside the pool: bounds checks of the kernel."""
    x = P.problem([6], 1, 2, 32, slots=4, seed=1)
    p = la.params_for(x["q"], x["k"], x["v"], x["g"], x["pool"], 2, T=4)
    before = x["pool"].clone()
    y = torch.full((6, 2, 32), 7.0, device="cuda")
    la.la_forward(p, x["q"], x["k"], x["v"], x["g"], i32(cu), x["pool"], i32(slots), i32([2, 3]), y, None)
    bad = [n for n in range(2) if not (0 <= cu[n] <= cu[n + 1] <= 6 and cu[n + 1] - cu[n] <= 4 and -1 <= slots[n] < 4)]
    assert bad and gdn.device_status() == 1 and b"la_forward" in gdn.library().gdn_last_error()
    for n in bad:
        assert torch.equal(x["pool"][2 + n], before[2 + n])
    assert gdn.device_status() == 0


def test_states_move_between_steps():
    """The pool is gdn_states_move's: beams change places between two steps."""
    x = P.problem([1] * 4, 2, 2, 64, slots=4, seed=2)
    pool = x["pool"].clone()
    src = [2, 2, 0, 1]
    decode.gdn_states_move(pool[None], i32(src), i32([0, 1, 2, 3]), group=4)
    a = la.forward(x["q"], x["k"], x["v"], x["g"], pool, i32([0, 1, 2, 3]))
    b = la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], i32(src), i32([-1] * 4))
    assert torch.equal(a, b)


def test_another_stream_and_a_graph():
    x = P.problem([2] * 6, 2, 4, 64, slots=12, dtype=BF16, seed=4)
    s_in, s_out = i32(range(6)), i32(range(6, 12))
    step = lambda stream=None: (la.forward(x["q"], x["k"], x["v"], x["g"], x["pool"], s_in, s_out, stream=stream),
                                *la.backward(x["q"], x["k"], x["v"], x["g"], x["pool"], s_in, x["dy"], x["dstate"], stream=stream))
    direct = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(direct, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    x["v"].copy_(torch.randn(x["v"].shape, device="cuda"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))
    assert not torch.equal(captured[0], direct[0])
