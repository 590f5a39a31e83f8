"""The serving form of the gated delta rule (include/gdn_decode.h) on the GPU, against the token
recurrence in 64 bits.

Tolerance.  A token's dots over S_k <= 256 columns round about 40 times at 2^-24 of |M_j| |k|; with
|k| = 1 and rows of length up to about 5 that is 1.2e-5, and the decay and the correction (both contractions)
keep the earlier tokens' errors from growing beyond a small factor; errors of random sign stay well
below it.  Hence 2e-5 (1 + |ref|) for fp32.  A 16-bit y has no tolerance of its own: it has to be
the fp32 y of the same call, rounded once."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import decode, gdn  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def problem(counts, H_k, H_v, S, SV, kda=False, dtype=F32, gate=F32, slots=None, seed=0, g_std=1.0, shift=0):
    """Token rows of a packed qkv buffer (`shift` elements off its start), gates and a pool."""
    gen = torch.Generator().manual_seed(seed)
    n = sum(counts)
    def unit(*s):
        x = torch.randn(*s, generator=gen, dtype=torch.float64)
        return x / x.square().sum(-1, keepdim=True).sqrt()
    width = 2 * H_k * S + H_v * SV
    buf = torch.zeros(n * width + shift, dtype=dtype)
    qkv = buf[shift:].view(n, width)
    qkv[:, : 2 * H_k * S] = unit(n, 2 * H_k, S).reshape(n, 2 * H_k * S).to(dtype)
    qkv[:, 2 * H_k * S:] = torch.randn(n, H_v * SV, generator=gen, dtype=torch.float64).to(dtype)
    g = -torch.nn.functional.softplus(torch.randn(*((n, H_v, S) if kda else (n, H_v)), generator=gen, dtype=torch.float64) * g_std)
    beta = torch.sigmoid(torch.randn(n, H_v, generator=gen, dtype=torch.float64))
    pool = 0.1 * torch.randn(len(counts) if slots is None else slots, H_v, SV, S, generator=gen)
    dev = buf.cuda()[shift:].view(n, width)
    return dict(q=dev[:, : H_k * S].view(n, H_k, S), k=dev[:, H_k * S: 2 * H_k * S].view(n, H_k, S), v=dev[:, 2 * H_k * S:].view(n, H_v, SV),
                g=g.to(gate).cuda(), beta=beta.to(gate).cuda(), pool=pool.cuda())


def plain(x, counts, slot_in, scale):
    """Token by token in 64 bits: (y, the state after each sequence)."""
    f = lambda t: t.double().cpu().numpy()
    q, k, v, g, beta, pool = (f(x[n]) for n in ("q", "k", "v", "g", "beta", "pool"))
    H_v = v.shape[1]
    head = np.arange(H_v) % q.shape[1]
    y, after, row = np.zeros(v.shape), [], 0
    for n, c in enumerate(counts):
        M = pool[slot_in[n]].copy() if slot_in[n] >= 0 else np.zeros(pool.shape[1:])
        for _ in range(c):
            a = np.exp(g[row])
            M *= a[:, None, :] if a.ndim == 2 else a[:, None, None]
            kk, qq = k[row][head], q[row][head]
            delta = beta[row][:, None] * (v[row] - np.einsum("hji,hi->hj", M, kk))
            M += delta[:, :, None] * kk[:, None, :]
            y[row] = scale * np.einsum("hji,hi->hj", M, qq)
            row += 1
        after.append(M)
    return y, after


def near(got, ref, tol=2e-5):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= tol * (1 + np.abs(ref))).all(), float((err / (1 + np.abs(ref))).max())


def check(counts, H_k, H_v, S, SV, kda=False, dtype=F32, gate=F32, y_dtype=F32, ragged=True, slot_in=None, slot_out=None, slots=None, **kw):
    N = len(counts)
    slot_in = list(range(N)) if slot_in is None else slot_in
    slot_out = slot_in if slot_out is None else slot_out
    x = problem(counts, H_k, H_v, S, SV, kda, dtype, gate, slots, **kw)
    before = x["pool"].clone()
    y_ref, after = plain(x, counts, slot_in, S ** -0.5)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    cu = i32(np.concatenate([[0], np.cumsum(counts)]).tolist()) if ragged else None
    call = lambda pool, ty: decode.decode(x["q"], x["k"], x["v"], x["g"], x["beta"], pool, i32(slot_in), i32(slot_out), cu_tokens=cu, y_dtype=ty)
    y = call(x["pool"], F32)
    if y_dtype != F32:
        assert torch.equal(call(before.clone(), y_dtype), y.to(y_dtype))
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    near(y, y_ref)
    for n, s in enumerate(slot_out):
        if s >= 0:
            near(x["pool"][s], after[n])
    for s in set(range(before.shape[0])) - set(slot_out):
        assert torch.equal(x["pool"][s], before[s])  # nothing else is touched


@pytest.mark.parametrize("kda", [False, True], ids=["scalar", "kda"])
@pytest.mark.parametrize("S,SV", [(16, 16), (32, 32), (64, 64), (128, 128), (256, 256), (128, 48), (16, 240), (256, 16)])
def test_head_sizes(S, SV, kda):
    check([1, 0, 3, 2], 2, 6, S, SV, kda)


@pytest.mark.parametrize("kda", [False, True], ids=["scalar", "kda"])
@pytest.mark.parametrize("dtype,gate,y_dtype", [(BF16, F32, BF16), (F16, F32, F16), (BF16, BF16, F32), (F16, F16, BF16), (F32, F32, F16)])
def test_types(dtype, gate, y_dtype, kda):
    check([2, 1, 4], 2, 4, 128, 128, kda, dtype, gate, y_dtype)


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_off_their_alignment(dtype, shift):
    check([1, 2], 1, 3, 64, 64, dtype=dtype, shift=shift)


@pytest.mark.parametrize("N,T", [(1, 1), (3, 1), (2, 7), (70, 1)])
def test_same_number_of_tokens(N, T):
    """Without cu_tokens; 70 sequences of 48 heads take the wide layout, the others the narrow one."""
    check([T] * N, 16, 48, 128, 128, dtype=BF16, ragged=False)


def test_wide_layouts():
    for S, kda in ((16, False), (32, True), (64, False), (64, True), (128, True), (256, False), (256, True)):
        check([1, 2, 0] * 14, 8, 16 if S > 64 else 32, S, max(S, 32), kda)


def test_long_sequences():
    check([300, 17], 1, 2, 128, 128)
    check([300, 17], 1, 2, 64, 64, kda=True, g_std=2.0)


def test_slots():
    # one parent's slot read by three sequences, a zero start, a state that is not kept, a copy without tokens
    check([1, 2, 1, 3, 0, 1], 2, 4, 64, 64, slot_in=[2, 2, 2, -1, 5, 4], slot_out=[7, 8, 9, 10, 11, -1], slots=12)


def test_all_sequences_empty():
    check([0, 0], 2, 4, 64, 64, slot_in=[1, -1], slot_out=[3, 2], slots=4)


def test_follows_the_training_forward():
    """Prefill by gdn_forward, then the next tokens by the serving form: the forward's outputs on the whole sequence."""
    x = problem([40], 2, 4, 128, 128)
    q, k, v, g, beta = (x[n] for n in ("q", "k", "v", "g", "beta"))
    lead = lambda t, a, b: t[None, a:b].contiguous()
    state0 = torch.zeros(1, 4, 128, 128, device="cuda")
    y, sT, _, _ = gdn.forward(*[lead(t, 0, 40) for t in (q, k, v, g, beta)], state0)
    _, s32, _, _ = gdn.forward(*[lead(t, 0, 32) for t in (q, k, v, g, beta)], state0)
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    y2 = decode.decode(q[32:], k[32:], v[32:], g[32:].contiguous(), beta[32:].contiguous(), s32, slot)
    near(y2, y[0, 32:].double().cpu().numpy(), tol=2e-4)   # the chunked forward's own tolerance
    near(s32, sT.double().cpu().numpy(), tol=2e-4)


@pytest.mark.parametrize("kda", [False, True], ids=["scalar", "kda"])
def test_bits_do_not_depend_on_the_batch_or_the_steps(kda):
    T, N = 4, 50
    x = problem([T] * N, 8, 16, 128, 128, kda, BF16)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    whole, steps = x["pool"].clone(), x["pool"].clone()
    args = lambda rows: [x[n][rows].contiguous() for n in ("q", "k", "v", "g", "beta")]
    y = decode.decode(*args(slice(None)), whole, i32(range(N)))
    for n in (0, 17, 49):
        for t in range(T):
            row = slice(n * T + t, n * T + t + 1)
            y1 = decode.decode(*args(row), steps, i32([n]))
            assert torch.equal(y1, y[row])
        assert torch.equal(steps[n], whole[n])


def test_strong_gates():
    x = problem([3, 3], 2, 2, 64, 64, kda=True)
    x["g"][1] = -200.0   # exp underflows: the state is forgotten
    x["g"][2] = 0.0
    x["beta"][4] = 0.0
    y_ref, after = plain(x, [3, 3], [0, 1], 0.125)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    y = decode.decode(*[x[n] for n in ("q", "k", "v", "g", "beta", "pool")], torch.tensor([0, 1], dtype=torch.int32, device="cuda"), cu_tokens=cu)
    near(y, y_ref)
    near(x["pool"], np.stack(after))


def test_bad_slots_and_ranges_are_skipped_and_reported():
    x = problem([1, 1, 1, 1], 2, 4, 64, 64)
    before = x["pool"].clone()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    y = torch.full((4, 4, 64), 7.0, device="cuda")
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    p = decode.params_for(*args, x["pool"], 4)
    y_ref, after = plain(x, [1] * 4, [0, 1, 2, 3], 0.125)
    decode.gdn_decode(p, *args, i32([0, 1, 2, 3, 4]), x["pool"], i32([0, 4, -2, 3]), i32([0, 1, 2, 9]), y)
    assert gdn.device_status() == gdn.library().gdn_decode_supported(None) == 1
    assert gdn.device_status() == 0
    near(y[0], y_ref[0])
    near(x["pool"][0], after[0])
    assert torch.equal(x["pool"][1:], before[1:]) and (y[1:] == 7.0).all()
    x["pool"].copy_(before)
    decode.gdn_decode(p, *args, i32([0, 1, 0, 2, 5]), x["pool"], i32([0, 1, 2, 3]), i32([0, 1, 2, 3]), y)
    assert gdn.device_status() == 1   # sequence 1 ends before it starts, sequence 3 leaves the rows
    assert torch.equal(x["pool"][1], before[1]) and torch.equal(x["pool"][3], before[3])
    near(x["pool"][0], after[0])


def test_pool_beyond_32_bit_offsets_and_another_stream():
    H_v, S = 2, 64
    n, stride = 3, 1_200_000_000   # elements between slots: the last slot starts past 2^31 elements
    big = torch.empty(2 * stride + H_v * S * S, device="cuda")
    pool = big.as_strided((n, H_v, S, S), (stride, S * S, S, 1))
    x = problem([1, 2, 1], 1, H_v, S, S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    cu, slots = i32([0, 1, 3, 4]), i32([0, 1, 2])
    with torch.cuda.stream(side):
        pool.copy_(x["pool"])
        y = decode.decode(*[x[n] for n in ("q", "k", "v", "g", "beta")], pool, slots, cu_tokens=cu)
    side.synchronize()
    y_ref, after = plain(x, [1, 2, 1], [0, 1, 2], S ** -0.5)
    near(y, y_ref)
    near(pool, np.stack(after))


# ---- moves -------------------------------------------------------------------------------------

def moved(pool, src, dst):
    out = pool.clone()
    for s, d in zip(src, dst):
        if d >= 0:
            out[:, d] = 0 if s < 0 else pool[:, s]
    return out


def run_moves(pool, src, dst, group):
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    decode.gdn_states_move(pool, i32(src), i32(dst), group=group)
    torch.cuda.synchronize()
    return pool


@pytest.mark.parametrize("shape,dtype", [((1, 16), F32), ((3, 4, 64, 64), F32), ((2, 7, 48), BF16), ((1, 8200), torch.uint8), ((2, 40001, 4), F32)])
@pytest.mark.parametrize("group", [1, 2, 3, 8, 24])
def test_groups_change_places(group, shape, dtype):
    """Every group permutes its slots, with copies, clears and moves of nothing among them."""
    slots, gen = 24, np.random.default_rng(group)
    shape = (shape[0], slots) + shape[1:]
    pool = torch.randint(0, 100, shape, device="cuda").to(dtype)
    if pool[0, 0].numel() * pool.element_size() % 16:
        pool = pool[..., : pool.shape[-1] // 16 * 16].contiguous()
    src, dst = [], []
    for lo in range(0, slots, group):
        own = list(range(lo, min(lo + group, slots)))
        src += [int(gen.choice(own + [-1])) for _ in own]
        dst += [int(d) if gen.random() < 0.85 else -1 for d in gen.permutation(own)]
    want = moved(pool, src, dst)
    assert torch.equal(run_moves(pool, src, dst, group), want)


def test_large_groups():
    for n in (257, 1024):
        pool = torch.randn(2, n, 1000, device="cuda")
        perm = np.random.default_rng(n).permutation(n).tolist()
        want = moved(pool, perm, range(n))
        assert torch.equal(run_moves(pool, perm, list(range(n)), n), want)


def test_moves_only_the_states():
    """Layers inside one another's slots, gaps after every state: the gaps and the other slots stay."""
    big = torch.randn(5, 3, 20, device="cuda")              # [slot][layer][state 16 | gap 4]
    pool, before = big.transpose(0, 1)[..., :16], big.clone()
    want = moved(pool.contiguous(), [4, 0, -1], [0, 4, 2])
    run_moves(pool, [4, 0, -1], [0, 4, 2], 3)
    assert torch.equal(pool.contiguous(), want) and torch.equal(big[..., 16:], before[..., 16:])


def test_bad_moves_are_skipped_and_reported():
    pool = torch.randn(2, 4, 64, device="cuda")
    want = moved(pool, [0], [1])
    assert torch.equal(run_moves(pool, [0, 4, 1, -2], [1, 2, 7, 3], 4), want)
    assert gdn.device_status() == 1 and gdn.device_status() == 0


def test_moves_beyond_32_bit_offsets():
    stride = 2_200_000_000   # bytes between slots
    big = torch.empty(2 * stride + 4096, dtype=torch.uint8, device="cuda")
    pool = big.as_strided((1, 3, 4096), (0, stride, 1))
    pool.copy_(torch.randint(0, 255, (1, 3, 4096), device="cuda", dtype=torch.uint8))
    want = moved(pool.contiguous(), [2, 0, 1], [0, 1, 2])
    assert torch.equal(run_moves(pool, [2, 0, 1], [0, 1, 2], 3).contiguous(), want)
