"""The beam selection (include/beam.h) on the GPU against its definition in 64 bits.

Tolerance.  The sum of exponentials is off by a few 2^-22 at most (the exponential's own error; the
sums round less), its logarithm by 1e-6, and the rest rounds three times at the magnitude of the score:
|error| <= 2e-6 + 4 2^-24 |score| + 4 2^-24 |logit - max|.  Below, 2e-6 (1 + |score|) + 3e-7 |logit - max|.
The choice has to be the definition's wherever its own gaps are above that; ties are made of equal logits and
scores, where both sides are equal to the last bit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import beam  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = float("inf")


def plain(logits, scores, done, n, pad):
    """(score, flat index) of the n best, and every candidate's score, in 64 bits."""
    N, K = scores.shape
    x = logits.double().cpu().numpy().reshape(N, K, -1).copy()
    V = x.shape[2]
    x[np.isnan(x)] = -INF
    s = scores.double().cpu().numpy().copy()
    s[np.isnan(s)] = -INF
    top = x.max(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.where(x == top, np.where(np.isneginf(top), -INF, 0.0), x - top)
        c = s[..., None] + (d - np.log(np.exp(d).sum(-1, keepdims=True)))
    c[np.isnan(c)] = -INF
    if done is not None:
        for i, k in zip(*np.nonzero(done.cpu().numpy())):
            c[i, k] = -INF
            c[i, k, pad] = s[i, k]
    c[np.isneginf(s)] = -INF
    flat = c.reshape(N, K * V)
    order = np.argsort(-flat, axis=1, kind="stable")[:, :n]
    return np.take_along_axis(flat, order, 1), order, flat


def check(logits, scores, done=None, n=None, pad=0, exact_ties=False):
    N, K = scores.shape
    V = logits.shape[1]
    n = K if n is None else n
    slots = torch.arange(100, 100 + N * K, dtype=torch.int32, device="cuda").view(N, K).flip(1).contiguous()
    got, parent, token, src = beam.select(logits, scores, done, slots, n_out=n, pad_token=pad)
    ref, order, flat = plain(logits, scores, done, n, pad)
    g, at = got.double().cpu().numpy(), (parent.long() * V + token).cpu().numpy()
    assert ((token >= 0) & (token < V) & (parent >= 0) & (parent < K)).all()
    assert torch.equal(src, slots.gather(1, parent.long()))
    assert (np.isneginf(g) == np.isneginf(ref)).all()
    fine = np.isfinite(ref)
    tol = 2e-6 * (1 + np.abs(np.where(fine, ref, 0))) + 3e-7 * 40
    assert (np.abs(g[fine] - ref[fine]) <= tol[fine]).all()
    assert (np.sort(at, 1)[:, 1:] != np.sort(at, 1)[:, :-1]).all()          # nothing twice
    own = np.take_along_axis(flat, at, 1)                                   # what the chosen are worth
    assert (np.abs(own[fine] - ref[fine]) <= 2 * tol[fine]).all()
    clear = np.ones_like(fine)                                              # far from both neighbours in the whole order
    more = -np.sort(-flat, axis=1)[:, : n + 1]
    if more.shape[1] == n:
        more = np.concatenate([more, np.full((N, 1), -INF)], 1)
    with np.errstate(invalid="ignore"):
        gap = more[:, :-1] - more[:, 1:]
    clear = (gap > 4 * tol) & (np.concatenate([np.full((N, 1), INF), gap[:, :-1]], 1) > 4 * tol)
    if exact_ties:
        clear = np.ones_like(clear)
    clear |= ~fine
    assert (at == order)[clear].all()
    again = beam.select(logits, scores, done, slots, n_out=n, pad_token=pad)
    assert all(torch.equal(a, b) for a, b in zip(again, (got, parent, token, src)))
    return got, parent, token


def make(N, K, V, dtype=F32, seed=0, std=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(N * K, V, generator=gen, device="cuda") * std).to(dtype), -4 * torch.randn(N, K, generator=gen, device="cuda").abs()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,K,V,n", [(1, 1, 1, 1), (2, 1, 5, 5), (1, 4, 3, 12), (3, 2, 17, 4), (2, 3, 257, 6), (1, 4, 32000, 4), (5, 5, 4099, 10),
                                     (1, 1, 700, 32), (2, 8, 8193, 64), (1, 64, 1000, 64), (40, 4, 50001, 4), (3, 16, 130000, 32)])
def test_sizes(N, K, V, n, dtype):
    check(*make(N, K, V, dtype, seed=V), n=n)


def test_row_strides_and_alignment():
    for dtype in (F32, BF16):
        for stride, shift in ((5000, 0), (4999, 1), (5003, 5)):
            x, s = make(2, 3, 4990, dtype)
            buf = torch.full((6 * stride + shift,), 99.0, device="cuda", dtype=dtype)   # what lies between rows would win
            view = buf[shift:].view(6, stride)[:, :4990]
            view.copy_(x)
            got = check(view, s, n=7)
            for a, b in zip(got, beam.select(x, s, n_out=7)):
                assert torch.equal(a, b) or a.dtype == F32


def test_masked_tokens_and_rows():
    x, s = make(3, 4, 3001)
    x[:, 10:] = -INF            # ten tokens allowed
    x[0] = -INF                 # a beam without any
    x[4:8] = -INF               # a sequence without any: the lowest indices at -inf
    check(x, s, n=8)
    x[8:12] = -INF
    x[9, 2000] = 1.0            # a single candidate, and fillers around it
    x[10, 1] = -1.0
    check(x, s, n=8)
    check(x[8:12], s[2:], n=64)


def test_first_step_and_dead_beams():
    x, s = make(4, 5, 50001, F16)
    s[:, 1:] = -INF
    got, parent, _ = check(x, s, n=10)
    assert (parent == 0).all()
    s[1, 0] = -INF              # nothing alive
    s[2, 0] = float("nan")
    check(x, s, n=10)


def test_finished_beams():
    x, s = make(3, 4, 1000)
    done = torch.zeros(3, 4, dtype=torch.uint8, device="cuda")
    done[0, 1] = done[1] = 1
    done[2, 3] = 7
    s[2, 3] = -INF
    got, parent, token = check(x, s, done, n=8, pad=13)
    assert (token[1, :4] == 13).all() and torch.isneginf(got[1, 4:]).all()
    check(x, s, done.bool(), n=4, pad=999)


def test_infinite_and_nan_logits():
    x, s = make(2, 2, 5000)
    x[0, 7] = x[0, 4000] = INF
    x[1, ::2] = float("nan")
    x[2] = float("nan")
    x[3, 1] = INF
    check(x, s, n=6)


@pytest.mark.parametrize("value", [0.0, -0.0, 3.5])
def test_ties_go_to_the_lowest_index(value):
    for V in (40, 300, 9000, 40000):
        x = torch.full((4, V), value, device="cuda", dtype=BF16)
        if value == 0.0:
            x[:, ::3] = -0.0
        s = torch.zeros(2, 2, device="cuda")
        _, parent, token = beam.select(x, s, n_out=20)
        assert (parent == 0).all() and (token == torch.arange(20, device="cuda")).all()
        x[:, V // 2] = x[:, V - 1] = 5.0
        _, parent, token = beam.select(x, s, n_out=7)
        assert parent.tolist() == [[0, 0, 1, 1, 0, 0, 0]] * 2
        assert token.tolist() == [[V // 2, V - 1, V // 2, V - 1, 0, 1, 2]] * 2


def test_few_distinct_values():
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(0, 3, (6, 30016), generator=gen, device="cuda").to(BF16)
    x[1::3] = x[0::3]          # two equal beams: equal candidates, the lower beam first
    s = torch.tensor([[-1.0, -1.0, -2.0]] * 2, device="cuda")
    check(x, s, n=40, exact_ties=True)


def test_large_scores_and_logits():
    x, s = make(2, 3, 2000, std=2000.0)
    check(x, s * 1e4, n=6)


def test_rows_beyond_32_bit_offsets_and_another_stream():
    V, stride = 1000, 1_100_000_000
    big = torch.empty(2 * stride + V, dtype=BF16, device="cuda")
    rows = big.as_strided((3, V), (stride, 1))
    x, s = make(1, 3, V, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rows.copy_(x)
        out = beam.select(rows, s)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, beam.select(x, s)))
