"""Distillation from a teacher's top logits (include/distill.h) on the GPU against its definition in 64 bits.

Tolerance.  A student's exponential is off by 2^-22 and by what its argument, (x - m) L in one rounding with L rounded once,
is off by: 2 2^-24 |x - m| log2(e) / tau, so its logarithm's error is at most 2^-22 + 2^-23 |x - m| / tau; weighted by q, |x - m| / tau
is below 20 for the tensors here (normal logits, |x - m| up to 14 sigma at 1 / tau of 2: bound 60 for single elements).  So
lse is within 4e-6 + 3 2^-24 |lse|, a q within 60 2^-23 + 2^-21 + 2^-23 |lse| <= 1.2e-5 relative.  The loss adds
K terms p (log p - log q): 4e-6 + 2^-22 (|log p| + |log q|), below 2e-5 for the magnitudes here (|log q| <= 40).
dlogits: scale (q - p), each factor within 1.2e-5 relative, and half a unit of the stored type."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import distill  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = float("inf")


def plain(x, idx, t, dloss, tau):
    """(loss, lse, dlogits, q, p on the listed tokens) in 64 bits."""
    V = x.shape[1]
    x, t = x.double() / tau, t.double() / tau
    entry = (idx >= 0) & (idx < V) & (t != -INF)
    has = entry.any(1)
    at = idx.long().clamp(0, V - 1)
    lse = torch.logsumexp(x, 1)
    t = t.masked_fill(~entry, -INF).masked_fill(~has[:, None], 0.0)
    logp = torch.log_softmax(t, 1)
    p = logp.exp().masked_fill(~entry, 0.0)
    xs = x.gather(1, at)
    logq = torch.where(xs == -INF, -INF, xs - lse[:, None])
    loss = torch.where(p == 0, 0.0, p * (logp - logq)).sum(1)
    q = torch.where(x == -INF, 0.0, (x - lse[:, None]).exp())
    full = torch.zeros_like(x).scatter_add_(1, at, p)
    scale = (dloss.double() / tau)[:, None]
    bad = torch.isnan(lse) | torch.isnan(loss) | (lse == INF)
    d = torch.where(has[:, None], scale * (q - full), 0.0)
    size = lambda a: torch.where(has[:, None], a * scale.abs(), 0.0)
    return torch.where(has, torch.where(bad, float("nan"), loss), 0.0), torch.where(has, lse, 0.0), d, size(q), size(full)


def check(x, idx, t, tau=1.0, seed=0, in_place=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N = x.shape[0]
    dloss = torch.randn(N, generator=gen, device="cuda")
    keep = x.clone()
    loss, lse = distill.forward(x, idx, t, tau)
    both = distill.forward(x, idx, t, tau, dloss=dloss)
    d = distill.backward(x, idx, t, lse, dloss, tau)
    assert torch.equal(x, keep) or torch.isnan(keep).any()
    alike = lambda a, b: torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    assert alike(loss, both[0]) and alike(lse, both[1])
    r_loss, r_lse, r_d, q, p = plain(x, idx, t, dloss, tau)
    fine = torch.isfinite(r_loss)
    assert torch.equal(torch.isnan(r_loss), torch.isnan(loss)) and torch.equal(r_loss == INF, loss == INF)
    assert ((loss - r_loss).abs()[fine] <= 2e-5).all(), float((loss - r_loss).abs()[fine].max())
    good = torch.isfinite(r_lse) & fine
    assert ((lse - r_lse).abs() <= 4e-6 + 2e-7 * r_lse.abs())[good].all()
    half = 0.0 if x.dtype == F32 else torch.finfo(x.dtype).eps / 2
    least = 2.0 ** -24 if x.dtype == F16 else 1e-37
    rows = ~torch.isnan(r_loss)
    for got in (both[2], d):
        err = (got.double() - r_d).abs()[rows]
        bound = (1.2e-5 * (q + p) + half * r_d.abs() + least)[rows]
        assert (err <= bound).all(), float((err / bound).max())
    if in_place:
        y = x.clone()
        out = distill.forward(y, idx, t, tau, dloss=dloss, in_place=True)
        assert out[2] is y and torch.equal(y[rows], both[2][rows]) and torch.equal(out[0][fine], loss[fine])
        y = x.clone()
        distill.backward(y, idx, t, lse, dloss, tau, in_place=True)
        assert torch.equal(y[rows], d[rows])
    again = distill.forward(x, idx, t, tau, dloss=dloss)
    assert all(torch.equal(a[rows], b[rows]) for a, b in zip(both, again))
    return loss, lse, both[2]


def make(N, V, K, dtype=F32, seed=0, std=2.0, teacher=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, V, generator=gen, device="cuda") * std
    t, idx = (0.7 * x + torch.randn(N, V, generator=gen, device="cuda")).topk(min(K, V), 1)
    return x.to(dtype), idx.to(torch.int32).contiguous(), t.to(teacher).contiguous()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (2, 7, 3), (5, 31, 31), (7, 1000, 5), (400, 1023, 20), (2, 4099, 64), (1, 32000, 64), (350, 8191, 33),
                                   (3, 50001, 20), (2, 128257, 100), (310, 33000, 128), (1, 151937, 256), (320, 1, 1), (4, 2000, 1000)])
def test_sizes(N, V, K, dtype):
    check(*make(N, V, K, dtype, seed=V), tau=1.0 if N % 2 else 1.5)


@pytest.mark.parametrize("dtype,V", [(F32, 140001), (F32, 131073), (BF16, 300001), (BF16, 262145)])
def test_rows_longer_than_the_registers(dtype, V):
    check(*make(3, V, 50, dtype, seed=1))


def test_row_strides_alignment_and_types_of_the_teacher():
    for dtype in (F32, BF16, F16):
        for stride, shift in ((5000, 0), (4999, 1), (5003, 5)):
            x, idx, t = make(6, 4990, 12, dtype, teacher=BF16 if shift == 1 else F16 if shift else F32)
            buf = torch.full((6 * stride + shift,), 50.0, device="cuda", dtype=dtype)   # what lies between rows would win
            view = buf[shift:].view(6, stride)[:, :4990]
            view.copy_(x)
            check(view, idx, t, in_place=False)
            before = buf.clone()
            dloss = torch.ones(6, device="cuda")
            out = distill.forward(view, idx, t, dloss=dloss, in_place=True)
            dense = distill.forward(x, idx, t, dloss=dloss)
            assert ((out[2].float() - dense[2].float()).abs() <= 2e-5 + 0.01 * dense[2].float().abs()).all()
            inside = torch.zeros_like(buf, dtype=torch.bool)
            inside[shift:].view(6, stride)[:, :4990] = True
            assert torch.equal(buf[~inside], before[~inside])
            # a gradient whose rows lie otherwise than the logits'
            p = distill.params_for(x, idx, t, dlogits=view)
            loss, lse = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
            distill.distill_forward(p, x, idx, t, loss, lse, dloss, view)
            assert torch.equal(view, dense[2]) and torch.equal(loss, dense[0]) and torch.equal(buf[~inside], before[~inside])


def test_short_lists_padding_and_empty_rows():
    x, idx, t = make(9, 3001, 16)
    idx[1, 5:] = -1
    idx[2] = -1                      # a token without a teacher
    idx[3, 0] = 3001                 # outside: no entry
    idx[4, ::2] = -7
    t[5, 3:] = -INF                  # no entries either
    t[6] = -INF
    x[2] = float("nan")              # whatever such a row holds
    loss, lse, d = check(x, idx, t)
    for n in (2, 6):
        assert loss[n] == 0 and lse[n] == 0 and (d[n] == 0).all()
    empty = idx[:, :0].contiguous(), t[:, :0].contiguous()
    loss, lse, d = distill.forward(x, *empty, dloss=torch.ones(9, device="cuda"))
    assert (loss == 0).all() and (lse == 0).all() and (d == 0).all()


def test_tokens_listed_twice():
    x, idx, t = make(4, 2500, 32, BF16)
    idx[:, 1::2] = idx[:, ::2]
    idx[2] = idx[2, 0]
    check(x, idx, t)


def test_masked_infinite_and_nan_logits():
    x, idx, t = make(8, 5000, 10)
    x[0, idx[0].long().max() + 1:] = -INF
    x[1, 100:] = -INF                # most of the listed ones masked: the loss is infinite, the gradient is not
    x[2] = -INF
    x[3, 17] = float("nan")
    x[4, 4000] = INF
    x[5] = float("nan")
    x[6, :] = torch.finfo(F32).min   # masks of the type's lowest value
    x[6, 5:9] = torch.arange(4, device="cuda").float()
    idx[6] = -1
    idx[6, :4] = torch.tensor([5, 8, 6, 5])
    t[7, 2] = float("nan")
    loss, lse, d = check(x, idx, t, in_place=False)
    assert torch.isnan(loss[[3, 4, 5, 7]]).all() and (loss[[1, 2]] == INF).all() and lse[2] == -INF
    assert torch.isnan(d[[3, 4, 5]]).all() and torch.isfinite(d[[0, 1, 2, 6]]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_rows_of_nothing_but_the_lowest_value(dtype):
    """Finite, so every token is as likely as any other; in fp32 the logits times log2(e) leave the range."""
    x, idx, t = make(3, 700, 4, dtype)
    x[0] = torch.finfo(dtype).min
    x[2, 300:] = torch.finfo(dtype).min
    loss, lse, d = distill.forward(x, idx, t, dloss=torch.ones(3, device="cuda"))
    r = plain(x, idx, t, torch.ones(3, device="cuda"), 1.0)
    p = torch.softmax(t[0].double(), 0)
    assert abs(float(loss[0]) - float((p * (p.log() + torch.log(torch.tensor(700.0).double()))).sum())) <= 2e-5
    half = 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    assert ((d.double() - r[2]).abs()[1:] <= 2e-5 + half * r[2].abs()[1:]).all()
    others = torch.ones(700, dtype=torch.bool, device="cuda")
    others[idx[0].long()] = False
    assert ((d[0][others].double() - 1 / 700).abs() <= (1.2e-5 + half) / 700).all()


def test_temperatures_and_large_logits():
    for tau in (0.5, 1.0, 4.0, 100.0):
        check(*make(5, 2000, 20, seed=3), tau=tau)
    x, idx, t = make(3, 2000, 8)
    big = x * 1e4                     # one token holds everything
    loss, lse, d = distill.forward(big, idx, t, dloss=torch.ones(3, device="cuda"))
    r = plain(big, idx, t, torch.ones(3, device="cuda"), 1.0)
    assert ((loss - r[0]).abs() <= 4e-7 * (lse.abs() + r[0].abs())).all() and ((lse - r[1]).abs() <= 4e-7 * r[1].abs()).all()


def test_gradient_against_differences():
    """Central differences of the 64-bit loss (third derivatives of a log-sum-exp are below 1: h^2 of it)."""
    x, idx, t = make(2, 60, 6, seed=9)
    dloss = torch.tensor([1.0, -0.5], device="cuda")
    d = distill.forward(x, idx, t, 1.3, dloss=dloss)[2]
    h = 1e-4
    for n, w in ((0, 3), (0, int(idx[0, 0])), (1, int(idx[1, 2])), (1, 59)):
        y = x.double()
        val = []
        for s in (h, -h):
            z = y.clone()
            z[n, w] += s
            val.append(float((plain(z, idx, t, dloss, 1.3)[0] * dloss).sum()))
        assert abs((val[0] - val[1]) / (2 * h) - float(d[n, w])) <= 1e-5


def test_rows_beyond_32_bit_offsets_another_stream_and_a_graph():
    V, stride = 1000, 1_100_000_000
    x, idx, t = make(3, V, 8, BF16)
    big = torch.empty(2 * stride + V, dtype=BF16, device="cuda")
    rows = big.as_strided((3, V), (stride, 1))
    dloss = torch.ones(3, device="cuda")
    want = distill.forward(x, idx, t, dloss=dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rows.copy_(x)
    got = distill.forward(rows, idx, t, dloss=dloss, in_place=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = distill.forward(x, idx, t, dloss=dloss)
    x.copy_(torch.randn(3, V, device="cuda"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(captured, distill.forward(x, idx, t, dloss=dloss)))
