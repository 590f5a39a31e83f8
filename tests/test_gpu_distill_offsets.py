"""Distillation (include/distill.h) of logits that lie far from zero: a softmax does not change when all logits of a row are shifted, however far.

Tolerance.  With D = (m - x) / tau >= 0 (m the row's largest logit), a student's exponential is exp(-D): x - m is rounded once, log2(e) / tau once and their product
once, 3 2^-24 D, and 2^x is off by 2^-22; the sum over the row adds what test_gpu_distill.py derives.  So q is within 1.2e-5 + 2^-22 D relative, and the teacher's
p within 1.2e-5 + 2^-22 D_t with its own distances.  None of it depends on where the row lies: the gradient alone
goes by lse up to 32 in size, where its fp32 number adds 2^-24 |lse| and its product with log2(e) the same, 3.8e-6 within the 1.2e-5.  lse is one fp32 number: 4e-6 + 2e-7 |lse|.
The loss is the sum of p (log p - log q): p's error times what it weighs, and 2^-22 of the terms D, D_t and log V that make up the logarithms, and 1e-5 for the two sums'."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import distill  # noqa: E402
from test_gpu_distill import BF16, F16, F32, make, plain  # noqa: E402
from test_gpu_distill_clusters import padded  # noqa: E402


def far_rows(dtype, V, K, N=None):
    """Rows of normal logits a long way off, rows of one value, and rows spread over a wide range: those of fp32, as far as the type holds them."""
    most = torch.finfo(dtype).max
    offsets = [0.0] + [s * o for o in (40.0, 1e3, 1e4, 6e4, 1e6, 1e9, 1e30) for s in (1, -1) if o < most]
    flat = [-most, most] + [s * o for o in (300.0, 1e4, 1e9, 5.1e9, 1e10, 1e12, 1e30) for s in (1, -1) if o < most]
    n = len(offsets) + len(flat) + 2
    x, idx, t = make(n, V, K, F32, seed=V + K)
    x[: len(offsets)] += torch.tensor(offsets, device="cuda")[:, None]
    x[len(offsets): -2] = torch.tensor(flat, device="cuda")[:, None]
    x[-2] *= 1e4 if dtype != F16 else 1e3
    x[-1, V // 2:] = -most                       # a masked half
    x = x.to(dtype)
    if N is not None:                            # the same rows over and over
        order = torch.arange(N, device="cuda") % n
        x, idx, t = x[order].contiguous(), idx[order].contiguous(), t[order].contiguous()
    return x, idx, t


FORMS = {"rows": dict(V=1003, K=20), "wide rows": dict(V=33001, K=12, N=80), "clusters": dict(V=1003, K=20, pad=True), "larger clusters": dict(V=70000, K=12, pad=True),
         "clusters that read again": dict(V=140001, K=12, dtypes=[F32])}
CASES = [(form, dtype) for form, kw in FORMS.items() for dtype in kw.get("dtypes", [F32, BF16, F16])]


def problem(form, dtype):
    kw = dict(FORMS[form])
    kw.pop("dtypes", None)
    pad = kw.pop("pad", False)
    x = far_rows(dtype, **kw)
    return padded(*x) if pad else x


def bounds(x, idx, t, dloss, tau):
    """(loss, its bound, lse, dlogits, their bound) in 64 bits, which at 1e30 hold no log of a sum beside the largest logit: so from the distances to it."""
    V = x.shape[1]
    m = x.double().amax(1, keepdim=True)
    X, T = (x.double() - m) / tau, t.double() / tau
    loss, lse, d, q, p = plain(x.double() - m, idx, t, dloss, tau)
    entry = idx >= 0
    at = idx.long().clamp(0, V - 1)
    D = -X
    T = T.masked_fill(~entry, -math.inf)
    Dt = (T.amax(1, keepdim=True) - T).masked_fill(~entry, 0.0)
    P = torch.softmax(T, 1).masked_fill(~entry, 0.0)
    logs = (torch.log_softmax(T, 1).masked_fill(~entry, 0.0) - (X.gather(1, at) - lse[:, None])).abs()
    off = (P * ((1.2e-5 + 2.0 ** -22 * Dt) * logs + 2.0 ** -22 * (D.gather(1, at) + Dt + math.log(V)))).sum(1) + 1e-5
    # p of an unlisted token is 0; of one listed twice, each entry's error
    err = q * (1.2e-5 + 2.0 ** -22 * D) + p * (1.2e-5 + 2.0 ** -22 * Dt.amax(1, keepdim=True))
    half = 0.0 if x.dtype == F32 else torch.finfo(x.dtype).eps / 2
    # the hardware's 2^x gives 0 below 2^-126: a q or p of a listed token that is lost there counts |dloss| / tau times
    err = err + 2.0 ** -125 * dloss.double().abs()[:, None] / tau
    return loss, off, lse + m[:, 0] / tau, d, err * (1 + half) + half * d.abs() + (2.0 ** -24 if x.dtype == F16 else 1e-37)


def within(got, want, bound, what):
    over = ~((got.double() - want).abs() <= bound)
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} off, in rows {sorted(set(over.nonzero()[:, 0].tolist()))[:20]}, by up to {float((got.double() - want).abs()[over].max()):.3e}"


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0, 4.0])
@pytest.mark.parametrize("form,dtype", CASES)
def test_loss(form, dtype, tau):
    x, idx, t = problem(form, dtype)
    loss, lse = distill.forward(x, idx, t, tau)
    r_loss, off, r_lse, _, _ = bounds(x, idx, t, torch.ones(len(x), device="cuda"), tau)
    held = torch.isfinite(r_lse.float())        # fp32 holds it
    within(lse[held, None], r_lse[held, None], (4e-6 + 2e-7 * r_lse.abs())[held, None], "lse")
    assert torch.isinf(lse[~held]).all()
    within(loss[:, None], r_loss[:, None], off[:, None], "loss")


def test_a_sum_whose_correction_would_leave_the_range():
    """Values whose product with log2(e) is off by just over 126 powers of two when it is rounded: neither the product's 2^x nor the correction's is infinite."""
    m = torch.tensor([3000016896.0, 3000146432.0, 3000164352.0, 3000244736.0, 3000293888.0, 3000374272.0, 3000392192.0, 3000521728.0])
    product = m.double() * torch.tensor(1 / math.log(2)).double()
    off = (product - product.float().double()).abs()
    assert (off > 126.2).all() and (off < 127.8).all()
    found = m.tolist()
    x, idx, t = make(16, 700, 6)
    x[:] = torch.tensor(found + [-v for v in found], device="cuda")[:, None]
    for lists in ((idx, t), padded(x, idx, t)[1:]):
        loss, lse = distill.forward(x, *lists)
        r_loss, off, r_lse, _, _ = bounds(x, *lists, torch.ones(16, device="cuda"), 1.0)
        within(loss[:, None], r_loss[:, None], off[:, None], "loss")
        within(lse[:, None], r_lse[:, None], (4e-6 + 2e-7 * r_lse.abs())[:, None], "lse")


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0, 4.0])
@pytest.mark.parametrize("form,dtype", CASES)
def test_gradient_with_the_loss(form, dtype, tau):
    x, idx, t = problem(form, dtype)
    dloss = torch.linspace(-1.5, 1.0, len(x), device="cuda")
    loss, lse, d = distill.forward(x, idx, t, tau, dloss=dloss)
    alone = distill.forward(x, idx, t, tau)
    assert torch.equal(loss, alone[0]) and torch.equal(lse, alone[1])
    _, _, _, r_d, bound = bounds(x, idx, t, dloss, tau)
    within(d, r_d, bound, "dlogits")
    y = x.clone()
    distill.forward(y, idx, t, tau, dloss=dloss, in_place=True)
    assert torch.equal(y, d)
    if dtype == F32:                                 # what moves all logits alike changes nothing
        assert (d.double().sum(1).abs() <= bound.sum(1)).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_shift_changes_nothing(dtype):
    """Logits that are whole multiples of 64 stay exact under shifts by multiples of 2^20 within 24 (bf16: 8) bits: the gradient keeps its bits."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    step = 64.0 if dtype == F32 else 2.0 ** 14
    x = torch.randint(0, 4, (40, 900), generator=gen, device="cuda").float() * step
    _, idx, t = make(40, 900, 8)
    for lists in ((idx, t), padded(x, idx, t)[1:]):
        want = distill.forward(x.to(dtype), *lists, step, dloss=torch.ones(40, device="cuda"))
        for shift in (2.0 ** 20, -2.0 ** 20, 2.0 ** 20 + 4 * step):
            y = (x + shift).to(dtype)
            assert torch.equal(y.float() - shift, x)
            got = distill.forward(y, *lists, step, dloss=torch.ones(40, device="cuda"))
            assert torch.equal(got[2], want[2])


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0, 4.0])
@pytest.mark.parametrize("form,dtype", CASES)
def test_gradient_alone(form, dtype, tau):
    x, idx, t = problem(form, dtype)
    dloss = torch.linspace(-1.5, 1.0, len(x), device="cuda")
    loss, lse = distill.forward(x, idx, t, tau)
    d = distill.backward(x, idx, t, lse, dloss, tau)
    _, _, r_lse, r_d, bound = bounds(x, idx, t, dloss, tau)
    within(d, r_d, bound, "dlogits")
    within(distill.backward(x, idx, t, r_lse.float(), dloss, tau), r_d, bound, "dlogits from an lse of 64 bits")
    y = x.clone()
    distill.backward(y, idx, t, lse, dloss, tau, in_place=True)
    assert torch.equal(y, d)
    lse[::2] = float("nan")
    d = distill.backward(x, idx, t, lse, dloss, tau)
    assert torch.isnan(d[::2]).all() and torch.isfinite(d[1::2].float()).all()


@pytest.mark.parametrize("tau", [0.5, 0.01, 100.0])
@pytest.mark.parametrize("form,dtype", CASES)
def test_other_temperatures(form, dtype, tau):
    """Small ones bring losses of listed but masked tokens near fp32's limit: those that it holds are given, others are infinite."""
    x, idx, t = problem(form, dtype)
    dloss = torch.linspace(-1.5, 1.0, len(x), device="cuda")
    loss, lse, d = distill.forward(x, idx, t, tau, dloss=dloss)
    r_loss, off, r_lse, r_d, bound = bounds(x, idx, t, dloss, tau)
    held = r_loss + off < torch.finfo(F32).max
    within(loss[held, None], r_loss[held, None], off[held, None], "loss")
    assert (loss[r_loss - off > torch.finfo(F32).max * (1 + 2.0 ** -24)] == math.inf).all()
    held = torch.isfinite(r_lse.float())
    within(lse[held, None], r_lse[held, None], (4e-6 + 2e-7 * r_lse.abs())[held, None], "lse")
    assert torch.isinf(lse[~held]).all()
    within(d, r_d, bound, "dlogits")
    within(distill.backward(x, idx, t, lse, dloss, tau), r_d, bound, "dlogits alone")


@pytest.mark.parametrize("pad", [False, True])
def test_a_masked_token_that_counts_for_little(pad):
    """Its distance to the largest logit, over the temperature, is beyond fp32's range; what it adds to the loss is not."""
    x, idx, t = make(4, 800, 6)
    x[torch.arange(4, device="cuda")[:, None], idx[:, 2:3].long()] = torch.finfo(F32).min
    t[:] = torch.tensor([3.0, 2.0, 1.0, 0.0, -1.0, -2.0], device="cuda")
    if pad:
        x, idx, t = padded(x, idx, t)
    loss = distill.forward(x, idx, t, 0.5)[0]
    r_loss, off, _, _, _ = bounds(x, idx, t, torch.ones(4, device="cuda"), 0.5)
    assert (r_loss < 3e38).all() and (r_loss > 1e36).all()
    within(loss[:, None], r_loss[:, None], off[:, None], "loss")
