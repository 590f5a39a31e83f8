"""The norm's gradient with rows enough that every place of its ring of asynchronous copies is written three times and more, in
each of its forms: whole packs, rows that packs cut, the longest rows (weights in shared memory, the ring read twice), one row
or several a CTA, tensors off their 16 bytes, and rows beyond the ring's.

Tolerance.  fp32 arithmetic: 4e-6 of the sum of the terms' magnitudes, as in test_gpu_rms.py, t below.  The rounding to the
type has none: dx has to lie between what reference - t and reference + t round to (rounding is monotone).  dweight: 1e-5 of
the sum of magnitudes."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import rms  # noqa: E402
from test_gpu_rms import inputs  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SMS = 152
# (type, columns, rows of a CTA's threads at most): with 13 turns of SMS CTAs a ring of four is gone round three times
FORMS = [(BF16, 2048, 4), (BF16, 8192, 1), (F32, 4096, 2), (F32, 8192, 1), (F16, 512, 16), (BF16, 96, 16),       # whole
         (BF16, 2047, 3), (BF16, 4095, 1), (BF16, 8185, 1), (F32, 4095, 1), (F32, 1001, 5), (F16, 509, 8),       # cut
         (BF16, 12288, 1), (BF16, 8200, 1), (BF16, 12281, 1), (F16, 8193, 1),                                    # longest
         (BF16, 16384, 1), (F32, 8190, 1)]                                                                       # beyond


def check_rows(rows, D, dtype, w_dtype=F32, with_dh=True, stride=None, shift=0, seed=3):
    h, dy, w = inputs(rows, D, dtype, w_dtype, stride, shift, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    dh = torch.randn(rows, D, generator=gen, device="cuda").to(dtype) if with_dh else None
    rstd = torch.cat([h[at: at + 4096].double().square().mean(1) for at in range(0, rows, 4096)]).add(1e-6).rsqrt().float()
    dx, dw = rms.backward(h, rstd, dy, w, dh)
    again, dw2 = rms.backward(h, rstd, dy, w, dh)
    assert torch.equal(again, dx) and torch.equal(dw2, dw)   # run to run
    total, size = 0, 0
    for at in range(0, rows, 4096):   # some rows at a time, in 64 bits
        some = slice(at, at + 4096)
        r = rstd[some, None].double()
        n, g = h[some].double() * r, dy[some].double()
        t, d = g * w.double(), 0 if dh is None else dh[some].double()
        c = (t * n).mean(1, keepdim=True)
        ref = r * (t - n * c) + d
        off = 4e-6 * (r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True)) + (0 if dh is None else d.abs()))
        assert ((ref - off).to(dtype) <= dx[some]).all() and (dx[some] <= (ref + off).to(dtype)).all()
        total, size = total + (g * n).sum(0), size + (g * n).abs().sum(0)
    assert ((dw.double() - total).abs() <= 1e-5 * size).all()


@pytest.mark.parametrize("dtype,D,most", FORMS)
def test_rings_go_round(dtype, D, most):
    check_rows(SMS * most * 13 + 5, D, dtype, BF16 if D % 2 else F32, with_dh=D % 3 != 0)


@pytest.mark.parametrize("dtype,D", [(BF16, 1024), (BF16, 1001), (F32, 777)])
def test_without_a_ring(dtype, D):
    check_rows(SMS * 8 * 4 + 3, D, dtype, shift=1)


@pytest.mark.parametrize("dtype,D,stride", [(BF16, 2048, 2064), (BF16, 4095, 4103), (BF16, 12281, 12289), (F32, 1001, 1005)])
def test_rings_of_strided_rows(dtype, D, stride):
    check_rows(SMS * 13 + 1, D, dtype, stride=stride)


@pytest.mark.parametrize("dtype,D", [(BF16, 2048), (BF16, 4095), (BF16, 12288), (BF16, 12281), (F32, 4095)])
def test_a_row_is_the_same_early_and_late(dtype, D):
    """dx of rows far down a CTA's list, to the bit, as in a call of their own (at the same place within 16 bytes, and
    with as many rows a CTA)."""
    rows, few = SMS * 24, SMS * 4
    gen = torch.Generator(device="cuda").manual_seed(D)
    h, dy, dh = (torch.randn(rows, D, generator=gen, device="cuda").to(dtype) for _ in range(3))
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    rstd = (h.float().square().mean(1) + 1e-6).rsqrt()
    dx, _ = rms.backward(h, rstd, dy, w, dh)
    for at in (0, SMS * 7 + 8, rows - few):
        part = slice(at, at + few)
        assert torch.equal(rms.backward(h[part], rstd[part], dy[part], w, dh[part])[0], dx[part])
