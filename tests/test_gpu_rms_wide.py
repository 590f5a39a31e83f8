"""The norm's gradient on the widest rows.

Tolerance.  A thread of the long rows' kernel adds D / 1024 products one after the other, and a row's sum rounds some 45 times more:
(D / 1024 + 45) 2^-24 of the sum of magnitudes in c, four roundings of each term beside it."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import rms  # noqa: E402


@pytest.mark.parametrize("rows,D", [(1, 65535 * 256), (2, 65535 * 256 + 1), (1, 70001 * 256)])
def test_more_columns_than_a_grid_has_rows_of(rows, D):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    h, dy = (torch.randn(rows, D, generator=gen, device="cuda") for _ in range(2))
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = rms.backward(h, rstd, dy, w)
    for i in range(rows):   # a row at a time, in 64 bits
        r = rstd[i].double()
        n, t = h[i].double() * r, dy[i].double() * w.double()
        c = (t * n).mean()
        err = (dx[i].double() - r * (t - n * c)).abs()
        sums = (t * n).abs().mean()
        assert (err <= 4 * 2.0**-23 * r * (t.abs() + n.abs() * c.abs()) + (D / 1024 + 45) * 2.0**-24 * r * n.abs() * sums).all()
    terms = dy.double() * (h.double() * rstd.double()[:, None])
    assert ((dw.double() - terms.sum(0)).abs() <= 1e-5 * terms.abs().sum(0)).all()
