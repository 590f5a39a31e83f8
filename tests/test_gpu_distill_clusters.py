"""Distillation of rows that clusters of CTAs hold (test_gpu_distill.py's checks and tolerances): lists of more entries than a CTA has threads, here
by padding, send rows of any length there, and so does a row of more than 64 KB."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import distill  # noqa: E402
from test_gpu_distill import BF16, F16, F32, INF, check, make, plain  # noqa: E402


def padded(x, idx, t, K=300):
    n = K - idx.shape[1]
    fill = lambda a, v: torch.cat([a, torch.full((a.shape[0], n), v, dtype=a.dtype, device="cuda")], 1)
    return x, fill(idx, -1), fill(t, 0.0)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (2, 7, 3), (5, 31, 31), (7, 1000, 5), (400, 1023, 20), (2, 4099, 64), (1, 32000, 64), (350, 8191, 33),
                                   (620, 2048, 200)])
def test_sizes(N, V, K, dtype):
    check(*padded(*make(N, V, K, dtype, seed=V)), tau=1.0 if N % 2 else 1.5)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,K", [(5000, 300), (70000, 12)])
def test_special_rows(dtype, V, K):
    x, idx, t = make(10, V, 12, dtype, seed=V)
    idx[1, 5:] = -1                  # a short list
    idx[2] = -1                      # no list, whatever the row holds
    x[2] = float("nan")
    idx[3, 1::2] = idx[3, ::2]       # tokens listed twice
    x[4, 100:] = -INF                # most listed ones masked
    x[5] = -INF
    x[6, 17] = float("nan")
    x[7] = torch.finfo(dtype).min
    idx[7] = -1
    idx[7, :4] = torch.tensor([5, 8, 6, 5])
    x[7, 5:9] = torch.arange(4, device="cuda").to(dtype)
    t[8, 2] = float("nan")
    t[9, 3:] = -INF
    idx[9, 0] = V                    # outside: no entry
    loss, lse, d = check(*padded(x, idx, t, K), tau=1.5, in_place=False)
    assert loss[2] == 0 and (d[2] == 0).all() and torch.isnan(loss[8]) and torch.isnan(d[6]).all()
    assert torch.isfinite(d[[0, 1, 2, 3, 4, 5, 7, 9]].float()).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_rows_of_nothing_but_the_lowest_value(dtype):
    x, idx, t = make(3, 700, 4, dtype)
    x[0] = torch.finfo(dtype).min
    x[2, 300:] = torch.finfo(dtype).min
    x, idx, t = padded(x, idx, t)
    dloss = torch.ones(3, device="cuda")
    loss, lse, d = distill.forward(x, idx, t, dloss=dloss)
    r = plain(x, idx, t, dloss, 1.0)
    p = torch.softmax(t[0, :4].double(), 0)
    assert abs(float(loss[0]) - float((p * (p.log() + torch.log(torch.tensor(700.0).double()))).sum())) <= 2e-5
    half = 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    assert ((d.double() - r[2]).abs()[1:] <= 2e-5 + half * r[2].abs()[1:]).all()


def test_row_strides_and_places():
    for dtype in (F32, BF16):
        for stride, shift in ((5000, 0), (4999, 1), (5003, 5)):
            x, idx, t = padded(*make(6, 4990, 12, dtype))
            buf = torch.full((6 * stride + shift,), 50.0, device="cuda", dtype=dtype)   # what lies between rows would win
            view = buf[shift:].view(6, stride)[:, :4990]
            view.copy_(x)
            check(view, idx, t, in_place=False)
            inside = torch.zeros_like(buf, dtype=torch.bool)
            inside[shift:].view(6, stride)[:, :4990] = True
            distill.forward(view, idx, t, dloss=torch.ones(6, device="cuda"), in_place=True)
            assert (buf[~inside] == 50).all()


def test_a_graph():
    x, idx, t = padded(*make(20, 4000, 16, BF16))
    dloss = torch.randn(20, device="cuda")
    distill.forward(x, idx, t, dloss=dloss)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = distill.forward(x, idx, t, dloss=dloss)
    x.copy_(torch.randn(20, 4000, device="cuda"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(captured, distill.forward(x, idx, t, dloss=dloss)))
