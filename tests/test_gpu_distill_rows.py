"""Distillation over many rows, where CTAs walk them (test_gpu_distill.py's checks and tolerances): every special row among hundreds,
at places that different CTAs and different turns of one CTA take."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import distill  # noqa: E402
from test_gpu_distill import BF16, F16, F32, INF, check, make, plain  # noqa: E402


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,V,K", [(304, 8, 3), (305, 9, 9), (2000, 100, 17), (1000, 1023, 256), (700, 8191, 33), (640, 16380, 100), (1300, 32000, 64),
                                   (400, 32761, 1), (330, 32768, 5), (310, 4097, 257), (200, 50001, 100), (160, 65522, 256),
                                   (170, 32760, 64)])
def test_sizes(N, V, K, dtype):
    check(*make(N, V, K, dtype, seed=V), tau=1.0 if N % 2 else 1.5)


def special(dtype, V=5000, K=12, times=120):
    """Rows of every kind, over and over."""
    x, idx, t = make(10, V, K, dtype, seed=V)
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
    order = torch.randperm(10 * times, generator=torch.Generator().manual_seed(1)).cuda() % 10
    return x[order].contiguous(), idx[order].contiguous(), t[order].contiguous(), order


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [5000, 4999, 1003, 32000, 40001])
def test_special_rows_among_others(dtype, V):
    x, idx, t, order = special(dtype, V)
    loss, lse, d = check(x, idx, t, tau=1.5, in_place=False)
    first = torch.stack([(order == k).nonzero()[0, 0] for k in range(10)])
    same = lambda a: torch.equal(a.nan_to_num(7.0), a[first][order].nan_to_num(7.0))
    if V * x.element_size() % 16 == 0:   # the same row, the same place within 16 bytes: the same bits
        assert same(loss) and same(lse)
    assert (loss[order == 2] == 0).all() and (d[order == 2] == 0).all() and torch.isnan(loss[order == 8]).all() and torch.isnan(d[order == 6]).all()
    assert torch.isfinite(d[(order != 6) & (order != 8)].float()).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_the_lowest_value_and_large_logits(dtype):
    x, idx, t = make(400, 700, 4, dtype)
    x[::3] = torch.finfo(dtype).min
    x[1::3] *= 1e4
    dloss = torch.ones(400, device="cuda")
    loss, lse, d = distill.forward(x, idx, t, dloss=dloss)
    r = plain(x, idx, t, dloss, 1.0)
    half = 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    p = torch.softmax(t[::3].double(), 1)
    want = (p * (p.log() + torch.log(torch.tensor(700.0).double()))).sum(1)
    assert ((loss[::3] - want).abs() <= 2e-5).all()
    others = torch.ones(700, dtype=torch.bool, device="cuda")
    others[idx[0].long()] = False
    assert ((d[0][others].double() - 1 / 700).abs() <= (1.2e-5 + half) / 700).all()
    assert ((loss[1::3] - r[0][1::3]).abs() <= 4e-7 * (lse[1::3].abs() + r[0][1::3].abs())).all()
    assert ((d.double() - r[2]).abs()[2::3] <= 2e-5 + half * r[2].abs()[2::3]).all()


def test_row_strides_places_and_gradients_elsewhere():
    for dtype in (F32, BF16):
        for stride, shift in ((2504, 0), (2499, 1), (2503, 5)):
            x, idx, t = make(350, 2490, 12, dtype)
            buf = torch.full((350 * stride + shift,), 50.0, device="cuda", dtype=dtype)   # what lies between rows would win
            view = buf[shift:].view(350, stride)[:, :2490]
            view.copy_(x)
            check(view, idx, t, in_place=False)
            inside = torch.zeros_like(buf, dtype=torch.bool)
            inside[shift:].view(350, stride)[:, :2490] = True
            dloss = torch.linspace(-1, 1, 350, device="cuda")
            distill.forward(view, idx, t, dloss=dloss, in_place=True)
            dense = distill.forward(x, idx, t, dloss=dloss)
            assert ((view.float() - dense[2].float()).abs() <= 2e-5 + 0.01 * dense[2].float().abs()).all() and (buf[~inside] == 50).all()
            p = distill.params_for(x, idx, t, dlogits=view)   # rows that lie otherwise than the logits'
            loss, lse = torch.empty(350, device="cuda"), torch.empty(350, device="cuda")
            distill.distill_forward(p, x, idx, t, loss, lse, dloss, view)
            assert torch.equal(view, dense[2]) and torch.equal(loss, dense[0]) and (buf[~inside] == 50).all()


def test_both_kernels_agree_and_a_weight_of_nothing():
    """A list of more than 256 entries, here padding, sends rows to clusters."""
    x, idx, t = make(310, 6000, 40, BF16)
    dloss = torch.randn(310, device="cuda")
    dloss[::7] = 0.0
    padded = torch.cat([idx, torch.full((310, 260), -1, dtype=torch.int32, device="cuda")], 1), torch.cat([t, torch.zeros(310, 260, device="cuda")], 1)
    a, b = distill.forward(x, idx, t, dloss=dloss), distill.forward(x, *padded, dloss=dloss)
    assert ((a[0] - b[0]).abs() <= 4e-5).all() and ((a[1] - b[1]).abs() <= 1e-5).all()
    assert ((a[2].float() - b[2].float()).abs() <= 2.0 ** -7 * b[2].float().abs() + 1e-7).all()
    assert (a[2][::7] == 0).all() and (b[2][::7] == 0).all()


def test_another_stream_and_a_graph():
    x, idx, t = make(500, 4000, 16, BF16)
    dloss = torch.randn(500, device="cuda")
    want = distill.forward(x, idx, t, dloss=dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = distill.forward(x, idx, t, dloss=dloss, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = (*distill.forward(x, idx, t, dloss=dloss), distill.backward(x, idx, t, want[1], dloss))
    x.copy_(torch.randn(500, 4000, device="cuda"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(captured, (*distill.forward(x, idx, t, dloss=dloss), distill.backward(x, idx, t, want[1], dloss))))
