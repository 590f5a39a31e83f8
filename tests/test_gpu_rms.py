"""The root-mean-square norm (include/rms.h) on the GPU against its definition in 64 bits.

Tolerances.  A row's sum rounds at most about 40 times a term's way up at 2^-24 (2.4e-6 of a sum of
squares, half of it in rstd) and a product chain 4 times: 4e-6 of the value for y, rstd and scales.  dx
is a difference, so 4e-6 of the sum of its terms' magnitudes, plus half a unit in the last place of its type
(2^-8 of the value in bf16, 2^-11 in fp16).  dweight sums up to a few hundred terms one after the
other: 1e-5 of the sum of magnitudes.  16-bit y, h and the 8-bit codes have no tolerance: they must be what the
fp32 values of the same call round to."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import gdn, rms  # noqa: E402

F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn
UNIT = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}


def rows_of(gen, rows, D, dtype, std, stride, shift):
    """[rows, D] values, `stride` elements apart, `shift` elements off an aligned start."""
    buf = torch.zeros(rows * stride + shift, device="cuda", dtype=dtype)
    t = buf[shift: shift + rows * stride].view(rows, stride)[:, :D]
    t.copy_(torch.randn(rows, D, generator=gen, device="cuda") * std)
    return t


def inputs(rows, D, dtype=F32, w_dtype=F32, stride=None, shift=0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = D if stride is None else stride
    return (rows_of(gen, rows, D, dtype, 1.0, s, shift), rows_of(gen, rows, D, dtype, 2.0, s, shift),
            (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(w_dtype))


def plain(x, r, w, eps):
    h = x.double() + (0 if r is None else r.double())
    rstd = (h.square().mean(1) + eps).rsqrt()
    return h, h * rstd[:, None] * (1 if w is None else w.double()), rstd


def near(got, ref, tol):
    assert got.shape == ref.shape and torch.isfinite(got.double()).all()
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())


def check_forward(x, r, w, eps=1e-6):
    h_ref, y_ref, rstd_ref = plain(x, r, w, eps)
    y, h, rstd = rms.forward(x, w, r, eps, y_dtype=F32)
    near(y, y_ref, 4e-6 * y_ref.abs() + 1e-37)
    near(rstd, rstd_ref, 4e-6 * rstd_ref)
    assert torch.equal(h, x if r is None else (x.float() + r.float()).to(x.dtype))
    for dtype in (BF16, F16):
        assert torch.equal(rms.forward(x, w, r, eps, y_dtype=dtype)[0], y.to(dtype))
    D = x.shape[1]
    for group in [0] + [g for g in (16, 32, 64, 128) if D % g == 0]:
        q, scales, h8, rstd8 = rms.forward(x, w, r, eps, y_dtype=E4M3, group=group)
        parts = y.view(x.shape[0], -1, group or D)
        want = (y_ref.view(parts.shape).abs().amax(-1) / 448).clamp(min=2.0 ** -126)
        near(scales.view(want.shape), want, 4e-6 * want)
        codes = (parts * (1.0 / scales.view(want.shape)[..., None])).to(E4M3).view(x.shape)
        assert torch.equal(q.view(torch.uint8), codes.view(torch.uint8))
        assert torch.equal(h8, h) and torch.equal(rstd8, rstd)
    return y, h, rstd


SIZES = [(1, 1), (3, 7), (1, 64), (5, 128), (300, 96), (7, 1000), (2, 2048), (333, 1024), (4, 6144), (2, 8191), (3, 8192), (2, 16384), (1, 20000), (2, 33000)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,D", SIZES)
def test_forward(rows, D, dtype):
    check_forward(*inputs(rows, D, dtype))


@pytest.mark.parametrize("w_dtype", [None, F32, BF16, F16])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_without_parts(residual, w_dtype):
    x, r, w = inputs(5, 384, BF16, w_dtype or F32)
    check_forward(x, r if residual else None, w if w_dtype else None)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("stride,shift", [(264, 0), (256, 1), (259, 3), (300, 8)])
def test_forward_strides_and_alignment(stride, shift, dtype):
    check_forward(*inputs(6, 256, dtype, stride=stride, shift=shift))


@pytest.mark.parametrize("D", [1024, 1001, 40000])
def test_forward_in_place(D):
    x, r, w = inputs(4, D, BF16)
    y, h, rstd = rms.forward(x, w, r)
    for buf in (x.clone(), r.clone()):
        y2, rstd2 = torch.empty_like(y), torch.empty_like(rstd)
        a, b = (buf, r) if torch.equal(buf, x) else (x, buf)
        rms.rms_forward(rms.params_for(x, w), a, b, w, buf, y2, None, rstd2)
        assert torch.equal(buf, h) and torch.equal(y2, y) and torch.equal(rstd2, rstd)


def test_forward_special_values():
    x = torch.zeros(4, 256, device="cuda")
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 1e-30
    y, _, rstd = rms.forward(x, eps=1e-6)
    assert (y[0] == 0).all() and abs(float(rstd[0]) - 1e3) <= 4e-3
    assert torch.isnan(y[1, 3]) and (y[1, :3] == 0).all() and torch.isnan(y[2]).all()
    near(y[3].double(), torch.full((256,), 1e-27, dtype=torch.float64, device="cuda"), 4e-33)
    q, scales, _, _ = rms.forward(x, eps=1e-6, y_dtype=E4M3)
    assert (q[0].float() == 0).all() and scales[0] == 2.0 ** -126      # a row of zeros
    assert (q[3].float() == 448).all()


def check_backward(rows, D, dtype=F32, w_dtype=F32, with_dh=True, with_w=True, stride=None, shift=0, seed=3):
    h, dy, w = inputs(rows, D, dtype, w_dtype, stride, shift, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    dh = torch.randn(rows, D, generator=gen, device="cuda").to(dtype) if with_dh else None
    if not with_w:
        w = None
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = rms.backward(h, rstd, dy, w, dh)
    r, n = rstd.double()[:, None], h.double() * rstd.double()[:, None]
    t = dy.double() * (1 if w is None else w.double())
    ref = r * (t - n * (t * n).mean(1, keepdim=True)) + (0 if dh is None else dh.double())
    size = r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True)) + (0 if dh is None else dh.double().abs())
    near(dx, ref, 4e-6 * size + UNIT[dtype] * ref.abs() * 1.01)
    if with_w:
        near(dw, (dy.double() * n).sum(0), 1e-5 * (dy.double() * n).abs().sum(0))
        again, dw2 = rms.backward(h, rstd, dy, w, dh)
        assert torch.equal(again, dx) and torch.equal(dw2, dw)   # run to run


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,D", SIZES + [(5000, 256), (2000, 1000)])
def test_backward(rows, D, dtype):
    check_backward(rows, D, dtype)


@pytest.mark.parametrize("with_dh,with_w,w_dtype", [(False, True, BF16), (True, False, F32), (False, False, F32), (True, True, F16)])
def test_backward_without_parts(with_dh, with_w, w_dtype):
    check_backward(40, 512, BF16, w_dtype, with_dh, with_w)


@pytest.mark.parametrize("stride,shift", [(264, 0), (256, 1), (259, 3)])
def test_backward_strides_and_alignment(stride, shift):
    check_backward(6, 256, BF16, stride=stride, shift=shift)


def test_backward_without_rows():
    h = torch.zeros(0, 32, device="cuda")
    dx, dw = rms.backward(h, torch.zeros(0, device="cuda"), h, torch.ones(32, device="cuda"))
    assert dx.shape == (0, 32) and (dw == 0).all()


def test_backward_against_differences():
    """d/dx of sum(gy y + gh h) by central differences of the forward's definition in 64 bits."""
    x, r, w = inputs(3, 200, F32)
    gen = torch.Generator(device="cuda").manual_seed(9)
    gy, gh = (torch.randn(3, 200, generator=gen, device="cuda") for _ in range(2))
    _, h, rstd = rms.forward(x, w, r)
    dx, dw = rms.backward(h, rstd, gy, w, gh)

    def loss(x, w):
        hh, y, _ = plain(x, r, w, 1e-6)
        return float((gy.double() * y).sum() + (gh.double() * hh).sum())

    for i, j in [(0, 0), (1, 17), (2, 199)]:
        step = torch.zeros(3, 200, dtype=torch.float64, device="cuda")
        step[i, j] = 1e-5
        diff = (loss(x.double() + step, w) - loss(x.double() - step, w)) / 2e-5
        assert abs(diff - float(dx[i, j])) <= 2e-5 * (1 + abs(diff))
        diff = (loss(x, w.double() + step[i]) - loss(x, w.double() - step[i])) / 2e-5
        assert abs(diff - float(dw[j])) <= 2e-5 * (1 + abs(diff))


def test_another_stream():
    x, r, w = inputs(64, 2048, BF16)
    y, h, rstd = rms.forward(x, w, r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, h2, rstd2 = rms.forward(x, w, r)
    y3 = rms.forward(x, w, r, stream=side)[0]
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(rstd, rstd2) and torch.equal(y, y3)


def test_rows_beyond_32_bit_offsets():
    D, stride = 64, 1_200_000_000
    big = torch.empty(2 * stride + D, dtype=BF16, device="cuda")
    x = big.as_strided((3, D), (stride, 1))
    dense = torch.randn(3, D, device="cuda").to(BF16)
    x.copy_(dense)
    y, rstd = torch.empty(3, D, device="cuda"), torch.empty(3, device="cuda")
    rms.rms_forward(rms.params_for(x, y_dtype=F32), x, None, None, None, y, None, rstd)
    assert torch.equal(y, rms.forward(dense, y_dtype=F32)[0])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D", [1, 2, 3, 5, 7, 9])
def test_rows_shorter_than_a_pack(D, dtype):
    """A pack may hold several rows, and what follows the last one is not theirs (here NaN)."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    for rows in (1, 2, 3, 9, 40):
        bufs = [torch.full((rows * D + 64,), float("nan"), device="cuda", dtype=dtype) for _ in range(2)]
        x, r = (b[: rows * D].view(rows, D) for b in bufs)
        for t in (x, r):
            t.copy_(1 + torch.rand(rows, D, generator=gen, device="cuda"))
        w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        y, h, rstd = check_forward(x, r, w)
        dx, dw = rms.backward(x, rstd, r, w)
        assert torch.isfinite(dx.float()).all() and torch.isfinite(dw).all()
        for b in bufs:
            assert torch.isnan(b[rows * D:]).all()


def test_each_call_sees_what_the_one_before_it_wrote():
    """Launches overlap the end of the kernel before them; none may read ahead of its writes."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    x, w = torch.randn(600, 2048, generator=gen, device="cuda"), torch.ones(2048, device="cuda")

    def chain(pause):
        h, g, ws = x.clone(), torch.ones_like(x), w.clone()
        for _ in range(6):
            y, h, rstd = rms.forward(h, ws, g, y_dtype=F32)
            pause()
            g, dw = rms.backward(h, rstd, y, ws)
            pause()
            ws.copy_(1 + 0.01 * torch.tanh(dw))
            pause()
        return h, g, ws

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))
