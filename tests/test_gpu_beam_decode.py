"""The serving operators together (examples/beam_decode.py): the search's scores against a plain
model in 64 bits, and a step replayed from a CUDA graph.

Tolerance of the scores: with fp32 activations a step's logits are off by the chunked prefill's error (2e-4 of
the state's magnitude, bounds of gdn_forward) and fp32 rounding; five steps' log-probabilities add
up: 5 x 5e-4."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beam_decode  # noqa: E402
from gated_delta_rule_backward_gb300 import beam, decode, gdn, rms  # noqa: E402


def plain_scores(model, prompt, tokens):
    """log p(tokens | prompt) of a model of fp32 weights, token by token in 64 bits."""
    D = lambda t: t.double()
    H_k, H_v, S = model.H_k, model.H_v, model.S
    M = [torch.zeros(H_v, S, S, dtype=torch.float64, device="cuda") for _ in range(model.L)]
    head = torch.arange(H_v, device="cuda") % H_k
    norm = lambda h, w: h * (h.square().mean() + 1e-6).rsqrt() * D(w)
    total, sequence = 0.0, prompt.tolist() + tokens.tolist()
    for t, tok in enumerate(sequence[:-1]):
        h = D(model.embed[tok])
        for i in range(model.L):
            p = norm(h, model.norms[i]) @ D(model.w_in[i])
            qk = p[: 2 * H_k * S].view(2 * H_k, S)
            qk = qk / qk.square().sum(-1, keepdim=True).sqrt()
            q, k, v = qk[:H_k][head], qk[H_k:][head], p[2 * H_k * S: (2 * H_k + H_v) * S].view(H_v, S)
            a, beta = (-torch.nn.functional.softplus(p[-2 * H_v: -H_v])).exp(), torch.sigmoid(p[-H_v:])
            M[i] = M[i] * a[:, None, None]
            delta = beta[:, None] * (v - torch.einsum("hji,hi->hj", M[i], k))
            M[i] = M[i] + delta[..., None] * k[:, None]
            y = torch.einsum("hji,hi->hj", M[i], q) * S ** -0.5
            h = h + y.reshape(-1) @ D(model.w_out[i])
        if t >= len(prompt) - 1:
            logits = norm(h, model.norms[model.L]) @ D(model.head)
            total += float(torch.log_softmax(logits, 0)[sequence[t + 1]])
    return total


def test_scores_are_the_sequences_probabilities():
    model = beam_decode.Model(layers=2, D=128, H_k=2, H_v=4, S=32, vocab=500, dtype=torch.float32, eight_bit=False, seed=3)
    prompts = torch.randint(1, 500, (2, 33), device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    scores, tokens = beam_decode.search(model, prompts, 3, 5)
    assert gdn.device_status() == 0
    assert (scores[:, :-1] >= scores[:, 1:]).all()
    for n in range(2):
        assert len({tuple(t) for t in tokens[n].tolist()}) == 3
        for b in range(3):
            t = tokens[n, b]
            ends = (t == 0).nonzero()
            t = t[: int(ends[0]) + 1] if len(ends) else t   # what follows the end is not scored
            assert abs(plain_scores(model, prompts[n], t) - float(scores[n, b])) <= 5 * 5e-4


@pytest.mark.parametrize("eight_bit", [False, True])
def test_runs_in_16_and_8_bits(eight_bit):
    model = beam_decode.Model(layers=2, vocab=3001, eight_bit=eight_bit)
    prompts = torch.randint(1, 3001, (3, 20), device="cuda")
    scores, tokens = beam_decode.search(model, prompts, 5, 6)
    assert gdn.device_status() == 0
    assert tokens.shape == (3, 5, 6) and torch.isfinite(scores).all() and ((tokens >= 0) & (tokens < 3001)).all()


def test_a_step_in_a_cuda_graph():
    """Every operator of a step captured and replayed on new values gives what direct calls give."""
    N, K, V, D, H, S = 3, 4, 2000, 256, 4, 64
    gen = torch.Generator("cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    unit = lambda *s: torch.nn.functional.normalize(rnd(*s), dim=-1)
    rows = N * K
    x, res, w = rnd(rows, D), rnd(rows, D), rnd(D)
    q, k, v, g, beta = unit(rows, 2, S), unit(rows, 2, S), rnd(rows, H, S), -rnd(rows, H).abs(), torch.sigmoid(rnd(rows, H))
    pool = rnd(2, 2 * rows, H, S, S)
    logits, scores = rnd(rows, V), rnd(N, K)
    i32 = dict(dtype=torch.int32, device="cuda")
    src, dst = torch.arange(rows, **i32), torch.arange(rows, 2 * rows, **i32)

    def step():
        codes, scales, h, rstd = rms.forward(x, w, res, y_dtype=torch.float8_e4m3fn, group=128)
        y = decode.decode(q, k, v, g, beta, pool[0], src, dst)
        picked = beam.select(logits, scores, slots=dst.view(N, K))
        decode.gdn_states_move(pool, dst, src, group=K)
        dx, dw = rms.backward(h, rstd, x, w, res)
        return (codes.view(torch.uint8), scales, h, rstd, y, *picked, dx, dw)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for t in (x, res, v, logits, scores, pool):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
    before = pool.clone()
    graph.replay()
    graph_pool = pool.clone()
    pool.copy_(before)
    direct = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, direct)) and torch.equal(graph_pool, pool)
