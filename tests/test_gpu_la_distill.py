"""Linear attention and distillation together, as a student that learns and then answers uses them (la_student.py).

Tolerance, relative to a tensor's norm.  fp32: an operator is off by some (4 T + 48) 2^-24 of the magnitudes it sums, T = 40: 1.3e-5, and these
are up to ten times their signed sum: 1.3e-4; two layers forward and backward pass it four times, the products and norms less:
1e-3.  bf16: every tensor that is stored is rounded by up to 2^-8 of itself, 8 a layer in each direction: 2 x 2 x 8 x 2^-8 = 0.125."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import la_student as LS  # noqa: E402
from gated_delta_rule_backward_gb300 import gdn, la  # noqa: E402


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


CASES = [(torch.float32, [17, 0, 40, 3], 1e-3), (torch.bfloat16, [140, 0, 33, 1], 0.125)]


def student(dtype):
    return LS.Student(S=32 if dtype == torch.float32 else 64, dtype=dtype)


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("dtype,counts,tol", CASES)
def test_gradients_of_a_lesson(dtype, counts, tol):
    m = student(dtype)
    tokens, indices, teacher, cu = LS.lesson(counts)
    loss, grads = m.learn(tokens, indices, teacher, 2.0, m.states(1), i32([-1] * len(counts)), cu, max(counts))
    assert gdn.device_status() == 0
    params = {k: v.double().requires_grad_() for k, v in m.p.items()}
    want = LS.plain_loss(LS.plain(m, params, tokens, counts), indices, teacher, 2.0)
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= tol * float(want.detach())
    for name, w in params.items():
        assert off(grads[name], w.grad) <= tol, (name, off(grads[name], w.grad))
    # and against differences along one direction through all parameters (h^2 of the third derivative: far below tol)
    gen = torch.Generator(device="cuda").manual_seed(3)
    way = {k: torch.randn(v.shape, generator=gen, device="cuda", dtype=torch.float64) for k, v in params.items()}
    h, val = 1e-5, []
    with torch.no_grad():
        for s in (h, -h):
            val.append(float(LS.plain_loss(LS.plain(m, {k: v + s * way[k] for k, v in params.items()}, tokens, counts), indices, teacher, 2.0)))
    along = sum(float((grads[k].double() * way[k]).sum()) for k in way)
    size = sum(float(params[k].grad.square().sum()) for k in way) ** 0.5   # of the sum over a random direction, one sigma
    assert abs((val[0] - val[1]) / (2 * h) - along) <= 4 * tol * size


@pytest.mark.parametrize("dtype,counts,tol", CASES)
def test_answers_token_by_token(dtype, counts, tol):
    """A prompt at once and then single tokens, over the layers' pools, against one pass over all of them in 64 bits; the tokens' step
    captured once."""
    m = student(dtype)
    T, N, more = max(counts), 3, 5
    tokens = LS.lesson([T + more] * N)[0].view(N, T + more)
    want = LS.plain(m, {k: v.double() for k, v in m.p.items()}, tokens.flatten(), [T + more] * N).view(N, T + more, -1)
    pools, slots = m.states(N + 2), i32([3, 0, 2])
    logits, _ = m.forward(tokens[:, :T].flatten(), pools, slots)
    got = [logits.view(N, T, -1)]
    now = tokens[:, T].clone()
    keep = [p.clone() for p in pools]
    m.forward(now, pools, slots)                     # a first call outside the graph
    for p, k in zip(pools, keep):
        p.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = m.forward(now, pools, slots)[0]
    for t in range(T, T + more):
        now.copy_(tokens[:, t])
        graph.replay()
        got.append(step.clone().view(N, 1, -1))
    got = torch.cat(got, 1)
    assert off(got, want) <= tol and off(got[:, T:], want[:, T:]) <= tol and gdn.device_status() == 0
    assert all((p[[1, 4]] == 0).all() for p in pools)


def test_a_captured_lesson_and_a_second_graph_with_its_own_workspaces():
    """A step that updates the weights, captured twice (graphs that share no memory but the weights) and replayed in turn, gives what the same
    steps give outside."""
    counts = [140, 33]
    tokens, indices, teacher, cu = LS.lesson(counts)

    def step(m, pools, slots):
        loss, grads = m.learn(tokens, indices, teacher, 2.0, pools, slots, cu, 140)
        for k, w in m.p.items():
            if k != "embed":                          # index_add_'s order is not fixed
                w.sub_((0.1 * grads[k]).to(w.dtype))
        return loss

    results = []
    for captured in (False, True):
        m = student(torch.bfloat16)
        pools, slots = m.states(1), i32([-1, -1])
        if captured:
            before = {k: v.clone() for k, v in m.p.items()}
            step(m, pools, slots)
            graphs = []
            for _ in range(2):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    loss = step(m, pools, slots)
                graphs.append((graph, loss))
            for k, v in m.p.items():
                v.copy_(before[k])
            losses = []
            for turn in range(4):
                graphs[turn % 2][0].replay()
                losses.append(graphs[turn % 2][1].clone())
        else:
            losses = [step(m, pools, slots) for _ in range(4)]
        results.append((torch.stack(losses), *m.p.values()))
    assert all(torch.equal(a, b) for a, b in zip(*results)) and gdn.device_status() == 0


def test_two_threads_learn_and_answer():
    """Lessons and prompts at once, each on a stream of its own: each gives what it gives alone."""
    import threading
    m = student(torch.bfloat16)
    tokens, indices, teacher, cu = LS.lesson([140, 33])

    def lesson():
        loss, grads = m.learn(tokens, indices, teacher, 2.0, m.states(1), i32([-1, -1]), cu, 140)
        return [loss] + [g for k, g in grads.items() if k != "embed"]

    def prompt():
        pools = m.states(2)
        out = m.forward(tokens, pools, i32([0, 1]), None, cu, 140)[0]
        return [out, *pools]

    works, alone, errors = (lesson, prompt, lesson), [], []
    alone = [w() for w in works]
    torch.cuda.synchronize()
    start = threading.Barrier(len(works))

    def body(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(20):
                    got = works[k]()
                    torch.cuda.current_stream().synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, alone[k]))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=body, args=(k,)) for k in range(len(works))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and gdn.device_status() == 0


def test_the_forms_these_cases_take():
    for dtype, form in ((torch.float32, "token"), (torch.bfloat16, "chunked")):
        m = student(dtype)
        x = torch.zeros(140, (2 * m.H_k + m.H_v) * m.S + m.H_v, device="cuda", dtype=dtype)
        q, k, v, f = m.split(x)
        assert la.form(la.params_for(q, k, v, f.float(), m.states(1)[0], 1)) == form
