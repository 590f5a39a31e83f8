"""Selections one after the other, each reading what the one before it wrote, with nothing in between: the
kernels of a call start beside the end of those before them and may read none of it ahead."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import beam  # noqa: E402


@pytest.mark.parametrize("N,K,V", [(1, 4, 32000), (16, 8, 5001), (60, 5, 700), (3, 64, 1000)])
def test_each_selection_sees_the_scores_and_slots_of_the_one_before(N, K, V):
    gen = torch.Generator(device="cuda").manual_seed(V)
    steps = 8
    logits = [3 * torch.randn(N * K, V, generator=gen, device="cuda") for _ in range(steps)]
    i32 = dict(dtype=torch.int32, device="cuda")
    start = -torch.rand(N, K, generator=gen, device="cuda")
    first_slots = torch.arange(N * K, **i32).view(N, K)
    p = beam.params_for(logits[0], start)
    ws = beam.workspace(p, "cuda")

    def chain(pause):
        # two sets of buffers that change places, as in a search; every step's results are kept in buffers made before
        scores, slots = [start.clone(), torch.empty_like(start)], [first_slots.clone(), torch.empty_like(first_slots)]
        parent, token = [torch.empty(N, K, **i32) for _ in range(steps)], [torch.empty(N, K, **i32) for _ in range(steps)]
        torch.cuda.synchronize()
        for i, x in enumerate(logits):
            a, b = i % 2, 1 - i % 2
            beam.beam_select(p, x, scores[a], None, slots[a], scores[b], parent[i], token[i], slots[b], ws)
            pause()
        return [*scores, *slots, *parent, *token]

    want = chain(torch.cuda.synchronize)
    assert len({tuple(t.flatten().tolist()) for t in want[4: 4 + steps]}) > 1   # the choices do change
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))
