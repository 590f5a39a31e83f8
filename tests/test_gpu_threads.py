"""Calls from several host threads, each on a stream of its own, at sizes that ask one kernel for different amounts of shared
memory: no call may fail, and each gives what it gives alone."""
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gated_delta_rule_backward_gb300 import decode, rms  # noqa: E402


def run_threads(works, times):
    """Every work `times` times, all at once; the errors that they met."""
    errors, start = [], threading.Barrier(len(works))

    def body(work):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(times):
                    work()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=body, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def test_norm_gradients_of_different_lengths():
    works, results = [], []
    for rows, D in ((304, 768), (304, 8192), (304, 1536), (304, 4096)):   # one kernel with 48, 192, 72 and 192 KB
        gen = torch.Generator(device="cuda").manual_seed(D)
        h, dy, w = (torch.randn(*s, generator=gen, device="cuda") for s in ((rows, D), (rows, D), (D,)))
        h, dy, rstd = h.bfloat16(), dy.bfloat16(), torch.ones(rows, device="cuda")
        p = rms.params_for(h, w, residual=dy)
        outs = [(torch.empty_like(h), torch.empty_like(w)) for _ in range(2)]
        ws = rms.workspace(p, "cuda")
        call = lambda out, p=p, h=h, w=w, rstd=rstd, dy=dy, ws=ws: rms.rms_backward(p, h, w, rstd, dy, None, *out, ws)
        call(outs[0])
        works.append(lambda call=call, out=outs[1]: call(out))
        results.append(outs)
    assert run_threads(works, 2000) == []
    for alone, among in results:
        assert all(torch.equal(a, b) for a, b in zip(alone, among))


def test_moves_of_different_groups():
    works, results = [], []
    for group in (400, 1024, 513, 800):
        src = torch.randperm(group, generator=torch.Generator().manual_seed(group)).to(torch.int32).cuda()
        dst = torch.arange(group, dtype=torch.int32, device="cuda")
        before = torch.randn(1, group, 64, device="cuda")
        alone, among = before.clone(), before.clone()
        decode.gdn_states_move(alone, src, dst, group=group)
        works.append(lambda pool=among, a=before, src=src, dst=dst, group=group: (pool.copy_(a), decode.gdn_states_move(pool, src, dst, group=group)))
        results.append((alone, among))
    assert run_threads(works, 1500) == []
    assert all(torch.equal(a, b) for a, b in results)
