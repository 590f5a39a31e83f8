"""Beam search with a small random model of gated-delta-rule layers: the serving operators together.

A prompt goes through the training forward (gdn.forward) once; its states are forked to the slots of
K beams in every layer (gdn_states_move).  Each step then runs, for all beams of all sequences:

  rms_forward     the residual's addition and the norm before a layer, in 8 bits with one scale a
                  row where the projections take 8 bits
  gdn_decode      one token through the layer's states: read from the slots of the parent beams,
                  written to the other half of the pool, so that no state is copied to reorder beams
  beam_select     the K best continuations, their parents, and the parents' slots: the next slot_in

  python examples/beam_decode.py [--sequences 4] [--beams 4] [--steps 32] [--layers 4] [--plain16]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_delta_rule_backward_gb300 import beam, decode, gdn, rms  # noqa: E402


class Model:
    """Random weights; activations in `dtype`, states and gates in fp32."""

    def __init__(self, layers=4, D=512, H_k=4, H_v=8, S=64, vocab=4000, dtype=torch.bfloat16, eight_bit=True, seed=0):
        gen = torch.Generator().manual_seed(seed)
        w = lambda *shape: (torch.randn(*shape, generator=gen) / shape[0] ** 0.5).to("cuda", dtype)
        self.L, self.D, self.H_k, self.H_v, self.S, self.dtype, self.eight_bit = layers, D, H_k, H_v, S, dtype, eight_bit
        self.embed = torch.randn(vocab, D, generator=gen).to("cuda", dtype)
        self.head = w(D, vocab)
        self.norms = [(1 + 0.1 * torch.randn(D, generator=gen)).cuda() for _ in range(layers + 1)]
        self.w_in = [w(D, (2 * H_k + H_v) * S + 2 * H_v) for _ in range(layers)]
        self.w_out = [w(H_v * S, D) for _ in range(layers)]

    def normed_product(self, i, x, residual, weight):
        """(the sum of x and the residual stream, its norm times weight)."""
        if self.eight_bit:
            codes, scales, h, _ = rms.forward(x, self.norms[i], residual, y_dtype=torch.float8_e4m3fn)
            return h, (codes.to(self.dtype) @ weight).float() * scales[:, None]
        y, h, _ = rms.forward(x, self.norms[i], residual)
        return h, (y @ weight).float()

    def layer_inputs(self, p):
        """q, k (of length 1), v as row views of one buffer, log gates and correction strengths."""
        H_k, H_v, S = self.H_k, self.H_v, self.S
        n, nqk = p.shape[0], 2 * H_k * S
        qkv = torch.empty(n, nqk + H_v * S, device=p.device, dtype=self.dtype)
        qkv[:, :nqk] = torch.nn.functional.normalize(p[:, :nqk].view(n, 2 * H_k, S), dim=-1).view(n, nqk)
        qkv[:, nqk:] = p[:, nqk: nqk + H_v * S]
        g = -torch.nn.functional.softplus(p[:, -2 * H_v: -H_v]).contiguous()
        beta = torch.sigmoid(p[:, -H_v:]).contiguous()
        return qkv[:, : H_k * S].view(n, H_k, S), qkv[:, H_k * S: nqk].view(n, H_k, S), qkv[:, nqk:].view(n, H_v, S), g, beta

    def forward(self, tokens, rule):
        """Logits of each row's next token; rule(layer, q, k, v, g, beta) -> y [rows, H_v, S]."""
        x, h = self.embed[tokens], None
        for i in range(self.L):
            h, p = self.normed_product(i, x, h, self.w_in[i])
            y = rule(i, *self.layer_inputs(p))
            x = y.reshape(len(tokens), self.H_v * self.S).to(self.dtype) @ self.w_out[i]
        return self.normed_product(self.L, x, h, self.head)[1]


def search(model, prompts, beams, steps, end_token=0):
    """prompts: [N, T] tokens.  Returns (scores [N, beams], tokens [N, beams, steps])."""
    N, T = prompts.shape
    L, K, H_v, S = model.L, beams, model.H_v, model.S
    dev = prompts.device
    i32 = lambda x: x.to(torch.int32).contiguous()
    # slots: the beams' states before and after a step, changing places every step, and the prompts' own
    half = N * K
    pool = torch.zeros(L, 2 * half + N, H_v, S, S, device=dev)
    state0 = torch.zeros(N, H_v, S, S, device=dev)

    def prefill(i, q, k, v, g, beta):
        whole = [t.reshape(N, T, *t.shape[1:]).contiguous() for t in (q, k, v, g.to(q.dtype), beta.to(q.dtype))]
        y, state_T, _, _ = gdn.forward(*whole, state0)
        pool[i, 2 * half:] = state_T
        return y.reshape(N * T, H_v, S)

    logits = model.forward(prompts.reshape(-1), prefill).view(N, T, -1)[:, -1]
    # the first choice is made on the prompt's logits: one beam is alive, whose K copies get its states
    scores = torch.full((N, K), float("-inf"), device=dev)
    scores[:, 0] = 0
    scores, _, token = beam.select(logits.repeat_interleave(K, 0), scores)
    decode.gdn_states_move(pool, i32(2 * half + torch.arange(N, device=dev).repeat_interleave(K)), i32(torch.arange(half, device=dev)), group=K)

    src = i32(torch.arange(half, device=dev))
    out, other = src + half, src
    history = [token]
    done = token == end_token
    for _ in range(steps - 1):
        def step(i, q, k, v, g, beta):
            return decode.decode(q, k, v, g, beta, pool[i], src, out, y_dtype=model.dtype)

        logits = model.forward(token.reshape(-1).long(), step)
        scores, parent, token, src = beam.select(logits, scores, done, out.view(N, K), pad_token=end_token)
        src, out, other = src.view(-1), other, out
        parent = parent.long()
        done = done.gather(1, parent) | (token == end_token)
        history = [t.gather(1, parent) for t in history] + [token]
    return scores, torch.stack(history, 2)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--plain16", action="store_true", help="16-bit norms instead of 8-bit codes")
    a = ap.parse_args()
    model = Model(layers=a.layers, eight_bit=not a.plain16)
    prompts = torch.randint(1, 4000, (a.sequences, 50), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    search(model, prompts, a.beams, 4)
    torch.cuda.synchronize()
    began = time.perf_counter()
    scores, tokens = search(model, prompts, a.beams, a.steps)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    print(f"{a.steps} steps of {a.sequences} x {a.beams} beams in {1e3 * (time.perf_counter() - began):.1f} ms")
    for n in range(a.sequences):
        print(n, ["%.3f" % s for s in scores[n].tolist()], tokens[n, 0, :12].tolist())


if __name__ == "__main__":
    main()
