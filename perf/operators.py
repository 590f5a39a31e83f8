"""The operators of a decoding step with the gated delta rule, as cases to measure.

One decoding step of a model with gated-delta-rule layers runs, in this order: the root-mean-square
norm with the residual's addition (in 8 bits where the projections are 8-bit), the recurrent form of the rule over a
pool of states, the selection over beams and vocabulary, and the moves of states between the
pool's slots that the selection asks for.  Training adds the norm's backward pass.

The plain forms below compute in 32 bits with elementary torch operations and round once.
Every sequence's new tokens go through the rule together: with G the running sum of the log
gates, delta solves (I + A) delta = beta (v - (exp(G) k) M), A strictly lower triangular, and the
inverse of I + A is a finite product because A is nilpotent (up to 16 tokens a call).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
TINY = 2.0 ** -126


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one user's next token through one layer: 16 key heads over 48 value heads of size 128
        dict(name="decode_1", op="decode", N=1, T=1, ragged=False, H_k=16, H_v=48, d=128, kda=False, dtype="bf16"),
        # a serving batch's next tokens
        dict(name="decode_64", op="decode", N=64, T=1, ragged=False, H_k=16, H_v=48, d=128, kda=False, dtype="bf16"),
        # a large batch at the gate per key column, up to 5 drafted tokens a sequence, ragged
        dict(name="decode_200_drafts_kda", op="decode", N=200, T=5, ragged=True, H_k=16, H_v=48, d=128, kda=True, dtype="bf16"),
        # small heads, an odd batch, ragged with empty sequences
        dict(name="decode_121_small_heads", op="decode", N=121, T=16, ragged=True, H_k=4, H_v=4, d=64, kda=False, dtype="f32"),
        # one prompt's beams: four rows of logits
        dict(name="beam_1x4", op="beam", N=1, K=4, V=32000, n_out=4, dtype="f32", first=False),
        # a batch of beams over a large odd vocabulary, twice as many candidates as beams
        dict(name="beam_16x8", op="beam", N=16, K=8, V=128257, n_out=16, dtype="bf16", first=False),
        # the first step after the prompt: only one beam of each sequence is alive
        dict(name="beam_48x5_first", op="beam", N=48, K=5, V=50001, n_out=5, dtype="f16", first=True),
        # four sequences of four beams change places, one layer's states
        dict(name="move_beams", op="move", layers=1, heads=48, d=128, groups=4, group=4, kind="beams"),
        # prompts' states copied to the slots of eight beams each, in every layer of a small model
        dict(name="move_fork", op="move", layers=6, heads=16, d=128, groups=9, group=8, kind="fork"),
        # one token into an 8-bit projection
        dict(name="norm_1_e4m3", op="norm", rows=1, D=2048, dtype="bf16", out="e4m3", group=0, backward=False),
        # a prompt's tokens into an 8-bit projection, one scale for 128 columns
        dict(name="norm_4096_e4m3_groups", op="norm", rows=4096, D=6144, dtype="bf16", out="e4m3", group=128, backward=False),
        # training: the gradients of a norm over 8192 tokens
        dict(name="norm_backward_8192", op="norm", rows=8192, D=2048, dtype="bf16", out="bf16", group=0, backward=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "beam", "move", "norm"])
    if op == "decode":
        d = rng.choice([32, 64, 64, 128, 128])
        H_k, r = rng.choice([(16, 3), (16, 1), (4, 1), (2, 3), (5, 2), (8, 4)])
        cap = min(256, 200 * 48 * 128 * 128 // (H_k * r * d * d))
        N, T = _log(rng, 1, cap), rng.choice([1, 1, 1, 2, 3, 5, 8])
        kda = rng.random() < 0.4
        if kda:
            T = min(T, 5)
        return dict(op=op, N=N, T=T, ragged=T > 1 and rng.random() < 0.6, H_k=H_k, H_v=H_k * r, d=d, kda=kda, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "beam":
        K, V = rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), _log(rng, 1000, 130000)
        N = _log(rng, 1, max(1, min(48, 128 * 128257 // (K * V), 160 // K)))
        return dict(op=op, N=N, K=K, V=V, n_out=rng.choice([K, 2 * K]), dtype=rng.choice(["bf16", "f16", "f32"]), first=rng.random() < 0.2)
    if op == "move":
        d, heads = rng.choice([64, 128]), rng.choice([3, 4, 16, 48])
        group, layers = rng.choice([2, 3, 4, 5, 8, 16]), rng.choice([1, 2, 5])
        cap = 6 * 16 * 128 * 128 * 72 // (layers * heads * d * d * group)
        return dict(op=op, layers=layers, heads=heads, d=d, groups=_log(rng, 1, max(1, min(40, cap))), group=group, kind=rng.choice(["beams", "fork"]))
    backward = rng.random() < 0.4
    D = rng.choice([rng.randrange(64, 1024), 128 * rng.randrange(2, 48), 8 * rng.randrange(100, 700), _log(rng, 256, 8192) | 1])
    out = rng.choice(["e4m3", "e4m3", "same"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    rows = _log(rng, 1, max(1, min(16384, 8192 * 2048 // D)))
    return dict(op=op, rows=rows, D=D, dtype=dtype, out=dtype if backward or out == "same" else out, group=0 if backward or D % 128 else rng.choice([0, 128]), backward=backward)


def _counts(case):
    """Tokens of each sequence: all T, or ragged from 0 to T."""
    N, T = case["N"], case["T"]
    return [(7 * n + 3) % (T + 1) for n in range(N)] if case["ragged"] else [T] * N


def work(case):
    op = case["op"]
    if op == "decode":
        d, H_k, H_v, N = case["d"], case["H_k"], case["H_v"], case["N"]
        tokens, es = sum(_counts(case)), 4 if case["dtype"] == "f32" else 2
        gate = H_v * (d if case["kda"] else 1) + H_v
        return {"bytes": 2 * 4 * N * H_v * d * d + tokens * ((2 * H_k + 2 * H_v) * d * es + 4 * gate), "flops": 7 * d * d * H_v * tokens}
    if op == "beam":
        n, es = case["N"] * case["K"] * case["V"], 4 if case["dtype"] == "f32" else 2
        n = n // case["K"] if case["first"] else n
        return {"bytes": n * es + case["N"] * case["n_out"] * 16, "flops": 4 * n}
    if op == "move":
        slot = 4 * case["layers"] * case["heads"] * case["d"] ** 2
        read, written = _moved(case)
        return {"bytes": slot * (read + written), "flops": 0}
    n, es, eo = case["rows"] * case["D"], 4 if case["dtype"] == "f32" else 2, {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}[case["out"]]
    if case["backward"]:
        return {"bytes": n * 4 * es + 8 * case["D"] + 4 * case["rows"], "flops": 10 * n}
    scales = 0 if case["out"] != "e4m3" else case["rows"] * (case["D"] // case["group"] if case["group"] else 1)
    return {"bytes": n * (3 * es + eo) + 4 * case["D"] + 4 * (scales + case["rows"]), "flops": 6 * n}


# ---- inputs -----------------------------------------------------------------------------------

def _moves(case):
    """(src, dst) slots.  beams: the beams that go on stay where they are, and the others' slots get a copy of
    one of them; fork: a prompt's slot to its beams' slots."""
    src, dst, g = [], [], case["group"]
    for n in range(case["groups"]):
        for j in range(g):
            if case["kind"] == "beams":
                stays = j == n % g or (j * 5 + n) % 3 == 0
                dst.append(n * g + j)
                src.append(n * g + (j if stays else n % g))
            else:
                dst.append(case["groups"] + n * g + j)
                src.append(n)
    return src, dst


def _moved(case):
    pairs = [(s, t) for s, t in zip(*_moves(case)) if s != t]
    return len({s for s, _ in pairs}), len(pairs)


def prepare(case, seed):
    op, dev = case["op"], "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev) * std

    if op == "decode":
        N, H_k, H_v, d = case["N"], case["H_k"], case["H_v"], case["d"]
        counts = _counts(case)
        tokens, dt = sum(counts), DTYPES[case["dtype"]]
        qk = normal(tokens, 2 * H_k, d)
        qk = qk / qk.square().sum(-1, keepdim=True).sqrt()
        qkv = torch.cat([qk.reshape(tokens, 2 * H_k * d), normal(tokens, H_v * d)], 1).to(dt)  # a fused projection's rows
        g = -torch.nn.functional.softplus(normal(tokens, H_v, d) if case["kda"] else normal(tokens, H_v))
        beta = torch.sigmoid(normal(tokens, H_v))
        pool = torch.empty(2 * N, H_v, d, d, device=dev)  # the beams' states before and after the step
        pool[:N].normal_(0.0, 0.1, generator=gen)
        pool[N:].zero_()
        order = torch.randperm(N, generator=gen, device=dev).to(torch.int32)
        # the token rows of every sequence, padded, for the plain form
        cu = torch.tensor([0] + counts, device=dev).cumsum(0)
        pad = torch.arange(case["T"], device=dev)
        return dict(case=case, q=qkv[:, : H_k * d].view(tokens, H_k, d), k=qkv[:, H_k * d: 2 * H_k * d].view(tokens, H_k, d),
                    v=qkv[:, 2 * H_k * d:].view(tokens, H_v, d), g=g, beta=beta, pool=pool, slot_in=order,
                    slot_out=torch.arange(N, 2 * N, device=dev, dtype=torch.int32), cu=cu.to(torch.int32) if case["ragged"] else None,
                    rows=(cu[:-1, None] + pad).clamp(max=max(tokens - 1, 0)), real=pad < (cu[1:] - cu[:-1])[:, None],
                    y=torch.empty(tokens, H_v, d, device=dev, dtype=dt))
    if op == "beam":
        N, K, V = case["N"], case["K"], case["V"]
        logits = normal(N * K, V, std=3.0)
        logits.view(-1)[7::97] = -math.inf  # tokens that a mask forbids
        scores = -normal(N, K).abs() * 4
        done = torch.zeros(N, K, dtype=torch.uint8, device=dev)
        if case["first"]:
            scores[:, 1:] = -math.inf
        elif K > 2:
            done[1::3, 2] = 1
        n = case["n_out"]
        i32 = dict(dtype=torch.int32, device=dev)
        return dict(case=case, logits=logits.to(DTYPES[case["dtype"]]), scores=scores, done=done, pad=2, slots=torch.randperm(N * K, generator=gen, device=dev).to(torch.int32).view(N, K),
                    scores_out=torch.empty(N, n, device=dev), parent=torch.empty(N, n, **i32), token=torch.empty(N, n, **i32), src_slots=torch.empty(N, n, **i32))
    if op == "move":
        src, dst = _moves(case)
        slots = case["groups"] * (case["group"] + (1 if case["kind"] == "fork" else 0))
        pool = torch.empty(case["layers"], slots, case["heads"], case["d"], case["d"], device=dev).normal_(0.0, 0.1, generator=gen)
        return dict(case=case, pool=pool, src=torch.tensor(src, device=dev, dtype=torch.int32), dst=torch.tensor(dst, device=dev, dtype=torch.int32))
    rows, D, dt = case["rows"], case["D"], DTYPES[case["dtype"]]
    weight = 1.0 + normal(D, std=0.1)
    s = dict(case=case, eps=1e-6, weight=weight, x=normal(rows, D).to(dt), residual=normal(rows, D, std=2.0).to(dt))
    if case["backward"]:
        h = s.pop("x").float() + s.pop("residual").float()
        s |= dict(h=h.to(dt), rstd=torch.rsqrt(h.square().mean(1) + s["eps"]), dy=normal(rows, D).to(dt), dh=normal(rows, D).to(dt),
                  dx=torch.empty(rows, D, device=dev, dtype=dt), dweight=torch.empty(D, device=dev))
        return s
    scales = (rows, D // case["group"]) if case["group"] else (rows,)
    return s | dict(h=torch.empty(rows, D, device=dev, dtype=dt), y=torch.empty(rows, D, device=dev, dtype=DTYPES[case["out"]]),
                    scales=torch.empty(scales, device=dev) if case["out"] == "e4m3" else None, rstd=torch.empty(rows, device=dev))


# ---- the plain forms --------------------------------------------------------------------------

def _decode_plain(s):
    case, dt = s["case"], s["y"].dtype
    N, T, H_v, d, r = case["N"], case["T"], case["H_v"], case["d"], case["H_v"] // case["H_k"]
    real = s["real"][:, :, None]

    def padded(x):  # [N, H, T, d]: each sequence's tokens, the key heads repeated over their value heads
        return x[s["rows"]].float()

    q, k, v = (padded(s[n]) for n in "qkv")
    q, k, v = q.repeat(1, 1, r, 1).transpose(1, 2), k.repeat(1, 1, r, 1).transpose(1, 2), v.transpose(1, 2)
    beta = (padded(s["beta"]) * real).transpose(1, 2)[..., None]                 # padding tokens change nothing
    g = padded(s["g"])
    g = (g * real[..., None] if case["kda"] else (g * real)[..., None]).transpose(1, 2)  # [N, H, T, d or 1]
    M = s["pool"][s["slot_in"].long()]                                           # [N, H, rows (v), columns (k)]
    G = g.cumsum(2)
    decay = G.exp()
    u = (k * decay) @ M.transpose(2, 3)
    o = (q * decay) @ M.transpose(2, 3)
    if T == 1:
        delta = beta * (v - u)
        o = o + (q * k).sum(-1, keepdim=True) * delta
        tail = k
    else:
        lower = torch.ones(T, T, device=q.device).tril()
        between = (G[:, :, :, None] - G[:, :, None]).clamp(max=0.0).exp()        # [N, H, T, T, d or 1]
        if case["kda"]:
            kk = (k[:, :, :, None] * k[:, :, None] * between).sum(-1)
            qk = (q[:, :, :, None] * k[:, :, None] * between).sum(-1)
        else:
            kk, qk = (k @ k.transpose(2, 3)) * between[..., 0], (q @ k.transpose(2, 3)) * between[..., 0]
        one, X = torch.eye(T, device=q.device), -beta * kk * lower.tril(-1)
        X2 = X @ X
        X4 = X2 @ X2
        inverse = (one + X) @ (one + X2) @ (one + X4) @ (one + X4 @ X4)
        delta = inverse @ (beta * (v - u))
        o = o + (qk * lower) @ delta
        tail = k * (G[:, :, -1:] - G).exp()
    y = (o / math.sqrt(d)).transpose(1, 2)[s["real"]]
    s["pool"][s["slot_out"].long()] = M * decay[:, :, -1:] + delta.transpose(2, 3) @ tail
    return y.to(dt)


def _beam_plain(s):
    case = s["case"]
    N, K, V, n = case["N"], case["K"], case["V"], case["n_out"]
    x = s["logits"].float().view(N, K, V)
    top = x.amax(-1, keepdim=True)
    logp = (x - top) - (x - top).exp().sum(-1, keepdim=True).log()
    ended = torch.where(torch.arange(V, device=x.device) == s["pad"], 0.0, -math.inf)
    score = s["scores"][..., None] + torch.where(s["done"][..., None] != 0, ended, logp)
    # one whole number a candidate, ordered by score and then by the lowest index: bits of a float
    # order as whole numbers once the negative ones' are turned round
    bits = score.view(N, K * V).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = (order << 32) + (0x7FFFFFFF - torch.arange(K * V, device=x.device))
    at = 0x7FFFFFFF - (key.topk(n, 1).values & 0xFFFFFFFF)
    parent = at // V
    return (score.view(N, K * V).gather(1, at), parent.to(torch.int32), (at % V).to(torch.int32), s["slots"].gather(1, parent))


def _move_plain(s):
    s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return s["pool"]


def _norm_plain(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    D = case["D"]
    if case["backward"]:
        h, wdy, rstd = s["h"].float(), s["dy"].float() * s["weight"], s["rstd"][:, None]
        mean = (wdy * h).sum(1, keepdim=True) / D
        dx = rstd * (wdy - h * (rstd * rstd * mean)) + s["dh"].float()
        return dx.to(dt), (s["dy"].float() * h * rstd).sum(0)
    h = s["x"].float() + s["residual"].float()
    rstd = 1.0 / ((h * h).sum(1, keepdim=True) / D + s["eps"]).sqrt()
    y = h * rstd * s["weight"]
    if case["out"] != "e4m3":
        return h.to(dt), y.to(dt), rstd[:, 0]
    y = y.view(case["rows"], -1, case["group"] or D)
    scales = (y.abs().amax(-1, keepdim=True) / E4M3_MAX).clamp(min=TINY)
    codes = (y / scales).to(torch.float8_e4m3fn).view(case["rows"], D)
    return h.to(dt), codes, scales.view(s["scales"].shape), rstd[:, 0]


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "decode":
            return _decode_plain(s), s["pool"][case["N"]:]
        return {"beam": _beam_plain, "move": _move_plain, "norm": _norm_plain}[op](s)
    if op == "decode":
        from gated_delta_rule_backward_gb300 import decode
        if "p" not in s:
            s["p"] = decode.params_for(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], n_seq=case["N"], y_dtype=s["y"].dtype)
        decode.gdn_decode(s["p"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], s["pool"], s["slot_in"], s["slot_out"], s["y"])
        return s["y"], s["pool"][case["N"]:]
    if op == "beam":
        from gated_delta_rule_backward_gb300 import beam
        if "p" not in s:
            s["p"] = beam.params_for(s["logits"], s["scores"], n_out=case["n_out"], pad_token=s["pad"])
            s["ws"] = beam.workspace(s["p"], s["logits"].device)
        beam.beam_select(s["p"], s["logits"], s["scores"], s["done"], s["slots"], s["scores_out"], s["parent"], s["token"], s["src_slots"], s["ws"])
        return s["scores_out"], s["parent"], s["token"], s["src_slots"]
    if op == "move":
        from gated_delta_rule_backward_gb300 import decode
        decode.gdn_states_move(s["pool"], s["src"], s["dst"], group=case["group"])
        return s["pool"]
    from gated_delta_rule_backward_gb300 import rms
    if case["backward"]:
        if "p" not in s:
            s["p"] = rms.params_for(s["h"], s["weight"], eps=s["eps"])
            s["ws"] = rms.workspace(s["p"], s["h"].device)
        rms.rms_backward(s["p"], s["h"], s["weight"], s["rstd"], s["dy"], s["dh"], s["dx"], s["dweight"], s["ws"])
        return s["dx"], s["dweight"]
    if "p" not in s:
        s["p"] = rms.params_for(s["x"], s["weight"], eps=s["eps"], y_dtype=s["y"].dtype, group=case["group"])
    rms.rms_forward(s["p"], s["x"], s["residual"], s["weight"], s["h"], s["y"], s["scales"], s["rstd"])
    return (s["h"], s["y"], s["rstd"]) if s["scales"] is None else (s["h"], s["y"], s["scales"], s["rstd"])


# ---- the definitions in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "decode":
        N, H_k, H_v, d = case["N"], case["H_k"], case["H_v"], case["d"]
        counts = _counts(case)
        first = [sum(counts[:n]) for n in range(N)]
        head = torch.arange(H_v, device="cuda") % H_k
        out = torch.empty(sum(counts), H_v, d, dtype=torch.float64, device="cuda")
        after = torch.empty(N, H_v, d, d, dtype=torch.float64, device="cuda")
        slots = s["slot_in"].tolist()
        for lo in range(0, N, 32):  # some sequences at a time, token by token
            some = range(lo, min(N, lo + 32))
            M = s["pool"][[slots[n] for n in some]].double()
            for t in range(case["T"]):
                live = [i for i, n in enumerate(some) if t < counts[n]]
                if not live:
                    continue
                row = [first[some[i]] + t for i in live]
                q, k, v = s["q"][row][:, head].double(), s["k"][row][:, head].double(), s["v"][row].double()
                a, b = s["g"][row].double().exp(), s["beta"][row].double()
                S = M[live] * (a[:, :, None, :] if case["kda"] else a[:, :, None, None])
                delta = b[:, :, None] * (v - torch.einsum("nhji,nhi->nhj", S, k))
                S = S + delta[..., None] * k[:, :, None, :]
                M[live] = S
                out[row] = torch.einsum("nhji,nhi->nhj", S, q) / math.sqrt(d)
            after[lo: lo + len(some)] = M
        return out, after
    if op == "beam":
        N, K, V, n = case["N"], case["K"], case["V"], case["n_out"]
        got = []
        for i in range(N):
            rows = s["logits"][i * K: (i + 1) * K].double()
            c = s["scores"][i].double()[:, None] + (rows - torch.logsumexp(rows, 1, keepdim=True))
            for j in range(K):
                if s["done"][i, j]:
                    c[j] = -math.inf
                    c[j, s["pad"]] = s["scores"][i, j].double()
            best, at = c.reshape(-1).sort(descending=True, stable=True)
            got.append((best[:n], at[:n]))
        at = torch.stack([b for _, b in got])
        parent = at // V
        return torch.stack([a for a, _ in got]), parent, at % V, s["slots"].gather(1, parent)
    if op == "move":
        old = s["pool"].clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            s["pool"][:, b] = old[:, a]
        return s["pool"].double()
    D = case["D"]
    if case["backward"]:
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        n = h * r                                              # the normalised rows
        t = dy * s["weight"].double()
        return s["dh"].double() + r * (t - n * (t * n).mean(1, keepdim=True)), (dy * n).sum(0)
    h = s["x"].double() + s["residual"].double()
    r = (h.pow(2).mean(1) + s["eps"]).rsqrt()
    y = h * r[:, None] * s["weight"].double()
    if case["out"] != "e4m3":
        return h, y, r
    wide = y.reshape(case["rows"], -1, case["group"] or D)
    scales = (wide.abs().max(-1).values / E4M3_MAX).clamp(min=TINY)
    return h, (wide / scales[..., None]).reshape(case["rows"], D), scales.reshape(s["scales"].shape), r
