"""Linear attention with a decay for each head, and distillation from a teacher's top logits, as cases to measure.

Linear attention is the gated delta rule without the correction: M <- a M + v k', y = scale M q.  Its layers
stand between gated-delta-rule layers, share their pools of states, and are usually taught by a larger model: the
loss is the divergence from the teacher's distribution over its best tokens, with a gradient over the whole vocabulary.

The plain forms below compute in 32 bits with elementary torch operations and round once.  Every product
of linear attention and of its gradient is one core, forwards or backwards in time, with G the running sum of
the log decays:   out_t = sum_{s<=t} e^(G_t - G_s) (x_t . y_s) z_s + e^(G_t) S x_t
    y: (x, y, z) = (q, k, v);   dq: (dy, v, k);   dk: (v, dy, q) backwards;   dv: (k, q, dy) backwards.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one user's next token through one layer: 16 key heads over 48 value heads of size 128
        dict(name="la_token_1", op="la", N=1, T=1, ragged=False, H_k=16, H_v=48, d=128, dtype="bf16", constant=False, backward=False),
        # a serving batch's next tokens
        dict(name="la_tokens_64", op="la", N=64, T=1, ragged=False, H_k=16, H_v=48, d=128, dtype="bf16", constant=False, backward=False),
        # drafted tokens on small heads in 32 bits, ragged with empty sequences
        dict(name="la_drafts_121", op="la", N=121, T=16, ragged=True, H_k=4, H_v=4, d=64, dtype="f32", constant=False, backward=False),
        # one prompt
        dict(name="la_prompt_4096", op="la", N=1, T=4096, ragged=False, H_k=16, H_v=48, d=128, dtype="bf16", constant=False, backward=False),
        # a batch of prompts of odd lengths, decays that are the same for every token
        dict(name="la_prompts_23", op="la", N=23, T=701, ragged=True, H_k=16, H_v=16, d=128, dtype="bf16", constant=True, backward=False),
        # a long document
        dict(name="la_prompt_32768", op="la", N=1, T=32768, ragged=False, H_k=16, H_v=16, d=128, dtype="bf16", constant=False, backward=False),
        # training: the gradients of one sequence
        dict(name="la_gradients_4096", op="la", N=1, T=4096, ragged=False, H_k=16, H_v=48, d=128, dtype="bf16", constant=False, backward=True),
        # training on packed sequences of small heads
        dict(name="la_gradients_packed", op="la", N=9, T=500, ragged=True, H_k=8, H_v=8, d=64, dtype="bf16", constant=False, backward=True),
        # a training batch's loss with its gradients: 8192 tokens, the teacher's 64 best of 32000
        dict(name="distill_8192", op="distill", N=8192, V=32000, K=64, dtype="bf16", mode="both"),
        # the loss of a few tokens over a large odd vocabulary
        dict(name="distill_loss_5", op="distill", N=5, V=128257, K=100, dtype="f32", mode="loss"),
        # the batch's gradients behind a loss that other terms are added to
        dict(name="distill_gradients_8192", op="distill", N=8192, V=32000, K=64, dtype="bf16", mode="gradients"),
        # the gradients over an odd vocabulary, short lists
        dict(name="distill_gradients_300", op="distill", N=300, V=50001, K=20, dtype="f16", mode="gradients"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        H_k, r = rng.choice([(16, 3), (16, 1), (4, 1), (2, 3), (5, 2), (8, 4)])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
        d = rng.choice([64, 128, 128]) if dtype == "bf16" else rng.choice([32, 64, 128])
        backward = rng.random() < 0.35
        T = rng.choice([1, _log(rng, 2, 64), _log(rng, 64, 12000)])
        if backward:
            T = max(2, min(T, 4096))
        if dtype != "bf16":
            T = min(T, 200)
        tokens = (4096 * 48 if backward else 32768 * 16) * 128 // (H_k * r * d)  # with the states of as many sequences
        N = _log(rng, 1, max(1, min(64, tokens // (T + 256))))
        return dict(op="la", N=N, T=T, ragged=N > 1 and rng.random() < 0.6, H_k=H_k, H_v=H_k * r, d=d, dtype=dtype, constant=rng.random() < 0.25, backward=backward)
    V, K, dtype = _log(rng, 1000, 130000), _log(rng, 4, 256), rng.choice(["bf16", "bf16", "f16", "f32"])
    most = min(8192, 8192 * 32000 // (V * (2 if dtype == "f32" else 1)))
    return dict(op="distill", N=_log(rng, 1, most), V=V, K=K, dtype=dtype, mode=rng.choice(["loss", "gradients", "both"]))


def _counts(case):
    """Tokens of each sequence: all T, or ragged from 0 to T."""
    N, T = case["N"], case["T"]
    return [(n * 389 + T) % (T + 1) for n in range(N)] if case["ragged"] else [T] * N


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "la":
        N, H_k, H_v, d, tokens = case["N"], case["H_k"], case["H_v"], case["d"], sum(_counts(case))
        states = 4 * N * H_v * d * d
        if case["backward"]:
            return {"bytes": tokens * ((4 * H_k + 3 * H_v) * d * es + 8 * H_v) + 3 * states, "flops": 12 * d * d * H_v * tokens}
        return {"bytes": tokens * ((2 * H_k + 2 * H_v) * d * es + 4 * H_v) + 2 * states, "flops": 4 * d * d * H_v * tokens}
    N, V, K = case["N"], case["V"], case["K"]
    both = case["mode"] == "both"
    return {"bytes": (1 if case["mode"] == "loss" else 2) * N * V * es + (12 if both else 8) * N + 8 * N * K, "flops": (8 if both else 4) * N * V}


# ---- inputs -----------------------------------------------------------------------------------

def prepare(case, seed):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev) * std

    if case["op"] == "la":
        N, H_k, H_v, d, T = case["N"], case["H_k"], case["H_v"], case["d"], case["T"]
        counts = _counts(case)
        tokens = sum(counts)
        qkv = normal(tokens, (2 * H_k + H_v) * d).to(dt)  # a fused projection's rows
        if case["constant"]:  # from half a token's memory to that of thousands, by head
            g = torch.log1p(-torch.exp2(-1 - 11 * torch.rand(H_v, generator=gen, device=dev))).expand(tokens, H_v)
        else:
            g = -torch.exp(normal(tokens, H_v, std=1.5) - 3)
        pool = torch.empty(2 * N, H_v, d, d, device=dev)
        pool[:N].normal_(0.0, 1.0, generator=gen)
        pool[N:].zero_()
        cu = torch.tensor([0] + counts, device=dev).cumsum(0)
        pad = torch.arange(T, device=dev)
        s = dict(case=case, q=qkv[:, : H_k * d].view(tokens, H_k, d), k=qkv[:, H_k * d: 2 * H_k * d].view(tokens, H_k, d),
                 v=qkv[:, 2 * H_k * d:].view(tokens, H_v, d), g=g, pool=pool, slot_in=torch.randperm(N, generator=gen, device=dev).to(torch.int32),
                 slot_out=torch.arange(N, 2 * N, device=dev, dtype=torch.int32), cu=cu.to(torch.int32) if case["ragged"] else None,
                 # the token rows of every sequence, padded, for the plain form
                 rows=(cu[:-1, None] + pad).clamp(max=max(tokens - 1, 0)), real=pad < (cu[1:] - cu[:-1])[:, None])
        if not case["backward"]:
            return s | dict(y=torch.empty(tokens, H_v, d, device=dev, dtype=dt))
        like = lambda H: torch.empty(tokens, H, d, device=dev, dtype=dt)
        return s | dict(dy=normal(tokens, H_v, d).to(dt), dstate=normal(N, H_v, d, d), dq=like(H_k), dk=like(H_k), dv=like(H_v),
                        dg=torch.empty(tokens, H_v, device=dev), dstate0=torch.empty(N, H_v, d, d, device=dev))
    N, V, K = case["N"], case["V"], case["K"]
    logits = normal(N, V, std=2.0)
    teacher, indices = torch.empty(N, K, device=dev), torch.empty(N, K, dtype=torch.int64, device=dev)
    for lo in range(0, N, 1024):  # a teacher that partly agrees
        rows = logits[lo: lo + 1024]
        teacher[lo: lo + 1024], indices[lo: lo + 1024] = (0.7 * rows + normal(*rows.shape, std=2.0)).topk(K, 1)
    indices[1::5, K - K // 4:] = -1  # shorter lists
    indices[3::17] = -1              # padding: tokens without a teacher
    s = dict(case=case, logits=logits.to(dt), indices=indices.to(torch.int32), teacher=teacher, temperature=1.5,
             loss=torch.empty(N, device=dev), lse=torch.empty(N, device=dev))
    if case["mode"] == "gradients":
        x = (s["logits"].float() / s["temperature"]).double()
        s["lse"] = torch.cat([torch.logsumexp(r, 1) for r in x.split(1024)]).float()
        s["lse"][(s["indices"] < 0).all(1)] = 0.0
    if case["mode"] != "loss":
        s["dloss"] = torch.rand(N, generator=gen, device=dev) + 0.5
        s["dlogits"] = torch.empty(N, V, device=dev, dtype=dt)
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _core(x, y, z, g, S):
    """x, y [N, H, T, a], z [N, H, T, b], g [N, H, T], S [N, H, b, a].  Returns (out [N, H, T, b], S after)."""
    T, C = x.shape[2], 64
    lower = torch.ones(min(T, C), min(T, C), device=x.device).tril()
    out = torch.empty_like(z)
    for lo in range(0, T, C):
        at = slice(lo, min(lo + C, T))
        G = g[:, :, at].cumsum(2)
        xc, yc, zc, n = x[:, :, at], y[:, :, at], z[:, :, at], G.shape[2]
        weights = (xc @ yc.transpose(2, 3)) * (G[..., :, None] - G[..., None, :]).clamp(max=0.0).exp() * lower[:n, :n]
        out[:, :, at] = weights @ zc + G.exp()[..., None] * (xc @ S.transpose(2, 3))
        last = G[:, :, -1:]
        S = last.exp()[..., None] * S + ((last - G).exp()[..., None] * zc).transpose(2, 3) @ yc
    return out, S


def _la_plain(s):
    case = s["case"]
    H_k, d, r = case["H_k"], case["d"], case["H_v"] // case["H_k"]
    real, scale, dt = s["real"][:, :, None], 1.0 / math.sqrt(case["d"]), DTYPES[case["dtype"]]

    def padded(t):  # [N, H, T, ...]: each sequence's tokens, zeros after its last
        t = t[s["rows"]].float() * (real[..., None] if t.dim() == 3 else real)
        return t.transpose(1, 2)

    def rows_of(t):  # back to token rows
        return t.transpose(1, 2)[s["real"]]

    q, k, v, g = padded(s["q"]).repeat(1, r, 1, 1), padded(s["k"]).repeat(1, r, 1, 1), padded(s["v"]), padded(s["g"])
    M = s["pool"][s["slot_in"].long()]
    if not case["backward"]:
        y, after = _core(q, k, v, g, M)
        s["pool"][s["slot_out"].long()] = after
        return rows_of(scale * y).to(dt)
    dy = padded(s["dy"]) * scale
    dq, after = _core(dy, v, k, g, M.transpose(2, 3))
    # backwards in time: a token's gradient decays by the gate of the token behind it
    turn = lambda t: t.flip(2)
    behind = turn(torch.cat([g[:, :, 1:], torch.zeros_like(g[:, :, :1])], 2))
    D = s["dstate"]
    dk, _ = _core(turn(v), turn(dy), turn(q), behind, D.transpose(2, 3))
    dv, D = _core(turn(k), turn(q), turn(dy), behind, D)
    dk, dv = turn(dk), turn(dv)
    terms = ((q * dq).sum(-1) - (k * dk).sum(-1)).double()
    dg = (after.transpose(2, 3) * s["dstate"]).double().sum((2, 3))[..., None] + turn(turn(terms).cumsum(2))
    shared = lambda t: rows_of(t.unflatten(1, (r, H_k)).sum(1)).to(dt)
    return shared(dq), shared(dk), rows_of(dv).to(dt), rows_of(dg).float(), D * g[:, :, :1].exp()[..., None]


def _distill_plain(s):
    mode = s["case"]["mode"]
    x = s["logits"].float() / s["temperature"]
    listed_ = s["indices"] >= 0
    some = listed_.any(1)
    t = torch.where(listed_, s["teacher"] / s["temperature"], -math.inf)
    t = torch.where(some[:, None], t, 0.0)
    e = (t - t.amax(1, keepdim=True)).exp() * listed_
    total = e.sum(1, keepdim=True).clamp(min=1e-30)
    p, logp = e / total, (t - t.amax(1, keepdim=True)) - total.log()
    at = s["indices"].clamp(min=0).long()
    out, lse = (), s["lse"]
    if mode != "gradients":
        top = x.amax(1, keepdim=True)
        lse = (x - top).exp().sum(1).log() + top[:, 0]
        loss = (p * torch.where(listed_, logp - x.gather(1, at) + lse[:, None], 0.0)).sum(1)
        out = (loss, torch.where(some, lse, 0.0))
        if mode == "loss":
            return out
    scale = (s["dloss"] / s["temperature"] * some)[:, None]
    dx = (x - lse[:, None]).exp() * scale
    dx.scatter_add_(1, at, -p * scale)
    return *out, dx.to(s["dlogits"].dtype)


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if case["op"] == "la":
        if not own:
            out = _la_plain(s)
            return out if case["backward"] else (out, s["pool"][case["N"]:])
        from gated_delta_rule_backward_gb300 import la
        if "p" not in s:
            s["p"] = la.params_for(s["q"], s["k"], s["v"], s["g"], s["pool"], n_seq=case["N"], T=case["T"], y_dtype=s["v"].dtype)
            s["ws"] = la.backward_workspace(s["p"], s["q"].device) if case["backward"] else la.workspace(s["p"], s["q"].device)
        if case["backward"]:
            la.la_backward(s["p"], s["q"], s["k"], s["v"], s["g"], s["cu"], s["pool"], s["slot_in"], s["dy"], s["dstate"], s["dq"], s["dk"], s["dv"], s["dg"], s["dstate0"], s["ws"])
            return s["dq"], s["dk"], s["dv"], s["dg"], s["dstate0"]
        la.la_forward(s["p"], s["q"], s["k"], s["v"], s["g"], s["cu"], s["pool"], s["slot_in"], s["slot_out"], s["y"], s["ws"])
        return s["y"], s["pool"][case["N"]:]
    if not own:
        return _distill_plain(s)
    from gated_delta_rule_backward_gb300 import distill
    if "p" not in s:
        s["p"] = distill.params_for(s["logits"], s["indices"], s["teacher"], temperature=s["temperature"])
    if case["mode"] == "gradients":
        distill.distill_backward(s["p"], s["logits"], s["indices"], s["teacher"], s["lse"], s["dloss"], s["dlogits"])
        return s["dlogits"],
    # with dlogits, the gradients come with the loss: the logits are read once
    distill.distill_forward(s["p"], s["logits"], s["indices"], s["teacher"], s["loss"], s["lse"], s.get("dloss"), s.get("dlogits"))
    return (s["loss"], s["lse"]) if case["mode"] == "loss" else (s["loss"], s["lse"], s["dlogits"])


# ---- the definitions in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "distill":
        N, tau = case["N"], s["temperature"]
        loss, lse, dx = [], [], []
        for lo in range(0, N, 512):
            some = slice(lo, min(lo + 512, N))
            x, idx = s["logits"][some].double() / tau, s["indices"][some].long()
            whole = torch.logsumexp(x, 1)
            t = (s["teacher"][some].double() / tau).masked_fill(idx < 0, -math.inf)
            has = (idx >= 0).any(1)
            p = torch.softmax(t.masked_fill(~has[:, None], 0.0), 1).masked_fill(idx < 0, 0.0)
            if case["mode"] != "loss":
                full = torch.zeros_like(x).scatter_add_(1, idx.clamp(min=0), p)
                dx.append((torch.softmax(x, 1) - full) * (s["dloss"][some].double() / tau * has)[:, None])
            logq = x.gather(1, idx.clamp(min=0)) - whole[:, None]
            loss.append((torch.xlogy(p, p) - p * logq).sum(1))
            lse.append(whole.masked_fill(~has, 0.0))
        out = () if case["mode"] == "gradients" else (torch.cat(loss), torch.cat(lse))
        return out if case["mode"] == "loss" else (*out, torch.cat(dx))
    N, H_k, H_v, d, T = case["N"], case["H_k"], case["H_v"], case["d"], case["T"]
    counts, scale = _counts(case), 1.0 / math.sqrt(case["d"])
    order = sorted(range(N), key=lambda n: -counts[n])  # the longest first, so that the live ones are a prefix
    first = torch.tensor([sum(counts[:n]) for n in order], device="cuda")
    alive = [sum(c > t for c in counts) for t in range(T)]
    head = torch.arange(H_v, device="cuda") % H_k
    q, k, v, g = s["q"].double(), s["k"].double(), s["v"].double(), s["g"].double()
    M = s["pool"][s["slot_in"].long()[torch.tensor(order, device="cuda")]].double()
    y = torch.zeros_like(v)
    back = case["backward"]
    dy = s["dy"].double() if back else None
    dqh = torch.zeros_like(v) if back else None
    for t in range(T):
        n = alive[t]
        if n == 0:
            break
        r = first[:n] + t
        S = M[:n] * g[r].exp()[:, :, None, None] + v[r][..., None] * k[r][:, head][:, :, None, :]
        M[:n] = S
        y[r] = scale * (S @ q[r][:, head][..., None])[..., 0]
        if back:
            dqh[r] = scale * (dy[r][:, :, None, :] @ S)[:, :, 0]
    place = torch.argsort(torch.tensor(order, device="cuda"))
    if not back:
        return y, M[place]
    D = s["dstate"].double()[torch.tensor(order, device="cuda")]
    c = (M * D).sum((2, 3))           # the gate's gradient, carried to the sequence's start
    dkh, dv, dg = torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(g)
    for t in range(T - 1, -1, -1):
        n = alive[t]
        r = first[:n] + t
        D[:n] += scale * dy[r][..., None] * q[r][:, head][:, :, None, :]
        dv[r] = (D[:n] @ k[r][:, head][..., None])[..., 0]
        dkh[r] = (v[r][:, :, None, :] @ D[:n])[:, :, 0]
        c[:n] += (dy[r] * y[r]).sum(-1) - (v[r] * dv[r]).sum(-1)
        dg[r] = c[:n]
        D[:n] *= g[r].exp()[:, :, None, None]
    shared = lambda t: t.unflatten(1, (H_v // H_k, H_k)).sum(1)
    return shared(dqh), shared(dkh), dv, dg, D[place]
