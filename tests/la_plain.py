"""Linear attention in 64 bits, token by token, from the formulas of include/la.h; and the same on absolute values, which
bounds the sum of the magnitudes that a result is made of (what its rounding errors are relative to)."""
import torch


def problem(counts, H_k, H_v, S, SV=None, dtype=torch.float32, gate=torch.float32, slots=None, seed=0, constant=False, shift=0, strength=None,
            std=1.0):
    """Token rows of a packed qkv buffer (`shift` elements off its start), log decays, a pool, and what a backward pass gets."""
    SV = S if SV is None else SV
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    n, N = sum(counts), len(counts)
    width = 2 * H_k * S + H_v * SV
    buf = torch.zeros(n * width + shift, dtype=dtype)
    buf[shift:].view(n, width)[:] = (rnd(n, width) * std).to(dtype)
    dev = buf.cuda()[shift:].view(n, width)
    if strength is not None:
        g = torch.full((n, H_v), float(strength))
    else:
        g = -torch.exp(1.5 * rnd(n, H_v) - 3)
    g = g.to(gate).cuda()
    if constant:
        g = g[:1].expand(n, H_v) if n else g
    return dict(q=dev[:, : H_k * S].view(n, H_k, S), k=dev[:, H_k * S: 2 * H_k * S].view(n, H_k, S), v=dev[:, 2 * H_k * S:].view(n, H_v, SV), g=g,
                pool=rnd(N if slots is None else slots, H_v, SV, S).cuda(), dy=rnd(n, H_v, SV).to(dtype).cuda(), dstate=rnd(N, H_v, SV, S).cuda())


def forward(x, counts, slot_in, scale, absolute=False):
    """(y, the state after each sequence, the state after every token)."""
    f = (lambda t: t.double().abs()) if absolute else (lambda t: t.double())
    q, k, v, pool = f(x["q"]), f(x["k"]), f(x["v"]), f(x["pool"])
    a = x["g"].double().exp()
    H_v = v.shape[1]
    head = torch.arange(H_v, device=q.device) % q.shape[1]
    y, after, every, row = torch.zeros_like(v), [], [], 0
    for n, c in enumerate(counts):
        M = pool[slot_in[n]] if slot_in[n] >= 0 else torch.zeros_like(x["pool"][0]).double()
        for _ in range(c):
            M = M * a[row][:, None, None] + v[row][:, :, None] * k[row][head][:, None, :]
            y[row] = scale * (M * q[row][head][:, None, :]).sum(-1)
            every.append(M)
            row += 1
        after.append(M)
    return y, (torch.stack(after) if after else None), every


def backward(x, counts, slot_in, scale, with_state=True, absolute=False):
    """(dq, dk, dv, dg, dstate_0).  absolute: magnitudes; dg's is that of the running sum it is computed as."""
    f = (lambda t: t.double().abs()) if absolute else (lambda t: t.double())
    q, k, v, dy = f(x["q"]), f(x["k"]), f(x["v"]), f(x["dy"])
    a = x["g"].double().exp()
    H_k, H_v = q.shape[1], v.shape[1]
    head = torch.arange(H_v, device=q.device) % H_k
    _, after, every = forward(x, counts, slot_in, scale, absolute)
    dqh, dkh = (torch.zeros(q.shape[0], H_v, q.shape[2], dtype=torch.float64, device=q.device) for _ in range(2))
    dv, dg, first, end = torch.zeros_like(v), torch.zeros(v.shape[:2], dtype=torch.float64, device=q.device), [], 0
    for n, c in enumerate(counts):
        lo, end = end, end + c
        D = f(x["dstate"][n]) if with_state else torch.zeros_like(f(x["dstate"][n]))
        run = (D * after[n]).sum((1, 2))
        for t in range(end - 1, lo - 1, -1):
            kk, qq = k[t][head], q[t][head]
            D = D + scale * dy[t][:, :, None] * qq[:, None, :]
            dqh[t] = scale * (every[t] * dy[t][:, :, None]).sum(1)
            dkh[t] = (D * v[t][:, :, None]).sum(1)
            dv[t] = (D * kk[:, None, :]).sum(2)
            before = every[t - 1] if t > lo else (f(x["pool"][slot_in[n]]) if slot_in[n] >= 0 else torch.zeros_like(D))
            if absolute:
                run = run + (qq * dqh[t]).sum(1) + (kk * dkh[t]).sum(1)
                dg[t] = run
            else:
                dg[t] = a[t] * (D * before).sum((1, 2))
            D = D * a[t][:, None, None]
        first.append(D)
    shared = lambda t: t.unflatten(1, (H_v // H_k, H_k)).sum(1)
    return shared(dqh), shared(dkh), dv, dg, torch.stack(first) if first else None


def within(got, ref, magnitude, eps, what):
    """|got - ref| <= eps magnitude, and half a unit of got's own type."""
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    err = (got.double() - ref).abs()
    least = 2.0 ** -24 if got.dtype == torch.float16 else 1e-37   # below the smallest normal numbers
    over = err - (eps * magnitude + half * ref.abs() * (1 + eps) + least)
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    assert (over <= 0).all() if over.numel() else True, f"{what}: off by {float(err.max()):.3e}, {float((over > 0).double().mean()):.2%} of elements beyond the bound, worst ratio {float((err / (eps * magnitude + half * ref.abs() + least)).max()):.2f}"
