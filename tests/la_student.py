"""A small model of linear attention layers that learns from a teacher's top logits: its products are torch's, everything else the library's
operators, forward and backward; and the same in 64 bits, token by token, with torch's own gradients."""
import torch

from gated_delta_rule_backward_gb300 import distill, la, rms


class Student:
    def __init__(self, layers=2, D=96, H_k=2, H_v=4, S=32, vocab=300, dtype=torch.float32, seed=0):
        gen = torch.Generator().manual_seed(seed)
        w = lambda *shape: (torch.randn(*shape, generator=gen) / shape[0] ** 0.5).to("cuda", dtype)
        self.L, self.D, self.H_k, self.H_v, self.S, self.dtype = layers, D, H_k, H_v, S, dtype
        self.p = {"embed": torch.randn(vocab, D, generator=gen).to("cuda", dtype), "head": w(D, vocab)}
        for i in range(layers + 1):
            self.p[f"norm{i}"] = (1 + 0.1 * torch.randn(D, generator=gen)).cuda()
        for i in range(layers):
            self.p[f"in{i}"], self.p[f"out{i}"] = w(D, (2 * H_k + H_v) * S + H_v), w(H_v * S, D)

    def split(self, p):
        H_k, H_v, S = self.H_k, self.H_v, self.S
        n, a, b = p.shape[0], H_k * S, 2 * H_k * S + H_v * S
        return p[:, :a].view(n, H_k, S), p[:, a: 2 * a].view(n, H_k, S), p[:, 2 * a: b].view(n, H_v, S), p[:, b:]

    def states(self, slots):
        return [torch.zeros(slots, self.H_v, self.S, self.S, device="cuda") for _ in range(self.L)]

    def forward(self, tokens, pools, slot_in, slot_out=None, cu=None, T=None):
        """(logits, what the backward pass needs)."""
        x, h, kept = self.p["embed"][tokens], None, []
        for i in range(self.L):
            y, h, rstd = rms.forward(x, self.p[f"norm{i}"], h)
            p = y @ self.p[f"in{i}"]
            q, k, v, f = self.split(p)
            g = -torch.nn.functional.softplus(f.float())
            o = la.forward(q, k, v, g, pools[i], slot_in, slot_out, cu, T, y_dtype=self.dtype)
            kept.append((y, h, rstd, q, k, v, g, f, o))
            x = o.flatten(1) @ self.p[f"out{i}"]
        y, h, rstd = rms.forward(x, self.p[f"norm{self.L}"], h)
        return y @ self.p["head"], (kept, y, h, rstd)

    def backward(self, tokens, dlogits, kept, pools, slot_in, cu=None, T=None):
        kept, y, h, rstd = kept
        grads = {"head": y.t() @ dlogits}
        dx, grads[f"norm{self.L}"] = rms.backward(h, rstd, dlogits @ self.p["head"].t(), self.p[f"norm{self.L}"])
        for i in reversed(range(self.L)):
            y, h, rstd, q, k, v, g, f, o = kept[i]
            grads[f"out{i}"] = o.flatten(1).t() @ dx
            do = (dx @ self.p[f"out{i}"].t()).view_as(o)
            dq, dk, dv, dg, _ = la.backward(q, k, v, g, pools[i], slot_in, do, None, cu, T)
            df = -dg * torch.sigmoid(f.float())
            dp = torch.cat([t.flatten(1).to(self.dtype) for t in (dq, dk, dv, df)], 1)
            grads[f"in{i}"] = y.t() @ dp
            dx, grads[f"norm{i}"] = rms.backward(h, rstd, dp @ self.p[f"in{i}"].t(), self.p[f"norm{i}"], dx)
        grads["embed"] = torch.zeros_like(self.p["embed"]).index_add_(0, tokens, dx)
        return grads

    def learn(self, tokens, indices, teacher, tau, pools, slot_in, cu=None, T=None):
        """(mean loss over the tokens, gradients): the logits' gradient takes the logits' place."""
        drop = torch.full_like(slot_in, -1)
        logits, kept = self.forward(tokens, pools, slot_in, drop, cu, T)
        dloss = torch.full((len(tokens),), 1.0 / len(tokens), device="cuda")
        loss, _, d = distill.forward(logits, indices, teacher, tau, dloss=dloss, in_place=True)
        return loss.mean(), self.backward(tokens, d, kept, pools, slot_in, cu, T)


def plain(student, params, tokens, counts):
    """Logits in 64 bits from the formulas; every sequence starts from a state of zeros."""
    m, eps = student, 1e-6
    norm = lambda x, w: x * (x.square().mean(1, keepdim=True) + eps).rsqrt() * w
    h = params["embed"][tokens]
    head = torch.arange(m.H_v) % m.H_k
    for i in range(m.L):
        q, k, v, f = m.split(norm(h, params[f"norm{i}"]) @ params[f"in{i}"])
        a = (-torch.nn.functional.softplus(f)).exp()
        rows, row = [], 0
        for c in counts:
            M = torch.zeros(m.H_v, m.S, m.S, dtype=torch.float64, device="cuda")
            for _ in range(c):
                M = a[row][:, None, None] * M + v[row][:, :, None] * k[row][head][:, None, :]
                rows.append(m.S ** -0.5 * (M * q[row][head][:, None, :]).sum(-1))
                row += 1
        h = h + torch.stack(rows).flatten(1) @ params[f"out{i}"]
    return norm(h, params[f"norm{m.L}"]) @ params["head"]


def plain_loss(logits, indices, teacher, tau):
    t = torch.log_softmax(teacher.double() / tau, 1)
    s = torch.log_softmax(logits / tau, 1).gather(1, indices.long())
    return (t.exp() * (t - s)).sum(1).mean()


def lesson(counts, vocab=300, K=20, seed=1):
    gen = torch.Generator().manual_seed(seed)
    n = sum(counts)
    tokens = torch.randint(0, vocab, (n,), generator=gen).cuda()
    teacher, indices = (2 * torch.randn(n, vocab, generator=gen)).topk(K, 1)
    cu = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    return tokens, indices.to(torch.int32).cuda(), teacher.cuda(), cu
