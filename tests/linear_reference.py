"""Plain float64 references of linear attention with a decay for each head (torch on
the CPU): token after token, with gradients by automatic differentiation."""
import torch


def tokens(q, k, v, g, S, scale):
    """One sequence: q, k [n, hk, dk], v [n, hv, dv], g [n, hv], S [hv, dk, dv]; returns (o, S)."""
    rep = v.shape[1] // q.shape[1]
    outs = []
    for t in range(q.shape[0]):
        kt, qt = k[t].repeat_interleave(rep, 0), q[t].repeat_interleave(rep, 0)
        S = S * torch.exp(g[t])[:, None, None] + kt[:, :, None] * v[t][:, None, :]
        outs.append(scale * (qt[:, :, None] * S).sum(1))
    return (torch.stack(outs) if outs else v[:0]), S


def packed(q, k, v, g, cu, S0, scale):
    """Every sequence of a packed batch from S0 [n, hv, dk, dv] (or None); g [n, hv] or [hv]; rows behind cu[-1] are zero."""
    n = len(cu) - 1
    g = g if g.dim() == 2 else g.expand(q.shape[0], -1)
    S0 = torch.zeros(n, v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if S0 is None else S0
    outs, ends = [], []
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        o, S = tokens(q[a:b], k[a:b], v[a:b], g[a:b], S0[i], scale)
        outs.append(o)
        ends.append(S)
    o = torch.cat(outs + [torch.zeros_like(v[cu[-1]:])])
    return o, torch.stack(ends) if ends else S0


def packed_grads(q, k, v, g, cu, S0, dout, dS, scale):
    """Gradients (dq, dk, dv, dg, dS0) of sum(out dout) + sum(final dS)."""
    leaves = [t.clone().requires_grad_() for t in (q, k, v, g)]
    S0 = torch.zeros(len(cu) - 1, v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if S0 is None else S0
    leaves.append(S0.clone().requires_grad_())
    o, S = packed(*leaves[:4], cu, leaves[4], scale)
    loss = (o * dout)[: cu[-1]].sum() + (0 if dS is None else (S * dS).sum())
    got = torch.autograd.grad(loss, leaves, allow_unused=True)
    return [torch.zeros_like(x) if d is None else d for x, d in zip(leaves, got)]
