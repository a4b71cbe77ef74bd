"""Plain float64 references of the sequence operators (torch on the CPU): the
gated delta rule token after token with gradients by automatic
differentiation, and the group norm."""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def f64(t):
    return None if t is None else t.detach().double().cpu()


def tokens(q, k, v, g, beta, S):
    """One sequence: q, k [n, hk, dk], v [n, hv, dv], g, beta [n, hv], S [hv, dk, dv]; returns (o, S)."""
    rep = v.shape[1] // q.shape[1]
    outs = []
    for t in range(q.shape[0]):
        kt, qt = k[t].repeat_interleave(rep, 0), q[t].repeat_interleave(rep, 0)
        S = S * torch.exp(g[t])[:, None, None]
        u = beta[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", kt, S))
        S = S + kt[:, :, None] * u[:, None, :]
        outs.append(torch.einsum("hk,hkv->hv", qt, S))
    return (torch.stack(outs) if outs else v[:0]), S


def packed(q, k, v, g, beta, cu, S0):
    """Every sequence of a packed batch from S0 [n, hv, dk, dv] (or None); rows behind cu[-1] are zero."""
    n = len(cu) - 1
    S0 = torch.zeros(n, v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if S0 is None else S0
    outs, ends = [], []
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        o, S = tokens(q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], S0[i])
        outs.append(o)
        ends.append(S)
    o = torch.cat(outs + [torch.zeros_like(v[cu[-1]:])])
    return o, torch.stack(ends) if ends else S0


def packed_grads(q, k, v, g, beta, cu, S0, dout, dS):
    """Gradients (dq, dk, dv, dg, dbeta, dS0) of sum(out dout) + sum(final dS)."""
    leaves = [t.clone().requires_grad_() for t in (q, k, v, g, beta)]
    S0 = torch.zeros(len(cu) - 1, v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if S0 is None else S0
    leaves.append(S0.clone().requires_grad_())
    o, S = packed(*leaves[:5], cu, leaves[5])
    loss = (o * dout)[: cu[-1]].sum() + (0 if dS is None else (S * dS).sum())
    got = torch.autograd.grad(loss, leaves, allow_unused=True)
    return [torch.zeros_like(x) if d is None else d for x, d in zip(leaves, got)]


def act(name, u):
    if name == "silu":
        return u / (1 + torch.exp(-u))
    if name == "gelu":
        return 0.5 * u * (1 + torch.erf(u / math.sqrt(2)))
    return torch.relu(u) if name == "relu" else u


def group_norm(x, groups, weight, bias, gate, activation, center, eps):
    """x [n, s, c]; returns (out, mean, rstd)."""
    n, s, c = x.shape
    y = x.reshape(n, s, groups, c // groups)
    mean = y.mean((1, 3), keepdim=True) if center else torch.zeros(n, 1, groups, 1, dtype=x.dtype)
    rstd = 1 / torch.sqrt(((y - mean) ** 2).mean((1, 3), keepdim=True) + eps)
    u = ((y - mean) * rstd).reshape(n, s, c)
    u = u if weight is None else u * weight
    u = u if bias is None else u + bias
    out = act(activation, u) if gate is None else u * act(activation, gate)
    return out, mean[:, 0, :, 0], rstd[:, 0, :, 0]


def far(x, ref):
    """Relative 2-norm of x - ref, and the largest |x - ref| over max(|ref|, rms of ref)."""
    x, ref = f64(x), f64(ref)
    if not ref.numel():
        return 0.0, 0.0
    rms = max(ref.square().mean().sqrt().item(), 1e-300)
    d = (x - ref).abs()
    return (d.square().mean().sqrt() / rms).item(), (d / ref.abs().clamp_min(rms)).max().item()
