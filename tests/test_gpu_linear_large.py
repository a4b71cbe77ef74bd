"""GPU: linear attention and rotary positions over tensors of more than 2^31
elements.  An offset that wraps at 32 bits gives errors of the values' own size,
far above what the roundings of two calls differ by."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_frame_amd as G
    yield G
    torch.cuda.empty_cache()


def bounds(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def near(got, want, rel):
    return (got.float() - want.float()).norm().item() <= rel * want.float().norm().item()


def test_linear_attention(G):
    """The last sequence alone, and the last heads alone, are what they are in the whole call."""
    n, at, hv, dk, dv = 132001, 131500, 128, 16, 128
    assert (at + 1) * hv * dv > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    q, k, v, dout = r(n, 1, dk), r(n, 1, dk), r(n, hv, dv), r(n, hv, dv)
    g = -0.001 - 0.1 * torch.rand(n, hv, generator=gen, device="cuda")
    S0, dS = torch.randn(2, 3, hv, dk, dv, generator=gen, device="cuda")
    cu = [0, 1000, at, n]
    out, end = G.linear_forward(q, k, v, g, bounds(cu), S0, scale=0.25)
    dq, dk_, dv_, dg, d0 = G.linear_backward(q, k, v, g, bounds(cu), dout, S0, dS, scale=0.25)
    # bf16 results round to different neighbours where two calls' fp32 values differ: 2^-8 of few of them
    tail = [t[at:] for t in (q, k, v, g)]
    o, e = G.linear_forward(*tail, bounds([0, n - at]), S0[2:], scale=0.25)
    assert near(out[at:], o, 2.0 ** -18) and near(end[2:], e, 2.0 ** -18)
    got = G.linear_backward(*tail, bounds([0, n - at]), dout[at:], S0[2:], dS[2:], scale=0.25)
    for a, b in zip((dq[at:], dk_[at:], dv_[at:]), got):
        assert near(a, b, 2.0 ** -10)
    assert near(dg[at:], got[3], 2.0 ** -14) and near(d0[2:], got[4], 2.0 ** -18)
    heads = [t[:, -2:].contiguous() for t in (v, g, dout, S0, dS)]
    o, e = G.linear_forward(q, k, heads[0], heads[1], bounds(cu), heads[3], scale=0.25)
    assert near(out[:, -2:], o, 2.0 ** -18) and near(end[:, -2:], e, 2.0 ** -18)
    got = G.linear_backward(q, k, heads[0], heads[1], bounds(cu), heads[2], heads[3], heads[4], scale=0.25)
    assert near(dv_[:, -2:], got[2], 2.0 ** -10) and near(dg[:, -2:], got[3], 2.0 ** -14) and near(d0[:, -2:], got[4], 2.0 ** -18)


def test_rotary(G):
    n, at, hq, hk, width = 530001, 529900, 32, 8, 128
    assert at * hq * width > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k = (torch.randn(n, h, width, generator=gen, device="cuda", dtype=BF16) for h in (hq, hk))
    positions = torch.arange(n, dtype=torch.int32, device="cuda")
    f = G.rotary_frequencies(width)[0]
    gq, gk = G.rotary(q, k, positions, f)
    tq, tk = G.rotary(q[at:], k[at:], positions[at:].contiguous(), f)
    assert torch.equal(gq[at:], tq) and torch.equal(gk[at:], tk)
    assert G.rotary(q, k, positions, f, out=(q, k))[0] is q
    assert torch.equal(q[at:], tq) and torch.equal(k[at:], tk)
