"""GPU: digits of linear attention's results where few are left by cancellation
or by strong decays."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_frame_amd as G
    return G


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def bounds(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu,hk,hv,dk,dv", [([0, 1], 1, 1, 16, 16), ([0, 130, 130, 203], 2, 4, 112, 112), ([0, 700, 900], 1, 2, 64, 48),
                                            ([0, 65, 1000], 2, 2, 128, 128)])
def test_a_bf16_output_is_the_fp32_output_rounded_once(G, dtype, cu, hk, hv, dk, dv):
    n = cu[-1]
    x = [normal(1, n, hk, dk).to(dtype), normal(2, n, hk, dk).to(dtype), normal(3, n, hv, dv).to(dtype), -0.1 * normal(4, n, hv).abs()]
    S0 = normal(5, len(cu) - 1, hv, dk, dv)
    out, end = G.linear_forward(*x, bounds(cu), S0, scale=dk ** -0.5)
    short, same = G.linear_forward(*x, bounds(cu), S0, scale=dk ** -0.5, out_dtype=BF16)
    assert torch.equal(short, out.to(BF16)) and torch.equal(same, end)


def test_dk_takes_the_states_gradient_in_24_bits(G):
    """dk = R v of a single token, R the final state's gradient: two columns that cancel to 2^-14 of their values."""
    h, d = 16, 64
    r = 1 + torch.rand(h, d, generator=torch.Generator().manual_seed(1)).cuda()
    R = torch.zeros(1, h, d, d, device="cuda")
    R[0, :, :, 3] = r
    R[0, :, :, 41] = 2.0 ** -14 * normal(2, h, d) - r
    v = torch.zeros(1, h, d, dtype=BF16, device="cuda")
    v[:, :, 3] = v[:, :, 41] = 1.0
    z = torch.zeros_like(v)
    dk = G.linear_backward(normal(3, 1, h, d).to(BF16), normal(4, 1, h, d).to(BF16), v, torch.full((1, h), -0.1, device="cuda"),
                           bounds([0, 1]), z, None, R)[1][0].double()
    want = R[0].double().sum(-1)
    # six products of bf16 terms, exact, and their sums below 2: at most a step of 2^-23 each; then the result's half step
    assert ((dk - want).abs() / (6 * 2.0 ** -23 + 2.0 ** -8 * want.abs())).max().item() <= 1


def test_dk_takes_the_products_of_v_and_dout_in_24_bits(G):
    """dk of the first of two tokens, without a decay: (v.do) q of both, equal but for 2^-15 of their values, with opposite q."""
    h, d, n = 16, 16, 8
    rnd = lambda seed: (1 + torch.randint(0, 128, (n, h), generator=torch.Generator().manual_seed(seed)) / 128).cuda()  # noqa: E731
    v, do, q = (torch.zeros(2 * n, h, d, device="cuda") for _ in range(3))
    v[0::2, :, 0], v[0::2, :, 9] = rnd(1), rnd(2) / 256
    do[0::2, :, 0], do[0::2, :, 9] = rnd(3), rnd(4)
    do[1::2, :, 0], do[1::2, :, 9] = do[0::2, :, 0], rnd(5)
    sign = normal(6, n, h, d).sign()
    q[0::2], q[1::2] = sign, -sign
    x = [t.to(BF16) for t in (q, normal(7, 2 * n, h, d), v, do)]
    assert all(torch.equal(t.float(), u) for t, u in zip((x[0], x[2], x[3]), (q, v, do)))
    dk = G.linear_backward(*x[:3], torch.zeros(2 * n, h, device="cuda"), bounds(list(range(0, 2 * n + 1, 2))), x[3])[1][0::2].double()
    P = (v[0::2].double() * (do[0::2].double() - do[1::2].double())).sum(-1)
    want = P[..., None] * sign.double()
    # the products are below 4 + 2^-6 and exact in 24 bits; six products of their terms, whose sums have at most a step of 2^-21 each
    assert ((dk - want).abs() / (6 * 2.0 ** -21 + 2.0 ** -8 * want.abs())).max().item() <= 1


def gate_gradients(q, k, v, g, do, scale):
    """In 64 bits, of one sequence from zeros with heads of their own: e^g <R, S before> of each token and head, by the states
    themselves, and what its error goes by: the magnitudes of what each token reads from earlier ones and gives to later ones."""
    n, h, d = v.shape
    a, (Q, K, V, D) = torch.exp(g.double())[..., None, None], (t.double() for t in (q, k, v, do))
    outer = lambda x, y: x[:, :, None] * y[:, None, :]  # noqa: E731
    S = R = A = B = torch.zeros(h, q.shape[2], d, dtype=torch.float64, device="cuda")
    before, dg, mag = [], torch.zeros(n, h, dtype=torch.float64, device="cuda"), torch.zeros(n, h, dtype=torch.float64, device="cuda")
    for t in range(n):
        before.append(S * a[t])
        A = A * a[t]
        mag[t] += (scale * outer(Q[t].abs(), D[t].abs()) * A).sum((-1, -2)).square()
        S, A = before[-1] + outer(K[t], V[t]), A + outer(K[t].abs(), V[t].abs())
    for t in reversed(range(n)):
        mag[t] += (B * outer(K[t].abs(), V[t].abs())).sum((-1, -2)).square()
        R, B = R + scale * outer(Q[t], D[t]), B + scale * outer(Q[t].abs(), D[t].abs())
        dg[t] = (R * before[t]).sum((-1, -2))
        R, B = R * a[t], B * a[t]
    return dg, mag.flip(0).cumsum(0).flip(0)          # the squares of all tokens behind


STRONG = [-0.05, -1.0, -4.0, -8.0, -12.0, -16.0, -30.0, -60.0]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,dk,dv", [(60, 16, 16), (1500, 64, 64), (700, 128, 48)])
def test_gradients_of_strong_gates_have_digits(G, dtype, n, dk, dv):
    """One gate for all tokens of a head, and gates of every strength side by side.  What a token reads from earlier ones and what it
    gives to later ones have roundings of 2^-22 of their magnitudes in the 2-norm, independent ones, and a gate's gradient sums those
    behind it.  What a token reads of itself is in neither."""
    h, scale = len(STRONG), dk ** -0.5
    q, k, v, do = ((normal(i, n, h, d) / (8 if i < 3 else 1)).to(dtype) for i, d in ((1, dk), (2, dk), (3, dv), (4, dv)))
    g = torch.tensor(STRONG, device="cuda")
    want, var = gate_gradients(q, k, v, g.expand(n, h), do, scale)
    got = G.linear_backward(q, k, v, g.expand(n, h).contiguous(), bounds([0, n]), do, scale=scale)[3]
    assert ((got.double() - want).norm(dim=0) / (2.0 ** -22 * var.sum(0).sqrt())).max().item() <= 1
    assert ((got.double() - want).norm(dim=0) / want.norm(dim=0)).max().item() <= 1e-4
    got = G.linear_backward(q, k, v, g, bounds([0, n]), do, scale=scale)[3]
    # the sum over the tokens: a token's roundings count for every gate before it
    assert ((got.double() - want.sum(0)).abs() / (2.0 ** -22 * var.sqrt().sum(0))).max().item() <= 1
    mixed = -16 * torch.rand(n, h, generator=torch.Generator().manual_seed(9)).cuda() ** 3
    want, var = gate_gradients(q, k, v, mixed, do, scale)
    got = G.linear_backward(q, k, v, mixed, bounds([0, n]), do, scale=scale)[3]
    assert ((got.double() - want).norm(dim=0) / (2.0 ** -22 * var.sum(0).sqrt())).max().item() <= 1


@pytest.mark.parametrize("fixed", [False, True])
def test_gates_whose_exponential_rounds_to_0_have_no_gradient(G, fixed):
    """In fp32, e^g is 0 at g = -103.972084 and below, its smallest value at -103.972076: 150 ln 2 lies between."""
    n, d = 200, 32
    low = [-103.98, -103.97208404541016, -103.9721, -104.0]
    assert (torch.exp(torch.tensor(low, dtype=torch.float64)).float() == 0).all()
    assert torch.exp(torch.tensor(-103.97207641601562, dtype=torch.float64)).float() > 0
    x = [normal(i, n, 2, d) for i in (1, 2, 3)]
    S0, dS = normal(4, 1, 2, d, d), normal(5, 1, 2, d, d)
    for i, g in enumerate(low):
        gates = torch.full((n, 2), -0.05, device="cuda")
        gates[10 + 45 * i, 1] = g
        if fixed:
            gates = torch.tensor([-0.05, g], device="cuda")
        dg = G.linear_backward(*x, gates, bounds([0, n]), x[2] + 1, S0, dS)[3]
        assert (dg[1] if fixed else dg[10 + 45 * i, 1]).item() == 0
        assert torch.count_nonzero(dg).item() == dg.numel() - 1
