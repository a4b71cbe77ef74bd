"""GPU: one token of linear attention per row against the definition in 64 bits."""
import pytest
import torch

from tests import linear_reference as L
from tests import seq_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_frame_amd as G
    return G


def rows(n, hk, hv, dk, dv, dtype, seed, fixed=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = [r(n, hk, dk).to(dtype), r(n, hk, dk).to(dtype), r(n, hv, dv).to(dtype),
         -(0.001 + 0.3 * torch.rand((hv,) if fixed else (n, hv), generator=g))]
    return [x.cuda() for x in t]


def reference(q, k, v, g, state, slots, scale):
    """Rows in order; returns (out with None for padding rows, state, bounds of both by magnitude)."""
    q, k, v, g, state = (R.f64(x) for x in (q, k, v, g, state))
    g = g if g.dim() == 2 else g.expand(q.shape[0], -1)
    out, mag, state, smag = [], [], state.clone(), state.abs()
    for i, s in enumerate(slots):
        if not 0 <= s < state.shape[0]:
            out.append(None)
            mag.append(None)
            continue
        o, state[s] = L.tokens(q[i:i + 1], k[i:i + 1], v[i:i + 1], g[i:i + 1], state[s], scale)
        m, smag[s] = L.tokens(q[i:i + 1].abs(), k[i:i + 1].abs(), v[i:i + 1].abs(), g[i:i + 1], smag[s], abs(scale))
        out.append(o[0])
        mag.append(m[0])
    return out, state, mag, smag


@pytest.mark.parametrize("n,hk,hv,dk,dv,dtype,out_dtype,fixed", [
    (1, 1, 1, 16, 16, F32, F32, False), (1, 20, 20, 112, 112, BF16, BF16, True), (5, 2, 6, 48, 80, F32, F32, True),
    (7, 4, 4, 128, 16, BF16, F32, False), (3, 1, 4, 16, 128, BF16, BF16, False), (33, 2, 4, 128, 128, BF16, BF16, False),
    (2, 3, 3, 96, 112, F32, BF16, True)])
def test_decode(G, n, hk, hv, dk, dv, dtype, out_dtype, fixed):
    x, scale = rows(n, hk, hv, dk, dv, dtype, n, fixed), dk ** -0.5
    gen = torch.Generator().manual_seed(n)
    pool = n + 3
    state = torch.randn(pool, hv, dk, dv, generator=gen).cuda()
    slots = torch.randperm(pool, generator=gen)[:n]
    want, after, mag, smag = reference(*x, state, slots.tolist(), scale)
    got = G.linear_decode(*x, state, slots.to(torch.int32).cuda(), scale=scale, out_dtype=out_dtype)
    assert got.dtype == out_dtype and got.shape == (n, hv, dv)
    # a state value has a rounding of exp (two steps), of its product and of the sum: 4 of 2^-24 of its magnitude; an output is at
    # most two sums of d_k products and a few roundings away, each half a step of its magnitude; a bf16 output half a step more
    assert ((R.f64(state) - after).abs() <= 5 * R.HALF[F32] * smag).all()
    want, mag = torch.stack(want), torch.stack(mag)
    tol = (2 * dk + 16) * R.HALF[F32] * mag + (R.HALF[BF16] * want.abs() if out_dtype == BF16 else 0)
    assert ((R.f64(got) - want).abs() <= 1.01 * tol).all()


def test_padding_rows_repeated_slots_strides_and_no_slots(G):
    n, hk, hv, dk, dv, pool = 300, 1, 2, 32, 48, 40
    x = rows(n, hk, hv, dk, dv, F32, 11)
    gen = torch.Generator().manual_seed(5)
    slots = torch.randint(-2, pool + 3, (n,), generator=gen)
    slots[7], slots[8], slots[299] = 2 ** 31 - 1, -2 ** 31, 4
    state = torch.randn(pool, hv, dk, dv, generator=gen).cuda()
    want, after, mag, smag = reference(*x, state, slots.tolist(), 0.5)
    out = torch.full((n, hv, dv), 7.0, device="cuda")
    G.linear_decode(*x, state, slots.to(torch.int32).cuda(), scale=0.5, out=out)
    times = max(slots.tolist().count(s) for s in range(pool))        # tokens applied to one state
    assert ((R.f64(state) - after).abs() <= 5 * times * R.HALF[F32] * smag).all()
    for i in range(n):
        if want[i] is None:
            assert (out[i] == 7.0).all()
        else:
            assert ((R.f64(out[i]) - want[i]).abs() <= (5 * times + 2 * dk + 16) * R.HALF[F32] * mag[i]).all()
    # row order without slots, and slices of one projection
    n = 6
    x = rows(n, hk, hv, dk, dv, BF16, 3)
    s1 = torch.randn(n, hv, dk, dv, device="cuda")
    s2, s3 = s1.clone(), s1.clone()
    a = G.linear_decode(*x, s1)
    b = G.linear_decode(*x, s2, torch.arange(n, dtype=torch.int32, device="cuda"))
    row = torch.cat([t.reshape(n, -1) for t in x[:3]] + [torch.full((n, 8), float("nan"), dtype=BF16, device="cuda")], 1)
    q, k, v = (row[:, i:i + h * d].view(n, h, d) for i, h, d in ((0, hk, dk), (hk * dk, hk, dk), (2 * hk * dk, hv, dv)))
    c = G.linear_decode(q, k, v, x[3], s3)
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(s1, s2) and torch.equal(s1, s3)


def test_gates_at_their_ends(G):
    """A gate of -inf drops the old state; a NaN row stays in its own state."""
    n, d = 3, 32
    x = rows(n, 1, 1, d, d, F32, 2)
    x[3][0] = float("-inf")
    x[2][2] = float("nan")
    state = torch.randn(n, 1, d, d, device="cuda")
    out = G.linear_decode(*x, state)
    assert torch.equal(state[0, 0], x[1][0, 0][:, None] * x[2][0, 0][None, :])
    assert torch.isnan(out[2]).all() and torch.isfinite(out[:2]).all() and torch.isfinite(state[:2]).all()


def test_on_another_stream_and_in_a_graph(G):
    n, hk, hv, dk, dv = 9, 2, 2, 64, 64
    x = rows(n, hk, hv, dk, dv, BF16, 4)
    slots = torch.randperm(n).to(torch.int32).cuda()
    state = torch.randn(n, hv, dk, dv, device="cuda")
    eager, captured = state.clone(), state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = G.linear_decode(*x, eager, slots)
    torch.cuda.current_stream().wait_stream(side)
    out = torch.empty(n, hv, dv, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.linear_decode(*x, captured, slots, out=out)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = first if i == 0 else G.linear_decode(*x, eager, slots)
        assert torch.equal(out, want) and torch.equal(captured, eager)


def test_refusals(G):
    x = rows(4, 2, 4, 32, 32, BF16, 1)
    state = torch.zeros(4, 4, 32, 32, device="cuda")
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ((x[0], x[1][:, :1].contiguous(), *x[2:]), (x[0].float(), *x[1:]), (*x[:3], x[3].double()), (*x[:3], x[3][:3]),
                (*x[:3], x[3][0, :3].contiguous()), (*x[:3], x[3][:, 0]), (*x[:3], None), (x[0].half(), x[1].half(), x[2].half(), x[3]),
                (*x[:2], x[2][:, :3].contiguous(), x[3][:, :3].contiguous()), (x[0].cpu(), *x[1:])):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.linear_decode(*bad, state, slots)
    for bad in (state.double(), state[:, :2].contiguous(), state[:3].contiguous(), state.transpose(2, 3), state[0]):
        with pytest.raises(ValueError):
            G.linear_decode(*x, bad)
    for bad in (slots.long(), slots[:3], slots.cpu()):
        with pytest.raises(ValueError):
            G.linear_decode(*x, state, bad)
    for kw in (dict(scale=float("nan")), dict(out_dtype=torch.float16), dict(out=torch.zeros(4, 4, 32, device="cuda"), out_dtype=BF16)):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.linear_decode(*x, state, slots, **kw)
