"""GPU: rotary positions and their gradients against the turns in 64 bits."""
import math
from fractions import Fraction

import pytest
import torch

from tests import seq_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_frame_amd as G
    return G


def angles(positions, frequencies, sections, sign=1):
    """[tokens, pairs] in 64 bits on the CPU; exact enough where position times frequency is below 2^24."""
    p, f = positions.cpu().double(), frequencies.cpu()
    if p.dim() == 1:
        return sign * p[:, None] * f
    axis = torch.tensor(sum(([i] * n for i, n in enumerate(sections)), []))
    return sign * p[:, axis] * f


def turned(x, angle, layout, magnitude):
    """The turned heads in 64 bits and, for each value, |x| + |y| of its pair times the magnitude (0 where it is copied)."""
    x, pairs = R.f64(x), angle.shape[1]
    y, mag = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, pairs), slice(pairs, 2 * pairs)) if layout == "half" else (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2))
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y[..., a] = magnitude * (x[..., a] * c - x[..., b] * s)
    y[..., b] = magnitude * (x[..., a] * s + x[..., b] * c)
    mag[..., a] = mag[..., b] = abs(magnitude) * (x[..., a].abs() + x[..., b].abs())
    return y, mag


def near(got, x, angle, layout, magnitude, more=0.0):
    """A factor is off by the argument's rounding (2^-24 of at most pi/4), the polynomial's terms and evaluation (2) and its product
    with the magnitude (1), in units of 2^-24 of the magnitude; the two products and their sum add 2.  6 in all; a bf16 result half
    a step of its value more.  `more`: what the angle itself may be off."""
    want, mag = turned(x, angle, layout, magnitude)
    tol = (6 * R.HALF[F32] + more) * mag + (1.01 * R.HALF[BF16] * want.abs() if got.dtype == BF16 else 0)
    d = (R.f64(got) - want).abs()
    assert (d <= tol).all(), (d - tol).max().item()


def inputs(n, hq, hk, width, dtype, seed, sections=None, far=4096):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(n, h, width, generator=g).to(dtype).cuda() for h in (hq, hk))
    positions = torch.randint(-far, far + 1, (n,) if sections is None else (n, len(sections)), generator=g, dtype=torch.int32)
    return q, k, positions.cuda()


CASES = [  # tokens, heads_q, heads_k, width, pairs, dtype, layout, sections
    (1, 1, 1, 8, 4, F32, "half", None), (1, 20, 20, 112, 56, BF16, "interleaved", None), (48, 32, 16, 128, 64, BF16, "half", None),
    (5, 3, 2, 64, 16, BF16, "half", None), (5, 3, 2, 64, 16, F32, "interleaved", None), (7, 2, 1, 80, 33, F32, "half", None),
    (7, 2, 1, 80, 33, BF16, "half", None), (7, 2, 1, 80, 33, BF16, "interleaved", None), (9, 1, 3, 48, 1, BF16, "half", None),
    (9, 1, 3, 48, 1, F32, "interleaved", None), (33, 5, 4, 96, 12, F32, "half", None), (6, 2, 2, 112, 56, F32, "half", (24, 16, 16)),
    (6, 2, 2, 112, 56, BF16, "interleaved", (24, 16, 16)), (13, 1, 1, 24, 10, F32, "half", (3, 0, 5, 2)), (3, 2, 2, 1024, 512, BF16, "half", None),
    (2, 200, 1, 16, 8, F32, "half", (8,)), (4097, 2, 1, 40, 20, BF16, "half", None), (4099, 1, 2, 48, 24, F32, "interleaved", (8, 8, 8)),
    (5001, 1, 1, 32, 8, BF16, "half", None)]


@pytest.mark.parametrize("n,hq,hk,width,pairs,dtype,layout,sections", CASES)
def test_rotary_and_its_gradients(G, n, hq, hk, width, pairs, dtype, layout, sections):
    q, k, positions = inputs(n, hq, hk, width, dtype, n + pairs, sections)
    f = G.rotary_frequencies(2 * pairs)[0]
    for call, sign, m in ((G.rotary, 1, 1.0), (G.rotary_backward, -1, 1.25)):
        angle = angles(positions, f, sections, sign)
        gq, gk = call(q, k, positions, f, layout=layout, sections=sections, magnitude=m)
        assert gq.shape == q.shape and gk.shape == k.shape and gq.dtype == gk.dtype == dtype
        near(gq, q, angle, layout, m)
        near(gk, k, angle, layout, m)
        assert torch.equal(gq[..., 2 * pairs:], q[..., 2 * pairs:]) and torch.equal(gk[..., 2 * pairs:], k[..., 2 * pairs:])
        alone, none = call(q, None, positions, f, layout=layout, sections=sections, magnitude=m)
        assert none is None and torch.equal(alone, gq)
        iq, ik = q.clone(), k.clone()
        assert call(iq, ik, positions, f, layout=layout, sections=sections, magnitude=m, out=(iq, ik))[0] is iq
        assert torch.equal(iq, gq) and torch.equal(ik, gk)


def test_gradients_are_those_of_autograd_and_of_differences(G):
    n, pairs, width = 5, 12, 32
    q, k, positions = inputs(n, 2, 1, width, F32, 3)
    f = G.rotary_frequencies(2 * pairs)[0]
    angle = angles(positions, f, None)
    x = R.f64(q).requires_grad_()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x[..., :pairs], x[..., pairs: 2 * pairs]
    y = torch.cat([1.5 * (a * c - b * s), 1.5 * (a * s + b * c), x[..., 2 * pairs:]], -1)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(9)).cuda()
    (want,) = torch.autograd.grad(y, x, R.f64(do))
    got, _ = G.rotary_backward(do, None, positions, f, magnitude=1.5)
    assert ((R.f64(got) - want).abs() <= 6 * R.HALF[F32] * 1.5 * 2 * do.abs().max().item()).all()
    # the turn is linear: a difference along one component is its column of the Jacobian
    e = torch.zeros_like(q)
    e[2, 1, 7] = 1.0
    column, _ = G.rotary(e, None, positions, f, magnitude=1.5)
    assert math.isclose((column * do).sum().item(), got[2, 1, 7].item(), rel_tol=1e-5, abs_tol=1e-6)


def test_far_positions_turn_by_the_exact_angle(G):
    """Angles reduced with rational arithmetic: pi to 60 digits."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494")
    p = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 99999999, 7, 0]
    f = torch.tensor([1.0, 0.7853981633974483, 3.1e-3, 1e-4, 2.5, 1e-300, 6.283185307179586, 123456.789], dtype=torch.float64)
    positions = torch.tensor(p, dtype=torch.int32)
    angle = torch.tensor([[float((x * Fraction(y)) % (2 * pi)) for y in f.tolist()] for x in p], dtype=torch.float64)
    q = torch.randn(len(p), 2, 16, generator=torch.Generator().manual_seed(1)).cuda()
    got, _ = G.rotary(q, None, positions.cuda(), f.cuda())
    near(got, q, angle, "half", 1.0, 2.0 ** -40)


def test_strided_rows_and_outputs(G):
    """Slices of one projection, in place and into another; the values between them stay."""
    n, hq, hk, width = 11, 4, 2, 48
    q, k, positions = inputs(n, hq, hk, width, BF16, 5)
    f = G.rotary_frequencies(32)[0]
    want = G.rotary(q, k, positions, f, layout="interleaved")
    row = torch.full((n, (hq + hk) * width + 24), 7.0, dtype=BF16, device="cuda")
    sq, sk = row[:, 8: 8 + hq * width].unflatten(1, (hq, width)), row[:, 16 + hq * width: 16 + (hq + hk) * width].unflatten(1, (hk, width))
    sq.copy_(q)
    sk.copy_(k)
    got = G.rotary(sq, sk, positions, f, layout="interleaved")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    other = torch.full((n, 1024), 3.0, dtype=BF16, device="cuda")
    oq = other[:, : hq * width].unflatten(1, (hq, width))
    G.rotary(sq, sk, positions, f, layout="interleaved", out=(oq, sk))
    assert torch.equal(oq, want[0]) and torch.equal(sk, want[1]) and torch.equal(sq, q)
    assert (other[:, hq * width:] == 3.0).all()
    gaps = torch.cat([row[:, :8], row[:, 8 + hq * width: 16 + hq * width], row[:, 16 + (hq + hk) * width:]], 1)
    assert (gaps == 7.0).all()


def test_not_finite_values_stay_in_their_pair(G):
    q, k, positions = inputs(3, 2, 1, 32, BF16, 6)
    f = G.rotary_frequencies(16)[0]
    want, _ = G.rotary(q, None, positions, f)
    q[1, 0, 3], q[1, 1, 20], q[2, 0, 31] = float("nan"), float("inf"), float("-inf")
    got, _ = G.rotary(q, None, positions, f)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[1, 0, 3] = bad[1, 0, 11] = bad[1, 1, 20] = bad[2, 0, 31] = True
    assert torch.isnan(got[1, 0, 3]) and torch.isnan(got[1, 0, 11]) and got[1, 1, 20] == float("inf") and got[2, 0, 31] == float("-inf")
    assert torch.equal(got[~bad], want[~bad])


def test_on_another_stream_and_in_a_graph(G):
    q, k, positions = inputs(9, 4, 2, 64, BF16, 7)
    f = G.rotary_frequencies(64)[0]
    want = G.rotary(q, k, positions, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = G.rotary(q, k, positions, f)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    out = (torch.empty_like(q), torch.empty_like(k))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.rotary(q, k, positions, f, out=out)
    for i in range(3):
        positions.add_(i)
        want = G.rotary(q, k, positions, f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_no_tokens(G):
    q, k, positions = inputs(0, 2, 1, 32, BF16, 8)
    got = G.rotary(q, k, positions, G.rotary_frequencies(32)[0])
    assert got[0].shape == (0, 2, 32) and got[1].shape == (0, 1, 32)


def test_refusals(G):
    q, k, p = inputs(4, 2, 1, 32, BF16, 1)
    f = G.rotary_frequencies(32)[0]
    for bad in ((q.cpu(), k, p, f), (q.half(), k.half(), p, f), (q, k.float(), p, f), (q, k[:3].contiguous(), p, f), (q[0], None, p, f),
                (q, k[..., :16].contiguous(), p, f), (q, k, p.long(), f), (q, k, p[:3], f), (q, k, p.cpu(), f), (q, k, p, f.float()),
                (q, k, p, f.cpu()), (q, k, p, f[None]), (q, k, p, torch.cat([f, f])), (q, k, p, f[:0]), (q, k[:, :0], p, f),
                (q.transpose(0, 1), None, p[:2].contiguous(), f), (q[..., :30], None, p, f[:15].contiguous()), (q[..., ::2], None, p, f[:8].contiguous()),
                (q, k, p[:, None].expand(4, 2).contiguous(), f)):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.rotary(*bad)
    for kw in (dict(layout="other"), dict(sections=(8, 8)), dict(sections=(16,)), dict(sections=(8, 9)), dict(out=(q,)), dict(out=(q, k.float())),
               dict(out=(q[:3], k)), dict(magnitude=float("nan"))):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.rotary(q, k, p, f, **kw)
    with pytest.raises(ValueError):
        G.rotary(q, None, p, f, out=(q, k))
