"""GPU: calls of linear attention that differ in what they are given: with one of
the states alone, scales of either sign, captured with a gate for each head, on
two streams at once."""
import pytest
import torch

from tests import linear_reference as L
from tests import seq_reference as R
from tests.test_gpu_linear import G, bounds_of, check, cu_tensor, inputs, reference, states, steps  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("initial,final", [(True, False), (False, True)])
@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("dtype,lengths,scale", [(BF16, [90, 0, 1], -0.3), (F32, [700, 2, 130], 1.5), (BF16, [0, 1500, 64], 0.125)])
def test_one_of_the_states_alone(G, initial, final, fixed, dtype, lengths, scale):  # noqa: F811
    hk, hv, dk, dv = 1, 2, 32, 48
    cu = bounds_of(lengths)
    x = inputs(cu[-1], hk, hv, dk, dv, dtype, 61, fixed)
    S0 = states(len(lengths), hv, dk, dv, 1) if initial else None
    dS = states(len(lengths), hv, dk, dv, 2) if final else None
    eps = steps(dk, dv, lengths) + hv // hk
    o, end, mo, mend = reference(x, cu, S0, scale)
    got, last = G.linear_forward(*x, cu_tensor(cu), S0, scale=scale)
    check(got, o, mo, eps)
    check(last, end, mend, eps)
    dout = (x[2].float() * 0.5 + 1).to(dtype)
    args, z = [R.f64(t) for t in x], lambda t: None if t is None else R.f64(t).abs()  # noqa: E731
    want = L.packed_grads(*args, cu, R.f64(S0), R.f64(dout), R.f64(dS), scale)
    mag = L.packed_grads(*[t.abs() for t in args[:3]], args[3], cu, z(S0), z(dout), z(dS), abs(scale))
    dq, dk_, dv_, dg, d0 = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS, scale=scale)
    for a, w, m in ((dq, want[0], mag[0]), (dk_, want[1], mag[1]), (dv_, want[2], mag[2])):
        check(a, w, m, eps)
    if initial:
        check(d0, want[4], mag[4], eps)
    else:
        assert d0 is None
    terms = (args[2].abs() * mag[2]).sum(-1)
    m = torch.cat([terms[a:b].flip(0).cumsum(0).flip(0) + ((z(dS) * mend).sum((-1, -2))[i] if final else 0) for i, (a, b) in enumerate(zip(cu, cu[1:]))])
    m = 3 * (m.sum(0) if fixed else m)
    assert (R.f64(dg) - want[3]).norm() <= 2.0 ** -20 * m.norm()
    if not initial and not fixed:
        assert (dg[[a for a, b in zip(cu, cu[1:]) if b > a]] == 0).all()


def test_captured_with_a_gate_for_each_head(G):  # noqa: F811
    """Replays follow new lengths and gates; both directions on one workspace, with eager calls and synchronizations between."""
    n, hk, hv, d = 900, 2, 4, 64
    x = inputs(n, hk, hv, d, d, BF16, 71, True)
    cu, dout = cu_tensor([0, 300, n]), (x[2].float() + 1).to(BF16)
    S, dS = states(2, hv, d, d, 1), states(2, hv, d, d, 2)
    ws = torch.empty(max(G.linear_workspace_size(x[0], x[2], x[3], 2, gradient=b) for b in (False, True)), dtype=torch.uint8, device="cuda")
    out, end, grads = torch.zeros(n, hv, d, dtype=BF16, device="cuda"), torch.zeros_like(S), [torch.zeros_like(t) for t in x]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.linear_forward(*x, cu, S, out=out, final_state=end, workspace=ws)
        d0 = G.linear_backward(*x, cu, dout, S, dS, grads=grads, workspace=ws)[4]
    for lengths in ([0, 300, n], [0, 0, 64], [0, 899, n], [5, 6, 800]):
        cu.copy_(cu_tensor(lengths))
        x[3].mul_(1.3)
        ws.fill_(255)
        for t in (out, *grads):
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        o, e = G.linear_forward(*x, cu, S, out=torch.full_like(out, 5.0))
        w = G.linear_backward(*x, cu, dout, S, dS, grads=[torch.full_like(t, 5.0) for t in x])
        assert torch.equal(out, o) and torch.equal(end, e) and all(torch.equal(a, b) for a, b in zip((*grads, d0), w))


def test_two_streams_at_once(G):  # noqa: F811
    """Calls that overlap, each with a workspace of its own, give what they give alone."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for seed, lengths in ((1, [2000, 48, 4000]), (2, [5000, 0, 333])):
        cu = bounds_of(lengths)
        x = inputs(cu[-1], 2, 4, 64, 64, BF16, seed)
        S, dS = states(3, 4, 64, 64, seed), states(3, 4, 64, 64, seed + 5)
        run = lambda x=x, cu=cu_tensor(cu), S=S, dS=dS: (*G.linear_forward(*x, cu, S), *G.linear_backward(*x, cu, x[2], S, dS))  # noqa: E731
        jobs.append((run, run()))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for side, (run, _) in zip(sides, jobs):
            with torch.cuda.stream(side):
                got.append(run())
        torch.cuda.synchronize()
        for g, (_, want) in zip(got, jobs):
            assert all(torch.equal(a, b) for a, b in zip(g, want))
