"""GPU: linear attention and its gradients with more sequences than a wavefront
has lanes, and with many value heads to a key head, against the definition in
64 bits."""
import random

import pytest
import torch

from tests import linear_reference as L
from tests import seq_reference as R
from tests.test_gpu_linear import G, bounds_of, check, cu_tensor, inputs, reference, states, steps  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def lengths_of(n, seed):
    """Empty ones at both ends, short ones of 0 to 5 tokens, some of several segments among them."""
    rng = random.Random(seed)
    lengths = [rng.randint(0, 5) for _ in range(n)]
    for i in rng.sample(range(2, n - 2), 4):
        lengths[i] = rng.choice([129, 257, 300, 640])
    lengths[:2] = lengths[-2:] = [0, 0]
    return lengths


def gradients(G, x, cu, S0, dS, scale, eps, hv, hk):  # noqa: F811
    """Every gradient against the definition's, in the bounds of test_gpu_linear."""
    dout = (x[2].float() * 0.5 + 1).to(x[2].dtype)
    args, z = [R.f64(t) for t in x], lambda t: R.f64(t).abs()  # noqa: E731
    want = L.packed_grads(*args, cu, R.f64(S0), R.f64(dout), R.f64(dS), scale)
    mag = L.packed_grads(*[t.abs() for t in args[:3]], args[3], cu, z(S0), z(dout), z(dS), scale)
    dq, dk, dv, dg, d0 = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS, scale=scale)
    for got, w, m in ((dq, want[0], mag[0]), (dk, want[1], mag[1]), (dv, want[2], mag[2]), (d0, want[4], mag[4])):
        check(got, w, m, eps + hv // hk)
    terms = (args[2].abs() * mag[2]).sum(-1)
    tail = (z(dS) * reference(x, cu, S0, scale)[3]).sum((-1, -2))
    m = torch.cat([terms[a:b].flip(0).cumsum(0).flip(0) + tail[i] for i, (a, b) in enumerate(zip(cu, cu[1:]))])
    assert (R.f64(dg) - want[3]).norm() <= 2.0 ** -20 * 3 * m.norm()


@pytest.mark.parametrize("n,hk,hv,dtype", [(65, 1, 2, BF16), (130, 2, 2, F32), (700, 1, 1, BF16), (5000, 1, 2, BF16), (4097, 1, 1, F32)])
def test_many_sequences(G, n, hk, hv, dtype):  # noqa: F811
    d, scale = 16, 0.25
    lengths = lengths_of(n, n)
    cu = bounds_of(lengths)
    x = inputs(cu[-1], hk, hv, d, d, dtype, n)
    S0, dS = states(n, hv, d, d, 1), states(n, hv, d, d, 2)
    eps = steps(d, d, lengths)
    o, end, mo, mend = reference(x, cu, S0, scale)
    got, final = G.linear_forward(*x, cu_tensor(cu), S0, scale=scale)
    check(got, o, mo, eps)
    check(final, end, mend, eps)
    gradients(G, x, cu, S0, dS, scale, eps, hv, hk)
    # a pool in place, in any order, with padding and slots that two sequences share
    slots = torch.randperm(n + 9, generator=torch.Generator().manual_seed(n))[:n]
    long = max(range(n), key=lambda i: lengths[i])
    slots[3], slots[n - 4] = -1, slots[long] if long != n - 4 else slots[5]
    pool = states(n + 9, hv, d, d, 3)
    want, rows, mags, mrows = [], R.f64(pool).unbind(), [], R.f64(pool).abs().unbind()
    rows, mrows, args = list(rows), list(mrows), [R.f64(t) for t in x]
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        s, zero = slots[i].item(), torch.zeros(hv, d, d, dtype=torch.float64)
        y, S = L.tokens(*(t[a:b] for t in args), rows[s] if s >= 0 else zero, scale)
        my, mS = L.tokens(*(t[a:b].abs() for t in args[:3]), args[3][a:b], mrows[s] if s >= 0 else zero, scale)
        want.append(y)
        mags.append(my)
        if s >= 0:
            rows[s], mrows[s] = S, mS
    got, same = G.linear_forward(*x, cu_tensor(cu), pool, slots=slots.to(torch.int32).cuda(), scale=scale)
    assert same is pool
    check(got, torch.cat(want), torch.cat(mags), eps + 80)          # the shared slot has a few tokens more behind it
    check(pool, torch.stack(rows), torch.stack(mrows), eps + 80)


@pytest.mark.parametrize("hk,hv,dk,dv,dtype,lengths", [(1, 32, 32, 32, BF16, [500, 0, 40]), (1, 32, 16, 48, F32, [130]), (2, 16, 112, 64, BF16, [200, 190]),
                                                      (1, 8, 128, 128, BF16, [420])])
def test_many_value_heads_of_a_key_head(G, hk, hv, dk, dv, dtype, lengths):  # noqa: F811
    cu, scale = bounds_of(lengths), dk ** -0.5
    x = inputs(cu[-1], hk, hv, dk, dv, dtype, hv + dk)
    S0, dS = states(len(lengths), hv, dk, dv, 1), states(len(lengths), hv, dk, dv, 2)
    eps = steps(dk, dv, lengths)
    o, end, mo, mend = reference(x, cu, S0, scale)
    got, final = G.linear_forward(*x, cu_tensor(cu), S0, scale=scale)
    check(got, o, mo, eps)
    check(final, end, mend, eps)
    gradients(G, x, cu, S0, dS, scale, eps, hv, hk)
