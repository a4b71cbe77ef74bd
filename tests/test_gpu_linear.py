"""GPU: linear attention with a decay over packed sequences and its gradients
against the definition in 64 bits, at the sizes, masks and calls where they can
go wrong."""
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


def bounds_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def cu_tensor(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def inputs(n, hk, hv, dk, dv, dtype, seed, fixed=False, gate=(0.001, 0.1)):
    """q, k, v, log_gate on the GPU."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = [r(n, hk, dk).to(dtype), r(n, hk, dk).to(dtype), r(n, hv, dv).to(dtype),
         -(gate[0] + (gate[1] - gate[0]) * torch.rand((hv,) if fixed else (n, hv), generator=g))]
    return [x.cuda() for x in t]


def states(n, hv, dk, dv, seed):
    return torch.randn(n, hv, dk, dv, generator=torch.Generator().manual_seed(seed)).cuda()


def steps(dk, dv, lengths):
    """Roundings on the way to a value, in half steps of its terms' magnitudes: a dot product over a width, a sum over the 64 tokens
    of a chunk, the decay between two tokens or chunks (the exponent's rounding and exp2's), operands of 24 bits; and for each chunk
    before it that the state has passed, the sum over its tokens and its decay."""
    return 2 * max(dk, dv) + 64 + 40 + 70 * (max(lengths, default=0) // 64 + 1)


def check(got, want, mag, eps, two_terms=False):
    """Within the roundings; bf16 results half a step more, and 2^-16 of the magnitude where operands have two terms.  fp32 results:
    the roundings are independent, so that their 2-norm is far below their bound: 2^-20, 16 half steps."""
    d = (R.f64(got) - want).abs()
    tol = eps * R.HALF[F32] * mag
    if got.dtype == BF16:
        tol = tol + 1.01 * R.HALF[BF16] * want.abs() + (2.0 ** -16 * mag if two_terms else 0)
    assert (d <= tol).all(), (d / tol.clamp_min(1e-300)).max().item()
    if got.dtype == F32 and want.numel() and want.norm() > 0:
        assert d.norm() <= 2.0 ** -20 * mag.norm()


def reference(x, cu, S0, scale):
    args = [R.f64(t) for t in x]
    S = R.f64(S0)
    o, end = L.packed(*args, cu, S, scale)
    mo, mend = L.packed(*[t.abs() for t in args[:3]], args[3], cu, None if S is None else S.abs(), abs(scale))
    return o, end, mo, mend


CASES = [  # lengths, hk, hv, dk, dv, dtype, out_dtype, fixed, with a state
    ([1], 1, 1, 16, 16, F32, F32, False, False), ([5], 2, 2, 32, 64, BF16, F32, False, True),
    ([0, 5, 0, 1], 1, 3, 48, 80, F32, F32, False, True), ([63, 1, 130], 2, 4, 64, 64, BF16, BF16, True, True),
    ([64, 65], 1, 1, 112, 112, BF16, F32, False, False), ([31, 33, 32], 1, 2, 96, 32, F32, F32, True, True),
    ([200], 2, 2, 128, 128, BF16, BF16, False, True), ([129, 3], 1, 2, 128, 16, F32, BF16, False, False),
    ([70, 2], 1, 1, 16, 128, BF16, F32, True, False), ([90], 1, 4, 80, 96, BF16, F32, False, True),
    # several segments: bounds on, before and behind a segment's end, empty sequences between
    ([700], 1, 2, 64, 48, BF16, F32, False, True), ([300, 0, 257, 256, 1], 2, 2, 32, 32, F32, F32, False, True),
    ([255, 513, 0], 1, 2, 128, 112, BF16, F32, True, True), ([600, 40], 1, 1, 112, 128, F32, F32, False, False),
    ([10, 1100], 1, 1, 48, 16, BF16, BF16, False, False)]


@pytest.mark.parametrize("lengths,hk,hv,dk,dv,dtype,out_dtype,fixed,state", CASES)
def test_forward(G, lengths, hk, hv, dk, dv, dtype, out_dtype, fixed, state):
    cu, scale = bounds_of(lengths), dk ** -0.5
    x = inputs(cu[-1], hk, hv, dk, dv, dtype, cu[-1] + dk, fixed)
    S0 = states(len(lengths), hv, dk, dv, 5) if state else None
    o, end, mo, mend = reference(x, cu, S0, scale)
    got, final = G.linear_forward(*x, cu_tensor(cu), S0, scale=scale, out_dtype=out_dtype)
    assert got.dtype == out_dtype and got.shape == (cu[-1], hv, dv) and final.shape == end.shape
    eps = steps(dk, dv, lengths)
    check(got, o, mo, eps, two_terms=dtype == BF16)
    check(final, end, mend, eps)
    # nothing of the call before, and the same bits
    again, last = G.linear_forward(*x, cu_tensor(cu), S0, scale=scale, out_dtype=out_dtype)
    assert torch.equal(again, got) and torch.equal(last, final)


@pytest.mark.parametrize("lengths,hk,hv,dk,dv,dtype,out_dtype,fixed,state", CASES)
def test_backward(G, lengths, hk, hv, dk, dv, dtype, out_dtype, fixed, state):
    cu, scale = bounds_of(lengths), dk ** -0.5
    n = cu[-1]
    x = inputs(n, hk, hv, dk, dv, dtype, n + dk, fixed)
    gen = torch.Generator().manual_seed(n)
    dout = torch.randn(n, hv, dv, generator=gen).to(dtype).cuda()
    S0 = states(len(lengths), hv, dk, dv, 5) if state else None
    dS = states(len(lengths), hv, dk, dv, 6) if state else None
    args = [R.f64(t) for t in x]
    ab = [t.abs() for t in args[:3]] + [args[3]]
    zero = lambda t: None if t is None else R.f64(t).abs()  # noqa: E731
    want = L.packed_grads(*args, cu, R.f64(S0), R.f64(dout), R.f64(dS), scale)
    mag = L.packed_grads(*ab, cu, zero(S0), R.f64(dout).abs(), zero(dS), scale)
    dq, dk_, dv_, dg, d0 = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS, scale=scale)
    eps = steps(dk, dv, lengths) + hv // hk
    check(dq, want[0], mag[0], eps)
    check(dk_, want[1], mag[1], eps, two_terms=dtype == BF16)
    check(dv_, want[2], mag[2], eps)
    if state:
        check(d0, want[4], mag[4], eps)
    else:
        assert d0 is None
    # a gate's gradient: the sums behind its token of q.dq and v.dv of its value head, and <R, S> behind those
    terms = (ab[2] * mag[2]).sum(-1)                                         # [token, value head]; q.dq and v.dv sum to the same
    per_token = torch.cat([torch.stack([terms[t:b].sum(0) for t in range(a, b)]) if b > a else terms[:0] for a, b in zip(cu, cu[1:])])
    tail = 0.0
    if state:
        _, end, _, mend = reference([*x[:3], x[3]], cu, S0, scale)
        tail = (R.f64(dS).abs() * mend).sum((-1, -2))                        # [sequence, value head]
        per_token = per_token + torch.cat([tail[i].expand(b - a, -1) for i, (a, b) in enumerate(zip(cu, cu[1:]))])
    m = 3 * per_token
    if fixed:
        m = m.sum(0)
    assert ((R.f64(dg) - want[3]).abs() <= eps * R.HALF[F32] * m).all()
    assert (R.f64(dg) - want[3]).norm() <= 2.0 ** -20 * m.norm()
    if not state and not fixed:
        starts = [a for a, b in zip(cu, cu[1:]) if b > a]
        assert (dg[starts] == 0).all()
    again = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS, scale=scale)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk_, dv_, dg, d0)) if a is not None)


def test_gradients_are_those_of_differences(G):
    """Central differences in 64 bits of the definition, at values of every input."""
    lengths, hk, hv, dk, dv, scale = [3, 70], 1, 2, 16, 32, 0.3
    cu = bounds_of(lengths)
    x = inputs(cu[-1], hk, hv, dk, dv, F32, 8)
    dout, S0, dS = x[2] * 0.5 + 1, states(2, hv, dk, dv, 1), states(2, hv, dk, dv, 2)
    got = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS, scale=scale)
    args = [R.f64(t) for t in (*x, S0)]
    loss = lambda: sum((a * b).sum() for a, b in zip(L.packed(*args[:4], cu, args[4], scale), (R.f64(dout), R.f64(dS))))  # noqa: E731
    for t, d in zip(args, got):
        flat, h = t.view(-1), 1e-5
        for i in (0, flat.numel() // 3, flat.numel() - 1):
            at = flat[i].item()
            flat[i] = at + h
            up = loss()
            flat[i] = at - h
            diff = (up - loss()).item() / (2 * h)
            flat[i] = at
            # the difference has an error of h^2 and of 2^-53 of the loss over h; the gradient some hundred half steps
            assert abs(R.f64(d).view(-1)[i].item() - diff) <= 1e-4 * (1 + abs(diff))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompts_then_tokens_are_one_sequence(G, dtype):
    """A prompt in parts and then token by token over a pool gives what one call gives."""
    n, hk, hv, d, pool = 400, 1, 2, 64, 5
    x = inputs(n, hk, hv, d, d, dtype, 3)
    whole, end = G.linear_forward(*x, cu_tensor([0, n]), scale=0.1)
    state = states(pool, hv, d, d, 4)
    before = state.clone()
    slots = torch.tensor([3], dtype=torch.int32, device="cuda")
    state[3] = 0
    outs = []
    for a, b in ((0, 300), (300, 395)):
        o, p = G.linear_forward(*(t[a:b] for t in x), cu_tensor([0, b - a]), state, slots=slots, scale=0.1)
        assert p is state
        outs.append(o)
    for t in range(395, 400):
        outs.append(G.linear_decode(*(y[t:t + 1] for y in x), state, slots, scale=0.1))
    rel = (torch.cat(outs) - whole).double().norm() / whole.double().norm()
    assert rel <= 2.0 ** -20 and (state[3] - end[0]).double().norm() <= 2.0 ** -20 * end.double().norm()
    keep = [0, 1, 2, 4]
    assert torch.equal(state[keep], before[keep])


@pytest.mark.parametrize("lengths", [[40, 0, 7, 100, 3], [300, 0, 20, 700, 3]])
def test_pools_repeated_slots_and_padding(G, lengths):
    """Slots in any order; outside the pool: from zero, state dropped; repeated: one after another in place, each from the pool's row
    otherwise; the same with one segment and several."""
    hk, hv, dk, dv, pool = 1, 2, 32, 16, 6
    cu = bounds_of(lengths)
    x = inputs(cu[-1], hk, hv, dk, dv, F32, 12)
    state = states(pool, hv, dk, dv, 7)
    for slots in ([4, 2, 0, 1, 5], [4, 2, -1, 6, 2 ** 31 - 1], [3, 3, 3, 1, 3], [2, 2, 0, 2, 0], [5, 1, 5, 5, 1]):
        s = torch.tensor(slots, dtype=torch.int32, device="cuda")
        # in place
        want, rows = [], [R.f64(state[i]) for i in range(pool)]
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            inside = 0 <= slots[i] < pool
            o, S = L.tokens(*(R.f64(t[a:b]) for t in x), rows[slots[i]] if inside else torch.zeros(hv, dk, dv, dtype=torch.float64), 0.5)
            want.append(o)
            if inside:
                rows[slots[i]] = S
        want, rows = torch.cat(want), torch.stack(rows)
        p = state.clone()
        out, same = G.linear_forward(*x, cu_tensor(cu), p, slots=s, scale=0.5)
        assert same is p
        assert (R.f64(out) - want).norm() <= 2.0 ** -20 * want.norm() and (R.f64(p) - rows).norm() <= 2.0 ** -20 * rows.norm()
        unused = [i for i in range(pool) if i not in slots]
        assert torch.equal(p[unused], state[unused])
        # into another pool
        want, rows = [], {}
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            inside = 0 <= slots[i] < pool
            o, S = L.tokens(*(R.f64(t[a:b]) for t in x), R.f64(state[slots[i]]) if inside else torch.zeros(hv, dk, dv, dtype=torch.float64), 0.5)
            want.append(o)
            if inside:
                rows[slots[i]] = S
        want = torch.cat(want)
        q = torch.full_like(state, 9.0)
        out, _ = G.linear_forward(*x, cu_tensor(cu), state, slots=s, scale=0.5, final_state=q)
        assert (R.f64(out) - want).norm() <= 2.0 ** -20 * want.norm()
        for i in range(pool):
            if i in rows:
                assert (R.f64(q[i]) - rows[i]).norm() <= 2.0 ** -20 * rows[i].norm()
            else:
                assert (q[i] == 9.0).all()
        # without a final state nothing is written
        p = state.clone()
        G.linear_forward(*x, cu_tensor(cu), p, slots=s, scale=0.5, want_state=False)
        assert torch.equal(p, state)


def test_many_sequences_and_heads_with_a_long_one(G):
    """More states between segments than run at once: two vectors a lane in the chain; a pool in place, gradients against the formula's."""
    lengths, hv, d = [700] + [20 + i % 7 for i in range(32)], 16, 64
    cu, n = bounds_of(lengths), len(lengths)
    x = inputs(cu[-1], 8, hv, d, d, BF16, 41)
    S0, dS = states(n, hv, d, d, 1), states(n, hv, d, d, 2)
    o, end, mo, mend = reference(x, cu, S0, 0.125)
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(4)).to(torch.int32).cuda()
    pool = torch.empty_like(S0)
    pool[slots.long()] = S0
    eps = steps(d, d, lengths) + 2
    got, final = G.linear_forward(*x, cu_tensor(cu), pool, slots=slots, scale=0.125)
    assert final.data_ptr() == pool.data_ptr()
    check(got, o, mo, eps)
    check(final[slots.long()], end, mend, eps)
    dout = x[2] + 1
    args = [R.f64(t) for t in x]
    want = L.packed_grads(*args, cu, R.f64(S0), R.f64(dout), R.f64(dS), 0.125)
    mag = L.packed_grads(*[t.abs() for t in args[:3]], args[3], cu, R.f64(S0).abs(), R.f64(dout).abs(), R.f64(dS).abs(), 0.125)
    dq, dk, dv, _, d0 = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS, scale=0.125)
    check(dq, want[0], mag[0], eps)
    check(dk, want[1], mag[1], eps, two_terms=True)
    check(dv, want[2], mag[2], eps)
    check(d0, want[4], mag[4], eps)


def test_in_place_without_slots(G):
    cu, d = bounds_of([700, 0, 30]), 32
    x = inputs(cu[-1], 1, 1, d, d, F32, 2)
    S0 = states(3, 1, d, d, 3)
    want = G.linear_forward(*x, cu_tensor(cu), S0)
    S = S0.clone()
    out, same = G.linear_forward(*x, cu_tensor(cu), S, final_state=S)
    assert same is S and torch.equal(out, want[0]) and torch.equal(S, want[1])
    assert torch.equal(S[1], S0[1])


def test_padded_batches_strides_and_given_tensors(G):
    """Rows behind the last sequence and before the first are left alone; slices of one projection give the same bits."""
    lengths, hk, hv, dk, dv, pad = [300, 5, 290], 2, 4, 32, 48, 9
    cu = bounds_of(lengths)
    n = cu[-1] + pad
    x = inputs(n, hk, hv, dk, dv, BF16, 21)
    for t in x:
        t[cu[-1]:] = float("nan")
    S0, dS = states(3, hv, dk, dv, 1), states(3, hv, dk, dv, 2)
    dout = torch.randn(n, hv, dv, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    out = torch.full((n, hv, dv), 7.0, device="cuda")
    ws = torch.empty(G.linear_workspace_size(x[0], x[2], x[3], 3), dtype=torch.uint8, device="cuda")
    end = torch.empty_like(S0)
    got = G.linear_forward(*x, cu_tensor(cu), S0, out=out, final_state=end, workspace=ws)
    assert got[0] is out and got[1] is end and torch.isfinite(out).all() and (out[cu[-1]:] == 7.0).all()
    gws = torch.full((G.linear_workspace_size(x[0], x[2], x[3], 3, gradient=True),), 255, dtype=torch.uint8, device="cuda")
    grads = [torch.full_like(t, 3.0) for t in x]
    first = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS, grads=grads, workspace=gws)
    for d in grads:
        assert torch.isfinite(d[: cu[-1]]).all() and (d[cu[-1]:] == 3.0).all()
    y = [t[: cu[-1]].contiguous() for t in x]
    alone, last = G.linear_forward(*y, cu_tensor(cu), S0)
    assert torch.equal(alone, out[: cu[-1]]) and torch.equal(last, end)
    row = torch.cat([t.reshape(n, -1) for t in x[:3]] + [torch.full((n, 8), float("nan"), dtype=BF16, device="cuda")], 1)
    q, k, v = (row[:, i:i + h * d].view(n, h, d) for i, h, d in ((0, hk, dk), (hk * dk, hk, dk), (2 * hk * dk, hv, dv)))
    sliced = G.linear_forward(q, k, v, x[3], cu_tensor(cu), S0, out=out.clone())
    assert torch.equal(sliced[0], out) and torch.equal(sliced[1], end)
    grads2 = [torch.full_like(t, 3.0) for t in x]
    second = G.linear_backward(q, k, v, x[3], cu_tensor(cu), dout, S0, dS, grads=grads2)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    # the first sequence begins behind the first rows
    shifted = cu_tensor([c + 4 for c in cu])
    out2 = torch.full((n, hv, dv), 7.0, device="cuda")
    z = [torch.cat([torch.full_like(t[:4], float("nan")), t[:cu[-1]], t[:pad - 4]]) for t in x]
    G.linear_forward(*z, shifted, S0, out=out2)
    assert torch.equal(out2[4: cu[-1] + 4], alone) and (out2[:4] == 7.0).all() and (out2[cu[-1] + 4:] == 7.0).all()


def test_gates_at_their_ends(G):
    """-inf drops what was before, 0 keeps all; a fixed gate is the same as its rows; strong gates."""
    lengths, d = [130, 300], 32
    cu = bounds_of(lengths)
    x = inputs(cu[-1], 1, 2, d, d, F32, 5)
    S0, dS = states(2, 2, d, d, 1), states(2, 2, d, d, 2)
    x[3][7, 0] = x[3][129, 1] = x[3][200, 0] = x[3][cu[1], 1] = float("-inf")
    x[3][20:40] = 0.0
    x[3][300:303] = -50.0
    o, end, mo, mend = reference(x, cu, S0, 1.0)
    eps = steps(d, d, lengths)
    got, final = G.linear_forward(*x, cu_tensor(cu), S0)
    check(got, o, mo, eps)
    check(final, end, mend, eps)
    dout = x[2] + 1
    args = [R.f64(t) for t in x]
    want = L.packed_grads(*args, cu, R.f64(S0), R.f64(dout), R.f64(dS), 1.0)
    mag = L.packed_grads(*[t.abs() for t in args[:3]], args[3], cu, R.f64(S0).abs(), R.f64(dout).abs(), R.f64(dS).abs(), 1.0)
    dq, dk, dv, dg, d0 = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS)
    for a, w, m in ((dq, want[0], mag[0]), (dk, want[1], mag[1]), (dv, want[2], mag[2]), (d0, want[4], mag[4])):
        check(a, w, m, eps)
    assert torch.isfinite(dg).all()
    g = torch.tensor([-0.05, -0.3], device="cuda")
    a = G.linear_forward(*x[:3], g, cu_tensor(cu), S0)
    b = G.linear_forward(*x[:3], g.expand(cu[-1], 2).contiguous(), cu_tensor(cu), S0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = G.linear_backward(*x[:3], g, cu_tensor(cu), dout, S0, dS)
    b = G.linear_backward(*x[:3], g.expand(cu[-1], 2).contiguous(), cu_tensor(cu), dout, S0, dS)
    assert all(torch.equal(a[i], b[i]) for i in (0, 1, 2, 4)) and a[3].shape == (2,)
    assert torch.allclose(a[3].double(), b[3].double().sum(0), rtol=1e-5)


def test_gradients_without_the_initial_states(G):
    """The C entry may leave them out: the other gradients are the same, the gates' to what the sums of the first segments leave."""
    from gated_delta_rule_frame_amd import linear
    lengths, d = [100, 700], 32
    cu = bounds_of(lengths)
    x = inputs(cu[-1], 1, 2, d, d, BF16, 51)
    S0, dS = states(2, 2, d, d, 1), states(2, 2, d, d, 2)
    dout = x[2] + 1
    want = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS)
    bounds = cu_tensor(cu)
    p, device = linear._problem(*x, 1.0, F32, 2)[:2]
    ws, size = linear._space("gdn_linear_workspace_size", p, 1, None, device)
    got = [torch.empty_like(t) for t in want[:4]]
    linear._on(device, G.lib().gdn_linear_backward, p, *(t.data_ptr() for t in x), bounds.data_ptr(), S0.data_ptr(), dout.data_ptr(),
               dS.data_ptr(), *(t.data_ptr() for t in got), None, ws.data_ptr(), size)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want))
    # 2^-22 of q.dq and v.dv at each token, twice their sums' magnitude at most (as in test_backward: 2^-20 of the magnitudes)
    args = [R.f64(t) for t in x]
    mag = L.packed_grads(*[t.abs() for t in args[:3]], args[3], cu, R.f64(S0).abs(), R.f64(dout).abs(), R.f64(dS).abs(), 1.0)
    m = 3 * (args[2].abs() * mag[2]).sum(-1).sum(0)
    assert ((got[3] - want[3]).double().norm(dim=0).cpu() <= 2.0 ** -20 * m).all()


def test_gradients_of_fixed_gates_over_many_tokens(G):
    """Each token's q.dq and v.dv have roundings of 2^-22 of their size at most in the 2-norm, independent ones.  A gate's gradient sums
    what they leave behind every token, up to known ends of segments of at most 512 tokens: a bridge, whose sum has L^2 / 12 of a
    step's variance for each; the ends' own roundings, 2^-22, count L / 2 in the two segments beside them."""
    n, h, d = 20000, 32, 32
    g = torch.tensor([1 - 2.0 ** (-2 - 6 * i / h) for i in range(h)], dtype=torch.float64).log().float().cuda()
    q, k, v, _ = inputs(n, h, h, d, d, BF16, 77)
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(BF16) for t in (q, k))
    dout = inputs(n, h, h, d, d, BF16, 78)[2]
    got = G.linear_backward(q, k, v, g, cu_tensor([0, n]), dout)[3]
    a, (Q, K, V, D) = torch.exp(g.double())[:, None, None], (t.double() for t in (q, k, v, dout))
    S, R = torch.zeros(2, h, d, d, dtype=torch.float64, device="cuda")
    u, w = torch.empty(2, n, h, dtype=torch.float64, device="cuda")
    for t in range(n):
        S = S * a + K[t][:, :, None] * V[t][:, None, :]
        u[t] = (Q[t][:, :, None] * S * D[t][:, None, :]).sum((-1, -2))
        s = n - 1 - t
        R = R * a + Q[s][:, :, None] * D[s][:, None, :] if t else Q[s][:, :, None] * D[s][:, None, :]
        w[s] = (K[s][:, :, None] * R * V[s][:, None, :]).sum((-1, -2))
    dg = (u - w).flip(0).cumsum(0).flip(0)                     # of each token
    dg[0] = 0
    ends = dg[64::64].square().mean(0) * (n / 512)             # <R, S> of the segments' ends, by their mean square
    tol = 2.0 ** -22 * (512.0 ** 2 / 12 * (u * u + w * w).sum(0) + 512.0 ** 2 * ends).sum().sqrt()
    assert (got.double() - dg.sum(0)).norm() <= tol


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_that_drop_the_state_have_no_gradient(G, dtype):
    """exp(log_gate) is 0 in fp32: so is its gradient, exactly, in one segment, in several and for a fixed gate; the others keep theirs."""
    lengths, d = [130, 900], 32
    cu = bounds_of(lengths)
    x = inputs(cu[-1], 1, 2, d, d, dtype, 25)
    dropped = [(7, 0), (129, 1), (200, 0), (130, 1), (640, 1), (900, 0)]
    low = [float("-inf"), torch.finfo(F32).min, -1e4, -105.0, float("-inf"), -200.0]
    for (t, h), g in zip(dropped, low):
        x[3][t, h] = g
    S0, dS = states(2, 2, d, d, 1), states(2, 2, d, d, 2)
    dout = x[2] + 1
    dg = G.linear_backward(*x, cu_tensor(cu), dout, S0, dS)[3]
    args = [R.f64(t) for t in x]
    want = L.packed_grads(*args, cu, R.f64(S0), R.f64(dout), R.f64(dS), 1.0)[3]
    for t, h in dropped:
        assert dg[t, h].item() == 0
    # the sums of q.dq and v.dv behind a token and <R, S> at the end, as in test_backward
    mag = L.packed_grads(*[t.abs() for t in args[:3]], args[3], cu, R.f64(S0).abs(), R.f64(dout).abs(), R.f64(dS).abs(), 1.0)
    terms = (args[2].abs() * mag[2]).sum(-1)
    mend = reference(x, cu, S0, 1.0)[3]
    m = torch.cat([terms[a:b].flip(0).cumsum(0).flip(0) + (R.f64(dS).abs() * mend).sum((-1, -2))[i]
                   for i, (a, b) in enumerate(zip(cu, cu[1:]))])
    assert (R.f64(dg) - want).norm() <= 2.0 ** -20 * 3 * m.norm()
    fixed = torch.tensor([float("-inf"), -0.05], device="cuda")
    dg = G.linear_backward(*x[:3], fixed, cu_tensor(cu), dout, S0, dS)[3]
    assert dg[0].item() == 0 and dg[1].item() != 0


def test_not_finite_values_stay_where_they_are_documented(G):
    """A NaN reaches back at most to its chunk of 64, in the heads that read it and, in v, in its column; other sequences are whole."""
    lengths, hk, hv, d = [200, 90], 2, 4, 32
    cu = bounds_of(lengths)
    for dtype in (BF16, F32):
        x = inputs(cu[-1], hk, hv, d, d, dtype, 9)
        want, end = G.linear_forward(*x, cu_tensor(cu))
        for which, t in (("q", 0), ("k", 1), ("v", 2)):
            y = [a.clone() for a in x]
            y[t][100, 1, 3] = float("nan")
            got, fin = G.linear_forward(*y, cu_tensor(cu))
            same = torch.ones(cu[-1], hv, d, dtype=torch.bool, device="cuda")
            heads = [1] if which == "v" else [2, 3]
            cols = [3] if which == "v" else list(range(d))
            rows = range(100, 101) if which == "q" else range(100, 200) if which == "k" else range(64, 200)
            for h in heads:
                for r in rows:
                    same[r, h, cols] = False
            assert torch.equal(got[same], want[same])
            assert torch.isnan(got[100, heads][:, cols]).all()
            if which != "q":
                assert torch.isnan(got[199, heads][:, cols]).all() and torch.isnan(fin[0, heads][:, :, cols]).any()
            assert torch.equal(fin[1], end[1])
        for value in (float("nan"), float("inf")):             # in k: later tokens alone, also where its products are masked
            y = [a.clone() for a in x]
            y[1][100, 0, 5] = value
            got, _ = G.linear_forward(*y, cu_tensor(cu))
            assert torch.equal(got[:100], want[:100]) and torch.equal(got[200:], want[200:])
        y = [a.clone() for a in x]
        y[3][100, 2] = float("nan")
        got, fin = G.linear_forward(*y, cu_tensor(cu))
        assert torch.equal(got[:100], want[:100]) and torch.equal(got[200:], want[200:]) and torch.equal(got[:, [0, 1, 3]], want[:, [0, 1, 3]])
        assert torch.isnan(got[100:200, 2]).all() and torch.isnan(fin[0, 2]).all()


def test_malformed_offsets_stay_in_range(G):
    """Decreasing or outer offsets are clamped: nothing beside the tensors is written."""
    n, hv, d = 300, 2, 32
    x = inputs(n, 1, hv, d, d, BF16, 1)
    guard = torch.full((n + 128, hv, d), 7.0, device="cuda")
    S = states(3, hv, d, d, 1)
    for cu in ([0, 400, 300, 500], [-5, 10, 5, 300], [250, 20, 299, 1], [2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1]):
        G.linear_forward(*x, cu_tensor(cu), S, out=guard[64: 64 + n])
        grads = [torch.zeros_like(t) for t in x]
        G.linear_backward(*x, cu_tensor(cu), x[2], S, S, grads=grads)
        torch.cuda.synchronize()
        assert (guard[:64] == 7.0).all() and (guard[64 + n:] == 7.0).all()


def test_empty_batches(G):
    x = inputs(0, 1, 2, 32, 32, BF16, 1)
    S = states(2, 2, 32, 32, 1)
    out, end = G.linear_forward(*x, cu_tensor([0, 0, 0]), S)
    assert out.shape == (0, 2, 32) and torch.equal(end, S)
    _, zero = G.linear_forward(*x, cu_tensor([0, 0, 0]))
    assert (zero == 0).all()
    got = G.linear_backward(*x, cu_tensor([0, 0, 0]), x[2], S, S * 2)
    assert torch.equal(got[4], S * 2)
    g = torch.tensor([-0.1, -0.2], device="cuda")
    got = G.linear_backward(*x[:3], g, cu_tensor([0, 0, 0]), x[2])
    assert (got[3] == 0).all()
    got = G.linear_backward(*x[:3], g, cu_tensor([0]), x[2])
    assert (got[3] == 0).all()
    assert G.linear_forward(*x, cu_tensor([0]))[1].shape == (0, 2, 32, 32)


def test_on_another_stream_and_in_graphs(G):
    """Captured calls follow new lengths, gates and values; two graphs on one workspace, run one after the other."""
    n, hk, hv, d = 700, 1, 2, 48
    x = inputs(n, hk, hv, d, d, BF16, 4)
    cu = cu_tensor([0, 300, 700])
    S, dS = states(2, hv, d, d, 1), states(2, hv, d, d, 2)
    dout = (x[2].float() * 0.5).to(BF16)
    want = G.linear_forward(*x, cu, S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = G.linear_forward(*x, cu, S)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    size = max(G.linear_workspace_size(x[0], x[2], x[3], 2), G.linear_workspace_size(x[0], x[2], x[3], 2, gradient=True))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out, end = torch.zeros(n, hv, d, device="cuda"), torch.zeros_like(S)
    grads = [torch.zeros_like(t) for t in x]
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        G.linear_forward(*x, cu, S, out=out, final_state=end, workspace=ws)
    with torch.cuda.graph(b):
        d0 = G.linear_backward(*x, cu, dout, S, dS, grads=grads, workspace=ws)[4]
    for i, lengths in enumerate(([0, 300, 700], [0, 0, 690], [0, 650, 651], [0, 64, 128])):
        cu.copy_(cu_tensor(lengths))
        x[2].mul_(-1.0)
        x[3].mul_(1.1)
        out.fill_(5.0)
        for t in grads:
            t.fill_(5.0)
        a.replay()
        b.replay()
        torch.cuda.synchronize()
        o = torch.full_like(out, 5.0)
        o, e = G.linear_forward(*x, cu, S, out=o)
        w = G.linear_backward(*x, cu, dout, S, dS, grads=[torch.full_like(t, 5.0) for t in x])
        assert torch.equal(out, o) and torch.equal(end, e)
        assert all(torch.equal(s, t) for s, t in zip((*grads, d0), w))


def test_refusals(G):
    x = inputs(10, 2, 4, 32, 32, BF16, 1)
    cu = cu_tensor([0, 4, 10])
    S = states(2, 4, 32, 32, 1)
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in ((x[0], x[1][:, :1].contiguous(), *x[2:]), (x[0].float(), *x[1:]), (*x[:3], x[3].double()), (*x[:3], x[3][:3]),
                (*x[:3], x[3][0, :3].contiguous()), (x[0].half(), x[1].half(), x[2].half(), x[3]), (x[0].cpu(), *x[1:]),
                (x[0][..., :24].contiguous(), x[1][..., :24].contiguous(), *x[2:])):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.linear_forward(*bad, cu, S)
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.linear_backward(*bad, cu, x[2], S)
    for bad in (cu.long(), cu.cpu(), cu[None], cu[:0], cu[::2]):
        with pytest.raises(ValueError):
            G.linear_forward(*x, bad, None)
    for kw in (dict(initial_state=S.double()), dict(initial_state=S[:1].contiguous()), dict(final_state=S[:, :2].contiguous()),
               dict(slots=slots), dict(initial_state=S, slots=slots.long()), dict(initial_state=S, slots=slots[:1]),
               dict(out=torch.zeros(10, 4, 32, device="cuda"), out_dtype=BF16), dict(out=torch.zeros(9, 4, 32, device="cuda")),
               dict(scale=float("inf")), dict(out_dtype=torch.float16)):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.linear_forward(*x, cu, **kw)
    for kw in (dict(dfinal_state=S.double()), dict(grads=[x[0]]), dict(grads=[x[0], x[1], x[2], x[3].double()]), dict(scale=float("nan"))):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.linear_backward(*x, cu, x[2], **kw)
    with pytest.raises((ValueError, TypeError, G.GdnError)):
        G.linear_backward(*x, cu, x[2].float())
    y = inputs(700, 1, 1, 32, 32, BF16, 1)
    with pytest.raises(G.GdnError):
        G.linear_forward(*y, cu_tensor([0, 700]), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(G.GdnError):
        G.linear_backward(*y, cu_tensor([0, 700]), y[2], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
