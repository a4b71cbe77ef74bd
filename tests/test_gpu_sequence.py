"""GPU: the sequence operators against float64 references, at the sizes, masks
and calls where they can go wrong."""
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


def unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def rows(n, hk, hv, dk, dv, dtype, seed, gate=(0.001, 0.1)):
    """q, k, v, log_gate, beta on the GPU."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = [unit(r(n, hk, dk)).to(dtype), unit(r(n, hk, dk)).to(dtype), r(n, hv, dv).to(dtype),
         -(gate[0] + (gate[1] - gate[0]) * torch.rand(n, hv, generator=g)), torch.sigmoid(r(n, hv))]
    return [x.cuda() for x in t]


# ------------------------------------------------------------------ decode

def decode_reference(q, k, v, g, b, state, slots):
    """Rows in order; returns (out with None for padding rows, state, bounds of both by magnitude)."""
    q, k, v, g, b, state = (R.f64(x) for x in (q, k, v, g, b, state))
    rep = v.shape[1] // q.shape[1]
    out, mag = [], []
    state, smag = state.clone(), state.abs()
    for i, s in enumerate(slots):
        if not 0 <= s < state.shape[0]:
            out.append(None)
            mag.append(None)
            continue
        o, S = R.tokens(q[i:i + 1], k[i:i + 1], v[i:i + 1], g[i:i + 1], b[i:i + 1], state[s])
        kt, qt = k[i].repeat_interleave(rep, 0).abs(), q[i].repeat_interleave(rep, 0).abs()
        A = smag[s] * torch.exp(g[i])[:, None, None]
        U = b[i].abs()[:, None] * (v[i].abs() + (kt[:, :, None] * A).sum(1))
        smag[s] = A + kt[:, :, None] * U[:, None, :]
        out.append(o[0])
        mag.append((qt[:, :, None] * smag[s]).sum(1))
        state[s] = S
    return out, state, mag, smag


@pytest.mark.parametrize("n,hk,hv,dk,dv,dtype,out_dtype", [
    (1, 1, 1, 16, 16, F32, F32), (1, 20, 20, 112, 112, BF16, BF16), (5, 2, 6, 48, 80, F32, F32), (7, 4, 4, 128, 16, BF16, F32),
    (3, 1, 4, 16, 128, BF16, BF16), (33, 2, 4, 128, 128, BF16, BF16), (2, 3, 3, 96, 112, F32, BF16)])
def test_decode(G, n, hk, hv, dk, dv, dtype, out_dtype):
    x = rows(n, hk, hv, dk, dv, dtype, n)
    gen = torch.Generator().manual_seed(n)
    pool = n + 3
    state = torch.randn(pool, hv, dk, dv, generator=gen).cuda()
    slots = torch.randperm(pool, generator=gen)[:n]
    want, after, mag, smag = decode_reference(*x, state, slots.tolist())
    got = G.decode(*x, state, slots.to(torch.int32).cuda(), out_dtype=out_dtype)
    assert got.dtype == out_dtype and got.shape == (n, hv, dv)
    # every value is at most two sums of d_k products and a few roundings (and exp's two steps) away, each half a step of its
    # magnitude; a bf16 output half a step more
    eps = (2 * dk + 16) * R.HALF[F32]
    assert ((R.f64(state) - after).abs() <= eps * smag).all()
    want, mag = torch.stack(want), torch.stack(mag)
    tol = eps * mag + (R.HALF[BF16] * want.abs() if out_dtype == BF16 else 0)
    assert ((R.f64(got) - want).abs() <= 1.01 * tol).all()


def test_decode_without_slots_is_row_order_and_strided_inputs_give_the_same(G):
    n, hk, hv, dk, dv = 6, 2, 4, 64, 32
    x = rows(n, hk, hv, dk, dv, BF16, 3)
    state = torch.randn(n, hv, dk, dv, device="cuda")
    s1, s2, s3 = state.clone(), state.clone(), state.clone()
    a = G.decode(*x, s1)
    b = G.decode(*x, s2, torch.arange(n, dtype=torch.int32, device="cuda"))
    fused = torch.cat([t.reshape(n, -1) for t in x[:3]] + [torch.full((n, 8), float("nan"), dtype=BF16, device="cuda")], 1)
    q, k, v = (fused[:, i:i + w].view(n, h, d) for i, w, h, d in
               ((0, hk * dk, hk, dk), (hk * dk, hk * dk, hk, dk), (2 * hk * dk, hv * dv, hv, dv)))
    assert not q.is_contiguous()
    c = G.decode(q, k, v, x[3], x[4], s3)
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(s1, s2) and torch.equal(s1, s3)


def test_decode_padding_rows_and_repeated_slots(G):
    """Padding rows leave output and state alone; rows of one slot run in row order, across workgroups' strides."""
    n, hk, hv, dk, dv, pool = 300, 1, 2, 32, 48, 40
    x = rows(n, hk, hv, dk, dv, F32, 11)
    gen = torch.Generator().manual_seed(5)
    slots = torch.randint(-2, pool + 3, (n,), generator=gen)
    slots[7], slots[8], slots[299] = 2 ** 31 - 1, -2 ** 31, 4
    state = torch.randn(pool, hv, dk, dv, generator=gen).cuda()
    want, after, mag, smag = decode_reference(*x, state, slots.tolist())
    out = torch.full((n, hv, dv), 7.0, device="cuda")
    G.decode(*x, state, slots.to(torch.int32).cuda(), out=out)
    times = 8 + max(slots.tolist().count(s) for s in range(pool))   # tokens applied to one state
    eps = times * (2 * dk + 16) * R.HALF[F32]
    assert ((R.f64(state) - after).abs() <= eps * smag).all()
    for i in range(n):
        if want[i] is None:
            assert (out[i] == 7.0).all()
        else:
            assert ((R.f64(out[i]) - want[i]).abs() <= eps * mag[i]).all()


def test_decode_gates_at_their_ends(G):
    """A gate of -inf drops the old state; beta 0 writes nothing; a NaN row stays in its own state."""
    n, d = 4, 32
    x = rows(n, 1, 1, d, d, F32, 2)
    x[3][0] = float("-inf")
    x[4][1] = 0.0
    x[2][2] = float("nan")
    state = torch.randn(n, 1, d, d, device="cuda")
    before = state.clone()
    out = G.decode(*x, state)
    want = x[4][0, 0] * x[1][0, 0][:, None] * x[2][0, 0][None, :]
    assert torch.allclose(state[0, 0], want, rtol=1e-5, atol=1e-6)
    assert torch.allclose(state[1], before[1] * torch.exp(x[3][1, 0]), rtol=1e-6)
    assert torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 3]]).all() and torch.isfinite(state[3]).all()


def test_decode_on_another_stream_and_in_a_graph(G):
    n, hk, hv, dk, dv = 9, 2, 2, 64, 64
    x = rows(n, hk, hv, dk, dv, BF16, 4)
    slots = torch.randperm(n).to(torch.int32).cuda()
    state = torch.randn(n, hv, dk, dv, device="cuda")
    eager, captured = state.clone(), state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = G.decode(*x, eager, slots)
    torch.cuda.current_stream().wait_stream(side)
    out = torch.empty(n, hv, dv, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.decode(*x, captured, slots, out=out)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = first if i == 0 else G.decode(*x, eager, slots)
        assert torch.equal(out, want) and torch.equal(captured, eager)


def test_decode_refuses_what_does_not_fit(G):
    x = rows(4, 2, 4, 32, 32, BF16, 1)
    state = torch.zeros(4, 4, 32, 32, device="cuda")
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ((x[0], x[1][:, :1].contiguous(), *x[2:]), (x[0].float(), *x[1:]), (*x[:3], x[3].double(), x[4]),
                (*x[:2], x[2][:, :3].contiguous(), x[3][:, :3].contiguous(), x[4][:, :3].contiguous()),
                (*x[:4], x[4][:3]), (x[0].half(), x[1].half(), x[2].half(), *x[3:]),
                (x[0].transpose(1, 2).contiguous().transpose(1, 2), *x[1:]), (x[0].cpu(), *x[1:])):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            G.decode(*bad, state, slots)
    for bad in (state.double(), state[:, :2].contiguous(), state[:3].contiguous(), state.transpose(2, 3), state[0]):
        with pytest.raises(ValueError):
            G.decode(*x, bad)
    for bad in (slots.long(), slots[:3], slots.cpu()):
        with pytest.raises(ValueError):
            G.decode(*x, state, bad)
    with pytest.raises((ValueError, TypeError)):
        G.decode(*x, state, slots, out=torch.zeros(4, 4, 32, device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        G.decode(*x, state, slots, out=torch.zeros(4, 4, 32, device="cuda"), out_dtype=BF16)


# ------------------------------------------------------------------ group norm

def norm_inputs(n, s, c, dtype, gate, affine, seed, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *sh: torch.randn(*sh, generator=g)  # noqa: E731
    x = (r(n, s, c) * (0.5 + r(c).abs()) + offset * (1 + r(c).abs())).to(dtype).cuda()
    return (x, (1 + 0.2 * r(c)).cuda() if affine else None, (0.2 * r(c)).cuda() if affine else None,
            r(n, s, c).to(dtype).cuda() if gate else None, r(n, s, c).to(dtype).cuda())


NORMS = [  # n, s, c, groups, dtype, gate, affine, activation, center
    (1, 1, 16, 1, F32, False, True, "none", True), (5, 1, 4096, 32, BF16, True, True, "silu", False),
    (3, 1, 2240, 20, BF16, True, True, "silu", True), (7, 1, 33, 3, F32, False, False, "relu", True),
    (2, 1, 5120, 1, BF16, False, True, "none", False), (2, 1, 16384, 1, BF16, False, True, "gelu", True),
    (2, 1, 16392, 1, BF16, True, True, "silu", True), (300, 1, 258, 2, BF16, True, True, "gelu", True),
    (4, 1, 8, 8, F32, False, True, "none", False), (2, 880, 224, 2, BF16, False, True, "silu", True),
    (3, 7, 40, 5, F32, True, True, "gelu", True), (1, 1000, 129, 3, BF16, True, True, "relu", False),
    (40, 2, 64, 4, BF16, False, False, "silu", True), (2, 33, 2240, 20, F32, False, True, "silu", True),
    (1, 5, 4104, 1, F32, True, False, "silu", False), (1, 4097, 64, 8, BF16, True, True, "silu", True),
    # bands in registers: several n a workgroup, 512 lanes with five passes and with ten, odd widths, walks over n
    (500, 3, 48, 2, F32, True, True, "silu", True), (37, 130, 256, 2, BF16, True, True, "silu", True),
    (5, 200, 512, 4, BF16, False, True, "gelu", False), (200, 2, 1290, 10, BF16, True, True, "relu", True),
    (100, 2, 16384, 2048, BF16, False, True, "silu", True), (4, 64, 32, 4, F32, False, True, "none", False)]


@pytest.mark.parametrize("n,s,c,groups,dtype,gate,affine,activation,center", NORMS)
def test_group_norm_and_its_gradients(G, n, s, c, groups, dtype, gate, affine, activation, center):
    x, w, b, z, dy = norm_inputs(n, s, c, dtype, gate, affine, n * s + c)
    b = b if center else None
    shape = (n, c) if s == 1 else (n, s, c)
    view = lambda t: None if t is None else t.view(shape)  # noqa: E731
    out, mean, rstd = G.group_norm(view(x), groups, w, b, view(z), activation=activation, center=center, eps=1e-5)
    leaves = [None if t is None else R.f64(t).requires_grad_() for t in (x, w, b, z)]
    ro, rm, rr = R.group_norm(leaves[0], groups, *leaves[1:], activation, center, 1e-5)
    # fp32 statistics: a value passes through some 20 roundings and sums whose errors grow like the root of their length;
    # 2e-6 by 2-norm and 3e-5 at any place leave room for the steep part of the activations.  bf16 adds its half step.
    half = R.HALF[dtype] if dtype == BF16 else 0.0

    def near(got, ref, rounded):
        e, m = R.far(got, ref)
        assert e <= 2e-6 + (half if rounded else 0) and m <= 3e-5 + (half if rounded else 0), (e, m)

    assert out.dtype == dtype and out.shape == shape
    near(out.view(n, s, c), ro, True)
    near(rstd, rr, False)
    if center:
        near(mean, rm, False)
    else:
        assert mean is None
    have = [t for t in leaves if t is not None]
    ref = dict(zip([i for i, t in enumerate(leaves) if t is not None], torch.autograd.grad(ro, have, R.f64(dy))))
    got = G.group_norm_backward(view(dy), view(x), groups, mean, rstd, w, b, view(z), activation=activation, center=center)
    for i, (t, d) in enumerate(zip(leaves, got)):
        assert (t is None) == (d is None)
        if t is not None:
            near(d.view(t.shape), ref[i], i in (0, 3))


@pytest.mark.parametrize("s", [1, 50])
def test_group_norm_far_mean_and_constant_groups(G, s):
    """A mean of a thousand deviations does not cancel; a constant group has rstd 1 / sqrt(eps) and output bias."""
    n, c, groups = 4, 64, 4
    x = norm_inputs(n, s, c, F32, False, False, 3)[0] * 0.1 + 100.0
    x[1, :, :16] = 3.25
    w, b = torch.ones(c, device="cuda"), torch.full((c,), 0.5, device="cuda")
    out, mean, rstd = G.group_norm(x, groups, w, b, eps=1e-5)
    ro, rm, rr = R.group_norm(R.f64(x), groups, R.f64(w), R.f64(b), None, "none", True, 1e-5)
    assert R.far(mean, rm)[1] <= 1e-6
    # the mean's own rounding (half a step of 100, 3.8e-6) enters x - mean, which is about 0.1: relative 4e-5
    assert R.far(rstd, rr)[1] <= 1e-4 and R.far(out, ro)[1] <= 2e-4
    assert (out[1, :, :16] == 0.5).all()


def test_group_norm_keeps_nan_and_inf_in_their_group(G):
    for s in (1, 40):
        x = norm_inputs(3, s, 64, BF16, False, False, 9)[0]
        x[1, 0, 3], x[2, s - 1, 40] = float("nan"), float("inf")
        out, mean, rstd = G.group_norm(x, 4, activation="silu")
        bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
        bad[1, 0] = bad[2, 2] = True
        got = torch.isfinite(out.float()).view(3, s, 4, 16)
        assert (got.all(3).all(1) == ~bad).all()
        assert not got[1, :, 0].any() and not torch.isfinite(out[2, s - 1, 40])


def test_group_norm_gradients_against_differences(G):
    x, w, b, z, dy = norm_inputs(3, 6, 48, F32, True, True, 21)
    args = dict(activation="silu", center=True)
    out, mean, rstd = G.group_norm(x, 4, w, b, z, **args)
    grads = G.group_norm_backward(dy, x, 4, mean, rstd, w, b, z, **args)
    g = torch.Generator().manual_seed(1)
    for i, t in enumerate((x, w, b, z)):
        d = torch.randn(t.shape, generator=g).cuda()
        h = 2.0 ** -7
        at = lambda s: [u + s * h * d if j == i else u for j, u in enumerate((x, w, b, z))]  # noqa: E731
        up, dn = (G.group_norm(a[0], 4, *a[1:], **args)[0] for a in (at(1), at(-1)))
        slope = ((up.double() - dn.double()) * dy.double()).sum().item() / (2 * h)
        want = (grads[i].double() * d.double()).sum().item()
        size = (grads[i].double() ** 2).sum().sqrt().item() * (d.double() ** 2).sum().sqrt().item()
        # the third difference: h^2 / 6 times slopes of order one; fp32 steps of the outputs over 2 h
        assert abs(slope - want) <= 2e-3 * size


def test_group_norm_streams_graphs_and_two_calls_with_own_workspaces(G):
    x, w, b, z, dy = norm_inputs(4, 100, 128, BF16, True, True, 2)
    args = dict(activation="silu")
    want = G.group_norm(x, 8, w, b, z, **args)
    wantg = G.group_norm_backward(dy, x, 8, *want[1:], w, b, z, **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = G.group_norm(x, 8, w, b, z, **args)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = G.group_norm(x, 8, w, b, z, **args)
        gotg = G.group_norm_backward(dy, x, 8, *got[1:], w, b, z, **args)
    for _ in range(3):
        for t in (*got, *gotg):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((*got, *gotg), (*want, *wantg)))
        G.group_norm(x, 8, w, b, z, **args)


def test_group_norm_in_two_passes_in_a_graph(G):
    """A group that does not fit registers: several kernels over a workspace, replayed."""
    x, w, b, z, dy = norm_inputs(2, 6000, 32, BF16, True, True, 3)
    args = dict(activation="gelu")
    want = G.group_norm(x, 4, w, b, z, **args)
    wantg = G.group_norm_backward(dy, x, 4, *want[1:], w, b, z, **args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = G.group_norm(x, 4, w, b, z, **args)
        gotg = G.group_norm_backward(dy, x, 4, *got[1:], w, b, z, **args)
    for _ in range(3):
        for t in (*got, *gotg):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((*got, *gotg), (*want, *wantg)))
        G.group_norm(x, 4, w, b, z, **args)


@pytest.mark.parametrize("s", [1, 3, 200, 9000])
def test_group_norm_constant_groups_without_eps(G, s):
    """Nothing to divide by: a deviation of 0 or of its roundings, never the root of a negative number."""
    x = (torch.arange(1, 9, device="cuda").repeat_interleave(16) * 0.37 + 100).repeat(3, s, 1)
    _, mean, rstd = G.group_norm(x, 8, eps=0.0)
    assert (rstd >= 1e4).all() and not torch.isnan(rstd).any()      # inf, or 1 / (some half steps of 103)
    near32(mean, R.f64(x[:, 0].view(3, 8, 16).mean(2)))


def test_group_norm_refuses_what_does_not_fit(G):
    x, w, b, z, dy = norm_inputs(2, 3, 32, BF16, True, True, 1)
    ok = dict(activation="silu")
    for call in (lambda: G.group_norm(x, 5, w), lambda: G.group_norm(x, 4, w.bfloat16()), lambda: G.group_norm(x, 4, w[:16]),
                 lambda: G.group_norm(x, 4, gate=z.float()), lambda: G.group_norm(x, 4, gate=z[:1]),
                 lambda: G.group_norm(x.half(), 4), lambda: G.group_norm(x.transpose(0, 1), 4), lambda: G.group_norm(x[0, 0], 4),
                 lambda: G.group_norm(x, 4, activation="tanh"), lambda: G.group_norm(x, 4, eps=-1.0),
                 lambda: G.group_norm(x, 4, out=torch.empty_like(x.float())), lambda: G.group_norm(x, 0),
                 lambda: G.group_norm(torch.zeros(1, 6000, 32, device="cuda"), 4, workspace=torch.empty(8, device="cuda")),
                 lambda: G.group_norm_backward(dy, x, 4, None, torch.ones(2, 4, device="cuda"), **ok),
                 lambda: G.group_norm_backward(dy, x, 4, torch.ones(2, 4, device="cuda"), torch.ones(2, 4, device="cuda"),
                                               center=False),
                 lambda: G.group_norm_backward(dy.float(), x, 4, torch.ones(2, 4, device="cuda"),
                                               torch.ones(2, 4, device="cuda"))):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            call()


def test_group_norm_without_rows(G):
    x = torch.zeros(0, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    out, mean, rstd = G.group_norm(x, 4, w, w)
    assert out.shape == (0, 32) and rstd.shape == (0, 4)
    dx, dw, db, _ = G.group_norm_backward(x, x, 4, mean, rstd, w, w)
    assert dx.shape == (0, 32) and (dw == 0).all() and (db == 0).all()


# ------------------------------------------------------------------ packed sequences

def near32(got, ref, out_dtype=F32, times=1.0):
    """fp32 products and sums through a chunk: the largest of them sum 128 products, in matrix steps of 32 (errors grow
    like the root: some 12 half steps of the sum of magnitudes), five such products follow one another, and a state passes
    through all chunks, damped by its gates: 64 half steps by 2-norm (4e-6), ten times that at one place.  A bf16 result
    adds its half step."""
    half = R.HALF[out_dtype] if out_dtype == BF16 else 0.0
    e, m = R.far(got, ref)
    assert e <= 64 * R.HALF[F32] * times + half and m <= 640 * R.HALF[F32] * times + half, (e, m)


def cu_of(lengths, device="cuda"):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=device)


PACKED = [  # lengths, hk, hv, dk, dv, dtype, gate range, state
    ([1], 1, 1, 16, 16, BF16, (0.001, 0.1), False), ([64], 2, 2, 64, 64, BF16, (0.001, 0.1), True),
    ([0, 1, 63, 0, 65, 2, 0], 2, 4, 112, 112, BF16, (0.001, 0.1), True), ([200, 3], 1, 3, 128, 128, BF16, (0.0005, 0.02), True),
    ([129], 1, 1, 32, 48, F32, (0.001, 0.1), True), ([70, 130], 2, 2, 128, 96, F32, (0.001, 0.1), True),
    ([257], 1, 2, 80, 16, F32, (0.1, 6.0), False), ([300, 1, 20], 3, 3, 48, 128, BF16, (0.0, 30.0), True),
    ([1000], 1, 1, 64, 32, F32, (0.0, 0.0005), True),
    # more column strips than CUs, an odd number of them in a head: pairs of strips, the last one alone
    ([7, 0, 65, 130, 1] * 9, 2, 4, 48, 48, F32, (0.001, 0.1), True), ([70, 64, 1] * 8, 3, 6, 128, 80, BF16, (0.001, 0.1), True),
    # more pairs of strips than CUs; more sequences than are ordered by length
    ([64, 70, 0, 5, 200] * 6, 2, 4, 112, 112, BF16, (0.001, 0.1), True),
    ([1, 20, 66] * 23, 1, 4, 32, 32, BF16, (0.001, 0.1), True)]


@pytest.mark.parametrize("lengths,hk,hv,dk,dv,dtype,gate,with_state", PACKED)
def test_packed_forward(G, lengths, hk, hv, dk, dv, dtype, gate, with_state):
    n, pad = sum(lengths), 5
    x = rows(n + pad, hk, hv, dk, dv, dtype, n, gate)
    for t in x:
        t[n:] = float("nan")                     # rows behind the last sequence are not read
    S0 = torch.randn(len(lengths), hv, dk, dv, device="cuda") if with_state else None
    cu = cu_of(lengths)
    ro, rS = R.packed(*(R.f64(t) for t in x), cu.tolist(), R.f64(S0))
    for odt in (F32, BF16):
        out = torch.full((n + pad, hv, dv), 3.0, device="cuda", dtype=odt)
        _, S = G.packed_forward(*x, cu, S0, out=out)
        assert (out[n:] == 3.0).all()
        near32(out[:n], ro[:n], odt)
        near32(S, rS)


def test_packed_forward_equals_decode_and_the_dense_forward(G):
    """Token after token through decode, the packed call, and the layer's own forward scan agree."""
    n, h, d = 150, 2, 64
    x = rows(n, h, h, d, d, F32, 8)
    cu = cu_of([n])
    S0 = torch.randn(1, h, d, d, device="cuda")
    out, S = G.packed_forward(*x, cu, S0)
    state, outs = S0.clone(), []
    for t in range(n):
        outs.append(G.decode(*(y[t:t + 1] for y in x), state))
    near32(out, R.f64(torch.cat(outs)))
    near32(S, R.f64(state))
    dense, dS = G.forward(*(y.unsqueeze(0) for y in x), S0, "fwd")
    near32(out, R.f64(dense[0]))
    near32(S, R.f64(dS))


def test_packed_forward_strides_pools_and_repeated_slots(G):
    lengths, hk, hv, dk, dv, pool = [5, 70, 0, 64, 3, 90, 1], 1, 2, 48, 32, 6
    n = sum(lengths)
    x = rows(n, hk, hv, dk, dv, BF16, 6)
    fused = torch.cat([t.reshape(n, -1) for t in x[:3]], 1)
    q, k, v = fused[:, :48].view(n, 1, 48), fused[:, 48:96].view(n, 1, 48), fused[:, 96:].view(n, 2, 32)
    cu = cu_of(lengths)
    slots = [4, 1, 0, 4, -1, 4, 9]
    state = torch.randn(pool, hv, dk, dv, device="cuda")
    before = state.clone()
    ref = R.f64(state)
    outs, c = [], cu.tolist()
    for i, s in enumerate(slots):
        S = ref[s] if 0 <= s < pool else torch.zeros(hv, dk, dv, dtype=torch.float64)
        o, S = R.tokens(*(R.f64(t[c[i]:c[i + 1]]) for t in x), S)
        outs.append(o)
        if 0 <= s < pool:
            ref[s] = S
    st = torch.tensor(slots, dtype=torch.int32, device="cuda")
    out, final = G.packed_forward(q, k, v, x[3], x[4], cu, state, slots=st)
    assert final is state
    near32(out, torch.cat(outs))
    near32(state, ref)
    assert torch.equal(state[[0, 2, 3, 5]], before[[0, 2, 3, 5]])
    other = torch.full_like(state, 2.0)      # from zeros into a pool: the last sequence of a slot stays
    G.packed_forward(q, k, v, x[3], x[4], cu, None, slots=st, final_state=other)
    near32(other[4], R.tokens(*(R.f64(t[c[5]:c[6]]) for t in x), torch.zeros(hv, dk, dv, dtype=torch.float64))[1])
    assert (other[[2, 3, 5]] == 2.0).all() and (other[0] == 0).all()


@pytest.mark.parametrize("times", [2, 3])
def test_packed_forward_many_strips_into_a_pool(G, times):
    """More strips than CUs, an odd number a head, repeated and absent slots: as the sequences one after another."""
    lengths = [65, 3, 0, 128, 20, 1, 70, 64] * times
    hk, hv, dk, dv, pool = 4, 8, 64, 48, 16
    n, c = sum(lengths), cu_of(lengths).tolist()
    x = rows(n, hk, hv, dk, dv, BF16, 61)
    slots = [(5 * i) % 18 - 1 for i in range(len(lengths))]
    state = torch.randn(pool, hv, dk, dv, device="cuda")
    want, outs = state.clone(), []
    for i, s in enumerate(slots):
        at = s if 0 <= s < pool else None
        S = torch.zeros(1, hv, dk, dv, device="cuda") if at is None else want[at:at + 1].clone()
        o, S = G.packed_forward(*(t[c[i]:c[i + 1]] for t in x), cu_of(lengths[i:i + 1]), S)
        outs.append(o)
        if at is not None:
            want[at] = S[0]
    out, _ = G.packed_forward(*x, cu_of(lengths), state, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    near32(out, R.f64(torch.cat(outs)))
    near32(state, R.f64(want))


def test_packed_forward_hard_inputs(G):
    """-inf gates, beta 0, repeated keys and a NaN token: the first two exactly as the recurrence, NaN from its token on."""
    n, d = 140, 32
    x = rows(n, 1, 1, d, d, F32, 14)
    x[3][70], x[3][3] = float("-inf"), float("-inf")
    x[4][10:20] = 0.0
    x[1][30:60] = x[1][30]
    x[4][30:60] = 1.0
    cu = cu_of([n])
    ref = R.packed(*(R.f64(t) for t in x), cu.tolist(), None)
    out, S = G.packed_forward(*x, cu)
    near32(out, ref[0], times=4)       # thirty equal keys: the inverse's entries reach 1 at every distance
    near32(S, ref[1])
    y = [t.clone() for t in x]
    y[2][100] = float("nan")
    out2, S2 = G.packed_forward(*y, cu_of([90, 50]))
    near32(out2[:90], ref[0][:90], times=4)
    assert torch.isnan(out2[100:]).all() and torch.isnan(S2[1]).all()


def test_packed_forward_bad_offsets_stay_in_range(G):
    x = rows(130, 1, 1, 16, 16, BF16, 1)
    out = torch.zeros(130, 1, 16, device="cuda")
    for cu in ([0, 500, 130], [-9, 70, 130], [100, 20, 130], [0, 130, -5], [2 ** 31 - 1, -2 ** 31, 64]):
        G.packed_forward(*x, torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out)
    torch.cuda.synchronize()
    ref = R.packed(*(R.f64(t) for t in x), [0, 64, 130], None)
    near32(G.packed_forward(*x, cu_of([64, 66]))[0], ref[0])


def test_packed_forward_streams_and_graph(G):
    x = rows(333, 2, 4, 64, 64, BF16, 5)
    cu = cu_of([100, 133, 100])
    S0 = torch.randn(3, 4, 64, 64, device="cuda")
    want, wantS = G.packed_forward(*x, cu, S0)
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in sides:                               # two calls at once, each with a workspace of its own
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(G.packed_forward(*x, cu, S0))
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(o, want) and torch.equal(S, wantS) for o, S in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, S = G.packed_forward(*x, cu, S0)
    for _ in range(3):
        out.zero_(), S.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(S, wantS)
        G.packed_forward(*x, cu, S0)


def test_packed_forward_without_tokens_or_sequences(G):
    x = [t[:0] for t in rows(1, 1, 2, 32, 32, BF16, 1)]
    S0 = torch.randn(3, 2, 32, 32, device="cuda")
    out, S = G.packed_forward(*x, cu_of([0, 0, 0]), S0)
    assert out.shape == (0, 2, 32) and torch.equal(S, S0)
    assert (G.packed_forward(*x, cu_of([0]))[1] == 0).all()
    out, S = G.packed_forward(*x, cu_of([]))
    assert S.shape == (0, 2, 32, 32)


def test_packed_forward_refuses_what_does_not_fit(G):
    x = rows(10, 2, 4, 32, 32, BF16, 1)
    cu, S0 = cu_of([4, 6]), torch.zeros(2, 4, 32, 32, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: G.packed_forward(*x, cu.long(), S0), lambda: G.packed_forward(*x, cu.cpu(), S0),
                 lambda: G.packed_forward(*x, [0, 4, 10], S0), lambda: G.packed_forward(*x, cu[:0], S0),
                 lambda: G.packed_forward(*x, cu, S0[:1].contiguous()), lambda: G.packed_forward(*x, cu, S0.bfloat16()),
                 lambda: G.packed_forward(*x, cu, slots=slots), lambda: G.packed_forward(*x, cu, S0, slots=slots[:1]),
                 lambda: G.packed_forward(*x, cu, S0, slots=slots, final_state=torch.zeros(3, 4, 32, 32, device="cuda")),
                 lambda: G.packed_forward(*x, cu, S0, workspace=torch.empty(64, device="cuda")),
                 lambda: G.packed_forward(*(t.half() if i < 3 else t for i, t in enumerate(x)), cu, S0)):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            call()


# ------------------------------------------------------------------ packed gradients

NAMES = ("dq", "dk", "dv", "dlog_gate", "dbeta", "dinitial_state")


def check_grads(got, ref, n, dtype, times=1.0):
    for name, x, r in zip(NAMES, got, ref):
        if x is None:
            continue
        if name != "dinitial_state":
            x, r = x[:n], r[:n]
        try:
            near32(x, r, dtype if name in ("dq", "dk", "dv") else F32, times)
        except AssertionError as e:
            raise AssertionError(f"{name}: {e}") from None


@pytest.mark.parametrize("lengths,hk,hv,dk,dv,dtype,gate,with_state", PACKED)
def test_packed_backward(G, lengths, hk, hv, dk, dv, dtype, gate, with_state):
    n, pad = sum(lengths), 3
    x = rows(n + pad, hk, hv, dk, dv, dtype, n + 1, gate)
    gen = torch.Generator().manual_seed(n)
    x[4][n // 2] = 0.0
    dout = torch.randn(n + pad, hv, dv, generator=gen).to(dtype).cuda()
    for t in (*x, dout):
        t[n:] = float("nan")
    S0 = torch.randn(len(lengths), hv, dk, dv, generator=gen).cuda() if with_state else None
    dS = torch.randn(len(lengths), hv, dk, dv, generator=gen).cuda() if with_state else None
    cu = cu_of(lengths)
    ref = R.packed_grads(*(R.f64(t) for t in x), cu.tolist(), R.f64(S0), R.f64(dout).nan_to_num(), R.f64(dS))
    got = G.packed_backward(*x, cu, dout, S0, dS)
    assert (got[5] is None) == (S0 is None)
    assert [t.dtype for t in got[:5]] == [dtype] * 3 + [F32] * 2
    # a gate's gradient is the difference of sums over its chunk's tokens: some eight times its own size
    check_grads(got, ref, n, dtype, 8.0)


def test_packed_backward_hard_inputs(G):
    """-inf gates (gradient 0), beta 0 and equal keys."""
    n, d = 140, 32
    x = rows(n, 1, 1, d, d, F32, 14)
    x[3][70], x[3][3] = float("-inf"), float("-inf")
    x[4][10:20] = 0.0
    x[1][30:60] = x[1][30]
    x[4][30:60] = 1.0
    cu, dout = cu_of([n]), torch.randn(n, 1, d, device="cuda")
    finite = [t.clone() for t in x]
    finite[3][finite[3] < -1e4] = -1e4         # exp is 0 either way; automatic differentiation needs a finite gate
    ref = R.packed_grads(*(R.f64(t) for t in finite), cu.tolist(), None, R.f64(dout), None)
    got = G.packed_backward(*x, cu, dout)
    check_grads(got, ref, n, F32, 32.0)
    # sums that cancel to zero: within their terms' roundings
    assert got[3][[3, 70]].abs().max() <= 1e-4 * got[3].abs().max()


def test_packed_gradients_against_differences(G):
    """Directional differences of the forward call, with shared heads and states."""
    lengths, hk, hv, dk, dv = [70, 5, 90], 2, 4, 32, 48
    n = sum(lengths)
    x = rows(n, hk, hv, dk, dv, F32, 31)
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    S0, dS, dout, cu = r(3, hv, dk, dv), r(3, hv, dk, dv), r(n, hv, dv), cu_of(lengths)
    grads = G.packed_backward(*x, cu, dout, S0, dS)
    leaves = [*x, S0]
    for i, t in enumerate(leaves):
        d = r(*t.shape) * (0.05 if i in (3, 4) else 1.0)
        h = 2.0 ** -8

        def loss(s):
            y = [u + s * h * d if j == i else u for j, u in enumerate(leaves)]
            out, S = G.packed_forward(*y[:5], cu, y[5])
            return (out.double() * dout).sum().item() + (S.double() * dS).sum().item()

        slope = (loss(1) - loss(-1)) / (2 * h)
        want = (grads[i].double() * d).sum().item()
        size = grads[i].double().norm().item() * d.double().norm().item()
        # the third difference, h^2 / 6 of slopes that grow with the norms, and fp32 steps of the losses over 2 h
        assert abs(slope - want) <= 2e-3 * size, (NAMES[i], slope, want, size)


def test_packed_backward_streams_graph_and_repeats(G):
    x = rows(333, 2, 4, 64, 64, BF16, 5)
    cu = cu_of([100, 133, 100])
    S0, dS = torch.randn(3, 4, 64, 64, device="cuda"), torch.randn(3, 4, 64, 64, device="cuda")
    dout = torch.randn(333, 4, 64, device="cuda").bfloat16()
    want = G.packed_backward(*x, cu, dout, S0, dS)
    same = lambda a: all(torch.equal(i, j) for i, j in zip(a, want))  # noqa: E731
    sides, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(G.packed_backward(*x, cu, dout, S0, dS))
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    assert all(same(g) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = G.packed_backward(*x, cu, dout, S0, dS)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out)
        G.packed_backward(*x, cu, dout, S0, dS)


def test_packed_backward_without_tokens_and_refusals(G):
    x = [t[:0] for t in rows(1, 1, 2, 32, 32, BF16, 1)]
    S0 = torch.randn(2, 2, 32, 32, device="cuda")
    got = G.packed_backward(*x, cu_of([0, 0]), x[2], S0, S0)
    assert torch.equal(got[5], S0) and got[0].shape == (0, 1, 32)
    x = rows(10, 2, 4, 32, 32, BF16, 1)
    cu, S0, dout = cu_of([4, 6]), torch.zeros(2, 4, 32, 32, device="cuda"), torch.zeros(10, 4, 32, device="cuda", dtype=BF16)
    for call in (lambda: G.packed_backward(*x, cu, dout.float()), lambda: G.packed_backward(*x, cu, dout[:9]),
                 lambda: G.packed_backward(*x, cu, dout, S0[:1].contiguous()), lambda: G.packed_backward(*x, cu, dout, S0, S0.bfloat16()),
                 lambda: G.packed_backward(*x, cu.cpu(), dout),
                 lambda: G.packed_backward(*x, cu, dout, workspace=torch.empty(64, device="cuda"))):
        with pytest.raises((ValueError, TypeError, G.GdnError)):
            call()


def test_packed_backward_writes_into_given_tensors(G):
    """A padded batch: given zeroed tensors keep the rows behind the last sequence at zero."""
    x, cu = rows(140, 1, 2, 32, 48, BF16, 9), cu_of([30, 70])
    dout = torch.randn(140, 2, 48, device="cuda").bfloat16()
    want = G.packed_backward(*x, cu, dout)
    mine = [torch.zeros_like(t) for t in x]
    got = G.packed_backward(*x, cu, dout, grads=mine)
    for m, a, b in zip(mine, got, want):
        assert a is m and torch.equal(a[:100], b[:100]) and not a[100:].any()
    for bad in (mine[:4], [*mine[:4], mine[4].bfloat16()], [mine[0][:, :, :16], *mine[1:]], [mine[0].float(), *mine[1:]]):
        with pytest.raises(ValueError):
            G.packed_backward(*x, cu, dout, grads=bad)


def test_packed_backward_strided_inputs(G):
    """q, k and v as slices of one fused projection: the gradients of dense copies, bit for bit."""
    x, cu = rows(150, 2, 4, 48, 64, F32, 10), cu_of([1, 80, 69])
    fused = torch.cat([t.reshape(150, -1) for t in x[:3]], 1)
    q, k, v = fused[:, :96].view(150, 2, 48), fused[:, 96:192].view(150, 2, 48), fused[:, 192:].view(150, 4, 64)
    dout = torch.randn(150, 4, 64, device="cuda")
    for a, b in zip(G.packed_backward(q, k, v, *x[3:], cu, dout)[:5], G.packed_backward(*x, cu, dout)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ together

def test_serving_prompts_then_tokens(G):
    """Prompts into a pool of states, their gated norm, then decoding steps with padding rows and their norm."""
    lengths, hk, hv, d, pool, steps = [70, 1, 130], 2, 4, 64, 5, 3
    n, C = sum(lengths), 4 * 64
    x, cu = rows(n, hk, hv, d, d, BF16, 21), cu_of(lengths)
    gen = torch.Generator().manual_seed(22)
    z = torch.randn(n, C, generator=gen).bfloat16().cuda()
    weight = (1 + 0.1 * torch.randn(C, generator=gen)).cuda()
    state = torch.zeros(pool, hv, d, d, device="cuda")
    slots = [3, 0, 4]
    norm = dict(activation="silu", center=False, eps=1e-6)

    def check(got, o, gate):
        # the output is rounded to bf16 before the norm and after it, and its group's rms moves by at most as much:
        # three half steps; and near32's bound of fp32 errors, 4e-5 of the rms, times weight and gate up to 5
        ref = R.group_norm(o.reshape(-1, 1, C), hv, R.f64(weight), None, R.f64(gate).reshape(-1, 1, C), "silu", False, 1e-6)[0]
        err = (R.f64(got) - ref[:, 0]).abs()
        assert (err <= 3.1 * 2.0 ** -8 * ref[:, 0].abs() + 2e-4).all(), err.max()

    out, _ = G.packed_forward(*x, cu, state, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), out_dtype=BF16)
    y, _, _ = G.group_norm(out.view(n, C), hv, weight, None, z, **norm)
    ref, S = R.packed(*(R.f64(t) for t in x), cu.tolist(), None)
    check(y, ref, z)
    for i in range(steps):
        t = rows(4, hk, hv, d, d, BF16, 30 + i)
        gate = torch.randn(4, C, generator=gen).bfloat16().cuda()
        order = torch.tensor([4, -1, 3, 0], dtype=torch.int32, device="cuda")
        out = G.decode(*t, state, order, out=torch.zeros(4, hv, d, device="cuda", dtype=BF16))
        y, _, _ = G.group_norm(out.view(4, C), hv, weight, None, gate, **norm)
        want = torch.zeros(4, hv, d, dtype=torch.float64)
        for row, seq in ((0, 2), (2, 0), (3, 1)):
            o, S[seq] = R.tokens(*(R.f64(a[row:row + 1]) for a in t), S[seq])
            want[row] = o[0]
        check(y, want, gate)
    near32(state[slots], S, times=2)
    assert not state[[1, 2]].any()


def test_training_through_the_norm(G):
    """Gradients of sum(norm(rule(inputs)) w) through both backward calls, against differentiation in float64."""
    lengths, hk, hv, d = [33, 90], 1, 2, 32
    n, C = sum(lengths), 2 * 32
    x, cu = rows(n, hk, hv, d, d, F32, 41), cu_of(lengths)
    gen = torch.Generator().manual_seed(42)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    z, w, S0, weight = r(n, C), r(n, C), r(2, hv, d, d), 1 + 0.1 * r(C)
    out, _ = G.packed_forward(*x, cu, S0)
    y, mean, rstd = G.group_norm(out.view(n, C), hv, weight, None, z, activation="silu", center=False)
    dout, dw, _, dz = G.group_norm_backward(w, out.view(n, C), hv, None, rstd, weight, None, z, activation="silu", center=False)
    got = G.packed_backward(*x, cu, dout.view(n, hv, d), S0)
    leaves = [R.f64(t).requires_grad_() for t in (*x, S0, weight, z)]
    o, _ = R.packed(*leaves[:5], cu.tolist(), leaves[5])
    f = R.group_norm(o.reshape(n, 1, C), hv, leaves[6], None, leaves[7].reshape(n, 1, C), "silu", False, 1e-5)[0][:, 0]
    near32(y, f.detach())
    want = torch.autograd.grad((f * R.f64(w)).sum(), leaves)
    # the norm's rstd scales the rule's output up by 1 / rms of it: its errors count relative to small outputs
    check_grads(got, want[:6], n, F32, 32.0)
    near32(dw, want[6], times=8)
    near32(dz, want[7], times=8)


# ------------------------------------------------------------------ large tensors

def test_pools_past_32_bits(G):
    """State rows whose offsets pass 2^31 elements (8.8 GB): as in a small pool."""
    hv, d, pool = 32, 128, 4200
    assert (pool - 2) * hv * d * d > 2 ** 31
    state = torch.zeros(pool, hv, d, d, device="cuda")
    small = torch.randn(3, hv, d, d, device="cuda")
    far = [pool - 1, 5, pool - 2]
    state[far] = small
    x = rows(3, 16, hv, d, d, BF16, 51)
    at = lambda s: torch.tensor(s, dtype=torch.int32, device="cuda")  # noqa: E731
    assert torch.equal(G.decode(*x, state, at(far)), G.decode(*x, small, at([0, 1, 2])))
    assert torch.equal(state[far], small)
    x, cu = rows(100, 16, hv, d, d, BF16, 52), cu_of([64, 1, 35])
    a, b = (G.packed_forward(*x, cu, s, slots=at(i))[0] for s, i in ((state, far), (small, [0, 1, 2])))
    assert torch.equal(a, b) and torch.equal(state[far], small)
    assert not state[[0, 4, 6, pool - 3]].any()


def test_packed_rows_past_32_bits(G):
    """Rows whose offsets pass 2^31 elements: the last sequence as in a call of its own, forward and backward."""
    hv, d, each, count = 16, 128, 2048, 520
    n = each * count
    assert (n - each) * hv * d > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    x = [r(n, 1, 16), r(n, 1, 16), r(n, hv, d), torch.full((n, hv), -0.01, device="cuda"), torch.full((n, hv), 0.1, device="cuda")]
    cu, tail = cu_of([each] * count), slice(n - each, n)
    y, one = [t[tail].contiguous() for t in x], cu_of([each])
    out, S = G.packed_forward(*x, cu, out_dtype=BF16)
    want, wantS = G.packed_forward(*y, one, out_dtype=BF16)
    assert torch.equal(out[tail], want) and torch.equal(S[-1:], wantS)
    dout = out
    got = G.packed_backward(*x, cu, dout)
    for a, b in zip(got[:5], G.packed_backward(*y, one, dout[tail].contiguous())):
        assert torch.equal(a[tail], b)


@pytest.mark.parametrize("n,s,c,groups", [(530000, 1, 4096, 32), (300, 8000, 1024, 8)])
def test_group_norm_past_32_bits(G, n, s, c, groups):
    """The last item of more than 2^31 elements as in a call of its own."""
    assert (n - 1) * s * c > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(n, s, c, generator=gen, device="cuda", dtype=BF16)
    y = x[-1:].clone()
    out, mean, rstd = G.group_norm(x, groups)
    ref = R.group_norm(R.f64(y), groups, None, None, None, "none", True, 1e-5)
    near32(mean[-1:], ref[1], times=4)
    near32(rstd[-1:], ref[2], times=4)
    near32(out[-1:], ref[0], BF16)
    dx = G.group_norm_backward(out, x, groups, mean, rstd)[0]
    one = G.group_norm_backward(out[-1:].contiguous(), y, groups, mean[-1:].contiguous(), rstd[-1:].contiguous())[0]
    # both results are rounded to bf16, each by up to half a step of its own value.  Before that, dx cancels (dout is the
    # normalised x itself) and leaves the errors of the mean of dout x^, which is 1: fp32 sums over a million values, in
    # chains of some 1000 additions whose errors grow like the root, 32 half steps, in each call; times x^ up to 6
    a, b = dx[-1:].float(), one.float()
    assert ((a - b).abs() <= 2.0 ** -8 * (a.abs() + b.abs()) + 2 * 32 * 6 * 2.0 ** -24).all()
