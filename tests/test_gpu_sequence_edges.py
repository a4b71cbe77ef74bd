"""GPU: the sequence operators' calls at the edges: every kernel that the dispatch chooses, outputs of both types,
values at the ends of the types' ranges, bad offsets between guards."""
import pytest
import torch

from tests import seq_reference as R
from tests.test_gpu_sequence import BF16, F32, G, NAMES, PACKED, cu_of, near32, rows  # noqa: F401  (G: the fixture)

pytestmark = pytest.mark.gpu


# One, two and more than two strips of 16 columns per CU of 256: a forward kernel each (fp32 inputs share the last two)
STRIPS = [([70, 130], 1, 2, 48, 48), ([70, 1, 64, 90] * 3, 2, 4, 112, 112), ([200, 64, 3] * 10, 2, 4, 128, 96)]


@pytest.mark.parametrize("lengths,hk,hv,dk,dv", STRIPS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_forward_bf16_output_is_the_fp32_output_rounded(G, lengths, hk, hv, dk, dv, dtype):  # noqa: F811
    """The type of the output decides its one rounding and nothing before it."""
    x = rows(sum(lengths), hk, hv, dk, dv, dtype, 71)
    S0 = torch.randn(len(lengths), hv, dk, dv, generator=torch.Generator().manual_seed(72)).cuda()
    a, Sa = G.packed_forward(*x, cu_of(lengths), S0)
    b, Sb = G.packed_forward(*x, cu_of(lengths), S0, out_dtype=BF16)
    assert torch.equal(a.to(BF16), b) and torch.equal(Sa, Sb)


# ------------------------------------------------------------------ activations at the ends of the range

def act_limits(name, u):
    """Value and slope of the activation in float64, with their limits at +-inf."""
    big = u.abs() > 40.0                     # there both are their limits to far below fp32, but for SiLU's tail
    t = torch.where(big, torch.zeros_like(u), u)
    if name == "silu":
        big = u.abs() > 600.0
        t = torch.where(big, torch.zeros_like(u), u)
        s = 1 / (1 + torch.exp(-t))
        value, slope = t * s, s * (1 + t * (1 - s))
    elif name == "gelu":
        c = 0.5 * (1 + torch.erf(t / 2 ** 0.5))
        value, slope = t * c, c + t * torch.exp(-0.5 * t * t) / (2 * torch.pi) ** 0.5
    else:
        value, slope = torch.relu(t), (t > 0).double()
    return torch.where(big, torch.relu(u), value), torch.where(big, (u > 0).double(), slope)


def ends(dtype):
    m = torch.finfo(dtype).max
    return torch.tensor([[-30.0, -88.0, -90.0, -104.0, -1e30, -2.4e38, -m, float("-inf")],
                         [30.0, 88.0, 90.0, 104.0, 1e30, 2.4e38, m, float("inf")]])


def close(got, ref, dtype):
    """The group norm's bound at one place, 3e-5, of the value and of order one, and the output's own rounding."""
    got, ref = R.f64(got), ref.to(torch.float64)
    far = torch.isinf(ref)
    assert torch.equal(got[far], ref[far])
    ok = (got - ref)[~far].abs() <= (3e-5 + (R.HALF[dtype] if dtype == BF16 else 0.0)) * ref[~far].abs() + 3e-5
    assert ok.all(), int((~ok).sum())


@pytest.mark.parametrize("s", [1, 3, 6000])          # a row, a band in registers, two passes
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("activation", ["silu", "gelu", "relu"])
def test_group_norm_activations_at_the_ends_of_the_range(G, s, dtype, activation):  # noqa: F811
    """Gates and activated values up to the type's largest and lowest values and +-inf: a masked gate lets nothing through,
    forward or backward, and no value or slope is NaN."""
    n, c, groups = 2, 32, 4
    gen = torch.Generator().manual_seed(s)
    r = lambda *sh: torch.randn(*sh, generator=gen)  # noqa: E731
    x, dy, gate = r(n, s, c).to(dtype).cuda(), r(n, s, c).to(dtype).cuda(), r(n, s, c).to(dtype)
    gate[:, :, 8:16], gate[:, :, 24:] = ends(dtype)[0].to(dtype), ends(dtype)[1].to(dtype)
    gate = gate.cuda()
    # |x^| < 12 here, weights keep the largest gate's products in range
    w = torch.full((c,), 0.05).cuda()
    out, mean, rstd = G.group_norm(x, groups, w, None, gate, activation=activation)
    dx, dw, _, dz = G.group_norm_backward(dy, x, groups, mean, rstd, w, None, gate, activation=activation)
    X, Y, W, Z = R.f64(x).view(n, s, groups, 8), R.f64(dy).view(n, s, groups, 8), R.f64(w).view(groups, 8), R.f64(gate).view(n, s, groups, 8)
    M = X.mean((1, 3), keepdim=True)
    rs = 1 / torch.sqrt((X - M).square().mean((1, 3), keepdim=True) + 1e-5)
    h = (X - M) * rs
    value, slope = act_limits(activation, Z)
    flat = lambda t: t.reshape(n, s, c)  # noqa: E731
    close(out, flat(h * W * value), dtype)
    close(dz, flat(Y * h * W * slope), dtype)

    def inward(du):
        d = du * W
        return rs * (d - d.mean((1, 3), keepdim=True) - h * (d * h).mean((1, 3), keepdim=True))

    small = [0, 1, 2]                                  # the last group's gradients overflow with its gates
    close(dx.view(n, s, groups, 8)[:, :, small], inward(Y * value)[:, :, small], dtype)
    # ungated, the same values through the bias
    b = torch.cat([r(8), ends(F32)[0], r(8), ends(F32)[1]]).cuda()
    out, mean, rstd = G.group_norm(x, groups, w, b, activation=activation)
    dx, dw, db, _ = G.group_norm_backward(dy, x, groups, mean, rstd, w, b, activation=activation)
    u = (h * W + R.f64(b).view(groups, 8)).float().double()
    value, slope = act_limits(activation, u)
    if dtype == F32:                                   # in bf16 the largest fp32 values round to inf
        close(out, flat(value), dtype)
    else:
        close(out[:, :, :24], flat(value)[:, :, :24], dtype)
        assert not torch.isnan(out).any()
    close(dx, flat(inward(Y * slope)), dtype)
    terms = (Y * slope).abs().sum((0, 1)).reshape(c)
    assert ((R.f64(db) - (Y * slope).sum((0, 1)).reshape(c)).abs() <= 3e-5 * (1 + terms)).all()
    assert torch.isfinite(dw).all()


@pytest.mark.parametrize("s", [1, 3, 6000])
@pytest.mark.parametrize("activation", ["none", "silu", "gelu", "relu"])
def test_group_norm_gate_of_nan(G, s, activation):  # noqa: F811
    """A gate of NaN is NaN in its own place, forward and in the gate's gradient (ReLU's slope there is 0), and nowhere else."""
    x, z = torch.randn(2, s, 32).cuda(), torch.randn(2, s, 32).cuda()
    z[1, s - 1, 7] = float("nan")
    out, mean, rstd = G.group_norm(x, 4, None, None, z, activation=activation)
    bad = torch.isnan(z)
    assert torch.equal(torch.isnan(out), bad)
    dz = G.group_norm_backward(x, x, 4, mean, rstd, None, None, z, activation=activation)[3]
    assert not torch.isnan(dz[~bad]).any()
    assert torch.isnan(dz[bad]).all() == (activation in ("silu", "gelu"))


# ------------------------------------------------------------------ NaN and infinities in a packed batch

@pytest.mark.parametrize("lengths,hk,hv,dk,dv", STRIPS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("where", ["q", "k", "v", "log_gate", "beta"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_packed_forward_bad_value_stays_in_its_chunk_and_heads(G, lengths, hk, hv, dk, dv, dtype, where, value):  # noqa: F811
    """Earlier chunks, other sequences, other value heads and (for v) columns come out bit for bit as without it; from its
    token on it shows as in the recurrence (a q only in its own outputs)."""
    rep = hv // hk
    x = rows(sum(lengths), hk, hv, dk, dv, dtype, 81)
    cu = cu_of(lengths)
    c = cu.tolist()
    s = max(range(len(lengths)), key=lambda i: lengths[i])
    t = c[s] + (lengths[s] - 1) // 64 * 64 + 1                # a token of the last chunk
    want, wantS = G.packed_forward(*x, cu)
    i = ["q", "k", "v", "log_gate", "beta"].index(where)
    bad = [y.clone() for y in x]
    head = hk - 1 if i < 2 else hv - 1
    if i < 3:
        bad[i][t, head, 5] = value
    else:
        bad[i][t, head] = value
    got, gotS = G.packed_forward(*bad, cu)
    heads = slice(head * rep, (head + 1) * rep) if i < 2 else slice(head, head + 1)
    cols = slice(5, 6) if where == "v" else slice(0, dv)
    first = t if where == "q" else c[s] + (t - c[s]) // 64 * 64
    last = t + 1 if where == "q" else c[s + 1]
    reach = torch.zeros_like(got, dtype=torch.bool)
    reach[first:last, heads, cols] = True
    assert torch.equal(got[~reach], want[~reach])
    assert not torch.isfinite(got[t:last, heads, cols]).any()
    states = torch.zeros_like(gotS, dtype=torch.bool)
    states[s, heads, :, cols] = where != "q"
    assert torch.equal(gotS[~states], wantS[~states])
    assert where == "q" or not torch.isfinite(gotS[s, heads, :, cols]).any()


def test_packed_backward_bad_value_stays_in_its_sequence(G):  # noqa: F811
    lengths, hk, hv, dk, dv = [70, 130, 40], 2, 4, 48, 32
    x, cu = rows(240, hk, hv, dk, dv, BF16, 82), cu_of(lengths)
    dout = torch.randn(240, hv, dv).to(BF16).cuda()
    want = G.packed_backward(*x, cu, dout)
    for i in range(6):
        bad = [y.clone() for y in (*x, dout)]
        bad[i][100, 1] = float("nan")
        got = G.packed_backward(*bad[:5], cu, bad[5])
        for a, b in zip(got[:5], want[:5]):
            assert torch.equal(a[:70], b[:70]) and torch.equal(a[200:], b[200:])


# ------------------------------------------------------------------ every kernel that the dispatch chooses

# 257 to 512 strips (the forward scan's pairs, the reverse scan's single strips) at every padded d_k; then key heads enough
# for the gradients' preparation by key head (tokens / 64 + sequences times heads_k from 1024 on), at every padded d_k
CHOSEN = [([1, 20, 66] * 8, 2, 4, 32, 48), ([3, 70, 129] * 3, 4, 8, 64, 64), ([70, 1, 64, 90] * 3, 2, 4, 112, 112),
          ([65, 30] * 5, 4, 4, 128, 128),
          ([1] * 1020 + [70, 2, 140], 1, 2, 16, 16), ([1] * 500 + [64, 0, 130] * 5, 2, 4, 64, 32),
          ([1] * 340 + [70, 3], 3, 6, 112, 48), ([2, 0] * 129 + [65], 4, 16, 128, 16)]


def near_grads(got, ref, q):
    """near32's bound for each gradient but the gates'.  A gate's is the suffix sum over its chunk of q dq + k rows - k cols
    per token, which cancel (one token without a state: to 0).  Its error is that of its terms, so it is counted against
    their size: q dq's, |q dq| summed over d_k, at each place that near32's 64 half steps are for; three terms in place of
    one, and a suffix of up to 64 tokens whose errors grow like the root: 3 sqrt 64 = 24; or, where the gradient is larger,
    eight times against itself, as everywhere."""
    for name, x, r in zip(NAMES, got, ref):
        if x is None:
            continue
        try:
            if name != "dlog_gate":
                near32(x, r, x.dtype)
            else:
                terms = (R.f64(q) * ref[0]).abs().sum(-1).square().mean().sqrt()
                d, own = (R.f64(x) - r).abs(), r.square().mean().sqrt()
                bound = 64 * R.HALF[F32] * max(8 * own, 24 * terms)
                assert d.square().mean().sqrt() <= bound and d.max() <= 10 * bound, (d.max().item(), bound.item())
        except AssertionError as e:
            raise AssertionError(f"{name}: {e}") from None


@pytest.mark.parametrize("lengths,hk,hv,dk,dv", CHOSEN)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_calls_of_every_chosen_kernel(G, lengths, hk, hv, dk, dv, dtype):  # noqa: F811
    n, gen = sum(lengths), torch.Generator().manual_seed(91)
    x, cu = rows(n, hk, hv, dk, dv, dtype, 90), cu_of(lengths)
    S0, dS = (torch.randn(len(lengths), hv, dk, dv, generator=gen).cuda() for _ in range(2))
    dout = torch.randn(n, hv, dv, generator=gen).to(dtype).cuda()
    leaves = [R.f64(t) for t in x]
    ro, rS = R.packed(*leaves, cu.tolist(), R.f64(S0))
    for odt in (F32, BF16):
        out, S = G.packed_forward(*x, cu, S0, out_dtype=odt)
        near32(out, ro, odt)
        near32(S, rS)
    near_grads(G.packed_backward(*x, cu, dout, S0, dS),
               R.packed_grads(*leaves, cu.tolist(), R.f64(S0), R.f64(dout), R.f64(dS)), x[0])


@pytest.mark.parametrize("lengths,hk,hv,dk,dv,dtype,gate,with_state", PACKED)
def test_packed_backward_to_the_last_term(G, lengths, hk, hv, dk, dv, dtype, gate, with_state):  # noqa: F811
    """Each gradient but the gates' to near32's own bound, below what a lost third term of the operands would cost."""
    n, gen = sum(lengths), torch.Generator().manual_seed(sum(lengths))
    x, cu = rows(n, hk, hv, dk, dv, dtype, n + 7, gate), cu_of(lengths)
    dout = torch.randn(n, hv, dv, generator=gen).to(dtype).cuda()
    S0, dS = (torch.randn(len(lengths), hv, dk, dv, generator=gen).cuda() if with_state else None for _ in range(2))
    ref = R.packed_grads(*(R.f64(t) for t in x), cu.tolist(), R.f64(S0), R.f64(dout), R.f64(dS))
    near_grads(G.packed_backward(*x, cu, dout, S0, dS), ref, x[0])


# ------------------------------------------------------------------ bad offsets, between guards

GUARD = 1 << 16


class Guarded:
    """Tensors that lie between bytes of a pattern, and whether those are as they were."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        whole = torch.full((2 * GUARD + (n + 255) // 256 * 256,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((whole, n))
        return whole[GUARD:GUARD + n].view(dtype).view(shape)

    def intact(self):
        return all((w[:GUARD] == 0xA5).all() and (w[GUARD + n:] == 0xA5).all() for w, n in self.all)


def offset_lists(sequences, n):
    gen = torch.Generator().manual_seed(sequences)
    yield torch.randint(-n, 2 * n, (sequences + 1,), generator=gen)
    yield torch.randint(0, n, (sequences + 1,), generator=gen).sort(descending=True)[0]
    yield torch.randint(-2 ** 31, 2 ** 31, (sequences + 1,), generator=gen)
    yield torch.full((sequences + 1,), 2 ** 31 - 1)
    yield torch.tensor([0, n] * sequences)[:sequences + 1]


@pytest.mark.parametrize("sequences,hk,hv,dk,dv", [(3, 1, 2, 16, 48), (40, 2, 4, 48, 64), (70, 2, 4, 112, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_calls_with_bad_offsets_write_nothing_else(G, sequences, hk, hv, dk, dv, dtype):  # noqa: F811
    """Offsets out of order and out of range, forward (with a pool, slots and final states) and backward: every write lies in
    its tensor, and a correct call afterwards gives what it gave before."""
    from gated_delta_rule_frame_amd import sequence as Q
    n, pool = 300, sequences + 2
    x = rows(n, hk, hv, dk, dv, dtype, 95)
    gen = torch.Generator().manual_seed(96)
    S0 = torch.randn(pool, hv, dk, dv, generator=gen).cuda()
    dout = torch.randn(n, hv, dv, generator=gen).to(dtype).cuda()
    slots = torch.randint(-1, pool + 1, (sequences,), generator=gen).to(torch.int32).cuda()
    good = cu_of([n // sequences] * sequences)
    want = G.packed_forward(*x, good, S0[:sequences])
    wantg = G.packed_backward(*x, good, dout, S0[:sequences], S0[:sequences])
    need = [G.packed_workspace_size(x[0], x[2], sequences, gradient=g) for g in (False, True)]
    for cu in offset_lists(sequences, n):
        cu, keep = cu.to(torch.int32).cuda(), Guarded()
        G.packed_forward(*x, cu, S0, slots=slots, out=keep((n, hv, dv), F32), final_state=keep(S0.shape, F32),
                         workspace=keep((need[0],), torch.uint8))
        p, _, _, _, _, _ = Q._problem(*x, F32)
        p.sequences = sequences
        grads = [keep(t.shape, t.dtype) for t in x]
        dS0, ws = keep((sequences, hv, dk, dv), F32), keep((need[1],), torch.uint8)
        assert G.lib().gdn_packed_backward(p, *(t.data_ptr() for t in (*x, cu, S0, dout, S0, *grads, dS0, ws)), need[1],
                                           torch.cuda.current_stream().cuda_stream) == G.OK
        torch.cuda.synchronize()
        assert keep.intact()
    again, againg = G.packed_forward(*x, good, S0[:sequences]), G.packed_backward(*x, good, dout, S0[:sequences], S0[:sequences])
    filled = good[-1].item()
    assert torch.equal(again[0][:filled], want[0][:filled]) and torch.equal(again[1], want[1])
    assert all(torch.equal(a[:filled], b[:filled]) for a, b in zip(againg[:5], wantg)) and torch.equal(againg[5], wantg[5])


# ------------------------------------------------------------------ the most sequences

@pytest.mark.parametrize("dtype,dv", [(BF16, 128), (F32, 128)])
def test_packed_forward_of_the_most_sequences(G, dtype, dv):  # noqa: F811
    """sequences * heads_v = 2^20 (65 to 76 GB of workspace): one token each, o = (q.k) beta v."""
    n, h, dk = 32768, 32, 16
    gen = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    q, k, v, beta = r(n, h, dk), r(n, h, dk), r(n, h, dv), torch.rand(n, h, generator=gen, device="cuda")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out, _ = G.packed_forward(q, k, v, -beta, beta, cu, want_state=False)
    qk = (q.double() * k.double()).sum(-1) * beta.double()
    size = (q.double() * k.double()).abs().sum(-1) * beta.double()
    err = (out.double() - qk[..., None] * v.double()).abs()
    # a product of d_k terms, its gate and beta, each rounded once or twice, on operands split to 24 bits
    assert (err <= (dk + 8) * 2.0 ** -24 * size[..., None] * v.double().abs() + 1e-30).all()
    del out, err
    with pytest.raises(G.GdnError):
        G.packed_forward(q, k, v, -beta, beta, torch.arange(n + 2, dtype=torch.int32, device="cuda"), want_state=False)


def test_packed_backward_of_the_most_sequences(G):  # noqa: F811
    """The same backward (91 GB): dq = beta (v.do) k, dk = beta (v.do) q, dv = beta (q.k) do, dbeta = (q.k) (v.do)."""
    n, h, d = 32768, 32, 16
    gen = torch.Generator(device="cuda").manual_seed(8)
    q, k, v, do = (torch.randn(n, h, d, generator=gen, device="cuda") for _ in range(4))
    beta = torch.rand(n, h, generator=gen, device="cuda")
    got = G.packed_backward(q, k, v, -beta, beta, torch.arange(n + 1, dtype=torch.int32, device="cuda"), do)
    dot = lambda a, b: (a.double() * b.double()).sum(-1)  # noqa: E731
    size = lambda a, b: (a.double() * b.double()).abs().sum(-1)  # noqa: E731
    b, eps = beta.double(), 2 * (d + 8) * 2.0 ** -24
    for x, want, scale in ((got[0], (b * dot(v, do))[..., None] * k.double(), (b * size(v, do))[..., None] * k.double().abs()),
                           (got[1], (b * dot(v, do))[..., None] * q.double(), (b * size(v, do))[..., None] * q.double().abs()),
                           (got[2], (b * dot(q, k))[..., None] * do.double(), (b * size(q, k))[..., None] * do.double().abs()),
                           (got[4], dot(q, k) * dot(v, do), size(q, k) * size(v, do)),
                           (got[3], torch.zeros_like(b), 4 * b * size(q, k) * size(v, do))):
        assert ((x.double() - want).abs() <= eps * scale + 1e-30).all()


# ------------------------------------------------------------------ graphs whose inputs change

def test_captured_calls_follow_new_lengths_slots_and_values(G):  # noqa: F811
    """A graph of a prefill into a pool, a decoding step, their norm and the packed gradients, replayed on other offsets,
    slots (padding and repeated ones among them) and values than it was captured with, two graphs on one workspace."""
    n, hk, hv, d, pool, batch = 300, 2, 4, 64, 9, 6
    gen = torch.Generator().manual_seed(5)
    fresh = lambda seed: (rows(n, hk, hv, d, d, BF16, seed), rows(batch, hk, hv, d, d, BF16, seed + 1))  # noqa: E731
    (x, y), z = fresh(1), torch.randn(batch, hv * d, generator=gen).to(BF16).cuda()
    dout = torch.randn(n, hv, d, generator=gen).to(BF16).cuda()
    cu, slots = cu_of([100, 0, 64, 136]), torch.tensor([3, 1, 0, 5], dtype=torch.int32, device="cuda")
    rows_of = torch.arange(batch, dtype=torch.int32, device="cuda")
    state, first = torch.randn(pool, hv, d, d, generator=gen).cuda(), torch.empty(pool, hv, d, d, device="cuda")
    size = max(G.packed_workspace_size(x[0], x[2], 4, gradient=True), G.packed_workspace_size(x[0], x[2], 4))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def serve(workspace):
        out, _ = G.packed_forward(*x, cu, state, slots=slots, out=torch.zeros(n, hv, d, device="cuda"), workspace=workspace)
        one = G.decode(*y, state, rows_of, out=torch.zeros(batch, hv, d, device="cuda", dtype=BF16))
        return (out, one, *G.group_norm(one.view(batch, hv * d), hv, None, None, z, activation="silu", center=False)[::2])

    def train(workspace):
        grads = [torch.zeros_like(t) for t in x]
        return G.packed_backward(*x, cu, dout, grads=grads, workspace=workspace)[:5]

    first.copy_(state)
    graphs = []
    for f in (serve, train):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = f(ws)
        graphs.append((graph, got))
    plans = [([100, 0, 64, 136], [3, 1, 0, 5], [0, 1, 2, 3, 4, 5]), ([1, 2, 3, 200], [8, 8, -1, 2], [4, -1, 9, 4, 8, 0]),
             ([0, 300, 0, 0], [0, 6, 6, 6], [6] * 6), ([0, 0, 0, 0], [1, 2, 3, 4], [-1] * 6), ([64, 64, 64, 64], [1, 2, 3, 4], [7, 7, 1, 1, 0, 2])]
    for i, (lengths, at, rows_at) in enumerate(plans):
        new = fresh(10 + 2 * i)
        for a, b in zip((*x, *y), (*new[0], *new[1])):
            a.copy_(b)
        cu.copy_(cu_of(lengths)), slots.copy_(torch.tensor(at)), rows_of.copy_(torch.tensor(rows_at))
        state.copy_(first)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        after = state.clone()
        state.copy_(first)
        want = (*serve(None), *train(None))
        for a, b in zip((*graphs[0][1], *graphs[1][1]), want):
            assert torch.equal(a, b)
        assert torch.equal(after, state)
