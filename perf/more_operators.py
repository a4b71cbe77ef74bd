"""Cases that measure the library's linear attention and rotary positions.

* ``decode``: one token of linear attention with a decay per row, over a pool of states picked by slot (``gdn.linear_decode``).
* ``forward``: the chunked form over sequences packed along the token axis (``gdn.linear_forward``).
* ``backward``: its gradients for every input (``gdn.linear_backward``).
* ``rotary``: rotary positions of queries and keys (``gdn.rotary``).
* ``rotary_grad``: their gradients (``gdn.rotary_backward``).

The recurrence per value head, with a state S of d_k x d_v, a = exp(log_gate) and the head's shared key and query:

    S <- a S + k v^T;   o = scale S^T q

The gate is one for each token and head, or one for each head. Rotary positions turn each pair of components (x, y) of a
query or key by the angle position * frequency of the pair.

``run`` computes it in elementary torch operations, or through the library where ``own`` is true.
"""
import math
import random

import torch

own = False

CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------
# Cases

def _linear(name, kind, tokens, seqs, cut, hk, hv, dk, dv, dtype, state=False, fixed=False, fused=False):
    """``seqs`` sequences of ``tokens`` tokens in all, cut at places that go by ``cut`` (decode: ``tokens`` rows); ``state``: with
    initial states; ``fixed``: one decay for each head; ``fused``: q, k and v are slices of one projection."""
    return {"name": name, "kind": kind, "tokens": tokens, "seqs": seqs, "cut": cut, "hk": hk, "hv": hv, "dk": dk, "dv": dv,
            "dtype": dtype, "state": state, "fixed": fixed, "fused": fused}


def _rotary(name, kind, tokens, hq, hk, d, width, layout, axes, scaling, far, dtype):
    """``width`` of ``d`` components are turned; positions on ``axes`` axes, up to ``far``."""
    return {"name": name, "kind": kind, "tokens": tokens, "hq": hq, "hk": hk, "d": d, "width": width, "layout": layout,
            "axes": axes, "scaling": scaling, "far": far, "dtype": dtype}


def listed():
    return [
        # one user's next token at the layer's own width: latency alone
        _linear("decode_one", "decode", 1, 1, 0, 20, 20, 112, 112, "bf16"),
        # a large serving batch with grouped heads, q, k and v from one projection
        _linear("decode_large", "decode", 440, 1, 0, 16, 32, 128, 128, "bf16", fused=True),
        # a few short prompts that arrived together, one of them a single token, on top of earlier states
        _linear("prompts_short", "forward", 203, 5, 3, 20, 20, 112, 112, "bf16", state=True),
        # a prefill batch of ragged prompts with grouped heads
        _linear("prompts_ragged", "forward", 8191, 13, 1, 16, 32, 128, 128, "bf16", state=True),
        # one long document, a fixed decay for each head
        _linear("document_long", "forward", 32768, 1, 0, 35, 35, 64, 64, "bf16", fixed=True),
        # a small training step in full precision: three clips of unequal length
        _linear("train_short", "backward", 880, 3, 2, 20, 20, 112, 112, "f32", state=True),
        # a packed training batch with grouped heads
        _linear("train_ragged", "backward", 8192, 6, 1, 16, 32, 128, 128, "bf16"),
        # a long training sequence, a fixed decay for each head
        _linear("train_long", "backward", 16384, 1, 0, 35, 35, 64, 64, "bf16", fixed=True),
        # the positions of one decoding step, far into a long context
        _rotary("rotary_tokens", "rotary", 48, 32, 16, 128, 128, "half", 1, "yarn", 1 << 20, "bf16"),
        # a minute of video latents: frame, row and column as three axes
        _rotary("rotary_frames", "rotary", 106480, 20, 20, 112, 112, "interleaved", 3, "none", 121, "bf16"),
        # a packed training batch that turns half of each head
        _rotary("rotary_grad_packed", "rotary_grad", 16384, 32, 16, 128, 64, "half", 1, "linear", 16384, "bf16"),
        # a short clip in full precision
        _rotary("rotary_grad_frames", "rotary_grad", 880, 20, 20, 112, 96, "interleaved", 1, "ntk", 18480, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "forward", "forward", "backward", "rotary", "rotary_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("rotary", "rotary_grad"):
        d = rng.choice([16, 48, 64, 80, 96, 112, 128, 256])
        axes = rng.choice([1, 1, 3])
        width = rng.choice([d, d, d // 2, d - 8])
        hq = rng.choice([1, 3, 8, 20, 32])
        hk = rng.choice([1, 2, hq])
        tokens = _log(rng, 1, (1 << 27) // ((hq + hk) * d))
        case = _rotary("", kind, tokens, hq, hk, d, width, rng.choice(["half", "interleaved"]), axes,
                       rng.choice(["none", "linear", "ntk", "yarn"]), _log(rng, 16, 1 << 21), dtype)
    else:
        hk = rng.choice([1, 2, 4, 8, 16, 20])
        hv = min(32, hk * rng.choice([1, 1, 2, 4]))
        hk = hk if hv % hk == 0 else 1
        dk = rng.choice([16, 48, 64, 80, 96, 112, 128])
        dv = rng.choice([dk, dk, 32, 64, 128])
        if kind == "decode":
            tokens, seqs = _log(rng, 1, 400), 1
        else:
            tokens = _log(rng, 1, 8000)
            seqs = _log(rng, 1, min(24, tokens))
        case = _linear("", kind, tokens, seqs, rng.randrange(1, 1000), hk, hv, dk, dv, dtype, rng.random() < 0.5,
                       rng.random() < 0.3, rng.random() < 0.5)
    del case["name"]
    return case


def _lengths(case):
    """Lengths of the packed sequences: cut at random places, so some are short and one may be empty."""
    r = random.Random(1000003 * case["cut"] + case["seqs"])
    at = sorted(r.randint(0, case["tokens"]) for _ in range(case["seqs"] - 1))
    at = [0] + at + [case["tokens"]]
    return [b - a for a, b in zip(at, at[1:])]


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    t = case["tokens"]
    if case["kind"] in ("rotary", "rotary_grad"):
        x = t * (case["hq"] + case["hk"])
        return {"bytes": 2 * x * case["d"] * b + 4 * t * case["axes"], "flops": 3 * x * case["width"]}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    gates = 4 * hv if case["fixed"] else 4 * hv * t
    qkvo = t * (2 * hk * dk + 2 * hv * dv) * b + gates
    step = t * hv * dk * dv * 2    # one product of a token's row with the state, or one rank-one update
    if case["kind"] == "decode":
        return {"bytes": 2 * t * hv * dk * dv * 4 + qkvo, "flops": 2 * step}
    states = case["seqs"] * hv * dk * dv * 4
    if case["kind"] == "forward":
        return {"bytes": qkvo + states * (2 if case["state"] else 1), "flops": 2 * step}
    grads = t * (2 * hk * dk + hv * dv) * b + gates
    return {"bytes": qkvo + grads + states * (3 if case["state"] else 0), "flops": 5 * step}


# ---------------------------------------------------------------------------------------------------------------
# Inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _unit(g, *shape):
    x = _normal(g, *shape)
    return x / x.square().sum(-1, keepdim=True).sqrt()


def _frequencies(case):
    """Radians per position of each pair and the factor of the turned values, by the way the context was lengthened 8 times."""
    pairs, factor, magnitude = case["width"] // 2, 8.0, 1.0
    i = torch.arange(pairs, dtype=torch.float64)
    base = 10000.0 * factor ** (case["width"] / (case["width"] - 2)) if case["scaling"] == "ntk" and pairs > 1 else 10000.0
    f = base ** (-i / pairs)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "yarn":
        # pairs that turn at most once in the 4096 positions of training are stretched, those of 32 turns and more are kept
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
        magnitude = 0.1 * math.log(factor) + 1
    return f.cuda(), magnitude


def _sections(case):
    """Pairs of each axis."""
    pairs, axes = case["width"] // 2, case["axes"]
    part = pairs // axes
    return [pairs - part * (axes - 1)] + [part] * (axes - 1)


def prepare(case, seed):
    g, ty = torch.Generator(device="cuda"), TYPES[case["dtype"]]
    g.manual_seed(int(seed))
    t = case["tokens"]
    if case["kind"] in ("rotary", "rotary_grad"):
        f, magnitude = _frequencies(case)
        top = torch.tensor([case["far"]] + [24, 44][: case["axes"] - 1], device="cuda")
        positions = (torch.rand((t, case["axes"]), generator=g, device="cuda") * top).to(torch.int32)
        return {"case": case, "q": _normal(g, t, case["hq"], case["d"]).to(ty), "k": _normal(g, t, case["hk"], case["d"]).to(ty),
                "positions": positions[:, 0].contiguous() if case["axes"] == 1 else positions, "frequencies": f,
                "magnitude": magnitude, "sections": _sections(case) if case["axes"] > 1 else None}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    q, k, v = _unit(g, t, hk, dk).to(ty), _unit(g, t, hk, dk).to(ty), _normal(g, t, hv, dv).to(ty)
    if case["fused"]:
        row = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        q, k = row[:, : hk * dk].unflatten(1, (hk, dk)), row[:, hk * dk: 2 * hk * dk].unflatten(1, (hk, dk))
        v = row[:, 2 * hk * dk:].unflatten(1, (hv, dv))
    st = {"case": case, "q": q, "k": k, "v": v, "scale": dk ** -0.5,
          "log_gate": -(0.001 + 0.099 * torch.rand((hv,) if case["fixed"] else (t, hv), generator=g, device="cuda"))}
    if case["kind"] == "decode":
        # a pool with a quarter more slots than rows, the rows' slots scattered over it
        pool = t + (t + 3) // 4
        st["state"] = 0.3 * _normal(g, pool, hv, dk, dv)
        st["slots"] = torch.randperm(pool, generator=g, device="cuda")[:t].to(torch.int32)
        return st
    cu = [0]
    for n in _lengths(case):
        cu.append(cu[-1] + n)
    st["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["longest"] = max(_lengths(case))
    st["initial_state"] = 0.3 * _normal(g, case["seqs"], hv, dk, dv) if case["state"] else None
    if case["kind"] == "backward":
        st["dout"] = _normal(g, t, hv, dv).to(ty)
        st["dfinal_state"] = 0.3 * _normal(g, case["seqs"], hv, dk, dv) if case["state"] else None
    return st


# ---------------------------------------------------------------------------------------------------------------
# Plain forms

def _plain_decode(st):
    rep = st["v"].shape[1] // st["q"].shape[1]
    q, k = (st[x].float().repeat_interleave(rep, 1) for x in ("q", "k"))
    at = st["slots"].long()
    S = st["state"][at] * torch.exp(st["log_gate"])[..., None, None] + k[..., None] * st["v"].float()[..., None, :]
    st["state"][at] = S
    return {"out": (st["scale"] * (q[..., None] * S).sum(2)).to(st["v"].dtype), "state": st["state"]}


def _t(x):
    return x.transpose(-1, -2)


def _chunks(st):
    """The packed rows as chunks [head, chunk, token of the chunk, ...] with zeros behind each sequence's end, what the gates make
    of them, and the state before each chunk: the chunks' own contributions times the matrix of the decays between them."""
    cu = st["cu_seqlens"].long()
    n, rows = cu.shape[0] - 1, st["q"].shape[0]
    slots = rows // CHUNK + n
    starts = cu[:-1] // CHUNK + torch.arange(n, device="cuda")
    slot = torch.arange(slots, device="cuda")
    seq = (torch.searchsorted(starts, slot, right=True) - 1).clamp_min(0)
    at = (cu[seq] + (slot - starts[seq]) * CHUNK)[:, None] + torch.arange(CHUNK, device="cuda")
    valid = (at < cu[seq + 1][:, None]) & (slot >= starts[seq])[:, None]
    index = torch.where(valid, at, torch.zeros_like(at))
    rep = st["v"].shape[1] // st["q"].shape[1]

    def lay(x, r):
        y = x.float()
        y = y.repeat_interleave(r, 1) if r > 1 else y
        y = y[index] * valid.view(valid.shape + (1,) * (x.dim() - 1))
        return y.permute((2, 0, 1) + tuple(range(3, y.dim()))).contiguous()

    def rows_of(y):
        return y.permute((1, 2, 0) + tuple(range(3, y.dim())))[valid]

    q, k, v = lay(st["q"], rep), lay(st["k"], rep), lay(st["v"], 1)
    gate = st["log_gate"] if st["log_gate"].dim() == 2 else st["log_gate"].expand(rows, -1)
    G = lay(gate, 1).double().cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    E = st["scale"] * torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf)).float()
    eG, eD = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    after = G[..., -1].cumsum(-1)                                      # [head, chunk]: gates up to each chunk's end
    before = after - G[..., -1]
    earlier = (seq[:, None] == seq) & (slot[:, None] > slot)
    D = torch.exp((before[..., :, None] - after[..., None, :]).masked_fill(~earlier, -math.inf)).float()
    first = before[:, starts]                                          # [head, sequence]
    last = torch.cat([starts[1:], torch.full_like(starts[:1], slots)]) - 1
    U = _t(k * eD) @ v
    S = (D @ U.flatten(2)).view_as(U)
    h, dk, dv = U.shape[0], U.shape[2], U.shape[3]
    S0 = st["initial_state"]
    if S0 is not None:
        S = S + torch.exp(before - first[:, seq]).float()[..., None, None] * S0.transpose(0, 1)[:, seq]
    own_chunks = seq == torch.arange(n, device="cuda")[:, None]       # [sequence, chunk]
    ends = torch.exp((after[:, last][..., None] - after[:, None, :]).masked_fill(~own_chunks, -math.inf)).float()
    final = (ends @ U.flatten(2)).view(h, n, dk, dv)
    if S0 is not None:
        final = final + torch.exp(after[:, last] - first).float()[..., None, None] * S0.transpose(0, 1)
    return lay, rows_of, rep, seq, last, first, before, after, q, k, v, E, eG, eD, D, U, S, final.transpose(0, 1).contiguous()


def _plain_forward(st):
    _, rows_of, _, _, _, _, _, _, q, k, v, E, eG, _, _, _, S, final = _chunks(st)
    out = st["scale"] * eG * (q @ S) + (E * (q @ _t(k))) @ v
    return {"out": rows_of(out).to(st["v"].dtype), "final_state": final}


def _plain_backward(st):
    lay, rows_of, rep, seq, last, first, before, after, q, k, v, E, eG, eD, D, U, S, _ = _chunks(st)
    do = lay(st["dout"], 1)
    W = st["scale"] * (_t(q * eG) @ do)
    R = (_t(D).contiguous() @ W.flatten(2)).view_as(W)                 # the gradient of the state after each chunk
    dfinal = st["dfinal_state"]
    if dfinal is not None:
        R = R + torch.exp(after[:, last][:, seq] - after).float()[..., None, None] * dfinal.transpose(0, 1)[:, seq]
    A, P = E * (do @ _t(v)), E * (q @ _t(k))
    dq = st["scale"] * eG * (do @ _t(S)) + A @ k
    dk = eD * (v @ _t(R)) + _t(A) @ q
    dv = eD * (k @ R) + _t(P) @ do
    dG = ((q * dq).double().sum(-1) - (v * dv).double().sum(-1))
    end = (R * (eG[:, :, -1:] * S + U)).double().sum((-1, -2))
    dg = rows_of(end[..., None] + dG.sum(-1, keepdim=True) - dG.cumsum(-1) + dG)
    if st["initial_state"] is None:                                    # the first gates of all scale a state of zeros
        starts = torch.zeros(dg.shape[0] + 1, device="cuda", dtype=torch.bool)
        starts[st["cu_seqlens"].long()] = True
        dg = dg * ~starts[:-1, None]
    ty = st["q"].dtype
    got = {"dq": rows_of(dq).unflatten(1, (-1, rep)).sum(2).to(ty), "dk": rows_of(dk).unflatten(1, (-1, rep)).sum(2).to(ty),
           "dv": rows_of(dv).to(ty), "dlog_gate": dg.float() if st["log_gate"].dim() == 2 else dg.sum(0).float()}
    if st["initial_state"] is not None:
        own_chunks = seq == torch.arange(last.shape[0], device="cuda")[:, None]
        whole = torch.exp(before - first[:, seq]).float()[:, None, :] * own_chunks
        d0 = (whole @ W.flatten(2)).unflatten(2, W.shape[2:])
        if dfinal is not None:
            d0 = d0 + torch.exp(after[:, last] - first).float()[..., None, None] * dfinal.transpose(0, 1)
        got["dinitial_state"] = d0.transpose(0, 1).contiguous()
    return got


def _turned(st, x, sign):
    c = st["case"]
    w, p = c["width"], st["positions"].double()
    if p.dim() == 2:
        p = p.repeat_interleave(torch.tensor(st["sections"], device="cuda"), 1)     # each pair's axis
    else:
        p = p[:, None]
    angle = sign * p * st["frequencies"]
    cos, sin = (st["magnitude"] * angle.cos()).float()[:, None], (st["magnitude"] * angle.sin()).float()[:, None]
    y, rest = x[..., :w].float(), x[..., w:]
    if c["layout"] == "half":
        a, b = y[..., : w // 2], y[..., w // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y.to(x.dtype), rest], -1)


def _plain_rotary(st):
    sign = -1 if st["case"]["kind"] == "rotary_grad" else 1
    return {"q": _turned(st, st["q"], sign), "k": _turned(st, st["k"], sign)}


PLAIN = {"decode": _plain_decode, "forward": _plain_forward, "backward": _plain_backward, "rotary": _plain_rotary,
         "rotary_grad": _plain_rotary}


# ---------------------------------------------------------------------------------------------------------------
# The library's calls

def _own_run(st):
    import gated_delta_rule_frame_amd as gdn
    c = st["case"]
    if c["kind"] in ("rotary", "rotary_grad"):
        call = gdn.rotary if c["kind"] == "rotary" else gdn.rotary_backward
        q, k = call(st["q"], st["k"], st["positions"], st["frequencies"], layout=c["layout"], magnitude=st["magnitude"],
                    sections=st["sections"])
        return {"q": q, "k": k}
    x = st["q"], st["k"], st["v"], st["log_gate"]
    if c["kind"] == "decode":
        out = gdn.linear_decode(*x, st["state"], st["slots"], scale=st["scale"], out_dtype=st["v"].dtype)
        return {"out": out, "state": st["state"]}
    if c["kind"] == "forward":
        out, final = gdn.linear_forward(*x, st["cu_seqlens"], st["initial_state"], scale=st["scale"], out_dtype=st["v"].dtype)
        return {"out": out, "final_state": final}
    dq, dk, dv, dg, dS = gdn.linear_backward(*x, st["cu_seqlens"], st["dout"], st["initial_state"], st["dfinal_state"],
                                             scale=st["scale"])
    got = {"dq": dq, "dk": dk, "dv": dv, "dlog_gate": dg}
    if dS is not None:
        got["dinitial_state"] = dS
    return got


def run(state):
    return _own_run(state) if own else PLAIN[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits: token after token, and the turns as products of complex numbers

def _exact_rotary(st):
    c = st["case"]
    p = st["positions"].double().reshape(c["tokens"], c["axes"])
    axis = torch.tensor(sum(([i] * n for i, n in enumerate(st["sections"] or [c["width"] // 2])), []), device="cuda")
    angle = p[:, axis] * st["frequencies"] * (-1 if c["kind"] == "rotary_grad" else 1)
    turn = torch.polar(torch.full_like(angle, st["magnitude"]), angle)[:, None]

    def turned(x):
        y, w = x.double(), c["width"]
        pairs = y[..., :w].unflatten(-1, (2, w // 2)).transpose(-1, -2) if c["layout"] == "half" else y[..., :w].unflatten(-1, (w // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = (z.transpose(-1, -2) if c["layout"] == "half" else z).flatten(-2)
        return torch.cat([z, y[..., w:]], -1)

    return {"q": turned(st["q"]), "k": turned(st["k"])}


def exact(case, seed):
    st = prepare(case, seed)
    rep = st["v"].shape[1] // st["q"].shape[1] if "v" in st else 1
    if case["kind"] in ("rotary", "rotary_grad"):
        return _exact_rotary(st)
    if case["kind"] == "decode":
        at = st["slots"].long()
        state = st["state"].double()
        q, k = (st[x].double().repeat_interleave(rep, 1) for x in ("q", "k"))
        state[at] = state[at] * st["log_gate"].double().exp()[..., None, None] + k[..., :, None] * st["v"].double()[..., None, :]
        return {"out": st["scale"] * (q[..., None, :] @ state[at])[..., 0, :], "state": state}

    # padded [token, sequence, head, ...] tensors; behind a sequence's end the gate is 1 and the rows are 0
    cu, T = st["cu_seqlens"].tolist(), max(1, st["longest"])

    def lay(x, r):
        y = torch.zeros((T, len(cu) - 1, x.shape[1] * r) + tuple(x.shape[2:]), dtype=torch.float64, device="cuda")
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            y[: b - a, i] = x[a:b].double().repeat_interleave(r, 1)
        return y

    def back(y):
        return torch.cat([y[: b - a, i] for i, (a, b) in enumerate(zip(cu, cu[1:]))])

    gate = st["log_gate"] if st["log_gate"].dim() == 2 else st["log_gate"].expand(case["tokens"], -1)
    q, k, v, a = lay(st["q"], rep) * st["scale"], lay(st["k"], rep), lay(st["v"], 1), lay(gate, 1).exp()[..., None, None]
    S = torch.zeros(v.shape[1:3] + (q.shape[-1], v.shape[-1]), dtype=torch.float64, device="cuda")
    S = S if st["initial_state"] is None else st["initial_state"].double()
    step = lambda S, t: S * a[t] + k[t][..., :, None] * v[t][..., None, :]  # noqa: E731
    if case["kind"] == "forward":
        o = torch.empty_like(v)
        for t in range(T):
            S = step(S, t)
            o[t] = (q[t][..., None, :] @ S)[..., 0, :]
        return {"out": back(o), "final_state": S}
    do = lay(st["dout"], 1)
    dS = torch.zeros_like(S) if st["dfinal_state"] is None else st["dfinal_state"].double()
    span, kept = 128, []
    for t in range(T):
        if t % span == 0:
            kept.append(S)
        S = step(S, t)
    dq, dk, dv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(a[..., 0, 0])
    for first in reversed(range(0, T, span)):
        states = [kept[first // span]]
        for t in range(first, min(T, first + span)):
            states.append(step(states[-1], t))
        for t in reversed(range(first, min(T, first + span))):
            dq[t] = (states[t - first + 1] @ do[t][..., None])[..., 0]
            dS = dS + q[t][..., :, None] * do[t][..., None, :]
            dk[t] = (dS @ v[t][..., None])[..., 0]
            dv[t] = (k[t][..., None, :] @ dS)[..., 0, :]
            dS = dS * a[t]
            dg[t] = (dS * states[t - first]).sum((-1, -2))
    shared = lambda x: back(x).unflatten(1, (-1, rep)).sum(2)  # noqa: E731
    dg = back(dg)
    got = {"dq": shared(dq) * st["scale"], "dk": shared(dk), "dv": back(dv),
           "dlog_gate": dg if st["log_gate"].dim() == 2 else dg.sum(0)}
    if st["initial_state"] is not None:
        got["dinitial_state"] = dS
    return got
