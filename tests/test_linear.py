"""Linear attention's host layer: argument checks, workspace sizes and calls
without work, through the C ABI with pointers that are never used (no GPU
needed), and the binding's refusals."""
import ctypes
import random

import pytest
import torch

import gated_delta_rule_frame_amd as G
from gated_delta_rule_frame_amd.sequence_abi import LinearProblem

FAKE = 0x10000


def problem(**kw):
    base = dict(abi_version=G.ABI_VERSION, heads_k=2, heads_v=4, d_k=64, d_v=64, qkv_dtype=G.BF16, out_dtype=G.BF16,
                state_rows=8, tokens=10, sequences=2, scale=1.0)
    base.update(kw)
    p = LinearProblem()
    for n, v in base.items():
        setattr(p, n, v)
    return p


BAD = [("abi_version", 1), ("heads_k", 0), ("heads_k", 3), ("heads_v", 0), ("heads_v", 70000), ("d_k", 8), ("d_k", 24), ("d_k", 144),
       ("d_v", 0), ("d_v", 129), ("qkv_dtype", 5), ("out_dtype", -1), ("tokens", -1), ("tokens", 1 << 31), ("q_stride", 127),
       ("q_stride", 64), ("k_stride", 132), ("v_stride", 255), ("v_stride", -256), ("k_stride", (1 << 23) + 8), ("gate_per_head", 2),
       ("gate_per_head", -1), ("scale", float("nan")), ("scale", float("inf"))]


def decode(p, q=FAKE, k=FAKE, v=FAKE, g=FAKE, state=FAKE, slots=FAKE, out=FAKE):
    return G.lib().gdn_linear_decode(p, q, k, v, g, state, slots, out, None)


def forward(p, ws=FAKE, ws_bytes=1 << 40, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, cu=FAKE, slots=FAKE, h0=FAKE, out=FAKE, hT=FAKE)
    a.update(kw)
    return G.lib().gdn_linear_forward(p, *a.values(), ws, ws_bytes, None)


def backward(p, ws=FAKE, ws_bytes=1 << 40, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, cu=FAKE, h0=FAKE, dout=FAKE, dhT=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, dh0=FAKE)
    a.update(kw)
    return G.lib().gdn_linear_backward(p, *a.values(), ws, ws_bytes, None)


def size(p, gradient):
    n = ctypes.c_size_t(12345)
    return G.lib().gdn_linear_workspace_size(p, gradient, ctypes.byref(n)), n.value


@pytest.mark.parametrize("field,value", BAD)
def test_bad_problems_are_refused(field, value):
    p = problem(**{field: value})
    assert decode(p) == forward(p) == backward(p) == size(p, 0)[0] == size(p, 1)[0] == G.ERR_INVALID_ARGUMENT
    assert G.lib().gdn_last_error_message()


def test_bad_counts_and_reserved_fields_are_refused():
    assert decode(problem(state_rows=-1)) == forward(problem(state_rows=-1)) == G.ERR_INVALID_ARGUMENT
    for n in (-1, 1 << 20):
        p = problem(sequences=n)
        assert forward(p) == backward(p) == size(p, 0)[0] == G.ERR_INVALID_ARGUMENT
    p = problem()
    p.reserved[4] = 1
    assert decode(p) == forward(p) == backward(p) == size(p, 1)[0] == G.ERR_INVALID_ARGUMENT
    assert G.lib().gdn_linear_decode(None, *[FAKE] * 7, None) == G.ERR_INVALID_ARGUMENT


def test_bad_pointers_and_workspaces_are_refused():
    p = problem(tokens=5000)
    for n in ("q", "k", "v", "g", "state", "out"):
        assert decode(p, **{n: None}) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "v", "state", "out"):
        assert decode(p, **{n: FAKE + 8}) == G.ERR_INVALID_ARGUMENT
    for n in ("g", "slots"):
        assert decode(p, **{n: FAKE + 2}) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "v", "g", "cu", "out"):
        assert forward(p, **{n: None}) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "v", "h0", "out", "hT", "ws"):
        assert forward(p, **{n: FAKE + 8}) == G.ERR_INVALID_ARGUMENT
    for n in ("g", "cu", "slots"):
        assert forward(p, **{n: FAKE + 2}) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "v", "g", "cu", "dout", "dq", "dk", "dv", "dg"):
        assert backward(p, **{n: None}) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "v", "h0", "dout", "dhT", "dq", "dk", "dv", "dh0", "ws"):
        assert backward(p, **{n: FAKE + 8}) == G.ERR_INVALID_ARGUMENT
    for n in ("g", "cu", "dg"):
        assert backward(p, **{n: FAKE + 2}) == G.ERR_INVALID_ARGUMENT
    assert G.lib().gdn_linear_workspace_size(p, 0, None) == G.ERR_INVALID_ARGUMENT
    for call, gradient in ((forward, 0), (backward, 1)):
        status, need = size(p, gradient)
        assert status == G.OK and need > 0
        assert call(p, ws_bytes=need - 1) == call(p, ws=None) == G.ERR_WORKSPACE_TOO_SMALL
    # one gate a head: its gradient is written even without tokens
    fixed = problem(gate_per_head=1, sequences=0)
    assert backward(fixed, dg=None) == backward(fixed, g=None) == G.ERR_INVALID_ARGUMENT


def test_calls_without_work_do_nothing():
    assert decode(problem(tokens=0), *[None] * 7) == G.OK
    assert decode(problem(state_rows=0), None, None, None, None, None, FAKE, None) == G.OK
    p = problem(sequences=0)
    assert forward(p, cu=None) == backward(p, cu=None) == G.OK
    assert G.lib().gdn_linear_forward(problem(sequences=0, tokens=0), *[None] * 9, None, 0, None) == G.OK


def test_workspaces_hold_what_the_plan_needs():
    """Short calls need none in the forward direction; what is kept between segments is a share of the tokens' own bytes."""
    assert size(problem(tokens=300), 0) == (G.OK, 0)
    rng = random.Random(2)
    for _ in range(300):
        hk = rng.choice([1, 2, 5, 16, 64])
        hv = hk * rng.choice([1, 2, 4])
        dk, dv = 16 * rng.randint(1, 8), 16 * rng.randint(1, 8)
        tokens, seqs = int(2 ** rng.uniform(0, 20)), int(2 ** rng.uniform(0, 12))
        p = problem(heads_k=hk, heads_v=hv, d_k=dk, d_v=dv, tokens=tokens, sequences=seqs, qkv_dtype=rng.randint(0, 1),
                    gate_per_head=rng.randint(0, 1))
        (s0, forward_bytes), (s1, backward_bytes) = size(p, 0), size(p, 1)
        assert s0 == s1 == G.OK
        bounds = tokens // 128                                   # segments have at least 128 tokens
        cell = hv * dk * dv * 4
        assert forward_bytes <= 2 * bounds * cell + (bounds + seqs) * hv * 4 + 1024
        assert backward_bytes <= 2 * (bounds * cell + (bounds + seqs) * hv * 8) + seqs * cell + tokens * (8 * hv + 8 * hk * dk) + 4096
        assert forward_bytes <= backward_bytes + bounds * cell


def test_cpu_tensors_are_refused():
    q, v, g = torch.zeros(4, 2, 32), torch.zeros(4, 4, 32), torch.zeros(4, 4)
    cu, S = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(1, 4, 32, 32)
    for call in (lambda: G.linear_decode(q, q, v, g, S), lambda: G.linear_forward(q, q, v, g, cu), lambda: G.linear_backward(q, q, v, g, cu, v)):
        with pytest.raises(ValueError):
            call()
    assert G.linear_workspace_size(q, v, g, 1) == 0
    with pytest.raises(TypeError):
        G.linear_workspace_size(q.half(), v.half(), g, 1)
    with pytest.raises(ValueError):
        G.linear_workspace_size(q, v, g, 1 << 31)
