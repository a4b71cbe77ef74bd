"""The sequence operators' host layer: argument checks, workspace sizes and
calls without work, through the C ABI with pointers that are never used (no
GPU needed), and the binding's refusals."""
import ctypes
import os
import random
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_frame_amd as G
from gated_delta_rule_frame_amd import sequence as Q

FAKE = 0x10000


def seq(**kw):
    base = dict(abi_version=G.ABI_VERSION, heads_k=2, heads_v=4, d_k=64, d_v=64, qkv_dtype=G.BF16, out_dtype=G.BF16,
                state_rows=8, tokens=10, sequences=2)
    base.update(kw)
    p = Q.SeqProblem()
    for n, v in base.items():
        setattr(p, n, v)
    return p


def message():
    return G.lib().gdn_last_error_message().decode()


BAD_SEQ = [("abi_version", 1), ("heads_k", 0), ("heads_k", 3), ("heads_v", 0), ("heads_v", 70000), ("d_k", 8), ("d_k", 24),
           ("d_k", 144), ("d_v", 0), ("d_v", 129), ("qkv_dtype", 5), ("out_dtype", -1), ("tokens", -1), ("tokens", 1 << 31),
           ("q_stride", 127), ("q_stride", 64), ("k_stride", 132), ("v_stride", 255), ("v_stride", -256), ("k_stride", (1 << 23) + 8)]


def call_decode(p, q=FAKE, k=FAKE, v=FAKE, g=FAKE, b=FAKE, state=FAKE, slots=FAKE, out=FAKE):
    return G.lib().gdn_decode(p, q, k, v, g, b, state, slots, out, None)


@pytest.mark.parametrize("field,value", BAD_SEQ + [("state_rows", -1)])
def test_decode_rejects_bad_problems(field, value):
    assert call_decode(seq(**{field: value})) == G.ERR_INVALID_ARGUMENT
    assert message()


def test_decode_rejects_bad_pointers():
    assert G.lib().gdn_decode(None, *[FAKE] * 8, None) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "v", "g", "b", "state", "out"):
        assert call_decode(seq(), **{n: None}) == G.ERR_INVALID_ARGUMENT
        assert call_decode(seq(), **{n: FAKE + 2}) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "v", "state", "out"):
        assert call_decode(seq(), **{n: FAKE + 8}) == G.ERR_INVALID_ARGUMENT
    assert call_decode(seq(), slots=FAKE + 1) == G.ERR_INVALID_ARGUMENT
    p = seq()
    p.reserved[4] = 1
    assert call_decode(p) == G.ERR_INVALID_ARGUMENT


def test_decode_without_rows_does_nothing():
    assert G.lib().gdn_decode(seq(tokens=0), *[None] * 8, None) == G.OK
    assert G.lib().gdn_decode(seq(state_rows=0), *[None] * 5, None, FAKE, None, None) == G.OK


def call_packed(p, ws=FAKE, ws_bytes=1 << 40, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, b=FAKE, cu=FAKE, slots=FAKE, h0=FAKE, out=FAKE, hT=FAKE)
    a.update(kw)
    return G.lib().gdn_packed_forward(p, *a.values(), ws, ws_bytes, None)


@pytest.mark.parametrize("field,value", BAD_SEQ + [("state_rows", -1), ("sequences", -1), ("sequences", 1 << 20)])
def test_packed_rejects_bad_problems(field, value):
    assert call_packed(seq(**{field: value})) == G.ERR_INVALID_ARGUMENT
    n = ctypes.c_size_t()
    assert field == "state_rows" or \
        G.lib().gdn_packed_workspace_size(seq(**{field: value}), 0, ctypes.byref(n)) == G.ERR_INVALID_ARGUMENT


def test_packed_rejects_bad_pointers_and_workspaces():
    for n in ("q", "k", "v", "g", "b", "cu", "out"):
        assert call_packed(seq(), **{n: None}) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "v", "h0", "out", "hT", "ws"):
        assert call_packed(seq(), **{n: FAKE + 8}) == G.ERR_INVALID_ARGUMENT
    for n in ("g", "b", "cu", "slots"):
        assert call_packed(seq(), **{n: FAKE + 2}) == G.ERR_INVALID_ARGUMENT
    n = ctypes.c_size_t()
    assert G.lib().gdn_packed_workspace_size(seq(), 0, None) == G.ERR_INVALID_ARGUMENT
    assert G.lib().gdn_packed_workspace_size(seq(), 0, ctypes.byref(n)) == G.OK and n.value > 0
    assert call_packed(seq(), ws_bytes=n.value - 1) == G.ERR_WORKSPACE_TOO_SMALL
    assert call_packed(seq(), ws=None) == G.ERR_WORKSPACE_TOO_SMALL
    assert call_packed(seq(sequences=0), cu=None) == G.OK


def norm(**kw):
    base = dict(abi_version=G.ABI_VERSION, dtype=G.BF16, batch=3, spatial=5, channels=64, groups=4, activation=1, center=1,
                eps=1e-5)
    base.update(kw)
    p = Q.NormProblem()
    for n, v in base.items():
        setattr(p, n, v)
    return p


@pytest.mark.parametrize("field,value", [
    ("abi_version", 3), ("dtype", 2), ("batch", -1), ("spatial", 0), ("spatial", (1 << 30) + 1), ("channels", 0), ("channels", 66), ("channels", 1 << 25),
    ("groups", 0), ("groups", 5), ("activation", 4), ("activation", -1), ("center", 2), ("eps", float("nan")), ("eps", -1e-5),
    ("batch", 1 << 41)])
def test_norm_rejects_bad_problems(field, value):
    n = ctypes.c_size_t()
    p = norm(**{field: value})
    assert G.lib().gdn_group_norm_workspace_size(p, 0, ctypes.byref(n)) == G.ERR_INVALID_ARGUMENT
    assert message()
    assert G.lib().gdn_group_norm(p, *[FAKE] * 8, 1 << 30, None) == G.ERR_INVALID_ARGUMENT
    assert G.lib().gdn_group_norm_backward(p, *[FAKE] * 12, 1 << 30, None) == G.ERR_INVALID_ARGUMENT


def test_norm_rejects_bad_pointers_and_workspaces():
    L, n = G.lib(), ctypes.c_size_t()
    args = dict(x=FAKE, w=FAKE, b=FAKE, z=FAKE, out=FAKE, mean=FAKE, rstd=FAKE)

    def fwd(p=None, ws=FAKE, ws_bytes=1 << 40, **kw):
        return L.gdn_group_norm(p or norm(), *{**args, **kw}.values(), ws, ws_bytes, None)

    for name in ("x", "out", "rstd", "mean"):
        assert fwd(**{name: None}) == G.ERR_INVALID_ARGUMENT
    for name in args:
        assert fwd(**{name: FAKE + 2}) == G.ERR_INVALID_ARGUMENT
    wide = norm(spatial=5000)            # does not fit registers
    assert L.gdn_group_norm_workspace_size(wide, 0, ctypes.byref(n)) == G.OK and n.value > 0
    assert fwd(wide, ws_bytes=n.value - 1) == G.ERR_WORKSPACE_TOO_SMALL
    assert fwd(wide, ws=None) == G.ERR_WORKSPACE_TOO_SMALL
    for s in (1, 5):
        assert L.gdn_group_norm_workspace_size(norm(spatial=s), 0, ctypes.byref(n)) == G.OK and n.value == 0
    back = dict(dout=FAKE, x=FAKE, w=FAKE, b=FAKE, z=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, db=FAKE, dz=FAKE)

    def bwd(ws_bytes=1 << 40, **kw):
        return L.gdn_group_norm_backward(norm(), *{**back, **kw}.values(), FAKE, ws_bytes, None)

    for name in ("dout", "x", "mean", "rstd", "dx", "z", "dz"):
        assert bwd(**{name: None}) == G.ERR_INVALID_ARGUMENT
    for name in back:
        assert bwd(**{name: FAKE + 8}) == G.ERR_INVALID_ARGUMENT
    assert L.gdn_group_norm_workspace_size(norm(), 1, ctypes.byref(n)) == G.OK
    assert bwd(ws_bytes=n.value - 1) == G.ERR_WORKSPACE_TOO_SMALL


def test_norm_without_rows_does_nothing():
    assert G.lib().gdn_group_norm(norm(batch=0), *[None] * 8, 0, None) == G.OK
    assert G.lib().gdn_group_norm_backward(norm(batch=0), *[None] * 12, 0, None) == G.OK


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 2, 16)
    g = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        G.decode(x, x, x, g, g, torch.zeros(4, 2, 16, 16))
    with pytest.raises(ValueError):
        G.group_norm(x, 2)
    with pytest.raises(ValueError):
        G.group_norm_backward(x, x, 2, g, g)


def test_host_calls_need_no_torch():
    """The library loads, and its host-only calls run, where torch cannot be imported."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "import gated_delta_rule_frame_amd as G\n"
            "p = G.make_problem(1, 2, 64, 64, 2, 880, G.BF16, G.F32)\n"
            "assert G.lib().gdn_abi_version() == G.ABI_VERSION\n"
            "print(G.workspace_size(p), G.segment_plan(p))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=os.path.dirname(os.path.dirname(__file__)))
    assert r.returncode == 0, r.stderr


def test_binding_refuses_sizes_beyond_the_abis_fields():
    """Sizes of 2^31 and more are refused, not cut off to 32 bits (tensors without memory: no GPU needed)."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        f = lambda *s: e(*s, dtype=torch.float32)  # noqa: E731
        i = lambda *s: e(*s, dtype=torch.int32)  # noqa: E731
        big = 2 ** 32 + 16
        for x, groups in ((e(1, big, 1), 1), (e(1, 2 ** 16, 2 ** 16 + 1, 1), 1), (e(1, big), 1), (e(1, 16), big)):
            with pytest.raises(ValueError, match="2.31"):
                G.group_norm(x, groups)
            with pytest.raises(ValueError, match="2.31"):
                G.group_norm_backward(x, x, groups, f(1, groups), f(1, groups))
        q, v, g = e(4, 2, 64), e(4, 2, 64), f(4, 2)
        for bad in ((e(1, big, 16), e(1, big, 16), f(1, big)), (e(1, 1, big), e(1, 1, 16), f(1, 1)), (e(1, 1, 16), e(1, 1, big), f(1, 1))):
            with pytest.raises(ValueError, match="2.31"):
                G.decode(bad[0], bad[0], bad[1], bad[2], bad[2], f(1, 1, 16, 16))
        with pytest.raises(ValueError, match="2.31"):
            G.decode(q, q, v, g, g, f(big, 2, 64, 64), i(4))
        with pytest.raises(ValueError, match="2.31"):
            G.packed_forward(q, q, v, g, g, i(big))
        with pytest.raises(ValueError, match="2.31"):
            G.packed_forward(q, q, v, g, g, i(3), f(big, 2, 64, 64), slots=i(2))
        with pytest.raises(ValueError, match="2.31"):
            G.packed_backward(q, q, v, g, g, i(big), v)
        with pytest.raises(ValueError, match="2.31"):
            G.packed_workspace_size(q, v, big)


def bounds(cu, s, tokens):
    """seq_bounds of gdn_packed.h."""
    a = min(max(cu[s], 0), tokens)
    return a, min(max(cu[s + 1], a), tokens)


def chunk_of(cu, sequences, tokens, slot):
    """find_chunk of gdn_packed.h: (sequence, first row, rows), or None."""
    lo, hi = 0, sequences - 1
    while lo < hi:
        mid = (lo + hi + 1) // 2
        if min(max(cu[mid], 0), tokens) // 64 + mid <= slot:
            lo = mid
        else:
            hi = mid - 1
    a, b = bounds(cu, lo, tokens)
    c = slot - (a // 64 + lo)
    return None if c < 0 or c * 64 >= b - a else (lo, a + c * 64, min(64, b - a - c * 64))


@pytest.mark.parametrize("seed", range(40))
def test_offsets_of_any_value_index_within_rows_and_workspace(seed):
    """The kernels' index arithmetic on offsets of any value: rows within the packed ones, chunk slots within the workspace's;
    on offsets in order every chunk has a slot of its own, and it is the one found from there."""
    r = random.Random(seed)
    tokens, sequences = r.choice([0, 1, 63, 64, 65, 1000]), r.choice([1, 2, 5, 64, 65, 200])
    for kind in range(4):
        cu = [r.choice([r.randint(-5, tokens + 5), r.randint(0, tokens), r.choice([-2 ** 31, 2 ** 31 - 1, -1, 0])])
              if kind else r.randint(0, tokens) for _ in range(sequences + 1)]
        if kind < 2:
            cu.sort()
        slots, seen = tokens // 64 + sequences, {}
        for s in range(sequences):
            a, b = bounds(cu, s, tokens)
            assert 0 <= a <= b <= tokens
            for c in range((b - a + 63) // 64):
                assert 0 <= a // 64 + s + c < slots
                if kind < 2:
                    assert (a // 64 + s + c) not in seen
                    seen[a // 64 + s + c] = (s, a + 64 * c, min(64, b - a - 64 * c))
        for slot in range(slots):
            found = chunk_of(cu, sequences, tokens, slot)
            if found:
                assert 0 <= found[0] < sequences and 0 <= found[1] and 0 < found[2] <= 64 and found[1] + found[2] <= tokens
            if kind < 2:
                assert found == seen.get(slot)


@pytest.mark.parametrize("dtype,t", [(G.BF16, 1), (G.F32, 3)])
def test_packed_workspace_is_what_the_header_says(dtype, t):
    n = ctypes.c_size_t()
    for tokens, sequences, hk, hv, dk, dv in ((1000, 1000, 16, 16, 128, 128), (64, 1, 1, 4, 16, 48), (63, 2, 2, 2, 48, 16), (0, 3, 1, 1, 80, 80)):
        p = seq(tokens=tokens, sequences=sequences, heads_k=hk, heads_v=hv, d_k=dk, d_v=dv, qkv_dtype=dtype)
        slots, D = tokens // 64 + sequences, 32 if dk <= 32 else 64 if dk <= 64 else 128
        for gradient, size in ((0, hv * 49920 + hk * 128 * t * D), (1, hv * (75008 + 512 * dv + 8 * D * dv) + hk * 256 * t * D)):
            assert G.lib().gdn_packed_workspace_size(p, gradient, ctypes.byref(n)) == G.OK and n.value == slots * size


def test_library_loaded_before_torch_shares_its_hip_runtime():
    """One HIP runtime in the process, whichever is loaded first: a second one sees no device."""
    code = ("import gated_delta_rule_frame_amd as G\n"
            "G.lib()\n"
            "import torch\n"
            "paths = {l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}\n"
            "assert len(paths) == 1, paths\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=os.path.dirname(os.path.dirname(__file__)))
    assert r.returncode == 0, r.stderr


def test_packed_workspace_size_refuses_other_types():
    x = torch.zeros(4, 2, 16)
    assert G.packed_workspace_size(x, x, 3) == 3 * (2 * 49920 + 2 * 128 * 3 * 32)
    with pytest.raises(TypeError):
        G.packed_workspace_size(x.half(), x.half(), 3)
