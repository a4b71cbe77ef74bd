"""Rotary positions on the host: argument checks through the C ABI with pointers
that are never used, the binding's refusals, and the frequencies (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_frame_amd as G
from gated_delta_rule_frame_amd.sequence_abi import RotaryProblem

FAKE = 0x10000


def problem(**kw):
    base = dict(abi_version=G.ABI_VERSION, dtype=G.BF16, tokens=10, heads_q=4, heads_k=2, width=64, pairs=32, layout=0, inverse=0,
                axes=1, sections=(32, 0, 0, 0), magnitude=1.0)
    base.update(kw)
    p = RotaryProblem()
    for n, v in base.items():
        setattr(p, n, (ctypes.c_int32 * 4)(*v) if n == "sections" else v)
    return p


def call(p, **kw):
    a = dict(q=FAKE, k=FAKE, positions=FAKE, frequencies=FAKE, qo=FAKE, ko=FAKE)
    a.update(kw)
    return G.lib().gdn_rotary(p, *a.values(), None)


@pytest.mark.parametrize("fields", [
    dict(abi_version=1), dict(dtype=2), dict(tokens=-1), dict(tokens=1 << 31), dict(heads_q=0), dict(heads_q=70000),
    dict(heads_k=-1), dict(heads_k=65536), dict(width=4), dict(width=60), dict(width=1032), dict(pairs=0), dict(pairs=33),
    dict(layout=2), dict(layout=-1), dict(inverse=2), dict(axes=0), dict(axes=5), dict(sections=(31, 0, 0, 0)),
    dict(sections=(16, 16, 0, 0)), dict(axes=2, sections=(33, -1, 0, 0)), dict(axes=2, sections=(2 ** 31 - 1, 33, 0, 0)),
    dict(magnitude=float("nan")), dict(magnitude=float("inf")), dict(q_stride=255), dict(q_stride=252), dict(k_stride=132),
    dict(q_out_stride=-256), dict(k_out_stride=(1 << 23) + 8)])
def test_bad_problems_are_refused(fields):
    assert call(problem(**fields)) == G.ERR_INVALID_ARGUMENT
    assert G.lib().gdn_last_error_message()


def test_bad_pointers_are_refused():
    assert G.lib().gdn_rotary(None, *[FAKE] * 6, None) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "positions", "frequencies", "qo", "ko"):
        assert call(problem(), **{n: None}) == G.ERR_INVALID_ARGUMENT
        assert call(problem(), **{n: FAKE + 2}) == G.ERR_INVALID_ARGUMENT
    for n in ("q", "k", "qo", "ko"):
        assert call(problem(), **{n: FAKE + 8}) == G.ERR_INVALID_ARGUMENT
    assert call(problem(), frequencies=FAKE + 4) == G.ERR_INVALID_ARGUMENT
    p = problem()
    p.reserved[3] = 1
    assert call(p) == G.ERR_INVALID_ARGUMENT
    assert call(problem(q_stride=512)) == G.ERR_INVALID_ARGUMENT        # in place with two strides
    assert call(problem(k_out_stride=512)) == G.ERR_INVALID_ARGUMENT
    assert call(problem(tokens=0), q=None, k=None, positions=None, frequencies=None, qo=None, ko=None) == G.OK


def test_frequencies():
    f, m = G.rotary_frequencies(64, 10000.0, device="cpu")
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert m == 1.0 and f.dtype == torch.float64 and torch.allclose(f, want, rtol=1e-14, atol=0)
    g, m = G.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert m == 1.0 and torch.allclose(g, want / 4, rtol=1e-14, atol=0)
    g, m = G.rotary_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert m == 1.0 and g[0] == 1.0 and math.isclose(g[-1], want[-1] / 4, rel_tol=1e-12) and (g[1:-1] > want[1:-1] / 4).all()
    assert G.rotary_frequencies(2, scaling="ntk", factor=4.0, device="cpu")[0].tolist() == [1.0]
    g, m = G.rotary_frequencies(64, scaling="yarn", factor=4.0, trained=4096, device="cpu")
    turns = 4096 * want / (2 * math.pi)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1) and torch.equal(g[turns >= 32], want[turns >= 32])
    assert torch.allclose(g[turns <= 1], want[turns <= 1] / 4, rtol=1e-14, atol=0)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (g[between] < want[between]).all() and (g[between] > want[between] / 4).all()
    assert (g[1:] < g[:-1]).all()
    for kw in (dict(width=3), dict(width=0), dict(width=64, scaling="other"), dict(width=64, base=0.0), dict(width=64, base=math.inf),
               dict(width=64, factor=0.5), dict(width=64, factor=math.nan), dict(width=64, scaling="yarn"),
               dict(width=64, scaling="yarn", trained=0), dict(width=64, scaling="yarn", trained=4096, slow=3.0, fast=3.0)):
        with pytest.raises(ValueError):
            G.rotary_frequencies(device="cpu", **kw)


def test_cpu_tensors_are_refused():
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        G.rotary(q, None, torch.zeros(4, dtype=torch.int32), G.rotary_frequencies(64, device="cpu")[0])


def test_host_arguments_that_are_no_numbers_are_refused():
    """Sections are counts: halves are not cut off.  A context of NaN positions has no frequencies."""
    from gated_delta_rule_frame_amd import positions as P
    assert P._sections((8, 0, 4), 12) == (8, 0, 4) and P._sections(None, 12) == (12,)
    for bad in ((8.5, 4.5), (8, 4.0), ("8", 4), (8, None), 12):
        with pytest.raises(TypeError):
            P._sections(bad, 12)
    for bad in ((), (8, 5), (13, -1), (4, 4, 2, 1, 1)):
        with pytest.raises(ValueError):
            P._sections(bad, 12)
    for trained in (math.nan, math.inf):
        with pytest.raises(ValueError):
            G.rotary_frequencies(64, scaling="yarn", factor=4.0, trained=trained, device="cpu")
