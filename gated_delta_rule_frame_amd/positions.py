"""Binding of libgdn's rotary positions (``include/gdn.h``, "Rotary positions of queries and keys").

``rotary`` wraps ``gdn_rotary``, ``rotary_backward`` its inverse turn, the
gradients; ``rotary_frequencies`` computes the pairs' frequencies on the host.
Checks, streams and errors are those of ``sequence``; results carry no autograd
graph.
"""
from __future__ import annotations

import functools
import math
import operator

import torch

from . import ABI_VERSION, lib
from .sequence import _CODE, _MAX, _dense, _on, _ptr, _rows
from .sequence_abi import RotaryProblem

LAYOUT = {"half": 0, "interleaved": 1}
_SCALING = ("none", "linear", "ntk", "yarn")


def rotary_frequencies(width, base=10000.0, *, scaling="none", factor=1.0, trained=None, slow=1.0, fast=32.0, device=None):
    """Frequencies of the width / 2 pairs of ``width`` turned components; returns (frequencies, magnitude).

    Pair i turns by base^(-2 i / width) radians per position.  ``scaling``
    stretches them for contexts ``factor`` >= 1 times as long as those of
    training: "linear" divides every frequency by factor; "ntk" raises the base
    to base factor^(width / (width - 2)), which keeps the first pair and divides
    the last by factor; "yarn" divides the frequency of pairs that turn at most
    ``slow`` times in the ``trained`` positions of training, keeps those of at
    least ``fast`` turns, goes from one to the other in between, linearly in the
    number of turns, and gives the magnitude 0.1 ln(factor) + 1 (1 otherwise).
    frequencies ([width / 2] fp64 on ``device``) and magnitude are ``rotary``'s.
    """
    if int(width) != width or width < 2 or width % 2:
        raise ValueError(f"width must be an even number >= 2 (got {width})")
    if scaling not in _SCALING:
        raise ValueError(f"unknown scaling {scaling!r}")
    if not (math.isfinite(base) and base > 0) or not (math.isfinite(factor) and factor >= 1):
        raise ValueError(f"base must be > 0 and factor >= 1 (got {base}, {factor})")
    pairs, magnitude = int(width) // 2, 1.0
    if scaling == "ntk" and pairs > 1:
        base = base * factor ** (width / (width - 2))
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -torch.arange(pairs, dtype=torch.float64) / pairs)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        if trained is None or not 1 <= trained < math.inf or not 0 <= slow < fast:
            raise ValueError(f"yarn needs trained >= 1 and 0 <= slow < fast (got {trained}, {slow}, {fast})")
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
        magnitude = 0.1 * math.log(factor) + 1
    return f.to("cuda" if device is None else device), magnitude


@functools.lru_cache(maxsize=1024)
def _problem(*fields):
    """The problem of these fields; kept, as making one takes longer than a small launch.  Calls only read it."""
    sections, rest = fields[0], fields[1:]
    p = RotaryProblem(ABI_VERSION, *rest[:9], sections + (0,) * (4 - len(sections)), rest[9])
    p.q_stride, p.k_stride, p.q_out_stride, p.k_out_stride = rest[10:]
    return p


def _sections(sections, pairs):
    """The numbers of pairs of the axes."""
    parts = (pairs,) if sections is None else tuple(operator.index(s) for s in sections)
    if not 1 <= len(parts) <= 4 or min(parts) < 0 or sum(parts) != pairs:
        raise ValueError(f"sections must be one to four numbers >= 0, {pairs} in all (got {parts})")
    return parts


def _turn(q, k, positions, frequencies, layout, magnitude, sections, out, inverse):
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be a tensor on a GPU")
    if q.dim() != 3 or (k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 3)):
        raise ValueError("q must be [tokens,heads_q,width] and k [tokens,heads_k,width] or None")
    if q.dtype not in _CODE:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if layout not in LAYOUT:
        raise ValueError(f"unknown layout {layout!r}")
    device, (n, hq, width) = q.device, q.shape
    hk = 0 if k is None else k.shape[1]
    if (hq | hk | width) > _MAX:
        raise ValueError(f"heads and width must be below 2^31 (got {hq}, {hk}, {width})")
    if k is not None and (k.dtype is not q.dtype or k.shape != (n, hk, width)):
        raise ValueError(f"k must be {q.dtype} of [{n},heads_k,{width}] (got {k.dtype}, {tuple(k.shape)})")
    if k is not None and hk == 0:
        raise ValueError("k must have heads")
    if not isinstance(frequencies, torch.Tensor) or frequencies.dim() != 1 or frequencies.shape[0] > width // 2:
        raise ValueError(f"frequencies must be a tensor of at most width / 2 = {width // 2} values")
    _dense("frequencies", frequencies, frequencies.shape, torch.float64, device)
    pairs = frequencies.shape[0]
    parts = _sections(sections, pairs)
    _dense("positions", positions, (n,) if sections is None else (n, len(parts)), torch.int32, device)
    if out is None:
        out = (None, None)
    elif len(out) != 2 or (k is None and out[1] is not None):
        raise ValueError("out must be a pair, the outputs of q and k")
    qs, ks, qos, kos = _rows("q", q, q.shape, q.dtype, device), 0, 0, 0
    qo, ko = out
    if qo is None:
        qo = torch.empty(q.shape, dtype=q.dtype, device=device)
    else:
        qos = _rows("q's output", qo, q.shape, q.dtype, device)
    if k is not None:
        ks = _rows("k", k, k.shape, q.dtype, device)
        if ko is None:
            ko = torch.empty(k.shape, dtype=q.dtype, device=device)
        else:
            kos = _rows("k's output", ko, k.shape, q.dtype, device)
    p = _problem(parts, _CODE[q.dtype], n, hq, hk, width, pairs, LAYOUT[layout], int(inverse), len(parts), float(magnitude),
                 qs, ks, qos, kos)
    _on(device, lib().gdn_rotary, p, q.data_ptr(), _ptr(k), positions.data_ptr(), frequencies.data_ptr(), qo.data_ptr(), _ptr(ko))
    return qo, ko


def rotary(q, k, positions, frequencies, *, layout="half", magnitude=1.0, sections=None, out=None):
    """Turns queries and keys by their positions (gdn_rotary); returns (q, k).

    q: [tokens,heads_q,width]; k: [tokens,heads_k,width] or None (fp32 or bf16,
    one dtype; width a multiple of 8 up to 1024; rows may be slices of one
    projection).  frequencies: [pairs] fp64, radians per position: the first 2
    pairs components of every head are turned, the others copied.  positions:
    [tokens] int32, or with ``sections``, the numbers of pairs of up to four
    axes, [tokens, axes] (frame, row and column, for instance).  ``layout``:
    pair i is components i and i + pairs ("half") or 2 i and 2 i + 1
    ("interleaved").  Turned values are scaled by ``magnitude``.  ``out``: a
    pair of outputs; (q, k) turns in place.
    """
    return _turn(q, k, positions, frequencies, layout, magnitude, sections, out, False)


def rotary_backward(dq, dk, positions, frequencies, *, layout="half", magnitude=1.0, sections=None, out=None):
    """Gradients of ``rotary``'s q and k from those of its results; returns (dq, dk).  The arguments are as given there."""
    return _turn(dq, dk, positions, frequencies, layout, magnitude, sections, out, True)
