"""Binding of libgdn's linear attention with a decay for each head (``include/gdn.h``, the section of that name).

``linear_decode`` wraps ``gdn_linear_decode``.  It stands beside ``decode``, whose
states, pools, checks and streams it shares; results carry no autograd graph.
"""
from __future__ import annotations

import torch

from . import ABI_VERSION, lib
from .sequence import _CODE, _MAX, _dense, _fits, _on, _output, _ptr, _rows
from .sequence_abi import LinearProblem


def _problem(q, k, v, log_gate, scale, out_dtype):
    """Checks the inputs the calls share; returns (problem, device, tokens, heads_v, d_k, d_v)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be a tensor on a GPU")
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q, k must be [tokens,heads_k,d_k] and v [tokens,heads_v,d_v]")
    if q.dtype not in _CODE or out_dtype not in _CODE:
        raise TypeError(f"unsupported dtype {q.dtype} or {out_dtype}")
    device, (n, hk, dk), (hv, dv) = q.device, q.shape, v.shape[1:]
    if (hk | hv | dk | dv) > _MAX:
        raise ValueError(f"heads and widths must be below 2^31 (got {hk}, {hv}, {dk}, {dv})")
    p = LinearProblem(ABI_VERSION, hk, hv, dk, dv, _CODE[q.dtype], _CODE[out_dtype], 0, n)
    p.q_stride = _rows("q", q, q.shape, q.dtype, device)
    p.k_stride = _rows("k", k, q.shape, q.dtype, device)
    p.v_stride = _rows("v", v, (n, hv, dv), q.dtype, device)
    p.scale = scale
    p.gate_per_head = int(isinstance(log_gate, torch.Tensor) and log_gate.dim() == 1)
    _dense("log_gate", log_gate, (hv,) if p.gate_per_head else (n, hv), torch.float32, device)
    return p, device, n, hv, dk, dv


def linear_decode(q, k, v, log_gate, state, slots=None, *, scale=1.0, out_dtype=None, out=None):
    """One token of linear attention per row, states updated in place (gdn_linear_decode); returns ``out``.

    Per value head: state <- exp(log_gate) state + k v^T, out = scale state^T q.
    q, k: [rows,heads_k,d_k]; v: [rows,heads_v,d_v] (fp32 or bf16, one dtype;
    heads_v a multiple of heads_k); log_gate: [rows,heads_v] fp32, or
    [heads_v], one decay for each head; state, ``slots`` and the output as in
    ``decode``.
    """
    odt = _output(out, out_dtype)
    p, device, n, hv, dk, dv = _problem(q, k, v, log_gate, scale, odt)
    rows = n
    if slots is not None:
        _dense("slots", slots, (n,), torch.int32, device)
        rows = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 4 else 0
        p.state_rows = _fits("the pool's rows", rows)
    _dense("state", state, (rows, hv, dk, dv), torch.float32, device)
    if out is None:
        out = torch.empty((n, hv, dv), dtype=odt, device=device)
    else:
        _dense("out", out, (n, hv, dv), odt, device)
    _on(device, lib().gdn_linear_decode, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(), state.data_ptr(),
        _ptr(slots), out.data_ptr())
    return out
