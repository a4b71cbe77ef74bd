"""Binding of libgdn's linear attention with a decay for each head (``include/gdn.h``, the section of that name).

``linear_decode`` wraps ``gdn_linear_decode``, ``linear_forward`` and
``linear_backward`` wrap ``gdn_linear_forward`` and its gradients.  They stand
beside ``decode``, ``packed_forward`` and ``packed_backward``, whose states,
pools, packed layout, checks and streams they share; results carry no autograd
graph.
"""
from __future__ import annotations

import functools

import torch

from . import ABI_VERSION, F32, lib
from . import sequence
from .sequence import _CODE, _MAX, _dense, _fits, _need, _on, _output, _ptr, _rows, _space
from .sequence_abi import LinearProblem


@functools.lru_cache(maxsize=1024)
def _fields(hk, hv, dk, dv, code, out_code, n, qs, ks, vs, per_head, scale, sequences, state_rows):
    """The problem of these fields; kept, as making one takes longer than a small launch.  Calls only read it."""
    return LinearProblem(ABI_VERSION, hk, hv, dk, dv, code, out_code, state_rows, n, qs, ks, vs, sequences, per_head, scale)


def _problem(q, k, v, log_gate, scale, out_dtype, sequences=0, state_rows=0):
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
    qs, ks = _rows("q", q, q.shape, q.dtype, device), _rows("k", k, q.shape, q.dtype, device)
    vs = _rows("v", v, (n, hv, dv), q.dtype, device)
    per_head = int(isinstance(log_gate, torch.Tensor) and log_gate.dim() == 1)
    _dense("log_gate", log_gate, (hv,) if per_head else (n, hv), torch.float32, device)
    p = _fields(hk, hv, dk, dv, _CODE[q.dtype], _CODE[out_dtype], n, qs, ks, vs, per_head, float(scale), sequences, state_rows)
    return p, device, n, hv, dk, dv


def _sequences(cu_seqlens, q):
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be a tensor on a GPU")
    return sequence._sequences(cu_seqlens, q.device)


def _pool(t):
    """Rows of a pool of states."""
    return _fits("the pool's rows", t.shape[0] if isinstance(t, torch.Tensor) and t.dim() == 4 else 0)


def linear_decode(q, k, v, log_gate, state, slots=None, *, scale=1.0, out_dtype=None, out=None):
    """One token of linear attention per row, states updated in place (gdn_linear_decode); returns ``out``.

    Per value head: state <- exp(log_gate) state + k v^T, out = scale state^T q.
    q, k: [rows,heads_k,d_k]; v: [rows,heads_v,d_v] (fp32 or bf16, one dtype;
    heads_v a multiple of heads_k); log_gate: [rows,heads_v] fp32, or
    [heads_v], one decay for each head; state, ``slots`` and the output as in
    ``decode``.
    """
    odt = _output(out, out_dtype)
    rows = 0 if slots is None else _pool(state)
    p, device, n, hv, dk, dv = _problem(q, k, v, log_gate, scale, odt, 0, rows)
    if slots is None:
        rows = n
    else:
        _dense("slots", slots, (n,), torch.int32, device)
    _dense("state", state, (rows, hv, dk, dv), torch.float32, device)
    if out is None:
        out = torch.empty((n, hv, dv), dtype=odt, device=device)
    else:
        _dense("out", out, (n, hv, dv), odt, device)
    _on(device, lib().gdn_linear_decode, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(), state.data_ptr(),
        _ptr(slots), out.data_ptr())
    return out


def linear_forward(q, k, v, log_gate, cu_seqlens, initial_state=None, *, slots=None, scale=1.0, out_dtype=None, out=None,
                   final_state=None, want_state=True, workspace=None):
    """Linear attention with a decay over packed sequences (gdn_linear_forward); returns (out, final_state).

    Per token of a value head: S <- exp(log_gate) S + k v^T, out = scale S^T q.
    q, k: [tokens,heads_k,d_k]; v: [tokens,heads_v,d_v] (fp32 or bf16, one
    dtype; heads_v a multiple of heads_k); log_gate: [tokens,heads_v] fp32, or
    [heads_v], one decay for each head.  cu_seqlens, slots, states and outputs
    are ``packed_forward``'s.  A NaN or infinity in v can make outputs of up to 63
    earlier tokens of its sequence NaN (those in its chunk of 64), in its head and
    column; in k or log_gate it reaches its own and later tokens alone.  An
    infinity may come out as a NaN (``linear_decode`` keeps it).
    """
    odt = _output(out, out_dtype)
    seqs, rows = _sequences(cu_seqlens, q), 0
    if slots is not None:
        if final_state is None:
            if initial_state is None:
                raise ValueError("a call with slots needs initial_state or final_state, the pool")
            if want_state:
                final_state = initial_state
        rows = _pool(initial_state if final_state is None else final_state)
    p, device, n, hv, dk, dv = _problem(q, k, v, log_gate, scale, odt, seqs, rows)
    if slots is not None:
        _dense("slots", slots, (seqs,), torch.int32, device)
    shape = (seqs if slots is None else rows, hv, dk, dv)
    if initial_state is not None:
        _dense("initial_state", initial_state, shape, torch.float32, device)
    if final_state is not None:
        _dense("final_state", final_state, shape, torch.float32, device)
    elif want_state and slots is None:
        final_state = torch.empty(shape, dtype=torch.float32, device=device)
    if out is None:
        out = torch.empty((n, hv, dv), dtype=odt, device=device)
    else:
        _dense("out", out, (n, hv, dv), odt, device)
    ws, ws_bytes = _space("gdn_linear_workspace_size", p, 0, workspace, device)
    _on(device, lib().gdn_linear_forward, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(), cu_seqlens.data_ptr(),
        _ptr(slots), _ptr(initial_state), out.data_ptr(), _ptr(final_state), _ptr(ws), ws_bytes)
    return out, final_state


def linear_backward(q, k, v, log_gate, cu_seqlens, dout, initial_state=None, dfinal_state=None, *, scale=1.0, grads=None,
                    workspace=None):
    """Gradients of ``linear_forward`` (gdn_linear_backward); returns (dq, dk, dv, dlog_gate, dinitial_state).

    The inputs are linear_forward's (without slots); dout: like v, dense, in
    its dtype (with bf16 inputs ask linear_forward for ``out_dtype`` bf16, or
    round the gradient of its fp32 output);
    dfinal_state: like the final state, or None (zeros).  dq, dk and dv have
    q's dtype and are dense, the others are fp32; dlog_gate has log_gate's
    shape, and an error of some 2^-22 of what the tokens behind a gate read from
    earlier ones and give to later ones, so that a gate stronger than those by
    e^-15 has no digits; dinitial_state is None where initial_state is.  Rows behind the
    last sequence are not written: for a padded batch give ``grads``, four
    tensors (dq, dk, dv, dlog_gate) to write into.
    """
    seqs = _sequences(cu_seqlens, q)
    p, device, n, hv, dk, dv = _problem(q, k, v, log_gate, scale, torch.float32, seqs)
    _dense("dout", dout, v.shape, q.dtype, device)
    shape = (seqs, hv, dk, dv)
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _dense(name, t, shape, torch.float32, device)
    inputs = {"dq": q, "dk": k, "dv": v, "dlog_gate": log_gate}
    if grads is None:
        grads = [torch.empty(t.shape, dtype=t.dtype, device=device) for t in inputs.values()]
    else:
        if len(grads) != 4:
            raise ValueError(f"grads must be four tensors (got {len(grads)})")
        for (name, t), d in zip(inputs.items(), grads):
            _dense(name, d, t.shape, t.dtype, device)
    ws, ws_bytes = _space("gdn_linear_workspace_size", p, 1, workspace, device)
    dstate = None if initial_state is None else torch.empty_like(initial_state)
    _on(device, lib().gdn_linear_backward, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(),
        cu_seqlens.data_ptr(), _ptr(initial_state), dout.data_ptr(), _ptr(dfinal_state), *(t.data_ptr() for t in grads),
        _ptr(dstate), _ptr(ws), ws_bytes)
    return (*grads, dstate)


def linear_workspace_size(q, v, log_gate, sequences, *, gradient=False):
    """Bytes of workspace of ``linear_forward`` (or ``linear_backward``) for inputs like q, v and log_gate."""
    if q.dtype not in _CODE:
        raise TypeError(f"unsupported dtype {q.dtype}")
    p = _fields(q.shape[1], v.shape[1], q.shape[2], v.shape[2], _CODE[q.dtype], F32, q.shape[0], 0, 0, 0, int(log_gate.dim() == 1),
                1.0, _fits("sequences", sequences), 0)
    return _need("gdn_linear_workspace_size", LinearProblem, bytes(p), int(gradient))
