"""Binding of the sequence operators of libgdn (``include/gdn.h``, "Sequences of tokens").

``decode`` wraps ``gdn_decode``; ``packed_forward`` and ``packed_backward``
wrap ``gdn_packed_forward`` and its gradients; ``group_norm`` and ``group_norm_backward``
wrap ``gdn_group_norm`` and its gradients.  As in the rest of the package the functions
check and marshal their arguments and launch the HIP kernels on the current
stream of the tensors' device; there is no CPU fallback, and results carry no
autograd graph, whether the inputs require gradients or not: a training step
calls ``packed_backward`` and ``group_norm_backward`` itself (a
``torch.autograd.Function`` around a pair of calls, for instance).
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import ABI_VERSION, BF16, F32, _check, lib
from .sequence_abi import NormProblem, SeqProblem

_MAX = 2 ** 31 - 1          # of the ABI's 32-bit sizes, which ctypes would cut off without an error
ACTIVATION = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}
_CODE = {torch.bfloat16: BF16, torch.float32: F32}


# The handle of a device's current stream, without the Stream object that the public call makes
# (1.8 us of a 12 us single-row decode step) where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _fits(name, n):
    if n > _MAX:
        raise ValueError(f"{name} must be below 2^31 (got {n})")
    return n


def _on(device, call, *args):
    """Runs a library call with the tensors' device current, on its current stream."""
    stream = _raw_stream(device.index)
    if device.index == _current():
        _check(call(*args, stream))
    else:
        with torch.cuda.device(device):
            _check(call(*args, stream))


def _rows(name, t, shape, dtype, device):
    """A packed [tokens, heads, width] input; returns its stride between tokens (0 = dense)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device.index:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.is_contiguous():
        return 0
    s = t.stride()
    if (shape[2] > 1 and s[2] != 1) or (shape[1] > 1 and s[1] != shape[2]) or s[0] < shape[1] * shape[2]:
        raise ValueError(f"the heads and widths of {name} must be dense and its rows must not overlap (strides {s})")
    return s[0]


def _dense(name, t, shape, dtype, device):
    """A contiguous tensor of this shape, type and device."""
    if (not isinstance(t, torch.Tensor) or t.get_device() != device.index or t.dtype is not dtype or t.shape != shape
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _problem(q, k, v, log_gate, beta, out_dtype):
    """Checks the inputs every sequence operator shares; returns (problem, device, tokens, heads_v, d_k, d_v)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be a tensor on a GPU")
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q, k must be [tokens,heads_k,d_k] and v [tokens,heads_v,d_v]")
    if q.dtype not in _CODE or out_dtype not in _CODE:
        raise TypeError(f"unsupported dtype {q.dtype} or {out_dtype}")
    device, (n, hk, dk), (hv, dv) = q.device, q.shape, v.shape[1:]
    if (hk | hv | dk | dv) > _MAX:
        raise ValueError(f"heads and widths must be below 2^31 (got {hk}, {hv}, {dk}, {dv})")
    p = SeqProblem(ABI_VERSION, hk, hv, dk, dv, _CODE[q.dtype], _CODE[out_dtype], 0, n)
    p.q_stride = _rows("q", q, q.shape, q.dtype, device)
    p.k_stride = _rows("k", k, q.shape, q.dtype, device)
    p.v_stride = _rows("v", v, (n, hv, dv), q.dtype, device)
    _dense("log_gate", log_gate, (n, hv), torch.float32, device)
    _dense("beta", beta, (n, hv), torch.float32, device)
    return p, device, n, hv, dk, dv


def _output(out, out_dtype):
    if out is None:
        return torch.float32 if out_dtype is None else out_dtype
    if not isinstance(out, torch.Tensor):
        raise ValueError("out must be a tensor")
    if out_dtype is not None and out_dtype != out.dtype:
        raise TypeError(f"out_dtype {out_dtype} differs from out's dtype {out.dtype}")
    return out.dtype


def decode(q, k, v, log_gate, beta, state, slots=None, *, out_dtype=None, out=None):
    """One token of the gated delta rule per row, states updated in place (gdn_decode); returns ``out``.

    q, k: [rows,heads_k,d_k]; v: [rows,heads_v,d_v] (fp32 or bf16, one dtype;
    heads_v a multiple of heads_k); log_gate, beta: [rows,heads_v] fp32;
    state: [state rows,heads_v,d_k,d_v] fp32.  ``slots`` ([rows] int32) picks
    each row's state; without it row i uses state row i.  A row whose slot is
    outside the pool is padding: its state and output rows stay as they were
    (a fresh output holds nothing there).  Rows of one slot are applied in row
    order.  The output is fp32 unless ``out_dtype`` or ``out`` says otherwise.
    """
    odt = _output(out, out_dtype)
    p, device, n, hv, dk, dv = _problem(q, k, v, log_gate, beta, odt)
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
    _on(device, lib().gdn_decode, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(), beta.data_ptr(),
        state.data_ptr(), None if slots is None else slots.data_ptr(), out.data_ptr())
    return out


def _sequences(cu_seqlens, device):
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be a tensor of sequences + 1 values")
    _dense("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, device)
    return _fits("sequences", cu_seqlens.shape[0] - 1)


def packed_forward(q, k, v, log_gate, beta, cu_seqlens, initial_state=None, *, slots=None, out_dtype=None, out=None,
                   final_state=None, want_state=True, workspace=None):
    """The gated delta rule over packed sequences (gdn_packed_forward); returns (out, final_state).

    q, k: [tokens,heads_k,d_k]; v: [tokens,heads_v,d_v] (fp32 or bf16, one
    dtype; heads_v a multiple of heads_k); log_gate, beta: [tokens,heads_v]
    fp32.  ``cu_seqlens`` ([sequences + 1] int32 on the GPU, not decreasing):
    sequence s is rows cu_seqlens[s] to cu_seqlens[s + 1]; output rows behind
    the last one stay as they were (a fresh output holds nothing there).
    initial_state, final_state: [sequences,heads_v,d_k,d_v] fp32, or with
    ``slots`` ([sequences] int32) pools of which each sequence uses one row; the
    final state of a call with ``slots`` goes into ``final_state``, by default
    into initial_state, in place.  The output is fp32 unless ``out_dtype`` or
    ``out`` says otherwise; it carries no autograd graph (``packed_backward``
    gives the gradients).  A NaN or infinity in a token's row can make outputs
    of up to 63 earlier tokens of its sequence NaN (those in its chunk of 64).
    """
    odt = _output(out, out_dtype)
    p, device, n, hv, dk, dv = _problem(q, k, v, log_gate, beta, odt)
    seqs = p.sequences = _sequences(cu_seqlens, device)
    states = seqs
    if slots is not None:
        _dense("slots", slots, (seqs,), torch.int32, device)
        if final_state is None:
            if initial_state is None:
                raise ValueError("a call with slots needs initial_state or final_state, the pool")
            if want_state:
                final_state = initial_state
        pool = initial_state if final_state is None else final_state
        states = pool.shape[0] if isinstance(pool, torch.Tensor) and pool.dim() == 4 else 0
        p.state_rows = _fits("the pool's rows", states)
    shape = (states, hv, dk, dv)
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
    L = lib()
    ws, ws_bytes = _space("gdn_packed_workspace_size", p, 0, workspace, device)
    _on(device, L.gdn_packed_forward, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(), beta.data_ptr(),
        cu_seqlens.data_ptr(), _ptr(slots), _ptr(initial_state), out.data_ptr(), _ptr(final_state), _ptr(ws), ws_bytes)
    return out, final_state


def packed_backward(q, k, v, log_gate, beta, cu_seqlens, dout, initial_state=None, dfinal_state=None, *, grads=None,
                    workspace=None):
    """Gradients of ``packed_forward`` (gdn_packed_backward); returns (dq, dk, dv, dlog_gate, dbeta, dinitial_state).

    The inputs are packed_forward's (without slots); dout: like v;
    dfinal_state: like the final state, or None (zeros).  dq, dk and dv have
    q's dtype and are dense, the others are fp32; dinitial_state is None
    where initial_state is.  Rows behind the last sequence are not written, so
    that in fresh tensors they hold nothing: for a padded batch give ``grads``,
    five zeroed tensors (dq, dk, dv, dlog_gate, dbeta) to write into.
    """
    p, device, n, hv, dk, dv = _problem(q, k, v, log_gate, beta, torch.float32)
    seqs = p.sequences = _sequences(cu_seqlens, device)
    _dense("dout", dout, v.shape, q.dtype, device)
    shape = (seqs, hv, dk, dv)
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _dense(name, t, shape, torch.float32, device)
    inputs = {"dq": q, "dk": k, "dv": v, "dlog_gate": log_gate, "dbeta": beta}
    if grads is None:
        grads = [torch.empty(t.shape, dtype=t.dtype, device=device) for t in inputs.values()]
    else:
        if len(grads) != 5:
            raise ValueError(f"grads must be five tensors (got {len(grads)})")
        for (name, t), d in zip(inputs.items(), grads):
            _dense(name, d, t.shape, t.dtype, device)
    L = lib()
    ws, ws_bytes = _space("gdn_packed_workspace_size", p, 1, workspace, device)
    dstate = None if initial_state is None else torch.empty_like(initial_state)
    _on(device, L.gdn_packed_backward, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(), beta.data_ptr(),
        cu_seqlens.data_ptr(), _ptr(initial_state), dout.data_ptr(), _ptr(dfinal_state), *(t.data_ptr() for t in grads),
        _ptr(dstate), _ptr(ws), ws_bytes)
    return (*grads, dstate)


def packed_workspace_size(q, v, sequences, *, gradient=False):
    """Bytes of workspace of ``packed_forward`` (or ``packed_backward``) for inputs like q and v."""
    if q.dtype not in _CODE:
        raise TypeError(f"unsupported dtype {q.dtype}")
    p = SeqProblem(ABI_VERSION, q.shape[1], v.shape[1], q.shape[2], v.shape[2], _CODE[q.dtype], F32, 0, q.shape[0])
    p.sequences = _fits("sequences", sequences)
    return _need("gdn_packed_workspace_size", SeqProblem, bytes(p), int(gradient))


def _ptr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=1024)
def _need(call, kind, fields, mode):
    """Bytes of workspace of the problem of these bytes; it depends on nothing else."""
    need = ctypes.c_size_t(0)
    _check(getattr(lib(), call)(kind.from_buffer_copy(fields), mode, ctypes.byref(need)))
    return need.value


def _space(call, problem, mode, workspace, device):
    """(tensor, bytes) of a call's workspace: the caller's, or a fresh one of the needed size."""
    need = _need(call, type(problem), bytes(problem), mode)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        return workspace, workspace.numel() * workspace.element_size()
    if need == 0:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=device), need


def _norm_problem(x, groups, weight, bias, gate, activation, center, eps):
    if not isinstance(x, torch.Tensor) or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous tensor on a GPU")
    if x.dim() < 2:
        raise ValueError("x must be [batch, ..., channels]")
    if x.dtype not in _CODE:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if activation not in ACTIVATION:
        raise ValueError(f"unknown activation {activation!r}")
    C = x.shape[-1]
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _dense(name, t, (C,), torch.float32, x.device)
    if gate is not None:
        _dense("gate", gate, x.shape, x.dtype, x.device)
    spatial = 1
    for n in x.shape[1:-1]:
        spatial *= n
    for name, n in (("the spatial size", spatial), ("channels", C), ("groups", groups)):
        _fits(name, n)
    return NormProblem(ABI_VERSION, _CODE[x.dtype], x.shape[0], spatial, C, groups, ACTIVATION[activation], int(bool(center)), eps)


def group_norm(x, groups, weight=None, bias=None, gate=None, *, activation="none", center=True, eps=1e-5, out=None,
               workspace=None):
    """Group norm with an activation or an activated gate, channels last (gdn_group_norm); returns (out, mean, rstd).

    x: [batch, ..., channels] (fp32 or bf16), statistics over the middle
    dimensions and the channels of each of ``groups`` groups; weight, bias:
    [channels] fp32 or None; gate: like x or None.  With u = weight h + bias
    the output is act(u), or u act(gate) where a gate is given; ``activation``
    is "none", "silu", "gelu" or "relu".  ``center=False`` normalises by the
    root mean square; its mean is None.  ``[tokens, heads * d_v]`` with the
    heads as groups is the norm of each token's heads.  mean and rstd
    ([batch, groups] fp32) are what ``group_norm_backward`` needs; nothing
    returned carries an autograd graph.
    """
    p = _norm_problem(x, groups, weight, bias, gate, activation, center, eps)
    if out is None:
        out = torch.empty_like(x)
    else:
        _dense("out", out, x.shape, x.dtype, x.device)
    ws, ws_bytes = _space("gdn_group_norm_workspace_size", p, 0, workspace, x.device)
    stats = (x.shape[0], groups)
    mean = torch.empty(stats, dtype=torch.float32, device=x.device) if center else None
    rstd = torch.empty(stats, dtype=torch.float32, device=x.device)
    _on(x.device, lib().gdn_group_norm, p, x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(gate), out.data_ptr(), _ptr(mean),
        rstd.data_ptr(), _ptr(ws), ws_bytes)
    return out, mean, rstd


def group_norm_backward(dout, x, groups, mean, rstd, weight=None, bias=None, gate=None, *, activation="none", center=True,
                        workspace=None):
    """Gradients of ``group_norm`` (gdn_group_norm_backward); returns (dx, dweight, dbias, dgate).

    dout: like x; mean (None without ``center``) and rstd: what ``group_norm``
    returned for x; the other arguments as given there.  dweight, dbias and
    dgate are None where weight, bias or gate are.
    """
    p = _norm_problem(x, groups, weight, bias, gate, activation, center, 0.0)
    _dense("dout", dout, x.shape, x.dtype, x.device)
    stats = (x.shape[0], groups)
    if center:
        _dense("mean", mean, stats, torch.float32, x.device)
    elif mean is not None:
        raise ValueError("mean must be None without center")
    _dense("rstd", rstd, stats, torch.float32, x.device)
    ws, ws_bytes = _space("gdn_group_norm_workspace_size", p, 1, workspace, x.device)
    dx = torch.empty_like(x)
    dw = None if weight is None else torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dz = None if gate is None else torch.empty_like(gate)
    _on(x.device, lib().gdn_group_norm_backward, p, dout.data_ptr(), x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(gate),
        _ptr(mean), rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(dz), _ptr(ws), ws_bytes)
    return dx, dw, db, dz
