"""Structures and argument types of the sequence operators' C ABI (``include/gdn.h``, "Sequences of tokens").

Apart from ``sequence``, whose marshalling needs torch, so that the library
loads, and its host-only calls run, without it.
"""
from __future__ import annotations

import ctypes


class SeqProblem(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_int32), ("heads_k", ctypes.c_int32), ("heads_v", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("qkv_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("state_rows", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("sequences", ctypes.c_int32), ("reserved", ctypes.c_int32 * 5)]


class NormProblem(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_int32), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int64),
                ("spatial", ctypes.c_int32), ("channels", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("center", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32 * 4)]


def declare(L):
    """Argument types of the sequence entry points of a loaded libgdn."""
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    P = ctypes.POINTER(SeqProblem)
    L.gdn_decode.restype = i32
    L.gdn_decode.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.gdn_packed_workspace_size.restype = i32
    L.gdn_packed_workspace_size.argtypes = [P, i32, ctypes.POINTER(ctypes.c_size_t)]
    L.gdn_packed_forward.restype = i32
    L.gdn_packed_forward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.gdn_packed_backward.restype = i32
    L.gdn_packed_backward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    N, sz = ctypes.POINTER(NormProblem), ctypes.c_size_t
    L.gdn_group_norm_workspace_size.restype = i32
    L.gdn_group_norm_workspace_size.argtypes = [N, i32, ctypes.POINTER(sz)]
    L.gdn_group_norm.restype = i32
    L.gdn_group_norm.argtypes = [N, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.gdn_group_norm_backward.restype = i32
    L.gdn_group_norm_backward.argtypes = [N, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
