"""ctypes mirror of include/kda_linear.h and include/kda_norm.h, on the library _abi.py loads."""
from __future__ import annotations

import ctypes
import struct

from . import _abi

KDA_DECAY_TOKEN = 0
KDA_DECAY_HEAD = 1

KDA_NORM_GATE_LINEAR = 0
KDA_NORM_GATE_SILU = 1
KDA_NORM_GATE_SIGMOID = 2


class LinearPrefillDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("n_seqs", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("n_k_heads", ctypes.c_int32),
        ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32),
        ("decay", ctypes.c_int32),
        ("t_total", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("state_dtype", ctypes.c_int32),
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("o", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("o_stride", ctypes.c_int64),
        ("h0", ctypes.c_void_p),
        ("ht", ctypes.c_void_p),
        ("cu_seqlens", ctypes.c_void_p),
        ("state_indices", ctypes.c_void_p),
        ("n_slots", ctypes.c_int32),
    ]


class LinearDecodeDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("n_seqs", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("n_k_heads", ctypes.c_int32),
        ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32),
        ("decay", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("state_dtype", ctypes.c_int32),
        ("state", ctypes.c_void_p),
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("o", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("o_stride", ctypes.c_int64),
        ("state_indices", ctypes.c_void_p),
        ("n_slots", ctypes.c_int32),
    ]


class GatedNormDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("gate", ctypes.c_int32),
        ("gate_first", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("rows", ctypes.c_int64),
        ("x", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64),
        ("y_stride", ctypes.c_int64),
    ]


class BlockNormDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("residual_dtype", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("gate", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("scale", ctypes.c_float),
        ("rows", ctypes.c_int64),
        ("x", ctypes.c_void_p),
        ("r", ctypes.c_void_p),
        ("w_post", ctypes.c_void_p),
        ("w_pre", ctypes.c_void_p),
        ("c", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("r_out", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64),
        ("r_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64),
        ("r_out_stride", ctypes.c_int64),
        ("y_stride", ctypes.c_int64),
    ]


# The same layouts for struct.pack, which fills a descriptor in a quarter of the
# time a ctypes structure takes (the calls of one token are short).
LINEAR_DECODE = struct.Struct("=I7ifi6Q4qQi4x")
GATED_NORM = struct.Struct("=I4ifq4Q3q")
BLOCK_NORM = struct.Struct("=I4i2f4xq8Q5q")
for _s, _d in ((LINEAR_DECODE, LinearDecodeDesc), (GATED_NORM, GatedNormDesc),
               (BLOCK_NORM, BlockNormDesc)):
    assert _s.size == ctypes.sizeof(_d)

_LIB = None


def lib():
    """The loaded libkda.so with these entry points' signatures set."""
    global _LIB
    if _LIB is None:
        L = _abi.lib()
        L.kda_linear_workspace_bytes.argtypes = [ctypes.POINTER(LinearPrefillDesc),
                                                 ctypes.POINTER(ctypes.c_int)]
        L.kda_linear_workspace_bytes.restype = ctypes.c_size_t
        L.kda_linear_prefill.argtypes = [ctypes.POINTER(LinearPrefillDesc), ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p]
        # descriptors as packed bytes or ctypes references
        for name in ("kda_linear_decode", "kda_gated_norm", "kda_block_norm"):
            getattr(L, name).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        for name in ("kda_linear_prefill", "kda_linear_decode", "kda_gated_norm", "kda_block_norm"):
            getattr(L, name).restype = ctypes.c_int
        _LIB = L
    return _LIB


def make(cls, **kw):
    """A descriptor with struct_size set and the named fields filled."""
    return cls(struct_size=ctypes.sizeof(cls), **kw)


def linear_workspace_bytes(desc: LinearPrefillDesc) -> int:
    st = ctypes.c_int(0)
    n = lib().kda_linear_workspace_bytes(ctypes.byref(desc), ctypes.byref(st))
    if st.value != _abi.KDA_OK:
        raise _abi.KdaError(st.value, "kda_linear_workspace_bytes")
    return int(n)
