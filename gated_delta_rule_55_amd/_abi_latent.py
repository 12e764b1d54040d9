"""ctypes mirror of include/kda_latent.h, on the library _abi.py loads."""
from __future__ import annotations

import ctypes

from . import _abi

KDA_ROTARY_HALF = 0
KDA_ROTARY_INTERLEAVED = 1

_i32, _i64, _f32, _ptr = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


def _fields(*groups):
    return [("struct_size", ctypes.c_uint32)] + [(n, t) for t, names in groups for n in names.split()]


class LatentPrefillDesc(ctypes.Structure):
    _fields_ = _fields((_i32, "dtype n_seqs n_heads dn dr dv"), (_f32, "scale"), (_i64, "q_total k_total"),
                       (_ptr, "q k k_pe v o"),
                       (_i64, "q_stride k_stride k_head_stride k_pe_stride v_stride v_head_stride o_stride"),
                       (_ptr, "cu_seqlens cu_seqlens_k"))


class LatentAttendDesc(ctypes.Structure):
    _fields_ = _fields((_i32, "dtype n_seqs n_heads dc dr page_size max_pages n_pages"), (_f32, "scale"),
                       (_i64, "t_total"), (_ptr, "q cache o"), (_i64, "q_stride page_stride row_stride o_stride"),
                       (_ptr, "block_table seq_lens cu_seqlens"))


class LatentAppendDesc(ctypes.Structure):
    _fields_ = _fields((_i32, "dtype n_seqs dc dr page_size max_pages n_pages rotary"), (_f32, "eps magnitude"),
                       (_i64, "t_total"), (_ptr, "latent k_pe cache rows_out"),
                       (_i64, "latent_stride k_pe_stride page_stride row_stride rows_out_stride"),
                       (_ptr, "weight frequencies block_table seq_lens cu_seqlens"))


class RotaryDesc(ctypes.Structure):
    _fields_ = _fields((_i32, "dtype n_heads dim rotary"), (_f32, "magnitude"), (_i64, "t_total"), (_ptr, "x y"),
                       (_i64, "x_stride x_head_stride y_stride y_head_stride"), (_ptr, "positions frequencies"))


_LIB = None


def lib():
    """The loaded libkda.so with these entry points' signatures set."""
    global _LIB
    if _LIB is None:
        L = _abi.lib()
        L.kda_latent_workspace_bytes.argtypes = [ctypes.POINTER(LatentAttendDesc), ctypes.POINTER(ctypes.c_int)]
        L.kda_latent_workspace_bytes.restype = ctypes.c_size_t
        L.kda_latent_attend.argtypes = [ctypes.POINTER(LatentAttendDesc), ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]
        L.kda_latent_prefill_workspace_bytes.argtypes = [ctypes.POINTER(LatentPrefillDesc),
                                                         ctypes.POINTER(ctypes.c_int)]
        L.kda_latent_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.kda_latent_prefill.argtypes = [ctypes.POINTER(LatentPrefillDesc), ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]
        L.kda_latent_append.argtypes = [ctypes.POINTER(LatentAppendDesc), ctypes.c_void_p]
        L.kda_rotary.argtypes = [ctypes.POINTER(RotaryDesc), ctypes.c_void_p]
        for name in ("kda_latent_attend", "kda_latent_prefill", "kda_latent_append", "kda_rotary"):
            getattr(L, name).restype = ctypes.c_int
        _LIB = L
    return _LIB


def make(cls, **kw):
    """A descriptor with struct_size set and the named fields filled."""
    return cls(struct_size=ctypes.sizeof(cls), **kw)


def _workspace_bytes(name, desc) -> int:
    st = ctypes.c_int(0)
    n = getattr(lib(), name)(ctypes.byref(desc), ctypes.byref(st))
    if st.value != _abi.KDA_OK:
        raise _abi.KdaError(st.value, name)
    return int(n)


def latent_workspace_bytes(desc: LatentAttendDesc) -> int:
    return _workspace_bytes("kda_latent_workspace_bytes", desc)


def latent_prefill_workspace_bytes(desc: LatentPrefillDesc) -> int:
    return _workspace_bytes("kda_latent_prefill_workspace_bytes", desc)
