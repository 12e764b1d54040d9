"""PyTorch-facing entry points of linear attention with a decay per head
(include/kda_linear.h) and of the norms around it (include/kda_norm.h):
argument marshalling only, as kda.py does for the KDA step.

Calls run on the device of their tensors, on `stream` or that device's current
stream; outputs and workspaces made here are allocated for that stream.

A call with dense tensors on the current device and stream goes through the
module _fast (csrc/kda_torch.cpp), which checks and launches it in 1 us above the
launch itself; it answers None to every other call, and to one that it would
have to refuse, which is then checked here, and made or refused.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import _abi
from . import _abi_layer as _al

try:
    from . import _fast
except ImportError:  # not built: every call is checked and made here
    _fast = None

_DTYPES = {torch.float32: _abi.KDA_DTYPE_F32, torch.bfloat16: _abi.KDA_DTYPE_BF16}


@contextlib.contextmanager
def _guard(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_HERE = contextlib.nullcontext()
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(dev, stream):
    """A context in which `dev` is current and `stream` (or the device's current
    stream) is the stream that torch allocates for."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    if stream is None and dev.index == _current_device():
        return _HERE
    return _guard(dev, stream)


# The current stream's handle: a torch.cuda.Stream object made for it would cost
# as much as the rest of a call's checks (2 us).
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(dev) -> int:
    if _current_handle is not None:
        return _current_handle(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _fail(t, name, shape, dtype, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous" if len(shape) != 3 else
                     f"{name} must be dense but for its first stride, got {t.stride()}")


def _dense(t, name, shape, dtype, dev) -> int:
    """Checks a contiguous tensor; its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == dev
            and t.shape == shape and t.is_contiguous()):
        _fail(t, name, shape, dtype, dev)
    return t.data_ptr()


def _rows3(t, name, shape, dtype, dev) -> Tuple[int, int]:
    """Checks a [rows, heads, d] tensor whose rows are dense; its address and
    the stride between rows (0: dense)."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == dev
            and t.shape == shape):
        _fail(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t.data_ptr(), 0
    s = t.stride()
    if s[2] != 1 or (shape[1] > 1 and s[1] != shape[2]) or s[0] < shape[1] * shape[2]:
        _fail(t, name, shape, dtype, dev)
    return t.data_ptr(), s[0]


def _linear_common(what, q, v):
    if not (isinstance(q, torch.Tensor) and isinstance(v, torch.Tensor)):
        raise TypeError(f"{what}: q and v must be tensors")
    dev, dtype = q.device, q.dtype
    if not q.is_cuda:
        raise ValueError(f"{what} runs on the GPU only")
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q and v must be [rows, heads, d], got {tuple(q.shape)}, {tuple(v.shape)}")
    return dev, dtype


def _decay(g, rows, H, dev):
    """g [rows, H] or [H] fp32: its kind and address."""
    if isinstance(g, torch.Tensor) and g.dim() == 1:
        return _al.KDA_DECAY_HEAD, _dense(g, "g", (H,), torch.float32, dev)
    return _al.KDA_DECAY_TOKEN, _dense(g, "g", (rows, H), torch.float32, dev)


def _scale(scale) -> float:
    """A scale as a descriptor holds it: 0 for the default."""
    if scale is None:
        return 0.0
    scale = float(scale)
    if scale != 0 and abs(scale) <= 2.0 ** -150:
        raise ValueError(f"scale {scale} is 0 in fp32, which stands for dk^-1/2")
    return scale


def linear_workspace_bytes(T: int, H: int, dk: int, dv: int, n_seqs: int = 1,
                           dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace linear_prefill needs for these sizes (0: none).  Not
    monotonic in T: a buffer for several sizes takes their maximum."""
    return _al.linear_workspace_bytes(_al.make(
        _al.LinearPrefillDesc, dtype=_DTYPES[dtype], n_seqs=n_seqs, n_heads=H, dk=dk, dv=dv,
        t_total=T))


def linear_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                   h0: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   ht: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   output_final_state: bool = True, stream=None,
                   state_indices: Optional[torch.Tensor] = None,
                   state_dtype: Optional[torch.dtype] = None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with one decay per head over packed sequences:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k: [T, Hk, dk] (each key head serves H / Hk consecutive value heads);
    v: [T, H, dv]; dk and dv each 32, 64 or 128; fp32 or bf16.  g: fp32
    log-decays [T, H], or [H] for one constant decay per head.  h0:
    [N, H, dk, dv] fp32 (or bf16 with bf16 inputs) or None; cu_seqlens: int32
    [N + 1] on the device or None (one sequence); scale: dk^-1/2 by default (and
    for 0).
    Returns (o [T, H, dv], ht [N, H, dk, dv] or None); ht may be h0 itself
    (in-place carry).  q, k, v and out may be slices of wider buffers: only
    their first stride may differ from a dense tensor's (a multiple of 16
    bytes).  state_indices (int32 [N] on the device): h0 and ht are pools
    [S, H, dk, dv] (ht defaults to h0: in place), sequence n uses slot
    state_indices[n], a negative slot skips it; no slot twice.  workspace: a buffer of
    linear_workspace_bytes bytes, one for each call that may overlap another
    (a captured graph keeps its own); allocated here when None.
    cu_seqlens is read on the device: contents that break its rules give
    unspecified results but no access out of bounds.  A sequence's bits do not
    depend on what it is packed with, but they may on T and N."""
    if _fast is not None and stream is None and (
            state_dtype is None or (h0 is None and ht is None and state_dtype in _DTYPES)):
        done = _fast.linear_prefill(q, k, v, g, h0, cu_seqlens, scale, out, ht, workspace,
                                    output_final_state, state_indices, state_dtype == torch.bfloat16)
        if done is not None:
            return done
    dev, dt = _linear_common("linear_prefill", q, v)
    T, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    if Hk < 1 or H % Hk:
        raise ValueError(f"q/k heads {Hk} must divide the value heads {H}")
    qp, qs = _rows3(q, "q", (T, Hk, dk), dt, dev)
    kp, ks = _rows3(k, "k", (T, Hk, dk), dt, dev)
    vp, vs = _rows3(v, "v", (T, H, dv), dt, dev)
    decay, gp = _decay(g, T, H, dev)
    N, cup, idxp, S = 1, None, None, 0
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be an int32 tensor [N + 1]")
        N = cu_seqlens.shape[0] - 1
        cup = _dense(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    pool = h0 if h0 is not None else ht
    sd = pool.dtype if pool is not None else (state_dtype or torch.float32)
    if sd not in _DTYPES or (state_dtype is not None and state_dtype != sd):
        raise TypeError(f"states must be fp32 or bf16 and of state_dtype, got {sd}, {state_dtype}")
    if state_indices is not None:
        idxp = _dense(state_indices, "state_indices", (N,), torch.int32, dev)
        if pool is None:
            raise ValueError("state_indices needs a state pool (h0 and/or ht)")
        if pool.dim() != 4:
            raise ValueError(f"a state pool is [S, H, dk, dv], got {tuple(pool.shape)}")
        S = pool.shape[0]
        if ht is None and output_final_state:
            ht = h0
    shape = (S if idxp is not None else N, H, dk, dv)
    h0p = None if h0 is None else _dense(h0, "h0", shape, sd, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(v) if vs == 0 else v.new_empty((T, H, dv))
            op, os_ = out.data_ptr(), 0
        else:
            op, os_ = _rows3(out, "out", (T, H, dv), dt, dev)
        if ht is None and output_final_state:
            ht = torch.empty(shape, dtype=sd, device=dev)
        htp = None if ht is None else _dense(ht, "ht", shape, sd, dev)
        desc = _al.LinearPrefillDesc(
            ctypes.sizeof(_al.LinearPrefillDesc), _DTYPES[dt], N, H, Hk, dk, dv, decay, T,
            _scale(scale), _DTYPES[sd], qp, kp, vp, gp, op, qs, ks, vs, os_,
            h0p, htp, cup, idxp, S)
        L = _al.lib()
        if workspace is None:
            need = _al.linear_workspace_bytes(desc)
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        wp, wn = (None, 0) if workspace is None else (
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
        st = L.kda_linear_prefill(ctypes.byref(desc), wp, wn, _raw_stream(dev))
    if st != _abi.KDA_OK:
        raise _abi.KdaError(st, "kda_linear_prefill")
    return out, ht


def linear_decode(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  g: torch.Tensor, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, stream=None,
                  state_indices: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token per sequence of linear_prefill's recurrence; `state`
    [N, H, dk, dv] (fp32, or bf16 with bf16 inputs) is updated in place.
    q, k: [N, Hk, dk]; v: [N, H, dv]; g: fp32 [N, H] or [H].  Returns o
    [N, H, dv].  state_indices (int32 [N] on the device): `state` is then a
    pool [S, H, dk, dv] and sequence n updates slot state_indices[n]; a
    negative slot skips it (its o is left as it was); no slot twice.  Strides as in
    linear_prefill."""
    if _fast is not None and stream is None:
        done = _fast.linear_decode(state, q, k, v, g, scale, out, state_indices)
        if done is not None:
            return done
    dev, dt = _linear_common("linear_decode", q, v)
    N, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    if Hk < 1 or H % Hk:
        raise ValueError(f"q/k heads {Hk} must divide the value heads {H}")
    if not isinstance(state, torch.Tensor) or state.dim() != 4 or state.dtype not in _DTYPES:
        raise TypeError("state must be an fp32 or bf16 tensor [N, H, dk, dv]")
    S, idxp = N, None
    if state_indices is not None:
        idxp = _dense(state_indices, "state_indices", (N,), torch.int32, dev)
        S = state.shape[0]
    sp = _dense(state, "state", (S, H, dk, dv), state.dtype, dev)
    qp, qs = _rows3(q, "q", (N, Hk, dk), dt, dev)
    kp, ks = _rows3(k, "k", (N, Hk, dk), dt, dev)
    vp, vs = _rows3(v, "v", (N, H, dv), dt, dev)
    decay, gp = _decay(g, N, H, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(v) if vs == 0 else v.new_empty((N, H, dv))
            op, os_ = out.data_ptr(), 0
        else:
            op, os_ = _rows3(out, "out", (N, H, dv), dt, dev)
        desc = _al.LINEAR_DECODE.pack(
            _al.LINEAR_DECODE.size, _DTYPES[dt], N, H, Hk, dk, dv, decay,
            _scale(scale), _DTYPES[state.dtype], sp, qp, kp, vp, gp, op,
            qs, ks, vs, os_, idxp or 0, S if idxp is not None else 0)
        st = _al.lib().kda_linear_decode(desc, _raw_stream(dev))
    if st != _abi.KDA_OK:
        raise _abi.KdaError(st, "kda_linear_decode")
    return out


_GATES = {None: _al.KDA_NORM_GATE_LINEAR, "none": _al.KDA_NORM_GATE_LINEAR,
          "silu": _al.KDA_NORM_GATE_SILU, "sigmoid": _al.KDA_NORM_GATE_SIGMOID}


def _norm_common(what, x, activation):
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a tensor [..., dim]")
    if not x.is_cuda:
        raise ValueError(f"{what} runs on the GPU only")
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if activation not in _GATES:
        raise ValueError(f"activation must be one of {list(_GATES)}")
    return x.device, x.dtype, x.shape[-1]


def _rows(t, name, shape, dtype, dev) -> Tuple[int, int]:
    """Checks a [..., dim] tensor whose rows lie at one stride; its address and
    that stride (0: dense)."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == dev
            and t.shape == shape):
        _fail(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t.data_ptr(), 0
    s = t.stride()
    row, below = None, 1  # the stride between rows, and the rows one step of a dimension spans
    for size, st in zip(reversed(shape[:-1]), reversed(s[:-1])):
        if size == 1:
            continue
        if row is None:
            row = st
        elif st != row * below:
            raise ValueError(f"{name}: rows must lie at one stride, got {s}")
        below *= size
    if (shape[-1] > 1 and s[-1] != 1) or row is None or row < shape[-1]:
        raise ValueError(f"{name}: rows must be dense and lie at one stride, got {s}")
    return t.data_ptr(), row


def _weight(w, name, dim, dev) -> int:
    return 0 if w is None else _dense(w, name, (dim,), torch.float32, dev)


def gated_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, activation=None, gate_first: bool = False,
               eps: float = 1e-6, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """RMSNorm over the last axis with a gate, the output norm of the recurrence
    ([T, H, dv]: every head of every token on its own): RMSNorm(x) * weight *
    act(gate), or with gate_first RMSNorm(x * act(gate)) * weight.

    x [..., dim] fp32 or bf16, dim up to 16384; weight fp32 [dim] or None
    (ones); gate as x, or None for the plain norm; activation None, "silu" or
    "sigmoid".  Rows may lie at any one stride.  out may be x or gate itself.
    Sums and everything up to the result's rounding are fp32."""
    if _fast is not None and stream is None:
        done = _fast.gated_norm(x, weight, gate, activation, gate_first, eps, out)
        if done is not None:
            return done
    dev, dt, dim = _norm_common("gated_norm", x, activation)
    shape = x.shape
    xp, xs = _rows(x, "x", shape, dt, dev)
    wp = _weight(weight, "weight", dim, dev)
    zp, zs = (0, 0) if gate is None else _rows(gate, "gate", shape, dt, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(x) if xs == 0 else x.new_empty(shape)
            yp, ys = out.data_ptr(), 0
        else:
            yp, ys = _rows(out, "out", shape, dt, dev)
        if dim == 0:
            return out
        desc = _al.GATED_NORM.pack(
            _al.GATED_NORM.size, _DTYPES[dt], dim, _GATES[activation], 1 if gate_first else 0, eps,
            x.numel() // dim, xp, wp, zp, yp, xs, zs, ys)
        st = _al.lib().kda_gated_norm(desc, _raw_stream(dev))
    if st != _abi.KDA_OK:
        raise _abi.KdaError(st, "kda_gated_norm")
    return out


def block_norm(x: torch.Tensor, residual: torch.Tensor,
               weight_post: Optional[torch.Tensor] = None,
               weight_pre: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               activation=None, channel_scale: Optional[torch.Tensor] = None, scale: float = 1.0,
               eps: float = 1e-6, residual_out: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, stream=None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """A block's output x joins the residual stream, and the sum's norm is the
    next block's input, in one pass:

        r = residual + scale * channel_scale * act(gate) * RMSNorm(x; weight_post)
        y = RMSNorm(r; weight_pre)

    Returns (r, y).  weight_post None: x as it is; weight_pre None: no y (None);
    gate (as x), channel_scale (fp32 [dim]) None: no such factor.  x, gate and y
    are [..., dim] fp32 or bf16, dim up to 16384; the residual is fp32, or bf16
    with bf16 x; weights fp32 [dim].  y comes from r before r is rounded.
    residual_out may be residual itself; out may be x or gate itself.  Rows may
    lie at any one stride."""
    if _fast is not None and stream is None:
        done = _fast.block_norm(x, residual, weight_post, weight_pre, gate, activation, channel_scale,
                                scale, eps, residual_out, out)
        if done is not None:
            return done
    dev, dt, dim = _norm_common("block_norm", x, activation)
    shape = x.shape
    rd = residual.dtype if isinstance(residual, torch.Tensor) else None
    if rd not in _DTYPES:
        raise TypeError("residual must be an fp32 or bf16 tensor")
    xp, xs = _rows(x, "x", shape, dt, dev)
    rp, rs = _rows(residual, "residual", shape, rd, dev)
    wpost = _weight(weight_post, "weight_post", dim, dev)
    wpre = _weight(weight_pre, "weight_pre", dim, dev)
    cp = _weight(channel_scale, "channel_scale", dim, dev)
    zp, zs = (0, 0) if gate is None else _rows(gate, "gate", shape, dt, dev)
    if out is not None and weight_pre is None:
        raise ValueError("out needs weight_pre")
    with _on(dev, stream):
        if residual_out is None:
            residual_out = torch.empty_like(residual) if rs == 0 else residual.new_empty(shape)
            rop, ros = residual_out.data_ptr(), 0
        else:
            rop, ros = _rows(residual_out, "residual_out", shape, rd, dev)
        yp, ys = 0, 0
        if weight_pre is not None:
            if out is None:
                out = torch.empty_like(x) if xs == 0 else x.new_empty(shape)
                yp = out.data_ptr()
            else:
                yp, ys = _rows(out, "out", shape, dt, dev)
        if dim == 0:
            return residual_out, out
        desc = _al.BLOCK_NORM.pack(
            _al.BLOCK_NORM.size, _DTYPES[dt], _DTYPES[rd], dim, _GATES[activation], eps, scale,
            x.numel() // dim, xp, rp, wpost, wpre, cp, zp, rop, yp, xs, rs, zs, ros, ys)
        st = _al.lib().kda_block_norm(desc, _raw_stream(dev))
    if st != _abi.KDA_OK:
        raise _abi.KdaError(st, "kda_block_norm")
    return residual_out, out
