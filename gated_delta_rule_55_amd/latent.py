"""PyTorch-facing entry points of latent attention and its paged cache
(include/kda_latent.h): argument marshalling only, as layer.py does for linear
attention.

A layer keeps one row per token for all heads, [c | k_pe]: a latent vector of dc
values and a positional part of dr.  Its serving path, call by call:

    latent_append    new tokens' rows into the pages (norm, rotation by position)
    rotary           the positional part of their queries
    latent_prefill   a prompt, on keys and values expanded per head
    latent_decode    one token per sequence, on the pages (absorbed queries)
    latent_extend    several new tokens per sequence, on the pages

The last two share three tables with the first: block_table int32 [N, MP] (the
pages of each sequence), seq_lens int32 [N] (its rows, new tokens among them) and,
where sequences have several new tokens, cu_seqlens int32 [N + 1].  All are read
on the device, so a captured graph follows their contents; a position without a
page of the cache (past the table, or a page number outside it) is neither
written nor seen.

Scores, softmax statistics and all sums are fp32.  In bf16 the softmax weights are rounded
to bf16 before they multiply the values, as the matrix cores take them (2^-8 of a weight at
most), and each output once more.

Calls run on the device of their tensors, on `stream` or that device's current
stream; outputs and workspaces made here are allocated for that stream.  Calls go
through the module _fast_latent (csrc/kda_latent_torch.cpp) where the device is the
current one and no stream is named; it answers None to every call that it does not
take or would have to refuse, which is then checked here, and made or refused.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _abi
from . import _abi_latent as _an
from .layer import _DTYPES, _on, _raw_stream

try:
    from . import _fast_latent
except ImportError:  # not built: every call is checked and made here
    _fast_latent = None


def _tensor(t, name, shape, dtype, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dense(t, name, shape, dtype, dev) -> int:
    """Checks a contiguous tensor; its address."""
    _tensor(t, name, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, shape, dtype, dev):
    """Checks a tensor whose rows (all but the first dimension) are dense; its address
    and the stride between rows (0: dense)."""
    _tensor(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t.data_ptr(), 0
    row = 1
    for size, st in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and st != row:
            raise ValueError(f"{name} must be dense but for its first stride, got {t.stride()}")
        row *= size
    if shape[0] == 1:
        return t.data_ptr(), 0
    if t.stride(0) < row:
        raise ValueError(f"{name}: rows must not overlap, got {t.stride()}")
    return t.data_ptr(), t.stride(0)


def _heads(t, name, shape, dtype, dev):
    """Checks a [rows, heads, d] tensor with dense d; its address, the stride between
    rows and the one between heads (0, 0: dense)."""
    _tensor(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t.data_ptr(), 0, 0
    s = t.stride()
    head = s[1] if shape[1] > 1 else shape[2]
    if s[2] != 1 or head < shape[2]:
        raise ValueError(f"{name}: heads must be dense and not overlap, got strides {s}")
    row = s[0] if shape[0] > 1 else shape[1] * head
    if row < (shape[1] - 1) * head + shape[2]:
        raise ValueError(f"{name}: rows must not overlap, got strides {s}")
    return t.data_ptr(), row, head


def _common(what, t, name, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} runs on the GPU only")
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    return t.device, t.dtype


def _positive(scale) -> float:
    scale = float(scale)
    if not (math.isfinite(scale) and scale >= 2.0 ** -126):
        raise ValueError(f"scale must be positive and finite in fp32, got {scale}")
    return scale


def _cu(cu, name, dev):
    """cu_seqlens: its sequences and address."""
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError(f"{name} must be an int32 tensor [N + 1]")
    return cu.shape[0] - 1, _dense(cu, name, cu.shape, torch.int32, dev)


def _workspace(given, need, dev):
    """Address and bytes of a call's workspace, and the tensor that holds it."""
    if given is None:
        n = need()
        if n == 0:
            return None, 0, None
        given = torch.empty(n, dtype=torch.uint8, device=dev)
    elif not isinstance(given, torch.Tensor) or given.device != dev or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return given.data_ptr(), given.numel() * given.element_size(), given


def latent_prefill_workspace_bytes(T: int, K: int, H: int, nope_dim: int, rope_dim: int, value_dim: int,
                                   n_seqs: int = 1, dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace latent_prefill needs for T queries and K keys in n_seqs sequences.  Not
    monotonic in these: a buffer for several sizes takes their maximum."""
    return _an.latent_prefill_workspace_bytes(_an.make(
        _an.LatentPrefillDesc, dtype=_DTYPES[dtype], n_seqs=n_seqs, n_heads=H, dn=nope_dim, dr=rope_dim,
        dv=value_dim, q_total=T, k_total=K, cu_seqlens_k=None if T == K else 16))


def latent_prefill(q: torch.Tensor, k: torch.Tensor, k_pe: torch.Tensor, v: torch.Tensor,
                   cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention over packed prompts on expanded keys and values:
    o_i = sum_j softmax_j(scale (q_i[:dn] . k_j + q_i[dn:] . k_pe_j)) v_j.

    q: [T, H, dn + dr]; k: [K, H, dn]; k_pe: [K, dr], shared by the heads; v:
    [K, H, dv]; dn and dv 64 or 128, dr 32 or 64; fp32 or bf16.  cu_seqlens: int32
    [N + 1] on the device, N at least 1, or None (one sequence).  cu_seqlens_k: the sequences'
    keys where they have more (or fewer) of them than queries, as in the end of a
    prompt whose beginning is expanded too: the last query stands beside the last
    key, and a query before the first key has output 0.  scale: (dn + dr)^-1/2 by
    default.  Returns o [T, H, dv].

    q and out may be slices of wider rows (their heads dense); k and v may be
    slices of one buffer [K, H, dn + dv], k_pe of wider rows; strides are multiples
    of 16 bytes.  cu_seqlens and cu_seqlens_k are read on the device: contents that
    do not ascend from 0 give unspecified results but no access out of bounds.
    Rows of out outside every sequence are left as they were.  workspace: a buffer of
    latent_prefill_workspace_bytes bytes (often 0), as in latent_decode."""
    if _fast_latent is not None and stream is None:
        done = _fast_latent.latent_prefill(q, k, k_pe, v, cu_seqlens, cu_seqlens_k, scale, out, workspace)
        if done is not None:
            return done
    dev, dt = _common("latent_prefill", q, "q", 3)
    for t, name in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a tensor [K, H, d]")
    T, H, dq = q.shape
    K, dn, dv = k.shape[0], k.shape[2], v.shape[2]
    dr = dq - dn
    qp, qs = _rows(q, "q", (T, H, dq), dt, dev)
    kp, ks, kh = _heads(k, "k", (K, H, dn), dt, dev)
    pp, ps = _rows(k_pe, "k_pe", (K, dr), dt, dev)
    vp, vs, vh = _heads(v, "v", (K, H, dv), dt, dev)
    N, cup, cukp = 1, None, None
    if cu_seqlens is not None:
        N, cup = _cu(cu_seqlens, "cu_seqlens", dev)
    if cu_seqlens_k is not None:
        if cu_seqlens is None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        cukp = _dense(cu_seqlens_k, "cu_seqlens_k", (N + 1,), torch.int32, dev)
    elif K != T:
        raise ValueError(f"{K} keys for {T} queries need cu_seqlens_k")
    with _on(dev, stream):
        if out is None:
            out = q.new_empty((T, H, dv))
        op, os_ = _rows(out, "out", (T, H, dv), dt, dev)
        desc = _an.LatentPrefillDesc(
            ctypes.sizeof(_an.LatentPrefillDesc), _DTYPES[dt], N, H, dn, dr, dv,
            0.0 if scale is None else _positive(scale), T, K, qp, kp, pp, vp, op, qs, ks, kh, ps, vs, vh, os_,
            cup, cukp)
        wp, wn, workspace = _workspace(workspace, lambda: _an.latent_prefill_workspace_bytes(desc), dev)
        st = _an.lib().kda_latent_prefill(ctypes.byref(desc), wp, wn, _raw_stream(dev))
    if st != _abi.KDA_OK:
        raise _abi.KdaError(st, "kda_latent_prefill")
    return out


def _tables(block_table, seq_lens, dev):
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be an int32 tensor [N, pages of a sequence]")
    N, MP = block_table.shape
    return (N, MP, _dense(block_table, "block_table", (N, MP), torch.int32, dev),
            _dense(seq_lens, "seq_lens", (N,), torch.int32, dev))


def _pages(cache, dev, dt):
    """A cache [P, page, W] whose rows are dense: its shape, address, page and row stride."""
    if not isinstance(cache, torch.Tensor) or cache.dim() != 3:
        raise ValueError("cache must be a tensor [pages, rows of a page, dc + dr]")
    P, page, W = cache.shape
    _tensor(cache, "cache", (P, page, W), dt, dev)
    if cache.is_contiguous():
        return P, page, W, cache.data_ptr(), 0, 0
    s = cache.stride()
    row = s[1] if page > 1 else W
    if s[2] != 1 or row < W or (P > 1 and s[0] < (page - 1) * row + W):
        raise ValueError(f"cache: rows must be dense and not overlap, got strides {s}")
    return P, page, W, cache.data_ptr(), s[0] if P > 1 else 0, row


def latent_workspace_bytes(T: int, H: int, latent_dim: int, rope_dim: int, n_seqs: int, max_pages: int,
                           page_size: int, dtype: torch.dtype = torch.bfloat16, extend: bool = False) -> int:
    """Bytes of workspace latent_decode (extend: latent_extend) needs for these sizes.  Not monotonic
    in these: a buffer for several sizes takes their maximum."""
    return _an.latent_workspace_bytes(_an.make(
        _an.LatentAttendDesc, dtype=_DTYPES[dtype], n_seqs=n_seqs, n_heads=H, dc=latent_dim, dr=rope_dim,
        page_size=page_size, max_pages=max_pages, scale=1.0, t_total=T, cu_seqlens=16 if extend else None))


def _attend(what, q, cache, block_table, seq_lens, cu_seqlens, latent_dim, scale, out, workspace, stream):
    if _fast_latent is not None and stream is None:
        done = _fast_latent.latent_attend(q, cache, block_table, seq_lens, cu_seqlens, latent_dim, scale, out, workspace)
        if done is not None:
            return done
    dev, dt = _common(what, q, "q", 3)
    T, H, W = q.shape
    N, MP, tp, lp = _tables(block_table, seq_lens, dev)
    P, page, _, cp, cps, crs = _pages(cache, dev, dt)
    if cache.shape[2] != W:
        raise ValueError(f"q has heads of {W}, the cache rows of {cache.shape[2]}")
    cup = None
    if cu_seqlens is not None:
        cup = _dense(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    elif T != N:
        raise ValueError(f"{what}: {T} tokens for {N} sequences")
    qp, qs = _rows(q, "q", (T, H, W), dt, dev)
    with _on(dev, stream):
        if out is None:
            out = q.new_empty((T, H, latent_dim))
        op, os_ = _rows(out, "out", (T, H, latent_dim), dt, dev)
        desc = _an.LatentAttendDesc(
            ctypes.sizeof(_an.LatentAttendDesc), _DTYPES[dt], N, H, latent_dim, W - latent_dim, page, MP, P,
            _positive(scale), T, qp, cp, op, qs, cps, crs, os_, tp, lp, cup)
        wp, wn, workspace = _workspace(workspace, lambda: _an.latent_workspace_bytes(desc), dev)
        st = _an.lib().kda_latent_attend(ctypes.byref(desc), wp, wn, _raw_stream(dev))
    if st != _abi.KDA_OK:
        raise _abi.KdaError(st, "kda_latent_attend")
    return out


def latent_decode(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  latent_dim: int, scale: float, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of one new token per sequence over the paged cache, in the absorbed
    form: o = sum_j softmax_j(scale q . row_j) row_j[:latent_dim].

    q: [N, H, dc + dr], the queries with the key projection multiplied in, then
    their (rotated) positional part; cache: [P, page, dc + dr]; dc = latent_dim 256
    or 512, dr 32 or 64; fp32 or bf16.  block_table: int32 [N, MP]; seq_lens: int32
    [N], the rows that each sequence's query sees (a sequence of length 0 has
    output 0).  scale: that of the expanded heads, (dn + dr)^-1/2.  Returns o [N, H,
    dc], to be multiplied by the value projection.

    q and out may be slices of wider rows, the cache's pages may lie apart and its
    rows be wider (strides are multiples of 16 bytes).  workspace: a buffer of
    latent_workspace_bytes bytes, one for each call that may overlap another (a
    captured graph keeps its own); allocated here when None.  Rounding depends on
    all sequences' lengths, which decide where the rows are shared out.  The host knows MP alone, not
    the lengths: a table much wider than they are can cost time, never a result."""
    return _attend("latent_decode", q, cache, block_table, seq_lens, None, latent_dim, scale, out, workspace, stream)


def latent_extend(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  cu_seqlens: torch.Tensor, latent_dim: int, scale: float, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """latent_decode for several new tokens per sequence, whose rows are in the cache
    already: new token i of the cu_seqlens[n + 1] - cu_seqlens[n] of sequence n sees
    its rows up to its own, the last new token all seq_lens[n].

    q: [T, H, dc + dr], packed; cu_seqlens: int32 [N + 1] on the device (contents
    that do not ascend from 0 give unspecified results but no access out of
    bounds).  Rows of out outside every sequence are left as they were.  Everything
    else as in latent_decode."""
    if cu_seqlens is None:
        raise ValueError("latent_extend needs cu_seqlens")
    return _attend("latent_extend", q, cache, block_table, seq_lens, cu_seqlens, latent_dim, scale, out, workspace,
                   stream)


def _frequencies(f, dim, dev) -> int:
    return _dense(f, "frequencies", (dim // 2,), torch.float64, dev)


def _magnitude(m) -> float:
    m = float(m)
    if m == 0 or not math.isfinite(m) or abs(m) <= 2.0 ** -150:
        raise ValueError(f"magnitude must be finite and not 0 in fp32, got {m}")
    return m


def latent_append(cache: torch.Tensor, latent: torch.Tensor, k_pe: torch.Tensor, block_table: torch.Tensor,
                  seq_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  frequencies: Optional[torch.Tensor] = None, interleaved: bool = False, magnitude: float = 1.0,
                  rows_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Writes new tokens' rows [RMSNorm(latent) * weight | R(k_pe)] into the paged
    cache: new token i of sequence n's L at position seq_lens[n] - L + i, the
    rotation R by that position.

    cache: [P, page, dc + dr], written in place and returned; latent: [T, dc] and
    k_pe: [T, dr], as they leave their projection (both may be slices of its rows);
    block_table, seq_lens (which counts the new tokens), cu_seqlens as in
    latent_extend, None: one token per sequence.  weight: fp32 [dc], or None (no
    norm); frequencies: fp64 [dr / 2] (rotary_frequencies), or None (no rotation);
    interleaved and magnitude as in rotary.  rows_out: [T, dc + dr], receives the
    same rows (latent_prefill's k_pe and the input of its keys and values); it may
    be the buffer that latent and k_pe are slices of.

    A token whose position has no page is not written; rows of the cache that no
    token stands at, and of rows_out outside every sequence, are left as they were.
    No position twice: a page that stands twice in the table of a call that writes
    both places is left with either's rows, mixed."""
    if _fast_latent is not None and stream is None:
        done = _fast_latent.latent_append(cache, latent, k_pe, block_table, seq_lens, cu_seqlens, weight, eps,
                                          frequencies, interleaved, magnitude, rows_out)
        if done is not None:
            return done
    dev, dt = _common("latent_append", latent, "latent", 2)
    T, dc = latent.shape
    P, page, W, cp, cps, crs = _pages(cache, dev, dt)
    N, MP, tp, lp = _tables(block_table, seq_lens, dev)
    dr = W - dc
    lat, ls = _rows(latent, "latent", (T, dc), dt, dev)
    pp, ps = _rows(k_pe, "k_pe", (T, dr), dt, dev)
    cup = None
    if cu_seqlens is not None:
        cup = _dense(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    elif T != N:
        raise ValueError(f"latent_append: {T} tokens for {N} sequences need cu_seqlens")
    wp = None if weight is None else _dense(weight, "weight", (dc,), torch.float32, dev)
    fp = None if frequencies is None else _frequencies(frequencies, dr, dev)
    rp, rs = (None, 0) if rows_out is None else _rows(rows_out, "rows_out", (T, W), dt, dev)
    with _on(dev, stream):
        desc = _an.LatentAppendDesc(
            ctypes.sizeof(_an.LatentAppendDesc), _DTYPES[dt], N, dc, dr, page, MP, P,
            _an.KDA_ROTARY_INTERLEAVED if interleaved else _an.KDA_ROTARY_HALF, eps, _magnitude(magnitude), T,
            lat, pp, cp, rp, ls, ps, cps, crs, rs, wp, fp, tp, lp, cup)
        st = _an.lib().kda_latent_append(ctypes.byref(desc), _raw_stream(dev))
    if st != _abi.KDA_OK:
        raise _abi.KdaError(st, "kda_latent_append")
    return cache


def rotary(x: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor, interleaved: bool = False,
           magnitude: float = 1.0, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x turned by its tokens' positions: each pair (a, b) of a head becomes
    magnitude (a cos t - b sin t, b cos t + a sin t), t = position * frequency.

    x: [T, H, dim], often the last columns of wider heads (q[..., dn:]); dim a
    multiple of 16 up to 256; fp32 or bf16.  Pairs are (x[i], x[i + dim / 2]), or
    (x[2 i], x[2 i + 1]) where interleaved.  positions: int32 [T]; frequencies: fp64
    [dim / 2] (rotary_frequencies).  out may be x itself, or a slice of another
    buffer (the positional part of the absorbed queries).  Angles are formed in
    fp64, so far positions lose nothing; sine and cosine are fp32."""
    if _fast_latent is not None and stream is None:
        done = _fast_latent.rotary(x, positions, frequencies, interleaved, magnitude, out)
        if done is not None:
            return done
    dev, dt = _common("rotary", x, "x", 3)
    T, H, dim = x.shape
    xp, xs, xh = _heads(x, "x", (T, H, dim), dt, dev)
    pp = _dense(positions, "positions", (T,), torch.int32, dev)
    fp = _frequencies(frequencies, dim, dev)
    with _on(dev, stream):
        if out is None:
            out = x.new_empty((T, H, dim))
        yp, ys, yh = _heads(out, "out", (T, H, dim), dt, dev)
        desc = _an.RotaryDesc(
            ctypes.sizeof(_an.RotaryDesc), _DTYPES[dt], H, dim,
            _an.KDA_ROTARY_INTERLEAVED if interleaved else _an.KDA_ROTARY_HALF, _magnitude(magnitude), T, xp, yp,
            xs, xh, ys, yh, pp, fp)
        st = _an.lib().kda_rotary(ctypes.byref(desc), _raw_stream(dev))
    if st != _abi.KDA_OK:
        raise _abi.KdaError(st, "kda_rotary")
    return out


def rotary_frequencies(dim: int, base: float = 10000.0, factor: float = 1.0,
                       original_length: Optional[int] = None, slow: float = 1.0, fast: float = 32.0,
                       device=None) -> torch.Tensor:
    """Frequencies of rotary and latent_append, in radians per position: fp64
    [dim / 2], f_i = base^(-2 i / dim).

    For contexts `factor` times the trained length.  Without original_length every
    frequency is divided by the factor (positions are interpolated).  With it, by
    parts: a pair that turns fewer than `slow` times over original_length positions
    is divided, one that turns more than `fast` times is kept, and between them the
    two are mixed in proportion to the turns (some models mix in proportion to i
    instead: such frequencies are the caller's to make)."""
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and positive, got {dim}")
    if not (base > 0 and factor > 0 and fast > slow >= 0) or (original_length is not None and original_length <= 0):
        raise ValueError("base, factor and original_length must be positive, and fast above slow")
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    if original_length is None:
        f = f / factor
    else:
        keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / factor
    return f.to(device)
