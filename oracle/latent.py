"""Latent attention, its cache rows and the rotation, in float64 with numpy; the
definitions row by row -- TEST INFRASTRUCTURE ONLY (see the package docstring).  Every attention also returns what an error bound needs:
the same with absolute values."""
import numpy as np


def attend(q, k, v, limit, scale):
    """q [R, d], k [L, d], v [L, e]; row r sees keys below limit[r].  Returns o [R, e],
    the weighted mean of |v|, and for each row the largest |scores|' sum of
    products over the keys it sees.  A row that sees none: 0."""
    o = np.zeros((len(q), v.shape[1]))
    mean, prod = np.zeros_like(o), np.zeros(len(q))
    for r in range(len(q)):
        n = int(min(max(limit[r], 0), len(k)))
        if n == 0:
            continue
        with np.errstate(all="ignore"):
            s = (k[:n] @ q[r]) * scale
            w = np.exp(s - s.max())
            w = w / w.sum()
            # 0 x inf would be NaN where a weight underflows; a visible row's values count as they are
            o[r], mean[r] = w @ v[:n], w @ np.abs(v[:n])
            prod[r] = (np.abs(k[:n]) @ np.abs(q[r])).max() * scale
    return o, mean, prod


def latent_prefill(q, k, k_pe, v, cu, cu_k, scale):
    """q [T, H, dn + dr], k [K, H, dn], k_pe [K, dr], v [K, H, dv]: o, mean and prod of
    attend for every token and head."""
    T, H, _ = q.shape
    o = np.zeros((T, H, v.shape[2]))
    mean, prod = np.zeros_like(o), np.zeros((T, H))
    for n in range(len(cu) - 1):
        t, j = slice(cu[n], cu[n + 1]), slice(cu_k[n], cu_k[n + 1])
        lq, lk = cu[n + 1] - cu[n], cu_k[n + 1] - cu_k[n]
        limit = np.arange(lq) + 1 + lk - lq
        for h in range(H):
            keys = np.concatenate([k[j, h], k_pe[j]], 1)
            o[t, h], mean[t, h], prod[t, h] = attend(q[t, h], keys, v[j, h], limit, scale)
    return o, mean, prod


def latent_rows(cache, table, length):
    """The rows of a sequence that exist, in order, and their positions."""
    pages, size = cache.shape[:2]
    at = [p for p in range(min(max(length, 0), len(table) * size)) if 0 <= table[p // size] < pages]
    rows = np.array([cache[table[p // size], p % size] for p in at]).reshape(len(at), cache.shape[2])
    return rows, np.array(at, dtype=np.int64)


def latent_attend(q, cache, table, lens, cu, dc, scale):
    """q [T, H, dc + dr] on cache [P, page, dc + dr]."""
    T, H, _ = q.shape
    o = np.zeros((T, H, dc))
    mean, prod = np.zeros_like(o), np.zeros((T, H))
    for n in range(len(lens)):
        rows, at = latent_rows(cache, table[n], lens[n])
        for t in range(cu[n], cu[n + 1]):
            limit = np.searchsorted(at, max(lens[n], 0) - (cu[n + 1] - t) + 1)
            o[t], mean[t], prod[t] = attend(q[t], rows, rows[:, :dc], np.full(H, limit), scale)
    return o, mean, prod


def rotary(x, positions, frequencies, interleaved=False, magnitude=1.0):
    """x [T, ..., dim]."""
    angle = np.asarray(positions, dtype=np.float64)[:, None] * frequencies
    angle = angle.reshape((len(x),) + (1,) * (x.ndim - 2) + (-1,))
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
    y = np.empty_like(x)
    half = x.shape[-1] // 2
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, half), slice(half, None))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def latent_new_rows(latent, k_pe, lens, cu, weight, eps, frequencies, interleaved, magnitude):
    """The rows that an append writes, [T, dc + dr], and each token's sequence and position."""
    T = len(latent)
    seq, at = np.full(T, -1), np.zeros(T, dtype=np.int64)
    for n in range(len(lens)):
        seq[cu[n]:cu[n + 1]] = n
        at[cu[n]:cu[n + 1]] = lens[n] - cu[n + 1] + np.arange(cu[n], cu[n + 1])
    c = latent
    if weight is not None:
        c = c / np.sqrt((c * c).mean(1, keepdims=True) + eps) * weight
    pe = k_pe if frequencies is None else rotary(k_pe, at, frequencies, interleaved, magnitude)
    return np.concatenate([c, pe], 1), seq, at
