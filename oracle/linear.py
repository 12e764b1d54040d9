"""Linear attention with one decay per head, token by token in fp64 -- TEST
INFRASTRUCTURE ONLY (see the package docstring).

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,     o_t = scale S_t^T q_t

per (sequence, head), value head h reading key head h / (H / Hk); the
definition in include/kda_linear.h.
"""
import numpy as np


def linear_attention(q, k, v, g, h0, cu_seqlens, scale):
    """q, k [T, Hk, dk]; v [T, H, dv]; g [T, H] or [H]; h0 [N, H, dk, dv] or
    None.  Returns (o [T, H, dv], ht [N, H, dk, dv])."""
    q, k, v, g = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g))
    T, H, dv = v.shape
    dk, N = q.shape[2], len(cu_seqlens) - 1
    head = np.arange(H) // (H // q.shape[1])
    g = np.broadcast_to(g, (T, H))
    o = np.zeros((T, H, dv))
    ht = np.zeros((N, H, dk, dv)) if h0 is None else np.array(h0, dtype=np.float64)
    for n in range(N):
        S = ht[n]
        for t in range(int(cu_seqlens[n]), int(cu_seqlens[n + 1])):
            S *= np.exp(g[t])[:, None, None]
            S += k[t, head][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", S, q[t, head])
    return o, ht


def linear_decode(state, q, k, v, g, scale):
    """One token per sequence; returns (o [N, H, dv], new state)."""
    N = state.shape[0]
    return linear_attention(q, k, v, g, state, np.arange(N + 1), scale)
