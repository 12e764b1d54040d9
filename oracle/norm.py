"""The norms around a layer's step in fp64 -- TEST INFRASTRUCTURE ONLY (see the
package docstring); the definitions in include/kda_norm.h."""
import numpy as np

from .conv import silu


def rmsnorm(u, w, eps):
    u = np.asarray(u, dtype=np.float64)
    y = u / np.sqrt(np.mean(u * u, axis=-1, keepdims=True) + eps)
    return y if w is None else y * np.asarray(w, dtype=np.float64)


def gate_activation(z, activation):
    z = np.asarray(z, dtype=np.float64)
    if activation in (None, "none"):
        return z
    return silu(z) if activation == "silu" else 1.0 / (1.0 + np.exp(-z))


def gated_norm(x, w, z, activation, gate_first, eps):
    x = np.asarray(x, dtype=np.float64)
    a = 1.0 if z is None else gate_activation(z, activation)
    return rmsnorm(x * a, w, eps) if gate_first else rmsnorm(x, w, eps) * a


def block_norm(x, r, w_post, w_pre, z, activation, c, scale, eps):
    """Returns (r', y), y None without w_pre."""
    p = np.asarray(x, dtype=np.float64)
    if w_post is not None:
        p = rmsnorm(p, w_post, eps)
    if z is not None:
        p = p * gate_activation(z, activation)
    if c is not None:
        p = p * np.asarray(c, dtype=np.float64)
    r = np.asarray(r, dtype=np.float64) + scale * p
    return r, (None if w_pre is None else rmsnorm(r, w_pre, eps))
