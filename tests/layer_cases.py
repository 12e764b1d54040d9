"""Inputs and error bounds shared by the tests of linear attention and of the
norms around it.

Bounds are derived from the operators' arithmetic, not from runs.  u is the
unit roundoff of a type (half a step: bf16 2^-8, fp32 2^-24).  A(...) is the
oracle run on absolute values, which bounds every partial sum the kernel forms.

o of a prefill (bf16): the decayed scores P and the copy of the state that q
meets are rounded once each (u_bf16 relative on their terms, which together
are at most A), the result once more (u_bf16 |o|); on top of that fp32 terms.
fp32 terms: a sum of m fp32 values in any order is off by at most m u_fp32
times the sum of their absolute values.  One output adds dk products per
score, 64 scored values, dk products with the state, and carries the state's
own error: each of the chunks before it multiplied the state once (the decay,
and an error of at most 4 steps in the exponential) and added 64 tokens in at
most three parts each.  (64 + dk) 2 + 200 + 8 chunks steps cover this.
The state itself: 200 + 8 chunks steps of A, plus its own rounding when it is
stored in bf16.
"""
import numpy as np
import torch

import oracle

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32 = 2.0 ** -24


def host64(t):
    return t.detach().cpu().double().numpy()


def linear_inputs(seed, lengths, H, Hk, dk, dv, dtype, decay="token", g_scale=1.0, n_states=None,
                  state_dtype=torch.float32, h0=True):
    """Seeded inputs on the CPU in their storage types."""
    gen = torch.Generator().manual_seed(seed)
    T = sum(lengths)

    def n(*shape):
        return torch.randn(shape, generator=gen)

    q, k, v = n(T, Hk, dk).to(dtype), (n(T, Hk, dk) * dk ** -0.5).to(dtype), n(T, H, dv).to(dtype)
    g = -g_scale * torch.nn.functional.softplus(n(T, H) if decay == "token" else n(H))
    N = len(lengths)
    st = (0.5 * n(n_states or N, H, dk, dv)).to(state_dtype) if h0 else None
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    return dict(q=q, k=k, v=v, g=g, h0=st, cu=cu)


def cuda(d):
    return {a: (b.cuda() if isinstance(b, torch.Tensor) else b) for a, b in d.items()}


def linear_reference(i, scale=None, h0="h0"):
    """Oracle results and the bounds' absolute runs: o, ht, A(o), A(ht)."""
    scale = i["q"].shape[2] ** -0.5 if scale is None else scale
    q, k, v, g = (host64(i[x]) for x in ("q", "k", "v", "g"))
    s = None if i[h0] is None else host64(i[h0])
    cu = i["cu"].cpu().numpy()
    o, ht = oracle.linear_attention(q, k, v, g, s, cu, scale)
    oa, ha = oracle.linear_attention(np.abs(q), np.abs(k), np.abs(v), g, None if s is None else np.abs(s),
                                     cu, abs(scale))
    return o, ht, oa, ha


def _chunks(i):
    cu = i["cu"].cpu().numpy()
    return int(max((cu[1:] - cu[:-1]).max(initial=0), 0)) // 64 + 1


def check_linear(i, o, ht, scale=None, ref=None):
    """Every element of o and ht within the bounds above."""
    ro, rh, ao, ah = linear_reference(i, scale) if ref is None else ref
    dk, ch = i["q"].shape[2], _chunks(i)
    u = U[i["q"].dtype]
    steps = 2 * (64 + dk) + 200 + 8 * ch
    if o is not None and ro.size:
        bound = steps * F32 * ao + 1.01 * u * np.abs(ro) + (1.01 * u * ao if u > F32 else 0.0)
        off = np.abs(host64(o) - ro)
        assert np.all(off <= bound), f"o off by {np.max(off / (bound + 1e-300)):.2f} of its bound"
    if ht is not None:
        us = U[ht.dtype]
        bound = (200 + 8 * ch) * F32 * ah + 1.01 * us * np.abs(rh)
        off = np.abs(host64(ht) - rh)
        assert np.all(off <= bound), f"state off by {np.max(off / (bound + 1e-300)):.2f} of its bound"
