"""Inputs and error bounds shared by the tests of latent attention and its cache.

Bounds are derived from the operators' arithmetic, not from runs.  u is half a
step of a type (bf16 2^-8, fp32 2^-24), F32 that of fp32.  With w the exact
weights of a query, mean = sum w |v| and prod the largest sum of |q| |k| scale
over the keys it sees (oracle.attend returns both):

A score is a sum of d products in any order, times scale log2(e), less the
maximum: off by at most (d + 8) F32 prod.  The exponential's argument carries
that into a weight's relative error, once above and once below the fraction
line; the exponential itself is off by at most 2 F32, a running sum of L terms
by L F32, twice.  Each of the at most L / 64 + 1 rescalings multiplies by a
factor that is off by 3 F32.  Pieces that are joined add a rescaling each.
(3 L + 200) F32 covers all but the scores.  In bf16 a weight is rounded once
before it multiplies its value (u mean), and the output once more (u |o|).
"""
import numpy as np
import torch

import oracle

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32 = 2.0 ** -24
BF = torch.bfloat16


def host64(t):
    return t.detach().cpu().double().numpy()


def cumulative(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def ints(x, dev="cuda"):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(dev)


def normal(seed, *shape, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def check_attention(got, ref, keys, d, where=None):
    """Every element of `got` [T, H, e] within the bounds above of ref = (o, mean, prod);
    keys: the largest number that a query sees."""
    o, mean, prod = ref
    u = U[got.dtype]
    bound = mean * (2 * (d + 8) * F32 * prod[..., None] + (3 * keys + 200) * F32) + 1.01 * u * np.abs(o)
    if u > F32:
        bound = bound + 1.01 * u * mean
    off = np.abs(host64(got) - o)
    if where is not None:
        off, bound = off[where], bound[where]
    assert np.all(off <= bound + 1e-300), f"off by {np.max(off / (bound + 1e-300)):.2f} of its bound"


def prefill_inputs(seed, new, keys, H, dn, dr, dv, dtype):
    """Packed prompts on the CPU; k and v are slices of one buffer."""
    T, K = sum(new), sum(keys)
    kv = normal(seed + 1, K, H, dn + dv, dtype=dtype)
    return dict(q=normal(seed, T, H, dn + dr, dtype=dtype), kv=kv, pe=normal(seed + 2, K, dr, dtype=dtype),
                cu=cumulative(new), cu_k=cumulative(keys), dn=dn)


def prefill_reference(i, scale):
    kv = host64(i["kv"])
    return oracle.latent_prefill(host64(i["q"]), kv[..., :i["dn"]], host64(i["pe"]), kv[..., i["dn"]:], i["cu"],
                                 i["cu_k"], scale)


def paged(seed, lens, dc, dr, page, dtype, spare=3, fill=None):
    """A cache on the CPU with the sequences' pages in a random order, and the table
    (-1 behind each sequence's pages).  fill: what rows that hold no token are filled
    with."""
    r = np.random.default_rng(seed)
    pages = [-(-max(n, 0) // page) for n in lens]
    pool = sum(pages) + spare
    order = r.permutation(pool)
    table = np.full((len(lens), max(pages) + 1), -1)
    cache = normal(seed, pool, page, dc + dr, dtype=dtype)
    live = np.zeros((pool, page), bool)
    at = 0
    for n, p in enumerate(pages):
        table[n, :p] = order[at:at + p]
        for j in range(max(lens[n], 0)):
            live[table[n, j // page], j % page] = True
        at += p
    if fill is not None:
        cache[torch.from_numpy(~live)] = fill
    return cache, table
