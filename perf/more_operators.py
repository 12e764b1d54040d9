"""Latent attention and its cache, as cases that can be timed and compared.

A layer of latent attention keeps one row per token for all heads: a latent vector of dc values and a
positional part of dr values that is rotated by the token's position.  Five operators, in a plain form
(elementary torch operations in 32 bits or more, rounded once) and through this package's entry points:

  prefill  the expanded form over packed prompts: per head a key of dn values beside the shared positional
           part, a value of dv; causal, the last query beside the last key
  decode   the absorbed form for one token per sequence: all heads' queries against the cached rows
           themselves, whose first dc values are the values too; rows found through a table of pages
  extend   the absorbed form for several new tokens per sequence, each seeing the rows up to its own
  append   new tokens' rows into the pages: RMSNorm of the latent vector, rotation of the positional part
  rotary   the rotation of the queries' positional part
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
SCORES = 1 << 28  # scores that a plain form holds at a time


def listed():
    return [
        # One long prompt at the prefill workload's size (32 heads of 128).  The largest case.
        dict(name="prefill-32k", op="prefill", dtype="bf16", tokens=32768, seqs=1, ragged=0.0, prefix=0, heads=32,
             dn=128, dr=64, dv=128),
        # Eight prompts of ragged lengths packed into one call.
        dict(name="prefill-varlen-8", op="prefill", dtype="bf16", tokens=33001, seqs=8, ragged=1.0, prefix=0,
             heads=32, dn=128, dr=64, dv=128),
        # The end of a prompt whose beginning was served before: 509 queries on 1,212 keys, in fp32 (the
        # parity path), smaller heads.
        dict(name="prefill-f32", op="prefill", dtype="f32", tokens=509, seqs=1, ragged=0.0, prefix=703, heads=16,
             dn=64, dr=32, dv=64),
        # The decode workload's batch: 64 sequences of ragged lengths, 8,192 cached rows on average.
        dict(name="decode-64", op="decode", dtype="bf16", seqs=64, context=64 * 8192, ragged=1.0, idle=0.0, heads=32,
             dc=512, dr=64, page=64),
        # A single long sequence: few rows of queries, one long axis.
        dict(name="decode-1", op="decode", dtype="bf16", seqs=1, context=32768, ragged=0.0, idle=0.0, heads=32,
             dc=512, dr=64, page=64),
        # A few short sequences in fp32, pages of an odd size, a row of the batch that holds no request: the
        # latency of one call.
        dict(name="decode-f32", op="decode", dtype="f32", seqs=4, context=700, ragged=1.0, idle=0.25, heads=16,
             dc=256, dr=32, page=7),
        # A prompt's next chunk over its cached beginning.
        dict(name="extend-2048", op="extend", dtype="bf16", seqs=1, tokens=2048, context=16384 + 2048, ragged=0.0,
             idle=0.0, heads=32, dc=512, dr=64, page=64),
        # Continuing sequences of a few tokens each, the serving step between prompts.
        dict(name="extend-24", op="extend", dtype="bf16", seqs=24, tokens=101, context=24 * 4096, ragged=1.0,
             idle=0.0, heads=32, dc=512, dr=64, page=16),
        # The cache rows of a long prompt.
        dict(name="append-32k", op="append", dtype="bf16", seqs=1, tokens=32768, context=32768, ragged=0.0, idle=0.0,
             dc=512, dr=64, page=64, norm=True, rotate=True, interleaved=True),
        # One row for each sequence of the decode batch.
        dict(name="append-64", op="append", dtype="bf16", seqs=64, tokens=64, context=64 * 512, ragged=1.0, idle=0.0,
             dc=512, dr=64, page=64, norm=True, rotate=True, interleaved=False),
        # The positional part of the queries of a long prompt, a slice of the projection's output.
        dict(name="rotary-32k", op="rotary", dtype="bf16", tokens=32768, heads=32, width=192, dr=64, far=32768,
             factor=1.0, interleaved=True),
        # The same for one decode step of 64 sequences at far positions, frequencies scaled for them.
        dict(name="rotary-64", op="rotary", dtype="bf16", tokens=64, heads=32, width=192, dr=64, far=1000000,
             factor=16.0, interleaved=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "decode", "extend", "extend", "append", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    big = dtype == "bf16"
    heads = rng.choice([1, 2, 3, 4, 8, 12, 16, 24, 32])
    dr = rng.choice([32, 64])
    case = dict(op=op, dtype=dtype)
    if op == "prefill":
        return dict(case, tokens=_spread(rng, 1, 16384 if big else 4096), seqs=_spread(rng, 1, 64),
                    ragged=rng.choice([0.0, 0.5, 1.0]), prefix=rng.choice([0, 0, _spread(rng, 1, 2000)]), heads=heads,
                    dn=rng.choice([64, 128]), dr=dr, dv=rng.choice([64, 128]))
    if op == "rotary":
        return dict(case, tokens=_spread(rng, 1, 32768), heads=heads, width=dr + rng.choice([0, 64, 128]), dr=dr,
                    far=_spread(rng, 100, 2000000), factor=rng.choice([1.0, 4.0, 32.0]),
                    interleaved=rng.random() < 0.5)
    case.update(seqs=_spread(rng, 1, 64), ragged=rng.choice([0.0, 0.5, 1.0]), idle=rng.choice([0.0, 0.0, 0.2]),
                dc=rng.choice([256, 512]), dr=dr, page=rng.choice([1, 7, 16, 64, 64, 100, 256]))
    if op == "decode":
        return dict(case, context=_spread(rng, 1, 300000 if big else 50000), heads=heads)
    if op == "extend":
        tokens = _spread(rng, 1, 1500 if big else 300)
        return dict(case, tokens=tokens, context=tokens + _spread(rng, 1, 30000 if big else 8000), heads=heads)
    tokens = _spread(rng, 1, 32768)
    return dict(case, tokens=tokens, context=tokens + _spread(rng, 1, 8000), norm=rng.random() < 0.7,
                rotate=rng.random() < 0.7, interleaved=rng.random() < 0.5)


def _parts(total, n, ragged, salt):
    """`total` in n parts: equal but for the remainder (ragged 0), or in proportion to uniform weights; where there
    is less than one for each, some are empty.  The same for every seed, so that the work is too."""
    rng = np.random.default_rng([total, n, salt])
    edges = np.cumsum(1 - ragged * rng.random(n))
    edges = np.floor(edges / edges[-1] * total + 1e-6).astype(np.int64)
    return np.diff(edges, prepend=0)


def _lengths(case):
    """New tokens and cached rows (the new ones among them) of each sequence."""
    N = case["seqs"]
    if case["op"] == "prefill":
        new = _parts(case["tokens"], N, case["ragged"], 1)
        return new, np.where(new > 0, new + case["prefix"], 0)
    if case["op"] == "decode":
        new, old = np.ones(N, np.int64), _parts(case["context"], N, case["ragged"], 2)
    else:
        new = _parts(case["tokens"], N, case["ragged"], 1)
        old = new + _parts(case["context"] - case["tokens"], N, case["ragged"], 2)
    idle = np.arange(N) < int(case["idle"] * N)  # rows of the batch that hold no request
    if case["op"] == "decode":
        return new, np.where(idle, 0, old)
    return np.where(idle, 0, new), np.where(idle, 0, old)


def _frequencies(case):
    """Radians per position: 10000^(-2 i / dr), for a longer context than the trained one (4,096) slowed by the
    factor where a dimension turns less than once over it, kept where it turns more than 32 times."""
    dr, factor = case["dr"], case.get("factor", 1.0)
    f = 10000.0 ** (-np.arange(0, dr, 2, dtype=np.float64) / dr)
    keep = np.clip((4096 * f / (2 * math.pi) - 1) / 31, 0, 1)
    return torch.from_numpy(keep * f + (1 - keep) * f / factor)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    host = np.random.default_rng([int(seed), 5])

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(dev)

    dt = DTYPES[case["dtype"]]
    s = dict(case=dict(case))
    if case["op"] == "rotary":
        T, H, dr = case["tokens"], case["heads"], case["dr"]
        s["q"] = normal(T, H, case["width"]).to(dt)
        s["x"] = s["q"][..., case["width"] - dr:]
        s["positions"] = ints(np.sort(host.integers(0, case["far"], T)))
        s["frequencies"] = _frequencies(case).to(dev)
        s["magnitude"] = 1.0 + 0.1 * math.log(case["factor"])
        return s
    new, old = _lengths(case)
    order = host.permutation(case["seqs"])  # the batch's order is the seed's
    new, old = new[order], old[order]
    s["new"], s["old"] = new.tolist(), old.tolist()  # the program that made the batch knows them
    s["cu"] = ints(np.concatenate([[0], np.cumsum(new)]))
    T = int(new.sum())
    if case["op"] == "prefill":
        H, dn, dr, dv = (case[x] for x in ("heads", "dn", "dr", "dv"))
        K = int(old.sum())
        s["q"] = normal(T, H, dn + dr).to(dt)
        kv = normal(K, H, dn + dv).to(dt)  # one projection's output
        s["k"], s["v"] = kv[..., :dn], kv[..., dn:]
        s["k_pe"] = normal(K, dr).to(dt)
        s["cu_k"] = ints(np.concatenate([[0], np.cumsum(old)])) if case["prefix"] else None
        s["scale"] = 1.5 * (dn + dr) ** -0.5
        return s
    dc, dr, page, N = case["dc"], case["dr"], case["page"], case["seqs"]
    pages = -(-old // page)
    pool = int(pages.sum()) + int(pages.sum()) // 8 + 2
    table = np.full((N, max(int(pages.max()), 1) + 1), -1)
    at = host.permutation(pool)
    for n in range(N):
        table[n, :pages[n]], at = at[:pages[n]], at[pages[n]:]
    s["table"], s["lens"] = ints(table), ints(old)
    s["cache"] = normal(pool, page, dc + dr).to(dt)
    if case["op"] == "append":
        rows = normal(T, dc + dr).to(dt)  # one projection's output
        s["latent"], s["k_pe"] = rows[:, :dc], rows[:, dc:]
        s["weight"] = 1 + 0.1 * normal(dc) if case["norm"] else None
        s["frequencies"] = _frequencies(case).to(dev) if case["rotate"] else None
        return s
    s["q"] = normal(T, case["heads"], dc + dr).to(dt)
    s["scale"] = 192 ** -0.5  # the expanded heads' width
    return s


# -- the plain forms ----------------------------------------------------------------------------


def _attend(q, k, v, seen, scale):
    """q [G, R, d], k [G, L, d], v [G, L, e] in fp32, seen [R, L] or [G, R, L]: softmax over the seen keys; a row that
    sees none is 0."""
    x = torch.matmul(q, k.transpose(1, 2).contiguous()) * scale
    x = torch.where(seen, x, torch.full((), -math.inf, device=x.device))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros((), device=x.device), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones((), device=x.device), total)


def _plain_prefill(s):
    case, dev = s["case"], s["q"].device
    H, dn = case["heads"], case["dn"]
    out = torch.empty(s["q"].shape[0], H, case["dv"], dtype=s["q"].dtype, device=dev)
    t0 = j0 = 0
    for n, L in zip(s["new"], s["old"]):
        step = max(1, SCORES // (H * max(L, 1)))
        q = s["q"][t0:t0 + n].float().transpose(0, 1)
        k = s["k"][j0:j0 + L].float().transpose(0, 1)
        pe = s["k_pe"][j0:j0 + L].float().expand(H, L, case["dr"])
        k, v = torch.cat([k, pe], -1), s["v"][j0:j0 + L].float().transpose(0, 1).contiguous()
        for a in range(0, n, step):
            b = min(n, a + step)
            end = L - n + b  # keys that the block's last query sees
            seen = torch.arange(end, device=dev) <= torch.arange(a, b, device=dev)[:, None] + (L - n)
            o = _attend(q[:, a:b].contiguous(), k[:, :end], v[:, :end], seen, s["scale"])
            out[t0 + a:t0 + b] = o.transpose(0, 1).to(out.dtype)
        t0, j0 = t0 + n, j0 + L
    return out


def _plain_decode(s):
    case, q, dev = s["case"], s["q"], s["q"].device
    N, H, W = q.shape
    dc, page, L = case["dc"], case["page"], max(max(s["old"]), 1)
    rows = s["cache"].view(-1, W)
    j = torch.arange(L, device=dev)
    out = torch.empty(N, H, dc, dtype=q.dtype, device=dev)
    step = max(1, SCORES // (L * W))
    for a in range(0, N, step):
        at = s["table"][a:a + step].long()[:, j // page]
        seen = (j < s["lens"][a:a + step, None]) & (at >= 0)
        c = rows[at.clamp(min=0) * page + j % page].float()
        o = _attend(q[a:a + step].float(), c, c[..., :dc], seen[:, None], s["scale"])
        out[a:a + step] = o.to(out.dtype)
    return out


def _plain_extend(s):
    case, dev = s["case"], s["q"].device
    T, H, W = s["q"].shape
    dc, page = case["dc"], case["page"]
    rows = s["cache"].view(-1, W)
    out = torch.empty(T, H, dc, dtype=s["q"].dtype, device=dev)
    t0 = 0
    for i, (n, L) in enumerate(zip(s["new"], s["old"])):
        j = torch.arange(L, device=dev)
        c = rows[s["table"][i].long()[j // page] * page + j % page].float()
        step = max(1, SCORES // (H * max(L, 1)))
        for a in range(0, n, step):
            b = min(n, a + step)
            end = L - n + b
            last = torch.arange(a, b, device=dev).repeat_interleave(H) + (L - n)
            q = s["q"][t0 + a:t0 + b].float().reshape(1, (b - a) * H, W)
            o = _attend(q, c[None, :end], c[None, :end, :dc], j[:end] <= last[:, None], s["scale"])
            out[t0 + a:t0 + b] = o.view(b - a, H, dc).to(out.dtype)
        t0 += n
    return out


def _turn(x, positions, frequencies, interleaved, magnitude):
    """x [T, ..., dr] in fp32 turned by position x frequency; angles in 64 bits."""
    angle = positions.double()[:, None] * frequencies
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (x.shape[-1] // 2,)
    cos = (magnitude * torch.cos(angle)).float().view(shape)
    sin = (magnitude * torch.sin(angle)).float().view(shape)
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    case, dev = s["case"], s["cache"].device
    page, W = case["page"], case["dc"] + case["dr"]
    cu = s["cu"].long()
    t = torch.arange(s["latent"].shape[0], device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    at = s["lens"].long()[seq] + t - cu[seq + 1]
    c, pe = s["latent"].float(), s["k_pe"].float()
    if s["weight"] is not None:
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["frequencies"] is not None:
        pe = _turn(pe, at, s["frequencies"], case["interleaved"], 1.0)
    slot = s["table"].long()[seq, at // page] * page + at % page
    s["cache"].view(-1, W)[slot] = torch.cat([c, pe], -1).to(s["cache"].dtype)
    return s["cache"]


def _plain_rotary(s):
    y = _turn(s["x"].float(), s["positions"], s["frequencies"], s["case"]["interleaved"], s["magnitude"])
    return y.to(s["x"].dtype)


# -- one pass -----------------------------------------------------------------------------------


def _own(s):
    import gated_delta_rule_55_amd as kda

    case = s["case"]
    if case["op"] == "prefill":
        return kda.latent_prefill(s["q"], s["k"], s["k_pe"], s["v"], cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"],
                                  scale=s["scale"])
    if case["op"] == "decode":
        return kda.latent_decode(s["q"], s["cache"], s["table"], s["lens"], case["dc"], s["scale"])
    if case["op"] == "extend":
        return kda.latent_extend(s["q"], s["cache"], s["table"], s["lens"], s["cu"], case["dc"], s["scale"])
    if case["op"] == "append":
        return kda.latent_append(s["cache"], s["latent"], s["k_pe"], s["table"], s["lens"], s["cu"],
                                 weight=s["weight"], eps=EPS, frequencies=s["frequencies"],
                                 interleaved=case["interleaved"])
    return kda.rotary(s["x"], s["positions"], s["frequencies"], interleaved=case["interleaved"],
                      magnitude=s["magnitude"])


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "extend": _plain_extend, "append": _plain_append,
            "rotary": _plain_rotary}[state["case"]["op"]](state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"] * case["dr"]
        return {"bytes": 2 * n * es + 4 * case["tokens"], "flops": 3 * n}
    new, old = _lengths(case)
    T, K = int(new.sum()), int(old.sum())
    pairs = int((new * (old - new) + new * (new + 1) // 2).sum())  # (query, key) that see each other
    if case["op"] == "prefill":
        H, dn, dr, dv = (case[x] for x in ("heads", "dn", "dr", "dv"))
        return {"bytes": es * (T * H * (dn + dr + dv) + K * (H * (dn + dv) + dr)),
                "flops": 2 * H * pairs * (dn + dr + dv)}
    dc, W = case["dc"], case["dc"] + case["dr"]
    if case["op"] == "append":
        return {"bytes": 2 * T * W * es + 4 * dc * case["norm"], "flops": T * (4 * dc + 3 * case["dr"])}
    if case["op"] == "decode":
        pairs = K
    H = case["heads"]
    return {"bytes": es * (K * W + T * H * (W + dc)), "flops": 2 * H * pairs * (W + dc)}


# -- the definitions in 64 bits -----------------------------------------------------------------


def _exact_rows(q, c, v, first, scale):
    """q [R, d] of one head (or of all, sharing the rows), keys c [L, d], values v [L, e]; row r sees the keys up to
    first[r].  In blocks of queries, with the sum of the weights beside the product."""
    R, L = q.shape[0], c.shape[0]
    o = torch.zeros(R, v.shape[1], dtype=torch.float64, device=q.device)
    j = torch.arange(L, device=q.device)[None, :]
    for a in range(0, R, 4096):
        n = int(first[a:a + 4096].max()) + 1
        if n < 1:
            continue
        w = (q[a:a + 4096] @ c[:n].t()).mul_(scale)
        w.masked_fill_(j[:, :n] > first[a:a + 4096, None], -1e300)
        w.sub_(w.max(1, keepdim=True).values).exp_()
        o[a:a + 4096] = (w @ v[:n]) / w.sum(1, keepdim=True) * (first[a:a + 4096, None] >= 0)
    return o


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        x = s["x"].double()
        z = torch.polar(torch.full((), s["magnitude"], dtype=torch.float64, device=x.device),
                        s["positions"].double()[:, None, None] * s["frequencies"])
        if case["interleaved"]:
            return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
        y = torch.complex(*x.chunk(2, -1)) * z
        return torch.cat([y.real, y.imag], -1)
    dev = s["cu"].device
    starts = np.concatenate([[0], np.cumsum(s["new"])])
    if case["op"] == "prefill":
        H, dn = case["heads"], case["dn"]
        ks = np.concatenate([[0], np.cumsum(s["old"])])
        out = torch.zeros(s["q"].shape[0], H, case["dv"], dtype=torch.float64, device=dev)
        for n, (lq, lk) in enumerate(zip(s["new"], s["old"])):
            tq, tk = slice(starts[n], starts[n + 1]), slice(ks[n], ks[n + 1])
            first = torch.arange(lq, device=dev) + (lk - lq)
            for h in range(H if lq else 0):
                c = torch.hstack([s["k"][tk, h].double(), s["k_pe"][tk].double()])
                out[tq, h] = _exact_rows(s["q"][tq, h].double(), c, s["v"][tk, h].double(), first, s["scale"])
        return out
    dc, page, table = case["dc"], case["page"], s["table"].tolist()
    where = [[(p, o) for p in table[n] for o in range(page)][:L] for n, L in enumerate(s["old"])]
    if case["op"] == "append":
        cache = s["cache"].double()
        latent, pe = s["latent"].double(), s["k_pe"].double()
        if s["weight"] is not None:
            latent = latent * (latent.pow(2).sum(1, keepdim=True) / dc + EPS).rsqrt() * s["weight"].double()
        for n, (lq, L) in enumerate(zip(s["new"], s["old"])):
            if lq == 0:
                continue
            p, o = torch.tensor(where[n][L - lq:], device=dev).t()
            tq = slice(starts[n], starts[n + 1])
            row = pe[tq]
            if s["frequencies"] is not None:
                z = torch.exp(1j * torch.arange(L - lq, L, device=dev).double()[:, None] * s["frequencies"])
                if case["interleaved"]:
                    y = torch.complex(row[:, 0::2], row[:, 1::2]) * z
                    row = torch.view_as_real(y).flatten(1)
                else:
                    y = torch.complex(*row.chunk(2, 1)) * z
                    row = torch.hstack([y.real, y.imag])
            cache[p, o] = torch.hstack([latent[tq], row])
        return cache
    out = torch.zeros(s["q"].shape[0], case["heads"], dc, dtype=torch.float64, device=dev)
    for n, (lq, L) in enumerate(zip(s["new"], s["old"])):
        if lq == 0 or L == 0:
            continue
        p, o = torch.tensor(where[n], device=dev).t()
        c = s["cache"][p, o].double()
        tq = slice(starts[n], starts[n + 1])
        q = s["q"][tq].double().flatten(0, 1)
        first = torch.arange(L - lq, L, device=dev).repeat_interleave(case["heads"])
        out[tq] = _exact_rows(q, c, c[:, :dc], first, s["scale"]).view(lq, case["heads"], dc)
    return out
