"""latent_prefill against the fp64 oracle."""
import itertools

import numpy as np
import pytest
import torch

from latent_cases import BF, check_attention, host64, ints, normal, prefill_inputs, prefill_reference

pytestmark = pytest.mark.gpu
DTYPES = [BF, torch.float32]


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


def call(kda, i, **kw):
    kv = i["kv"].cuda()
    same = np.array_equal(i["cu"], i["cu_k"])
    return kda.latent_prefill(i["q"].cuda(), kv[..., :i["dn"]], i["pe"].cuda(), kv[..., i["dn"]:],
                              cu_seqlens=ints(i["cu"]), cu_seqlens_k=None if same else ints(i["cu_k"]), **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dn,dr,dv", itertools.product((64, 128), (32, 64), (64, 128)))
def test_every_shape(kda, dtype, dn, dr, dv):
    i = prefill_inputs(10, [70, 1, 0, 133], [70, 1, 0, 133], 3, dn, dr, dv, dtype)
    ref = prefill_reference(i, (dn + dr) ** -0.5)
    check_attention(call(kda, i), ref, 133, dn + dr)


# one query block is 128 tokens, one wave's 32, one tile of keys 64
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 257, 700])
def test_lengths(kda, dtype, length):
    i = prefill_inputs(length, [length], [length], 2, 128, 64, 128, dtype)
    check_attention(call(kda, i), prefill_reference(i, 192 ** -0.5), length, 192)


@pytest.mark.parametrize("heads", [1, 2, 4, 5, 8, 12, 16, 24])
def test_heads_and_packing(kda, heads):
    """Every class of head counts that the workgroups are dealt out by; many short and
    empty sequences."""
    new = [0, 3, 130, 0, 0, 1, 64, 257, 2, 0]
    i = prefill_inputs(20 + heads, new, new, heads, 64, 32, 64, BF)
    check_attention(call(kda, i), prefill_reference(i, 96 ** -0.5), 257, 96)


def test_many_sequences(kda):
    """More sequences than one round of the search looks at."""
    r = np.random.default_rng(3)
    new = [int(x) for x in r.integers(0, 4, 4500)]
    i = prefill_inputs(30, new, new, 1, 64, 32, 64, BF)
    check_attention(call(kda, i), prefill_reference(i, 96 ** -0.5), 4, 96)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,keys", [
    ([5, 130, 1], [300, 131, 64]),        # the end of prompts
    ([40, 200, 7], [3, 0, 9]),            # queries before the first key: 0
    ([1, 0, 1], [0, 50, 513]),
])
def test_keys_of_their_own(kda, dtype, new, keys):
    i = prefill_inputs(40, new, keys, 3, 128, 64, 128, dtype)
    o = call(kda, i, scale=0.11)
    check_attention(o, prefill_reference(i, 0.11), max(keys), 192)
    for n, (a, b) in enumerate(zip(new, keys)):
        if a > b:
            assert torch.all(o[i["cu"][n]:i["cu"][n] + a - b] == 0)


def test_strides_scale_and_rows_outside(kda):
    """q, out and k_pe as slices of wider rows, k and v dense, tokens behind the last
    sequence left as they were."""
    T, H = 90, 3
    i = prefill_inputs(50, [60, 20], [60, 20], H, 64, 64, 128, BF)
    i["q"] = normal(51, T, H, 128)
    q = torch.full((T, H * 128 + 40), float("nan"), dtype=BF, device="cuda")
    q[:, 8:8 + H * 128] = i["q"].reshape(T, -1).cuda()
    pe = torch.full((T, 96), float("nan"), dtype=BF, device="cuda")
    pe[:80, 32:] = i["pe"].cuda()
    kv = torch.full((T, H, 192), float("nan"), dtype=BF, device="cuda")
    kv[:80] = i["kv"].cuda()
    out = torch.full((T, H * 128 + 16), 7.0, dtype=BF, device="cuda")
    o = out[:, 8:8 + H * 128].unflatten(1, (H, 128))
    got = kda.latent_prefill(q[:, 8:8 + H * 128].unflatten(1, (H, 128)), kv[..., :64].contiguous(), pe[:, 32:],
                             kv[..., 64:].contiguous(), cu_seqlens=ints(i["cu"]), scale=0.2, out=o)
    assert got is o
    i["q"] = i["q"][:80]
    check_attention(o[:80], prefill_reference(i, 0.2), 60, 128)
    assert torch.all(out[80:] == 7) and torch.all(out[:, :8] == 7) and torch.all(out[:, 8 + H * 128:] == 7)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_seen(kda, dtype, value):
    """A key or value that is not finite reaches the queries that see it and no other:
    not those before it, whose weights for it are 0 (0 x inf), nor the next sequence."""
    new = [150, 40]
    for part in ("k", "v", "pe"):
        i = prefill_inputs(60, new, new, 2, 64, 32, 64, dtype)
        clean = prefill_reference(i, 96 ** -0.5)
        if part == "k":
            i["kv"][100, 1, 5] = value
        elif part == "v":
            i["kv"][100, 1, 64 + 5] = value
        else:
            i["pe"][100, 3] = value
        o = call(kda, i)
        at = np.ones(o.shape, bool)
        at[100:150, (0 if part == "pe" else 1):] = False
        check_attention(o, clean, 150, 96, where=at)
        got = host64(o)[100:150, 1]
        if part == "v":
            other = np.arange(64) != 5
            assert not np.isfinite(got[:, 5]).any()
            if value == value:
                assert np.all((got[:, 5] == value) | np.isnan(got[:, 5])) and got[0, 5] == value
            check_attention(o[100:150, 1:, torch.from_numpy(other).cuda()], [x[100:150, 1:][..., other] if x.ndim == 3 else x[100:150, 1:]
                                                    for x in clean], 150, 96)
        elif value != value:
            assert np.isnan(got).all()


def test_a_query_that_is_not_finite(kda):
    i = prefill_inputs(61, [140], [140], 2, 128, 64, 128, BF)
    clean = prefill_reference(i, 192 ** -0.5)
    i["q"][70, 0, 9] = float("nan")
    i["q"][139, 1, 0] = float("inf")
    o = call(kda, i)
    at = np.ones(o.shape, bool)
    at[70, 0] = at[139, 1] = False
    check_attention(o, clean, 140, 192, where=at)
    assert torch.isnan(o[70, 0]).all() and not torch.isfinite(o[139, 1]).any()


def test_large_scores(kda):
    """Weights from 1 to 0 and a maximum that grows from tile to tile."""
    i = prefill_inputs(62, [400], [400], 2, 64, 32, 64, torch.float32)
    i["kv"][..., :64] *= torch.linspace(0.1, 12, 400)[:, None, None]
    check_attention(call(kda, i, scale=0.5), prefill_reference(i, 0.5), 400, 96)


def test_no_tokens(kda):
    q = torch.empty(0, 2, 96, dtype=BF, device="cuda")
    kv, pe = torch.empty(0, 2, 64, dtype=BF, device="cuda"), torch.empty(0, 32, dtype=BF, device="cuda")
    assert kda.latent_prefill(q, kv, pe, kv).shape == (0, 2, 64)
    q = torch.ones(3, 2, 96, dtype=BF, device="cuda")
    o = kda.latent_prefill(q, kv, pe, kv, cu_seqlens=ints([0, 3]), cu_seqlens_k=ints([0, 0]))
    assert torch.all(o == 0)


def test_a_long_prompt(kda):
    """Sampled queries of a prompt of many tiles and query blocks."""
    T, H = 9000, 8
    g = torch.Generator().manual_seed(5)
    q, kv, pe = (torch.randn(T, *s, generator=g).to(BF) for s in ((H, 192), (H, 256), (64,)))
    kvc = kv.cuda()
    o = kda.latent_prefill(q.cuda(), kvc[..., :128], pe.cuda(), kvc[..., 128:])
    import oracle

    for h, t in ((0, 8999), (7, 8998), (3, 4095), (5, 4096), (1, 127), (2, 6400)):
        keys = np.concatenate([host64(kv[:, h, :128]), host64(pe)], 1)
        ref = oracle.attend(host64(q[t:t + 1, h]), keys, host64(kv[:, h, 128:]), [t + 1], 192 ** -0.5)
        check_attention(o[t:t + 1, h:h + 1], [ref[0][:, None], ref[1][:, None], ref[2][:, None]], t + 1, 192)


def test_contents_that_break_the_rules(kda):
    """Tables that do not ascend or leave the tensors give some result and no fault."""
    i = prefill_inputs(63, [60, 60], [60, 60], 2, 64, 32, 64, BF)
    kv = i["kv"].cuda()
    for cu in ([0, 200, 120], [0, 100, 50], [30, -5, 120], [0, -2 ** 31, 2 ** 31 - 1]):
        o = kda.latent_prefill(i["q"].cuda(), kv[..., :64], i["pe"].cuda(), kv[..., 64:], cu_seqlens=ints(cu),
                               cu_seqlens_k=ints([0, 10 ** 9, 7]))
        torch.cuda.synchronize()
        assert o.shape == (120, 2, 64)


