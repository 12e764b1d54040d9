"""latent_prefill where a block of queries is shared by several workgroups: few queries
over many keys."""
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
    return kda.latent_prefill(i["q"].cuda(), kv[..., :i["dn"]], i["pe"].cuda(), kv[..., i["dn"]:],
                              cu_seqlens=ints(i["cu"]), cu_seqlens_k=ints(i["cu_k"]), **kw)


def workspace_bytes(kda, i):
    K, H, d = i["kv"].shape
    return kda.latent_prefill_workspace_bytes(i["q"].shape[0], K, H, i["dn"], i["pe"].shape[1], d - i["dn"],
                                              len(i["cu"]) - 1, i["q"].dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,keys,H", [
    ([1], [3000], 3), ([5, 130, 1], [2001, 131, 64], 2), ([200], [2500], 9), ([0, 33, 0, 129], [7, 1500, 0, 1000], 5),
    ([900], [700], 1),   # queries before the first key
    ([129], [129], 2), ([300], [300], 1),
])
def test_few_queries_many_keys(kda, dtype, new, keys, H):
    for dn, dr, dv in ((128, 64, 128), (64, 32, 64)):
        i = prefill_inputs(100, new, keys, H, dn, dr, dv, dtype)
        o = call(kda, i, scale=0.1)
        check_attention(o, prefill_reference(i, 0.1), max(keys), dn + dr)
        for n, (a, b) in enumerate(zip(new, keys)):
            if a > b:
                assert torch.all(o[i["cu"][n]:i["cu"][n] + a - b] == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [300, 1230])  # a key that all queries see, one that the last ones do
def test_rows_that_are_not_seen(kda, dtype, value, at):
    """A value that is not finite reaches the queries that see its row and no other, of
    its column alone."""
    new, keys, col = [100, 30], [1300, 1000], 5
    i = prefill_inputs(101, new, keys, 2, 64, 32, 64, dtype)
    clean = prefill_reference(i, 0.1)
    i["kv"][at, 1, 64 + col] = value
    o = call(kda, i, scale=0.1)
    first = max(at - 1200, 0)
    others = np.ones(o.shape, bool)
    others[first:100, 1, col] = False
    check_attention(o, clean, 1300, 96, where=others)
    got = host64(o)[first:100, 1, col]
    assert len(got) and not np.isfinite(got).any()
    if value == value:
        assert np.all((got == value) | np.isnan(got))


def test_scores_that_differ_much_between_parts(kda):
    i = prefill_inputs(102, [70], [2048], 2, 64, 32, 64, torch.float32)
    for down in (False, True):
        t = torch.linspace(0.1, 12, 2048)
        kv = i["kv"].clone()
        kv[..., :64] *= (t.flip(0) if down else t)[:, None, None]
        j = dict(i, kv=kv)
        check_attention(call(kda, j, scale=0.5), prefill_reference(j, 0.5), 2048, 96)


def test_a_query_that_is_not_finite(kda):
    i = prefill_inputs(103, [40], [1500], 2, 128, 64, 128, BF)
    clean = prefill_reference(i, 0.1)
    i["q"][7, 0, 9] = float("nan")
    i["q"][39, 1, 0] = float("inf")
    o = call(kda, i, scale=0.1)
    at = np.ones(o.shape, bool)
    at[7, 0] = at[39, 1] = False
    check_attention(o, clean, 1500, 192, where=at)
    assert torch.isnan(o[7, 0]).all() and not torch.isfinite(o[39, 1]).any()


def test_workspace(kda):
    """A caller's buffer with any contents, the same bits again; too small, of another
    alignment or on the host: refused.  Rows of out that no sequence has stay."""
    i = prefill_inputs(104, [60, 3], [2000, 900], 4, 128, 64, 128, BF)
    need = workspace_bytes(kda, i)
    assert need > 0
    want = call(kda, i)
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(call(kda, i, workspace=ws[:need]), want)
    with pytest.raises(kda.KdaError):
        call(kda, i, workspace=ws[:need - 1])
    with pytest.raises(kda.KdaError):
        call(kda, i, workspace=ws[16:])
    with pytest.raises(ValueError):
        call(kda, i, workspace=torch.empty(need, dtype=torch.uint8))
    out = torch.full((70, 4, 128), 7.0, dtype=BF, device="cuda")
    i["q"] = torch.cat([i["q"], normal(9, 7, 4, 192)])
    call(kda, i, out=out)
    assert torch.equal(out[:63], want) and torch.all(out[63:] == 7)


def test_a_call_that_fills_the_gpu_needs_no_workspace(kda):
    assert kda.latent_prefill_workspace_bytes(32768, 32768, 32, 128, 64, 128) == 0
    assert kda.latent_prefill_workspace_bytes(0, 1000, 32, 128, 64, 128) == 0


def test_contents_that_break_the_rules(kda):
    i = prefill_inputs(105, [60, 60], [2000, 60], 2, 64, 32, 64, BF)
    kv = i["kv"].cuda()
    assert workspace_bytes(kda, i) > 0
    for cu in ([0, 200, 120], [0, 100, 50], [30, -5, 120], [0, -2 ** 31, 2 ** 31 - 1]):
        for cu_k in ([0, 10 ** 9, 7], [0, 2060, 2060], [2060, 0, 1000]):
            o = kda.latent_prefill(i["q"].cuda(), kv[..., :64], i["pe"].cuda(), kv[..., 64:], cu_seqlens=ints(cu),
                                   cu_seqlens_k=ints(cu_k))
            torch.cuda.synchronize()
            assert o.shape == (120, 2, 64)
