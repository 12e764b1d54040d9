"""latent_decode and latent_extend in units of 64 queries, which calls with many queries
and long tables are made in, beside units of 32: the table's length alone chooses
(places without a page are not seen), so the same rows go through both."""
import itertools

import numpy as np
import pytest
import torch

import oracle
from latent_cases import BF, check_attention, cumulative, host64, ints, normal, paged

pytestmark = pytest.mark.gpu
NEW, LENS, PAGE = [40, 1, 0, 23], [300, 64, 5, 23], 16


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


def longer(table, columns):
    return np.concatenate([table, np.full((len(table), columns - table.shape[1]), -1)], 1)


def both(kda, q, cache, table, lens, cu, dc):
    """With the table as it is and as columns of a longer one: 64 tokens of 8 heads are 8 units of 64,
    which then have 400 tiles each."""
    cache, q, lens, cu = cache.cuda(), q.cuda(), ints(lens), ints(cu)
    for columns in (table.shape[1], 1600):
        yield kda.latent_extend(q, cache, ints(longer(table, columns)), lens, cu, dc, 0.07)


@pytest.mark.parametrize("dc,dr", itertools.product((256, 512), (32, 64)))
def test_every_shape(kda, dc, dr):
    cache, table = paged(40, LENS, dc, dr, PAGE, BF, fill=float("nan"))
    q, cu = normal(41, 64, 8, dc + dr), cumulative(NEW)
    ref = oracle.latent_attend(host64(q), host64(cache), table, LENS, cu, dc, 0.07)
    for o in both(kda, q, cache, table, LENS, cu, dc):
        check_attention(o, ref, 300, dc + dr)


@pytest.mark.parametrize("dc,dr", itertools.product((256, 512), (32, 64)))
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_seen(kda, dc, dr, value):
    """A new token's row that is not finite reaches the tokens from it on, of its sequence."""
    cache, table = paged(42, LENS, dc, dr, PAGE, BF)
    q, cu, at = normal(43, 64, 8, dc + dr), cumulative(NEW), 280
    ref = oracle.latent_attend(host64(q), host64(cache), table, LENS, cu, dc, 0.07)
    cache[table[0, at // PAGE], at % PAGE, 9] = value
    others = np.ones((64, 8, dc), bool)
    others[20:40] = False       # token i sees rows up to 260 + i
    for o in both(kda, q, cache, table, LENS, cu, dc):
        check_attention(o, ref, 300, dc + dr, where=others)
        if value != value:
            assert torch.isnan(o[20:40]).all()
        else:
            assert not torch.isfinite(o[20:40, :, 9]).all(1).any()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("dc,dr", itertools.product((256, 512), (32, 64)))
def test_values_that_no_query_sees(kda, dtype, dc, dr):
    """Rows past seq_lens that hold what is not finite in every place, in every kernel."""
    for fill in (float("nan"), float("inf")):
        cache, table = paged(44, [70, 130], dc, dr, PAGE, dtype, fill=fill)
        q = normal(45, 2, 40, dc + dr, dtype=dtype)
        ref = oracle.latent_attend(host64(q), host64(cache), table, [70, 130], [0, 1, 2], dc, 0.07)
        o = kda.latent_decode(q.cuda(), cache.cuda(), ints(table), ints([70, 130]), dc, 0.07)
        check_attention(o, ref, 130, dc + dr)


def test_decode_with_many_heads(kda):
    lens = [900, 0, 1, 64, 333, 1500]
    cache, table = paged(46, lens, 512, 64, 64, BF)
    q = normal(47, 6, 128, 576)
    ref = oracle.latent_attend(host64(q), host64(cache), table, lens, np.arange(7), 512, 0.07)
    for columns in (table.shape[1], 200):
        o = kda.latent_decode(q.cuda(), cache.cuda(), ints(longer(table, columns)), ints(lens), 512, 0.07)
        check_attention(o, ref, 1500, 576)
        assert torch.all(o[1] == 0)
