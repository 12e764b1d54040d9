"""Long sequences that are cut into pieces and joined, on marked rows (latent_marks): a piece
that is lost, doubled or scaled by a wrong maximum shows, whichever it is."""
import numpy as np
import pytest
import torch

import oracle
from latent_cases import BF, check_attention, cumulative, host64, ints, paged
from latent_marks import COURSES, mark_cache, queries, scores, values

pytestmark = pytest.mark.gpu
DTYPES = [BF, torch.float32]
SCALE = 1.0


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


def all_heads(ref, heads):
    """The oracle's answer for the first four heads, whose queries the others repeat."""
    return [np.concatenate([x] * (-(-heads // 4)), 1)[:, :heads] for x in ref]


def wider(table, columns):
    return np.concatenate([table, np.full((len(table), max(columns - table.shape[1], 0)), -1)], 1)


def marked(lens, dc, dtype, course, columns=0):
    cache, table = paged(50, lens, dc, 64, 64, dtype)
    mark_cache(cache, table, lens, dc, course)
    return cache, wider(table, columns)


# (lengths, heads, columns of the table): one unit over the whole GPU, two units of one sequence, a few sequences
# of very different lengths, more units than are counted one by one, and (columns) units of 64 rows
DECODE = [([32768], 4, 0), ([30011], 40, 0), ([20000, 9, 8000, 0, 65], 4, 0), ([1500 - 9 * i for i in range(70)], 8, 0),
          ([20000, 4001], 64, 800)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("course", COURSES)
@pytest.mark.parametrize("lens,heads,columns", DECODE)
def test_decode(kda, dtype, course, lens, heads, columns):
    dc = 512
    cache, table = marked(lens, dc, dtype, course, columns)
    q = queries(len(lens), heads, dc + 64, dc, dtype)
    o = kda.latent_decode(q.cuda(), cache.cuda(), ints(table), ints(lens), dc, SCALE)
    ref = oracle.latent_attend(host64(q[:, :4]), host64(cache), table, lens, np.arange(len(lens) + 1), dc, SCALE)
    check_attention(o, all_heads(ref, heads), max(lens), dc + 64)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("course", COURSES)
@pytest.mark.parametrize("new,lens,heads,columns", [([5, 0, 40], [9000, 70, 3000], 8, 0), ([12], [16000], 4, 0),
                                                    ([20, 12], [7000, 12000], 16, 3100)])
def test_extend(kda, dtype, course, new, lens, heads, columns):
    dc, cu = 256, cumulative(new)
    cache, table = marked(lens, dc, dtype, course, columns)
    q = queries(int(cu[-1]), heads, dc + 64, dc, dtype)
    o = kda.latent_extend(q.cuda(), cache.cuda(), ints(table), ints(lens), ints(cu), dc, SCALE)
    ref = oracle.latent_attend(host64(q[:, :4]), host64(cache), table, lens, cu, dc, SCALE)
    check_attention(o, all_heads(ref, heads), max(lens), dc + 64)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("course", COURSES)
@pytest.mark.parametrize("new,keys,heads", [([5], [8000], 2), ([100, 0, 30], [4000, 500, 3001], 4), ([300], [5000], 1)])
def test_prefill(kda, dtype, course, new, keys, heads):
    """Queries whose keys are shared by several workgroups."""
    dn, dr, dv, T, K = 64, 32, 128, sum(new), sum(keys)
    q = queries(T, heads, dn + dr, dn, dtype)
    k = torch.zeros(K, heads, dn, dtype=dtype)
    v = torch.from_numpy(np.concatenate([values(n, dv) for n in keys])).to(dtype)[:, None].repeat(1, heads, 1)
    pe = torch.zeros(K, dr, dtype=dtype)
    pe[:, 0] = torch.from_numpy(np.concatenate([scores(course, n) for n in keys])).to(dtype)
    cu, cu_k = cumulative(new), cumulative(keys)
    assert kda.latent_prefill_workspace_bytes(T, K, heads, dn, dr, dv, len(new), dtype) > 0
    o = kda.latent_prefill(q.cuda(), k.cuda(), pe.cuda(), v.cuda(), ints(cu), ints(cu_k), scale=SCALE)
    ref = oracle.latent_prefill(host64(q), host64(k), host64(pe), host64(v), cu, cu_k, SCALE)
    check_attention(o, ref, max(keys), dn + dr)
