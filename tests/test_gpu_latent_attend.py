"""latent_decode and latent_extend against the fp64 oracle."""
import itertools

import numpy as np
import pytest
import torch

import oracle
from latent_cases import BF, check_attention, cumulative, host64, ints, normal, paged

pytestmark = pytest.mark.gpu
DTYPES = [BF, torch.float32]
SCALE = 0.07


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


def decode(kda, q, cache, table, lens, dc, **kw):
    return kda.latent_decode(q.cuda(), cache.cuda(), ints(table), ints(lens), dc, SCALE, **kw)


def extend(kda, q, cache, table, lens, cu, dc, **kw):
    return kda.latent_extend(q.cuda(), cache.cuda(), ints(table), ints(lens), ints(cu), dc, SCALE, **kw)


def reference(q, cache, table, lens, cu, dc, scale=SCALE):
    return oracle.latent_attend(host64(q), host64(cache), np.asarray(table), lens, cu, dc, scale)


def each(lens):
    return np.arange(len(lens) + 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dc,dr", itertools.product((256, 512), (32, 64)))
def test_decode_every_shape(kda, dtype, dc, dr):
    lens = [100, 1, 0, 333]
    cache, table = paged(1, lens, dc, dr, 16, dtype, fill=float("nan"))
    q = normal(2, 4, 5, dc + dr, dtype=dtype)
    o = decode(kda, q, cache, table, lens, dc)
    check_attention(o, reference(q, cache, table, lens, each(lens), dc), 333, dc + dr)
    assert torch.all(o[2] == 0)


# a unit is 32 rows (token, head), a tile 64 rows of the cache
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [1, 15, 16, 31, 32, 33, 64, 70])
def test_decode_heads(kda, dtype, heads):
    lens = [65, 130, 7]
    cache, table = paged(3, lens, 256, 32, 64, dtype, fill=float("inf"))
    q = normal(4, 3, heads, 288, dtype=dtype)
    check_attention(decode(kda, q, cache, table, lens, 256), reference(q, cache, table, lens, each(lens), 256), 130, 288)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 64, 100, 1024])
def test_decode_lengths_and_pages(kda, page):
    lens = [1, 2, 63, 64, 65, 127, 128, 129, 500, 0, 31]
    cache, table = paged(5, lens, 512, 64, page, BF, fill=float("nan"))
    q = normal(6, len(lens), 4, 576)
    check_attention(decode(kda, q, cache, table, lens, 512), reference(q, cache, table, lens, each(lens), 512), 500, 576)


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_one_long_sequence(kda, dtype):
    """Cut into as many pieces as there are workgroups."""
    lens = [33000] if dtype == BF else [9001]
    cache, table = paged(7, lens, 512, 64, 64, dtype)
    q = normal(8, 1, 3, 576, dtype=dtype)
    check_attention(decode(kda, q, cache, table, lens, 512), reference(q, cache, table, lens, each(lens), 512), lens[0],
                    576)


def test_decode_a_large_ragged_batch(kda):
    """Runs that span several sequences, sequences that span several runs, and more
    sequences than threads look at in one round."""
    r = np.random.default_rng(9)
    lens = [int(x) for x in r.integers(0, 40, 600)]
    lens[17], lens[300], lens[599] = 5000, 3000, 1700
    cache, table = paged(9, lens, 256, 32, 16, BF, fill=float("nan"))
    q = normal(10, 600, 2, 288)
    check_attention(decode(kda, q, cache, table, lens, 256), reference(q, cache, table, lens, each(lens), 256), 5000, 288)


def test_pages_that_are_not_there(kda):
    """Page numbers outside the pool and lengths past the table: those rows are not seen."""
    lens = [200, 90, 1000, -5, 40]
    cache, table = paged(11, [200, 90, 320, 0, 40], 256, 64, 16, BF, fill=float("nan"))
    table = table[:, :20].copy()  # 320 positions
    table[0, 3] = -1
    table[0, 7] = cache.shape[0]
    table[1, 5] = 2 ** 31 - 1
    table[4] = -7  # none of its rows
    q = normal(12, 5, 6, 320)
    o = decode(kda, q, cache, table, lens, 256)
    check_attention(o, reference(q, cache, table, lens, each(lens), 256), 320, 320)
    assert torch.all(o[3:] == 0)
    # the table's last columns empty, in the midst of a batch of several tokens each
    cu = cumulative([3, 1, 4, 2, 5])
    q = normal(13, 15, 6, 320)
    o = extend(kda, q, cache, table, lens, cu, 256)
    check_attention(o, reference(q, cache, table, lens, cu, 256), 320, 320)
    # no pages at all
    o = kda.latent_decode(q[:5].cuda(), cache[:0].cuda(), ints(table), ints(lens), 256, SCALE)
    assert torch.all(o == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [1, 3, 8, 32, 40])
def test_extend(kda, dtype, heads):
    """Several tokens each, none, more than the sequence has rows (those see nothing)."""
    new, lens = [5, 1, 0, 70, 9, 2], [300, 1, 50, 70, 4, 129]
    cache, table = paged(14, lens, 256, 32, 16, dtype, fill=float("nan"))
    cu = cumulative(new)
    q = normal(15, cu[-1], heads, 288, dtype=dtype)
    o = extend(kda, q, cache, table, lens, cu, 256)
    check_attention(o, reference(q, cache, table, lens, cu, 256), 300, 288)
    assert torch.all(o[cu[4]:cu[4] + 5] == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dc,dr", itertools.product((256, 512), (32, 64)))
def test_extend_every_shape(kda, dtype, dc, dr):
    new, lens = [33, 40], [333, 40]
    cache, table = paged(16, lens, dc, dr, 64, dtype)
    cu = cumulative(new)
    q = normal(17, cu[-1], 4, dc + dr, dtype=dtype)
    check_attention(extend(kda, q, cache, table, lens, cu, dc), reference(q, cache, table, lens, cu, dc), 333, dc + dr)


@pytest.mark.parametrize("new,lens", [([600], [1500]), ([500], [500]), ([300, 1, 200], [301, 900, 2000])])
def test_extend_a_long_chunk(kda, new, lens):
    """Many units over few keys; sampled tokens are checked."""
    cache, table = paged(18, lens, 512, 64, 64, BF, fill=float("nan"))
    cu = cumulative(new)
    q = normal(19, cu[-1], 32, 576)
    o = extend(kda, q, cache, table, lens, cu, 512)
    for n, (a, L) in enumerate(zip(new, lens)):
        rows, _ = oracle.latent_rows(host64(cache), table[n], L)
        for t in {0, a // 2, a // 3, a - 1}:
            ref = oracle.attend(host64(q[cu[n] + t]), rows, rows[:, :512], np.full(32, L - a + t + 1), SCALE)
            check_attention(o[cu[n] + t], ref, L, 576)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_seen(kda, dtype, value):
    """A row that is not finite reaches the tokens that see it and none before it."""
    new, lens = [20, 3], [100, 50]
    cache, table = paged(20, lens, 256, 32, 16, dtype)
    cu = cumulative(new)
    q = normal(21, cu[-1], 3, 288, dtype=dtype)
    clean = reference(q, cache, table, lens, cu, 256)
    for column in (7, 260):  # of the latent vector, of the positional part
        bad = cache.clone()
        bad[table[0, 90 // 16], 90 % 16, column] = value  # seen by tokens 10 .. 19 of the first sequence
        o = extend(kda, q, bad, table, lens, cu, 256)
        at = np.ones(o.shape, bool)
        at[10:20] = False
        check_attention(o, clean, 100, 288, where=at)
        if value != value:
            assert torch.isnan(o[10:20]).all()


def test_a_query_that_is_not_finite(kda):
    lens = [100, 200]
    cache, table = paged(22, lens, 256, 32, 16, BF)
    q = normal(23, 2, 40, 288)
    clean = reference(q, cache, table, lens, each(lens), 256)
    q[0, 3, 0], q[1, 39, 280] = float("nan"), float("inf")
    o = decode(kda, q, cache, table, lens, 256)
    at = np.ones(o.shape, bool)
    at[0, 3] = at[1, 39] = False
    check_attention(o, clean, 200, 288, where=at)
    assert torch.isnan(o[0, 3]).all() and not torch.isfinite(o[1, 39]).any()


def test_scores_that_differ_much_between_pieces(kda):
    """Every piece of a long sequence has a maximum of its own."""
    lens = [9000]
    cache, table = paged(24, lens, 256, 32, 64, torch.float32)
    at = torch.arange(9000)
    growth = torch.linspace(0.01, 6, 9000)
    cache[torch.from_numpy(table[0])[at // 64], at % 64] *= growth[:, None]
    q = normal(25, 1, 8, 288, dtype=torch.float32)
    check_attention(decode(kda, q, cache, table, lens, 256), reference(q, cache, table, lens, [0, 1], 256), 9000, 288)


@pytest.mark.parametrize("several", [False, True])
def test_strides_and_rows_outside(kda, several):
    """Wider query, output and cache rows, pages that lie apart, tokens behind the last
    sequence."""
    lens = [40, 70]
    cache, table = paged(26, lens, 256, 64, 16, BF, fill=float("nan"))
    P = cache.shape[0]
    wide = torch.full((P, 3, 16, 328), float("nan"), dtype=BF, device="cuda")
    wide[:, 1, :, :320] = cache.cuda()
    view = wide[:, 1, :, :320]
    cu = cumulative([2, 3]) if several else each(lens)
    T = int(cu[-1]) + (4 if several else 0)
    q = normal(27, T, 3, 320)
    qw = torch.full((T, 1000), float("nan"), dtype=BF, device="cuda")
    qw[:, 8:968] = q.reshape(T, -1).cuda()
    ow = torch.full((T, 800), 7.0, dtype=BF, device="cuda")
    o, qv = ow[:, 16:784].unflatten(1, (3, 256)), qw[:, 8:968].unflatten(1, (3, 320))
    if several:
        got = kda.latent_extend(qv, view, ints(table), ints(lens), ints(cu), 256, SCALE, out=o)
    else:
        got = kda.latent_decode(qv, view, ints(table), ints(lens), 256, SCALE, out=o)
    assert got is o
    n = int(cu[-1])
    check_attention(o[:n], reference(q[:n], cache, table, lens, cu, 256), 70, 320)
    assert torch.all(ow[n:] == 7) and torch.all(ow[:, :16] == 7) and torch.all(ow[:, 784:] == 7)


def test_offsets_past_32_bits(kda):
    """A pool of more than 2^32 bytes and 2^31 values: pages at both ends."""
    page, W = 64, 576
    P = (2 ** 31 // (page * W)) + 1000
    cache = torch.zeros(P, page, W, dtype=BF, device="cuda")
    rows = normal(28, 200, W)
    table = np.array([[P - 1, 0, P - 2, P // 2 + 1]])
    full = torch.zeros(256, W, dtype=BF)
    full[:200] = rows
    for i, p in enumerate(table[0]):
        cache[int(p)] = full[64 * i:64 * i + 64].cuda()
    q = normal(29, 1, 8, W)
    o = kda.latent_decode(q.cuda(), cache, ints(table), ints([200]), 512, SCALE)
    small = full.view(4, 64, W)
    check_attention(o, reference(q, small, [[0, 1, 2, 3]], [200], [0, 1], 512), 200, W)


def test_the_same_page_in_two_sequences(kda):
    """A shared beginning: both sequences' tables name its pages."""
    lens = [100, 90]
    cache, table = paged(30, lens, 256, 32, 16, BF)
    table[1, :5] = table[0, :5]
    q = normal(31, 2, 4, 288)
    check_attention(decode(kda, q, cache, table, lens, 256), reference(q, cache, table, lens, each(lens), 256), 100, 288)


def test_the_same_call_has_the_same_bits(kda):
    lens = [3000, 70, 900]
    cache, table = paged(32, lens, 512, 64, 64, BF)
    q = normal(33, 3, 32, 576)
    a = decode(kda, q, cache, table, lens, 512)
    for _ in range(3):
        assert torch.equal(a, decode(kda, q, cache, table, lens, 512))


def test_workspace(kda):
    """A caller's buffer with any contents; too small or on the host: refused."""
    lens = [3000, 70]
    cache, table = paged(34, lens, 512, 64, 64, BF)
    q = normal(35, 2, 32, 576)
    want = decode(kda, q, cache, table, lens, 512)
    need = kda.latent_workspace_bytes(2, 32, 512, 64, 2, table.shape[1], 64)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    assert torch.equal(decode(kda, q, cache, table, lens, 512, workspace=ws), want)
    with pytest.raises(kda.KdaError):
        decode(kda, q, cache, table, lens, 512, workspace=ws[:-256])
    with pytest.raises(ValueError):
        decode(kda, q, cache, table, lens, 512, workspace=torch.empty(need, dtype=torch.uint8))


def test_contents_that_break_the_rules(kda):
    """Token counts that do not ascend or leave the tensors give some result and no fault."""
    lens = [40, 70]
    cache, table = paged(36, lens, 256, 32, 16, BF)
    q = normal(37, 12, 3, 288)
    for cu in ([0, 100, 12], [0, 12, 5], [7, -3, 12], [0, -2 ** 31, 2 ** 31 - 1], [12, 0, 0]):
        o = extend(kda, q, cache, table, lens, cu, 256)
        torch.cuda.synchronize()
        assert o.shape == (12, 3, 256)
