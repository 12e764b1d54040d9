"""latent_append and rotary against the fp64 oracle.

Bounds: an angle is exact to fp32 after its fp64 reduction, its sine and cosine
are off by at most 4 half steps of fp32 (of 1), so a rotated value by
(4 + 3) F32 magnitude (|a| + |b|) and its rounding.  A normed value: the sum of dc
squares in any order, a root, a division and two products, (dc / 2 + 8) F32
relative, and its rounding."""
import itertools

import numpy as np
import pytest
import torch

import oracle
from latent_cases import BF, F32, U, cumulative, host64, ints, normal, paged

pytestmark = pytest.mark.gpu
DTYPES = [BF, torch.float32]


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


def frequencies(dim):
    return 10000.0 ** (-np.arange(0, dim, 2) / dim)


def check_turned(got, x, want, interleaved, magnitude):
    x = np.abs(x)
    half = x.shape[-1] // 2
    both = x[..., 0::2] + x[..., 1::2] if interleaved else x[..., :half] + x[..., half:]
    both = np.repeat(both, 2, -1) if interleaved else np.concatenate([both, both], -1)
    bound = 7 * F32 * abs(magnitude) * both + 1.01 * U[got.dtype] * np.abs(want)
    assert np.all(np.abs(host64(got) - want) <= bound)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 128, 256])
def test_rotary(kda, dtype, interleaved, dim):
    T, H = 70, 5
    x = normal(dim, T, H, dim, dtype=dtype)
    at = np.random.default_rng(dim).integers(0, 40000, T)
    f = frequencies(dim)
    y = kda.rotary(x.cuda(), ints(at), torch.from_numpy(f).cuda(), interleaved=interleaved, magnitude=1.25)
    check_turned(y, host64(x), oracle.rotary(host64(x), at, f, interleaved, 1.25), interleaved, 1.25)


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 32), (3, 7), (5, 8), (2, 9), (1000, 3), (33, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_sizes(kda, tokens, heads, interleaved):
    x = normal(tokens, tokens, heads, 64)
    at, f = np.arange(tokens) * 3, frequencies(64)
    y = kda.rotary(x.cuda(), ints(at), torch.from_numpy(f).cuda(), interleaved=interleaved)
    check_turned(y, host64(x), oracle.rotary(host64(x), at, f, interleaved), interleaved, 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_far_positions(kda, interleaved):
    """To the ends of 32 bits, and behind 0."""
    at = np.array([0, 1, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31, 123456789])
    x, f = normal(1, 8, 3, 64, dtype=torch.float32), frequencies(64)
    y = kda.rotary(x.cuda(), ints(at), torch.from_numpy(f).cuda(), interleaved=interleaved, magnitude=-0.5)
    check_turned(y, host64(x), oracle.rotary(host64(x), at, f, interleaved, -0.5), interleaved, 0.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_a_part_of_the_heads(kda, dtype, interleaved):
    """In place on the last columns of wider heads, and from there into another buffer;
    the other columns stay."""
    T, H, at, f = 9, 4, np.arange(9) + 100, frequencies(32)
    q = normal(2, T, H, 96, dtype=dtype).cuda()
    x = host64(q[..., 64:])
    want = oracle.rotary(x, at, f, interleaved)
    fd = torch.from_numpy(f).cuda()
    out = torch.full((T, H, 200), 7.0, dtype=dtype, device="cuda")
    got = kda.rotary(q[..., 64:], ints(at), fd, interleaved=interleaved, out=out[..., 160:192])
    check_turned(got, x, want, interleaved, 1)
    assert torch.all(out[..., :160] == 7) and torch.all(out[..., 192:] == 7)
    before = q.clone()
    part = q[..., 64:]
    assert kda.rotary(part, ints(at), fd, interleaved=interleaved, out=part) is part
    assert torch.equal(part, got) and torch.equal(q[..., :64], before[..., :64])


def test_rotary_keeps_a_token_to_itself(kda):
    x = normal(3, 4, 2, 64)
    x[1, 0, 5] = float("nan")
    x[2, 1, 0] = float("inf")
    y = kda.rotary(x.cuda(), ints([1, 2, 3, 4]), torch.from_numpy(frequencies(64)).cuda(), interleaved=True)
    bad = ~torch.isfinite(y.cpu())
    assert bad[1, 0, 4:6].all() and bad[2, 1, :2].all() and bad.sum() == 4
    assert kda.rotary(x[:0].cuda(), ints([]), torch.from_numpy(frequencies(64)).cuda()).shape == (0, 2, 64)


def append(kda, cache, latent, pe, table, lens, cu, dtype, weight, f, interleaved, magnitude=1.0, **kw):
    return kda.latent_append(cache, latent, pe, ints(table), ints(lens), None if cu is None else ints(cu),
                             weight=None if weight is None else torch.from_numpy(weight).float().cuda(), eps=1e-5,
                             frequencies=None if f is None else torch.from_numpy(f).cuda(), interleaved=interleaved,
                             magnitude=magnitude, **kw)


def check_rows(got, latent, pe, want, dc, weight, f, interleaved, magnitude=1.0):
    """Rows [n, dc + dr] of `got` against the oracle's."""
    u = U[got.dtype]
    g = host64(got)
    if weight is None:
        assert np.array_equal(g[:, :dc], latent)
    else:
        w = want[:, :dc]
        assert np.all(np.abs(g[:, :dc] - w) <= ((dc / 2 + 8) * F32 + 1.01 * u) * np.abs(w))
    if f is None:
        assert np.array_equal(g[:, dc:], pe)
    else:
        check_turned(got[:, dc:], pe, want[:, dc:], interleaved, magnitude)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dc,dr", itertools.product((256, 512), (32, 64)))
@pytest.mark.parametrize("norm,turn,interleaved", [(True, True, False), (True, True, True), (False, True, True),
                                                   (True, False, False), (False, False, False)])
def test_append(kda, dtype, dc, dr, norm, turn, interleaved):
    new, lens = [3, 0, 70, 1], [40, 9, 70, 1]
    cache, table = paged(5, lens, dc, dr, 16, dtype)
    cu = cumulative(new)
    latent, pe = normal(6, cu[-1], dc, dtype=dtype), normal(7, cu[-1], dr, dtype=dtype)
    weight = 1 + 0.1 * np.random.default_rng(8).standard_normal(dc).astype(np.float32).astype(np.float64) if norm else None
    if weight is not None:
        weight = weight.astype(np.float32).astype(np.float64)
    f = frequencies(dr) if turn else None
    want, seq, at = oracle.latent_new_rows(host64(latent), host64(pe), lens, cu, weight, 1e-5, f, interleaved, 1.1)
    c = cache.cuda()
    rows = torch.full((cu[-1], dc + dr), 7.0, dtype=dtype, device="cuda")
    assert append(kda, c, latent.cuda(), pe.cuda(), table, lens, cu, dtype, weight, f, interleaved, 1.1,
                  rows_out=rows) is c
    page = torch.from_numpy(table[seq, at // 16])
    got = c.cpu()[page, torch.from_numpy(at % 16)]
    check_rows(got, host64(latent), host64(pe), want, dc, weight, f, interleaved, 1.1)
    assert torch.equal(rows.cpu(), got)
    rest = cache.clone()
    rest[page, torch.from_numpy(at % 16)] = got
    assert torch.equal(c.cpu(), rest)  # nothing else was written


@pytest.mark.parametrize("page", [1, 7, 64])
def test_append_one_token_each(kda, page):
    """The decode step: no cu_seqlens; empty sequences and full pages among them."""
    lens = [1, 7, 8, 64, 65, 0, 200]
    cache, table = paged(9, lens, 256, 64, page, BF)
    latent, pe, f = normal(10, 7, 256), normal(11, 7, 64), frequencies(64)
    want, _, at = oracle.latent_new_rows(host64(latent), host64(pe), lens, np.arange(8), np.ones(256), 1e-5, f, False, 1.0)
    c = cache.cuda()
    append(kda, c, latent.cuda(), pe.cuda(), table, lens, None, BF, np.ones(256), f, False)
    rest = cache.clone()
    for n, L in enumerate(lens):
        if L == 0:
            continue
        p, r = table[n, at[n] // page], at[n] % page
        check_rows(c[p, r][None].cpu(), host64(latent[n:n + 1]), host64(pe[n:n + 1]), want[n:n + 1], 256, np.ones(256), f,
                   False)
        rest[p, r] = c[p, r].cpu()
    assert torch.equal(c.cpu(), rest)


def test_append_where_there_is_no_page(kda):
    """Pages outside the pool, positions past the table and before 0, tokens behind the
    last sequence: nothing is written there; rows_out has the sequences' tokens all the
    same."""
    new, lens = [4, 5, 3], [18, 2, 70]
    cache, table = paged(12, [18, 2, 64], 256, 32, 16, BF)
    table = table[:, :4].copy()  # 64 positions
    table[0, 1] = cache.shape[0] if table[0, 1] >= 0 else -1
    cu = cumulative(new)
    latent, pe = normal(13, 20, 256), normal(14, 20, 32)
    c = cache.cuda()
    rows = torch.full((20, 288), 7.0, dtype=BF, device="cuda")
    append(kda, c, latent.cuda(), pe.cuda(), table, lens, cu, BF, None, None, False, rows_out=rows)
    rest = cache.clone()
    for n in range(3):
        for i in range(new[n]):
            p = lens[n] - new[n] + i
            if 0 <= p < 64 and 0 <= table[n, p // 16] < cache.shape[0]:
                rest[table[n, p // 16], p % 16] = torch.cat([latent[cu[n] + i], pe[cu[n] + i]])
    assert torch.equal(c.cpu(), rest)
    assert torch.equal(rows[:12].cpu(), torch.cat([latent, pe], 1)[:12]) and torch.all(rows[12:] == 7)


def test_append_slices_of_one_projection(kda):
    """latent and k_pe out of wider rows, rows_out over them, a cache of wider rows."""
    lens, T = [30, 25], 25
    cu = np.array([0, 20, 25])
    cache, table = paged(15, lens, 512, 64, 16, BF)
    wide = torch.full((cache.shape[0], 2, 16, 584), 7.0, dtype=BF, device="cuda")
    view = wide[:, 1, :, :576]
    view.copy_(cache.cuda())
    x = normal(16, T, 640).cuda()
    before = x.clone()
    f = frequencies(64)
    rows = x[:, 32:608]
    want, seq, at = oracle.latent_new_rows(host64(x[:, 32:544]), host64(x[:, 544:608]), lens, cu, np.ones(512), 1e-5, f,
                                           True, 1.0)
    append(kda, view, x[:, 32:544], x[:, 544:608], table, lens, cu, BF, np.ones(512), f, True, rows_out=rows)
    check_rows(rows, host64(before[:, 32:544]), host64(before[:, 544:608]), want, 512, np.ones(512), f, True)
    assert torch.equal(x[:, :32], before[:, :32]) and torch.equal(x[:, 608:], before[:, 608:])
    got = view[torch.from_numpy(table[seq, at // 16]).cuda(), torch.from_numpy(at % 16).cuda()]
    assert torch.equal(got, rows)
    assert torch.all(wide[:, 0] == 7) and torch.all(wide[:, 1, :, 576:] == 7)


def test_append_far_and_many(kda):
    """Positions past 2^24 turn exactly; more sequences than one round of the search."""
    n = 5000
    lens = np.full(n, 2 ** 24 + 77)
    table = np.full((n, 5), -1)
    table[:, 4] = np.arange(n) % 3  # pages of 2^22 + 1 rows would be needed: these are not read
    latent, pe, f = normal(17, n, 256, dtype=torch.float32), normal(18, n, 32, dtype=torch.float32), frequencies(32)
    rows = torch.empty(n, 288, dtype=torch.float32, device="cuda")
    cache = torch.zeros(3, 16, 288, dtype=torch.float32, device="cuda")
    cu = np.arange(n + 1)
    append(kda, cache, latent.cuda(), pe.cuda(), table, lens, cu, torch.float32, None, f, False, rows_out=rows)
    want = oracle.latent_new_rows(host64(latent), host64(pe), lens, cu, None, 0, f, False, 1.0)[0]
    check_rows(rows, host64(latent), host64(pe), want, 256, None, f, False)
    assert torch.all(cache == 0)


def test_append_contents_that_break_the_rules(kda):
    cache, table = paged(19, [40, 40], 256, 32, 16, BF)
    latent, pe = normal(20, 12, 256), normal(21, 12, 32)
    for cu in ([0, 100, 12], [0, 12, 5], [7, -3, 12], [0, -2 ** 31, 2 ** 31 - 1], [12, 0, 0]):
        for lens in ([40, 40], [-2 ** 31, 2 ** 31 - 1]):
            append(kda, cache.cuda(), latent.cuda(), pe.cuda(), table, lens, cu, BF, None, None, False)
            torch.cuda.synchronize()
