"""Rows that lie so far apart that their places pass 32 bits: the operators of latent attention
have the bits of the same calls on dense tensors.  (Where rows lie decides nothing else.)"""
import numpy as np
import pytest
import torch

from latent_cases import BF, cumulative, ints, normal

pytestmark = pytest.mark.gpu
FAR = 1 << 22      # the largest stride of k, v, out and positional parts, in elements
ROWS = 1100        # 4.6e9 elements


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


class Far:
    """A buffer of rows FAR apart, of which slices are given out one after the other."""

    def __init__(self, dtype, rows=ROWS):
        self.rows, self.at = torch.empty(rows, FAR, dtype=dtype, device="cuda"), 0

    def slice(self, *shape):
        n = int(np.prod(shape))
        part = self.rows[:, self.at:self.at + n]
        self.at += n + 64
        return part.unflatten(1, shape) if len(shape) > 1 else part

    def put(self, x):
        part = self.slice(*x.shape[1:])
        part.copy_(x)
        return part


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_prefill(kda, dtype):
    H, dn, dr, dv = 2, 64, 32, 64
    q, kv = normal(1, ROWS, H, dn + dr, dtype=dtype).cuda(), normal(2, ROWS, H, dn + dv, dtype=dtype).cuda()
    pe = normal(3, ROWS, dr, dtype=dtype).cuda()
    far = Far(dtype)
    fq, fkv, fpe, out = far.put(q), far.put(kv), far.put(pe), far.slice(H, dv)
    assert out[-1].data_ptr() - far.rows.data_ptr() > 1 << 32
    for cu in ([0, ROWS], [0, 300, 301, 1000, ROWS - 3]):
        n = cu[-1]
        want = kda.latent_prefill(q, kv[..., :dn], pe, kv[..., dn:], ints(cu))
        kda.latent_prefill(fq, fkv[..., :dn], fpe, fkv[..., dn:], ints(cu), out=out)
        assert torch.equal(out[:n], want[:n])


@pytest.mark.parametrize("several", [False, True])
def test_attend_and_append(kda, several):
    H, dc, dr, page = 3, 256, 32, 10
    W, pages = dc + dr, ROWS // page
    far, pool = Far(BF), Far(BF)
    table = np.random.default_rng(4).permutation(pages).reshape(10, 11)
    if several:
        new, lens = np.full(10, 60), np.array([110, 60, 61, 100, 70, 99, 109, 80, 90, 60])
    else:
        table = np.repeat(table, ROWS // 10, 0)  # every token a sequence of its own, which share their pages
        new, lens = np.ones(ROWS, np.int64), 1 + np.arange(ROWS) % 110
    cu = ints(cumulative(new)) if several else None
    T, tb, ln = int(new.sum()), ints(table), ints(lens)
    cache = normal(5, pages, page, W).cuda()
    fcache = pool.rows[:, :W].unflatten(0, (pages, page))
    fcache.copy_(cache)
    if several:
        row = normal(6, T, W).cuda()
        frow = far.put(torch.cat([row, row.new_zeros(ROWS - T, W)]))[:T]
        f, w = kda.rotary_frequencies(dr, device="cuda"), torch.rand(dc, device="cuda")
        kda.latent_append(cache, row[:, :dc], row[:, dc:], tb, ln, cu, weight=w, frequencies=f, rows_out=row)
        kda.latent_append(fcache, frow[:, :dc], frow[:, dc:], tb, ln, cu, weight=w, frequencies=f, rows_out=frow)
        assert torch.equal(frow, row) and torch.equal(fcache, cache)
    q = normal(7, T, H, W).cuda()
    fq = far.put(torch.cat([q, q.new_zeros(ROWS - T, H, W)]))[:T]
    out = far.slice(H, dc)[:T]
    if several:
        want = kda.latent_extend(q, cache, tb, ln, cu, dc, 0.1)
        kda.latent_extend(fq, fcache, tb, ln, cu, dc, 0.1, out=out)
    else:
        want = kda.latent_decode(q, cache, tb, ln, dc, 0.1)
        kda.latent_decode(fq, fcache, tb, ln, dc, 0.1, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(kda, interleaved):
    x, pos = normal(8, ROWS, 4, 64).cuda(), ints(np.arange(ROWS) * 7)
    f, far = kda.rotary_frequencies(64, device="cuda"), Far(BF)
    fx, out = far.put(x), far.slice(4, 64)
    want = kda.rotary(x, pos, f, interleaved=interleaved)
    kda.rotary(fx, pos, f, interleaved=interleaved, out=out)
    assert torch.equal(out, want)
    kda.rotary(fx, pos, f, interleaved=interleaved, out=fx)
    assert torch.equal(fx, want)
