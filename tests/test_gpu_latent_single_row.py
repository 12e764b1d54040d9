"""latent_append over its own inputs, and rotary in place, for calls of few tokens: the
decode step of one sequence and prompts of one token among them.  Bounds as in
test_gpu_latent_cache.py."""
import numpy as np
import pytest
import torch

import oracle
from latent_cases import BF, F32, U, host64, ints, normal, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_55_amd as m

    return m


@pytest.fixture(params=["native", "ctypes"])
def way(request, kda, monkeypatch):
    """The call by the native module, which has to take it, and by ctypes."""
    from gated_delta_rule_55_amd import latent

    if request.param == "ctypes":
        monkeypatch.setattr(latent, "_fast_latent", None)
    else:
        for name in ("latent_append", "rotary"):
            real = getattr(latent._fast_latent, name)

            def taken(*a, real=real):
                done = real(*a)
                assert done is not None
                return done

            monkeypatch.setattr(latent._fast_latent, name, taken)
    return request.param


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("tokens", [1, 2])
@pytest.mark.parametrize("several", [False, True])  # cu_seqlens given
@pytest.mark.parametrize("width,at", [(576, 0), (640, 32)])  # rows as they are, and out of wider ones
def test_append_over_its_inputs(kda, way, dtype, tokens, several, width, at):
    dc, dr, lens = 512, 64, [70, 5][:tokens]
    cache, table = paged(1, lens, dc, dr, 16, dtype)
    x = normal(2, tokens, width, dtype=dtype)
    f = 10000.0 ** (-np.arange(0, dr, 2) / dr)
    weight = torch.linspace(0.5, 1.5, dc)
    cu = np.arange(tokens + 1)
    latent, pe = host64(x[:, at:at + dc]), host64(x[:, at + dc:at + dc + dr])
    want, seq, pos = oracle.latent_new_rows(latent, pe, lens, cu, host64(weight), 1e-5, f, True, 1.0)
    y, c = x.cuda(), cache.cuda()
    rows = y[:, at:at + dc + dr]
    got = kda.latent_append(c, y[:, at:at + dc], y[:, at + dc:at + dc + dr], ints(table), ints(lens),
                            ints(cu) if several else None, weight=weight.cuda(), eps=1e-5,
                            frequencies=torch.from_numpy(f).cuda(), interleaved=True, rows_out=rows)
    assert got is c
    u, r = U[dtype], host64(rows)
    assert np.all(np.abs(r - want)[:, :dc] <= ((dc / 2 + 8) * F32 + 1.01 * u) * np.abs(want[:, :dc]))
    both = np.repeat(np.abs(pe[:, 0::2]) + np.abs(pe[:, 1::2]), 2, -1)
    assert np.all(np.abs(r - want)[:, dc:] <= 7 * F32 * both + 1.01 * u * np.abs(want[:, dc:]))
    place = torch.from_numpy(table[seq, pos // 16]), torch.from_numpy(pos % 16)
    rest = cache.clone()
    rest[place] = rows.cpu()
    assert torch.equal(c.cpu(), rest)
    assert torch.equal(y[:, :at].cpu(), x[:, :at]) and torch.equal(y[:, at + dc + dr:].cpu(), x[:, at + dc + dr:])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 4), (3, 1), (2, 4)])
def test_rotary_in_place(kda, way, dtype, tokens, heads):
    q = normal(3, tokens, heads, 192, dtype=dtype)
    f, pos = 10000.0 ** (-np.arange(0, 64, 2) / 64), np.arange(tokens) + 9
    x = host64(q[..., 128:])
    want = oracle.rotary(x, pos, f, False)
    d = q.cuda()
    kda.rotary(d[..., 128:], ints(pos), torch.from_numpy(f).cuda(), out=d[..., 128:])
    both = np.abs(x[..., :32]) + np.abs(x[..., 32:])
    bound = 7 * F32 * np.concatenate([both, both], -1) + 1.01 * U[dtype] * np.abs(want)
    assert np.all(np.abs(host64(d[..., 128:]) - want) <= bound)
    assert torch.equal(d[..., :128].cpu(), q[..., :128])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("tokens", [1, 5])
def test_rotary_into_other_columns(kda, way, dtype, tokens):
    """From some columns of the heads into others, in rows that hold more than the heads."""
    wide = normal(4, tokens, 4 * 192 + 576, dtype=dtype).cuda()
    before, heads = wide.clone(), wide[:, :4 * 192].unflatten(1, (4, 192))
    f, pos = 10000.0 ** (-np.arange(0, 64, 2) / 64), np.arange(tokens) + 9
    x = host64(heads[..., 128:])
    kda.rotary(heads[..., 128:], ints(pos), torch.from_numpy(f).cuda(), out=heads[..., 64:128])
    want, both = oracle.rotary(x, pos, f, False), np.abs(x[..., :32]) + np.abs(x[..., 32:])
    bound = 7 * F32 * np.concatenate([both, both], -1) + 1.01 * U[dtype] * np.abs(want)
    assert np.all(np.abs(host64(heads[..., 64:128]) - want) <= bound)
    heads[..., 64:128] = before[:, :4 * 192].unflatten(1, (4, 192))[..., 64:128]
    assert torch.equal(wide, before)
