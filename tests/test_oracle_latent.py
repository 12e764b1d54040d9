"""Pins of the latent attention oracle: the dense form with a mask, values worked by hand,
the equality of the expanded and the absorbed form, and mistakes planted in it, each of
which a pin must see."""
import types

import numpy as np
import pytest
import torch

import oracle
import oracle.latent as source


def draw(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def softmax_dense(q, k, v, scale):
    """[T, H, d] on [K, H, d] by whole matrices, the last query beside the last key."""
    T, K = len(q), len(k)
    s = torch.einsum("thd,khd->htk", torch.from_numpy(q), torch.from_numpy(k)) * scale
    mask = torch.arange(K)[None] > torch.arange(T)[:, None] + K - T
    w = torch.softmax(s.masked_fill(mask, -torch.inf), -1).nan_to_num(0.0)
    return torch.einsum("htk,khe->the", w, torch.from_numpy(v)).numpy()


def pin_prefill(o):
    q, k, pe, v = draw(1, 9, 2, 6), draw(2, 12, 2, 4), draw(3, 12, 2), draw(4, 12, 2, 3)
    cu, ck = [0, 4, 4, 9], [0, 7, 7, 12]   # the end of a prompt, nothing, a whole prompt
    got = o.latent_prefill(q, k, pe, v, cu, ck, 0.3)
    keys = np.concatenate([k, np.repeat(pe[:, None], 2, 1)], 2)
    for n in range(3):
        t, j = slice(cu[n], cu[n + 1]), slice(ck[n], ck[n + 1])
        assert np.allclose(got[0][t], softmax_dense(q[t], keys[j], v[j], 0.3), rtol=1e-12, atol=1e-13)
    # queries before the first key are 0, and the last one sees every key
    got = o.latent_prefill(q[:5], k[:3], pe[:3], v[:3], [0, 5], [0, 3], 0.3)[0]
    assert np.all(got[:2] == 0) and np.allclose(got[2], v[0]) and np.all(got[3] != 0)


def pin_pages(o):
    H, dc, dr = 2, 4, 2
    lens, cu, table = [7, 0, 7], [0, 2, 2, 5], np.array([[3, 1, 9], [0, 0, 0], [4, -1, 2]])
    cache, q = draw(5, 5, 3, dc + dr), draw(6, 5, H, dc + dr)
    got = o.latent_attend(q, cache, table, lens, cu, dc, 0.2)[0]
    for n, at in ((0, [(3, 0), (3, 1), (3, 2), (1, 0), (1, 1), (1, 2), None]), (2, [(4, 0), (4, 1), (4, 2), None, None, None, (2, 0)])):
        for t in range(cu[n], cu[n + 1]):
            rows = np.array([cache[p] for p in at[:lens[n] - (cu[n + 1] - 1 - t)] if p is not None])
            for h in range(H):
                s = rows @ q[t, h] * 0.2
                w = np.exp(s) / np.exp(s).sum()
                assert np.allclose(got[t, h], w @ rows[:, :dc], rtol=1e-12, atol=1e-13)


def pin_forms(o):
    """With keys c Wk and values c Wv, the absorbed queries on the rows themselves give the
    expanded form's output."""
    H, dn, dr, dv, dc, T = 2, 4, 2, 3, 6, 5
    c, pe, q = draw(7, T, dc), draw(8, T, dr), draw(9, T, H, dn + dr)
    wk, wv = draw(10, H, dn, dc), draw(11, H, dc, dv)
    a = o.latent_prefill(q, np.einsum("tc,hnc->thn", c, wk), pe, np.einsum("tc,hcv->thv", c, wv), [0, T], [0, T], 0.4)[0]
    absorbed = np.concatenate([np.einsum("thn,hnc->thc", q[..., :dn], wk), q[..., dn:]], 2)
    b = o.latent_attend(absorbed, np.concatenate([c, pe], 1)[None], [[0]], [T], [0, T], dc, 0.4)[0]
    assert np.allclose(a, np.einsum("thc,hcv->thv", b, wv), rtol=1e-10, atol=1e-12)


def pin_rotary(o):
    x = draw(12, 3, 2, 4)
    f, pos = np.array([1.0, 0.25]), [0, 2, 5]
    for inter in (False, True):
        y = o.rotary(x, pos, f, inter, 1.5)
        a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :2], x[..., 2:])
        z = 1.5 * (a + 1j * b) * np.exp(1j * np.outer(pos, f))[:, None]
        ya, yb = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :2], y[..., 2:])
        assert np.allclose(ya + 1j * yb, z, rtol=1e-13, atol=1e-14)
    # the product of two turned vectors depends on their positions' difference alone
    u, v = draw(13, 1, 4), draw(14, 1, 4)
    d = [float((o.rotary(u, [i + 3], f) * o.rotary(v, [i], f)).sum()) for i in (0, 11)]
    assert np.isclose(d[0], d[1], rtol=1e-12)


def pin_rows(o):
    latent, pe, w, f = np.array([[3.0, 4.0], [1.0, 1.0], [0.0, 2.0]]), draw(15, 3, 2), np.array([2.0, 1.0]), np.array([0.5])
    rows, seq, at = o.latent_new_rows(latent, pe, [7, 2], [0, 2, 3], w, 0.0, f, False, 1.0)
    assert list(seq) == [0, 0, 1] and list(at) == [5, 6, 1]
    assert np.allclose(rows[0, :2], [6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]) and np.allclose(rows[1, :2], w)
    for t in range(3):
        z = (pe[t, 0] + 1j * pe[t, 1]) * np.exp(0.5j * at[t])
        assert np.allclose(rows[t, 2:], [z.real, z.imag])
    plain = o.latent_new_rows(latent, pe, [7, 2], [0, 2, 3], None, 0.0, None, False, 1.0)[0]
    assert np.array_equal(plain, np.concatenate([latent, pe], 1))
    eps = o.latent_new_rows(latent, pe, [7, 2], [0, 2, 3], np.ones(2), 0.5, None, False, 1.0)[0]
    assert np.allclose(eps[1, :2], 1 / np.sqrt(1.5))


def pin_bounds(o):
    """What the error bounds are made of."""
    q, k, v = np.array([[1.0, -2.0]]), np.array([[1.0, 1.0], [2.0, 0.0], [9.0, 9.0]]), np.array([[-1.0], [1.0], [5.0]])
    out, mean, prod = o.attend(q, k, v, [2], 0.5)
    w = np.exp([-0.5, 1.0]) / np.exp([-0.5, 1.0]).sum()
    assert np.allclose(out, [[w[1] - w[0]]]) and np.allclose(mean, [[1.0]]) and np.allclose(prod, [1.5])
    assert not np.any(o.attend(q, k, v, [0], 0.5)[0]) and not np.any(o.attend(q, k, v, [-3], 0.5)[0])


PINS = [pin_prefill, pin_pages, pin_forms, pin_rotary, pin_rows, pin_bounds]

MUTANTS = {
    "no_scale": ("s = (k[:n] @ q[r]) * scale", "s = k[:n] @ q[r]"),
    "one_key_more": ("limit = np.arange(lq) + 1 + lk - lq", "limit = np.arange(lq) + 2 + lk - lq"),
    "first_key_beside_first_query": ("limit = np.arange(lq) + 1 + lk - lq", "limit = np.arange(lq) + 1"),
    "no_sum": ("w = w / w.sum()", "w = w / len(w)"),
    "mean_signed": ("w @ np.abs(v[:n])", "w @ v[:n]"),
    "prod_signed": ("np.abs(k[:n]) @ np.abs(q[r])", "k[:n] @ q[r]"),
    "missing_page_read": ("if 0 <= table[p // size] < pages]", "if table[p // size] < pages]"),
    "page_of_the_pool": ("cache[table[p // size], p % size]", "cache[p // size, p % size]"),
    "values_with_positions": ("rows, rows[:, :dc]", "rows, rows[:, -dc:]"),
    "new_tokens_late": ("(cu[n + 1] - t) + 1", "(cu[n + 1] - t)"),
    "turned_back": ("x[..., a] * c - x[..., b] * s", "x[..., a] * c + x[..., b] * s"),
    "magnitude_of_one_side": ("magnitude * np.sin(angle)", "np.sin(angle)"),
    "position_from_start": ("at[cu[n]:cu[n + 1]] = lens[n] - cu[n + 1] + np", "at[cu[n]:cu[n + 1]] = -cu[n] + np"),
    "no_eps": ("keepdims=True) + eps)", "keepdims=True))"),
    "norm_of_sum": ("(c * c).mean(1", "(c * c).sum(1"),
    "no_weight": (" * weight", ""),
}


@pytest.mark.parametrize("pin", PINS)
def test_pin(pin):
    pin(oracle)


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_mutant_is_caught(name):
    old, new = MUTANTS[name]
    text = open(source.__file__).read()
    assert text.count(old) >= 1, f"mutation site for {name} not found in the oracle source"
    m = types.ModuleType("mutant")
    exec(compile(text.replace(old, new, 1), "mutant", "exec"), m.__dict__)
    for pin in PINS:
        try:
            pin(m)
        except (AssertionError, IndexError, ValueError):
            return
    pytest.fail(f"no pin sees {name}")
