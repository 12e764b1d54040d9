"""Pins of the linear attention and norm oracles: the dense matrix form, the
split of a run into two, and norms worked by hand."""
import numpy as np
import pytest

import oracle


def _draw(seed, T, H, Hk, dk, dv, N):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, Hk, dk)), r.standard_normal((T, Hk, dk)), r.standard_normal((T, H, dv)),
            -np.abs(r.standard_normal((T, H))), r.standard_normal((N, H, dk, dv)))


def test_linear_equals_dense_form():
    q, k, v, g, h0 = _draw(1, 23, 4, 2, 5, 3, 1)
    o, ht = oracle.linear_attention(q, k, v, g, h0, [0, 23], 0.7)
    for h in range(4):
        G = np.cumsum(g[:, h])
        D = np.tril(np.exp(G[:, None] - G[None, :]))
        qh, kh = q[:, h // 2], k[:, h // 2]
        want = 0.7 * ((D * (qh @ kh.T)) @ v[:, h] + np.exp(G)[:, None] * (qh @ h0[0, h]))
        assert np.allclose(o[:, h], want, rtol=1e-12, atol=1e-12)
        end = np.exp(G[-1]) * h0[0, h] + (np.exp(G[-1] - G)[:, None] * kh).T @ v[:, h]
        assert np.allclose(ht[0, h], end, rtol=1e-12, atol=1e-12)


def test_linear_split_packed_and_decode():
    q, k, v, g, h0 = _draw(2, 9, 2, 2, 4, 4, 1)
    o, ht = oracle.linear_attention(q, k, v, g, h0, [0, 9], 1.0)
    o1, h1 = oracle.linear_attention(q[:8], k[:8], v[:8], g[:8], h0, [0, 8], 1.0)
    o2, h2 = oracle.linear_decode(h1, q[8:], k[8:], v[8:], g[8:], 1.0)
    assert np.array_equal(np.concatenate([o1, o2]), o) and np.array_equal(h2, ht)
    # two packed sequences with an empty one between them
    hh = np.concatenate([h0, h0 + 1, h0])
    op, hp = oracle.linear_attention(q, k, v, g, hh, [0, 4, 4, 9], 1.0)
    assert np.array_equal(op[:4], o[:4]) and np.array_equal(hp[1], h0[0] + 1)
    o3, h3 = oracle.linear_attention(q[4:], k[4:], v[4:], g[4:], h0, [0, 5], 1.0)
    assert np.array_equal(op[4:], o3) and np.array_equal(hp[2], h3[0])


def test_linear_constant_decay_is_a_row_of_g():
    q, k, v, g, h0 = _draw(3, 6, 3, 1, 4, 2, 1)
    a = oracle.linear_attention(q, k, v, g[0], h0, [0, 6], 1.0)
    b = oracle.linear_attention(q, k, v, np.tile(g[0], (6, 1)), h0, [0, 6], 1.0)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_norms_by_hand():
    x = np.array([[3.0, 4.0]])
    rms = np.sqrt(12.5)
    assert np.allclose(oracle.rmsnorm(x, None, 0.0), x / rms)
    y = oracle.gated_norm(x, [2.0, 1.0], np.array([[0.0, 0.0]]), "sigmoid", False, 0.0)
    assert np.allclose(y, [[3 / rms, 2 / rms]])
    y = oracle.gated_norm(x, None, np.array([[2.0, 0.0]]), None, True, 0.0)
    assert np.allclose(y, [[np.sqrt(2.0), 0.0]])
    r, y = oracle.block_norm(x, [[1.0, 1.0]], None, [1.0, 1.0], None, None, [0.0, 1.0], 2.0, 0.0)
    assert np.allclose(r, [[1.0, 9.0]]) and np.allclose(y, r / np.sqrt(41.0))
    assert oracle.block_norm(x, x, [1.0, 1.0], None, None, None, None, 1.0, 0.0)[1] is None


@pytest.mark.parametrize("name,value", [("silu", 2 / (1 + np.exp(-2.0))), ("sigmoid", 1 / (1 + np.exp(-2.0))),
                                        (None, 2.0)])
def test_gate_activations(name, value):
    y = oracle.gated_norm([[1.0, -1.0]], None, [[2.0, 2.0]], name, False, 0.0)
    assert np.allclose(y, [[value, -value]])
