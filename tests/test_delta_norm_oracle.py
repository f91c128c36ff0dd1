"""What pins the fp64 references of the trainable delta rule and of the block norm: the C oracle's recurrence, worked
values, and every gradient against differences of the forward pass."""
import numpy as np
import pytest

import oracle
from oracle import block_norm, delta


def _inputs(rng, T, Hk, Hv, dk, dv):
    k = rng.standard_normal((T, Hk, dk))
    return (rng.standard_normal((T, Hk, dk)), k / np.linalg.norm(k, axis=-1, keepdims=True), rng.standard_normal((T, Hv, dv)),
            -rng.random((T, Hv)), rng.random((T, Hv)), rng.standard_normal((Hv, dk, dv)))


def test_delta_is_the_gated_delta_rule(oracle_lib):
    """The same recurrence as the oracle of gdr_chunk_fwd, with the gate's logarithm and shared key heads."""
    rng = np.random.default_rng(1)
    q, k, v, g, b, S0 = _inputs(rng, 9, 2, 4, 8, 16)
    o, ST, states = delta.forward(q, k, v, g, b, S0)
    rep = lambda x: np.repeat(x, 2, axis=1)[None]  # noqa: E731
    o_c, S_c = oracle.forward(rep(q), rep(k), v[None], np.exp(g)[None], b[None], S0=S0[None])
    np.testing.assert_allclose(o, o_c[0], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(ST, S_c[0], rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(states[-1], ST)


def test_delta_one_token_by_hand():
    """a = 1/2, S = [[2], [4]], k = (1, 0), v = 5, beta = 1/4: X = [[1], [2]], e = 4, S' = [[2], [2]], o = 2 q0 + 2 q1."""
    o, ST, _ = delta.forward(np.array([[[3.0, -1.0]]]), np.array([[[1.0, 0.0]]]), np.array([[[5.0]]]), np.log([[0.5]]),
                             np.array([[0.25]]), np.array([[[2.0], [4.0]]]))
    np.testing.assert_allclose(ST, [[[2.0], [2.0]]])
    np.testing.assert_allclose(o, [[[4.0]]])


def test_delta_reset_forgets():
    rng = np.random.default_rng(2)
    q, k, v, g, b, S0 = _inputs(rng, 6, 1, 2, 4, 4)
    g[3] = -np.inf
    o, ST, _ = delta.forward(q, k, v, g, b, S0)
    o2, ST2, _ = delta.forward(q[3:], k[3:], v[3:], g[3:], b[3:])
    np.testing.assert_array_equal(o[3:], o2)
    np.testing.assert_array_equal(ST, ST2)
    assert (delta.backward(q, k, v, g, b, np.ones_like(v), np.ones_like(S0), S0)[3][3] == 0).all()


def _differences(loss, arrays, grads, rng, n=6, h=1e-6):
    """Differences along random directions: second order in h, so off by about h^2 and the loss's rounding over h."""
    for x, g in zip(arrays, grads):
        for _ in range(n):
            d = rng.standard_normal(x.shape)
            x += h * d
            up = loss()
            x -= 2 * h * d
            down = loss()
            x += h * d
            want = (g * d).sum()
            assert abs((up - down) / (2 * h) - want) <= 1e-6 * (1 + abs(want)) * 10


def test_delta_gradients_against_differences():
    rng = np.random.default_rng(3)
    q, k, v, g, b, S0 = _inputs(rng, 7, 2, 4, 5, 6)
    do, dST = rng.standard_normal(v.shape), rng.standard_normal(S0.shape)

    def loss():
        o, ST, _ = delta.forward(q, k, v, g, b, S0)
        return (o * do).sum() + (ST * dST).sum()
    _differences(loss, (q, k, v, g, b, S0), delta.backward(q, k, v, g, b, do, dST, S0), rng)


@pytest.mark.parametrize("norm", [None, "l2", "rms"])
@pytest.mark.parametrize("act", [None, "linear", "sigmoid", "silu"])
@pytest.mark.parametrize("next_norm", [None, "l2", "rms"])
def test_block_norm_gradients_against_differences(norm, act, next_norm):
    rng = np.random.default_rng(4)
    x, z, res, dy, dn = (rng.standard_normal((3, 8)) for _ in range(5))
    w, w2 = rng.standard_normal(8), rng.standard_normal(8)
    how = dict(norm=norm, weight=w, gate=z if act else None, act=act, scale=0.7, residual=res, res_scale=1.3, eps=1e-3,
               next_norm=next_norm, next_weight=w2 if next_norm else None)

    def loss():
        y, n = block_norm.forward(x, **how)
        return (y * dy).sum() + (0 if n is None else (n * dn).sum())
    grads = block_norm.backward(x, dy, dn=dn, **how)
    pairs = [(a, g) for a, g in zip((x, z, res, w, w2), grads) if g is not None]
    _differences(loss, [a for a, _ in pairs], [g for _, g in pairs], rng)


def test_block_norm_by_hand():
    """(3, 4): l2 norm 5; silu(0) = 0, so the residual alone is left; a row of zeros has r = 0 without eps."""
    y, n = block_norm.forward(np.array([[3.0, 4.0]]), norm="l2", eps=0.0, scale=10.0, next_norm="rms")
    np.testing.assert_allclose(y, [[6.0, 8.0]])
    np.testing.assert_allclose(n, np.array([[6.0, 8.0]]) / np.sqrt(50))
    y, _ = block_norm.forward(np.ones((1, 4)), gate=np.zeros((1, 4)), act="silu", residual=np.full((1, 4), 2.0), res_scale=0.5)
    np.testing.assert_allclose(y, np.ones((1, 4)))
    assert (block_norm.forward(np.zeros((1, 4)), eps=0.0)[0] == 0).all()
