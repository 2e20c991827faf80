"""Pins of the prompt-side oracle: the eager recurrence of the C oracle, closed forms, and gradients by differences."""
import numpy as np
import pytest

import oracle as c_oracle
from oracle import prompt as P


def _inputs(T, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    f = lambda x: x.astype(np.float32).astype(np.float64)  # noqa: E731
    return (f(unit(r.standard_normal((T, dk)))), f(unit(r.standard_normal((T, dk)))), f(r.standard_normal((T, dv))),
            -np.logaddexp(0, r.standard_normal(T)), f(r.random(T)), f(0.3 * r.standard_normal((dv, dk))), 0.25)


def test_delta_rule_is_the_eager_gdn_recurrence():
    q, k, v, g, beta, S0, _ = _inputs(9, 16, 32)
    alpha = np.exp(g).astype(np.float32)
    o, S, _ = P.delta_rule(q, k, v, np.log(alpha.astype(np.float64)), beta, S0, 1.0)
    Sc = S0[None].copy()
    one = lambda x: x.astype(np.float32)[None]  # noqa: E731
    out = c_oracle.gdn_round(Sc, one(alpha), one(beta), one(k), one(v), one(q), np.array([9], np.int32))
    out = out[0] if isinstance(out, tuple) else out
    np.testing.assert_allclose(np.asarray(out)[0], o, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(Sc[0], S, rtol=1e-12, atol=1e-13)


def test_delta_rule_with_unit_beta_stores_the_value():
    q, k, v, g, beta, S0, s = _inputs(7, 16, 16)
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    _, S, _ = P.delta_rule(q, k, v, g, np.ones(7), S0, s)
    np.testing.assert_allclose(S @ k[-1], v[-1], atol=1e-14)


def test_closed_gate_forgets():
    q, k, v, g, beta, S0, s = _inputs(6, 16, 16)
    g[3] = -np.inf
    _, S, _ = P.delta_rule(q, k, v, g, beta, S0, s)
    _, S2, _ = P.delta_rule(q[3:], k[3:], v[3:], g[3:], beta[3:], np.zeros_like(S0), s)
    np.testing.assert_array_equal(S, S2)


def test_delta_rule_gradients_by_differences():
    args = list(_inputs(5, 8, 6))
    r = np.random.default_rng(1)
    do, dS = r.standard_normal((5, 6)), r.standard_normal((6, 8))
    loss = lambda a: (lambda o, S, _: (o * do).sum() + (S * dS).sum())(*P.delta_rule(*a))  # noqa: E731
    grads = P.delta_rule_backward(*args, do, dS)
    for i, g in zip((0, 1, 2, 3, 4, 5), grads):
        num = np.zeros_like(g)
        for j in np.ndindex(*g.shape):
            up, down = [x.copy() if isinstance(x, np.ndarray) else x for x in args], [x.copy() if isinstance(x, np.ndarray) else x for x in args]
            up[i][j] += 1e-6
            down[i][j] -= 1e-6
            num[j] = (loss(up) - loss(down)) / 2e-6
        np.testing.assert_allclose(g, num, rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("inter", [False, True])
def test_qk_norm_lengths_and_relative_angles(norm, inter):
    r = np.random.default_rng(2)
    x = r.standard_normal((4, 3, 32))
    freq = 100.0 ** (-np.arange(8) / 8.0)
    y = P.qk_norm(x, None, norm, 0.0, 16, inter, np.array([0, 5, 1000, 7]), freq, 2.0, 2)
    assert y.shape == (4, 6, 32)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), 2.0 * (1 if norm == "l2" else 32 ** 0.5))
    np.testing.assert_array_equal(y[:, 0], y[:, 1])
    # a product of two rotated rows depends on the difference of their positions alone
    one = lambda p: P.qk_norm(x[:1, :2], None, norm, 0.0, 16, inter, np.array([p]), freq, 1.0, 1)[0]  # noqa: E731
    np.testing.assert_allclose(one(3)[0] @ one(10)[1], one(1003)[0] @ one(1010)[1], rtol=1e-10)


@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_qk_norm_gradients_by_differences(norm):
    r = np.random.default_rng(3)
    x, w, dy = r.standard_normal((2, 2, 16)), r.standard_normal(16), r.standard_normal((2, 4, 16))
    pos, freq = np.array([3, 9]), 10.0 ** (-np.arange(4) / 4.0)
    f = lambda x, w: (P.qk_norm(x, w, norm, 1e-3, 8, False, pos, freq, 0.5, 2) * dy).sum()  # noqa: E731
    dx, dw = P.qk_norm_backward(x, w, norm, 1e-3, 8, False, pos, freq, 0.5, 2, dy)
    for a, g, call in ((x, dx, lambda z: f(z, w)), (w, dw, lambda z: f(x, z))):
        num = np.zeros_like(g)
        for j in np.ndindex(*g.shape):
            up, down = a.copy(), a.copy()
            up[j] += 1e-6
            down[j] -= 1e-6
            num[j] = (call(up) - call(down)) / 2e-6
        np.testing.assert_allclose(g, num, rtol=1e-6, atol=1e-7)


def test_ragged_tables_by_hand():
    cu, cub, seq, pos, bseq = P.ragged_tables([3, 0, -2, 5], [10, 0, 0, 1], 4, 7)
    assert cu.tolist() == [0, 3, 3, 3, 7] and cub.tolist() == [0, 1, 1, 1, 2]
    assert seq.tolist() == [0, 0, 0, 3, 3, 3, 3] and pos.tolist() == [10, 11, 12, 1, 2, 3, 4]
    assert bseq.tolist() == [0, 3, -1, -1, -1]
