"""The fp64 oracle of a Mamba-2 layer's steps against closed forms and its gradients against differences (CPU)."""
import numpy as np
import pytest

from oracle import layer


def _differences(f, x, h=1e-6):
    """Central differences of the number f(x): off by h^2 |f'''| / 6 + 2^-53 |f| / h, below 1e-8 for the numbers here."""
    out = np.empty(x.shape)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        down = f()
        x[i] = keep
        out[i] = (up - down) / (2 * h)
    return out


def test_linear_is_the_quadratic_form():
    r = np.random.default_rng(1)
    T, dk, dv = 9, 5, 4
    q, k, v = r.standard_normal((T, dk)), r.standard_normal((T, dk)), r.standard_normal((T, dv))
    g, beta, S0 = -r.random(T), r.random(T), r.standard_normal((dv, dk))
    out, S, _ = layer.linear(q, k, v, g, beta, 0.7, S0, 0.5)
    G = np.cumsum(g)
    want = np.array([0.5 * (np.exp(G[t]) * S0 @ q[t] + sum(np.exp(G[t] - G[j]) * beta[j] * (q[t] @ k[j]) * v[j] for j in range(t + 1))) + 0.7 * v[t]
                     for t in range(T)])
    np.testing.assert_allclose(out, want, rtol=0, atol=1e-13)
    np.testing.assert_allclose(S, np.exp(G[-1]) * S0 + sum(np.exp(G[-1] - G[j]) * beta[j] * np.outer(v[j], k[j]) for j in range(T)), atol=1e-13)


def test_linear_gradients_against_differences():
    r = np.random.default_rng(2)
    T, dk, dv = 6, 4, 3
    a = {"q": r.standard_normal((T, dk)), "k": r.standard_normal((T, dk)), "v": r.standard_normal((T, dv)), "g": -r.random(T),
         "beta": r.random(T), "skip": np.array(0.3), "S0": r.standard_normal((dv, dk))}
    do, dS = r.standard_normal((T, dv)), r.standard_normal((dv, dk))

    def f():
        out, S, _ = layer.linear(**a, scale=0.6)
        return (out * do).sum() + (S * dS).sum()

    got = layer.linear_backward(**a, scale=0.6, do=do, dS=dS)
    for n in a:
        np.testing.assert_allclose(got["d" + n], _differences(f, a[n]), rtol=0, atol=1e-7)


@pytest.mark.parametrize("T,W,silu", [(0, 4, True), (1, 4, True), (2, 4, False), (7, 3, True), (5, 2, True), (4, 1, False)])
def test_conv_gradients_against_differences(T, W, silu):
    r = np.random.default_rng(T + W)
    D = 3
    a = {"x": r.standard_normal((T, D)), "w": r.standard_normal((D, W)), "bias": r.standard_normal(D), "first": r.standard_normal((W - 1, D))}
    dy, dlast = r.standard_normal((T, D)), r.standard_normal((W - 1, D))

    def f():
        y, last, _ = layer.conv(**a, silu=silu)
        return (y * dy).sum() + (last * dlast).sum()

    got = layer.conv_backward(**a, silu=silu, dy=dy, dlast=dlast)
    for n in a:
        np.testing.assert_allclose(got["d" + n], _differences(f, a[n]), rtol=0, atol=1e-7)


@pytest.mark.parametrize("gate", ["none", "before", "after"])
def test_norm_gradients_against_differences(gate):
    r = np.random.default_rng(5)
    a = {"x": r.standard_normal((4, 8)), "z": r.standard_normal((4, 8)), "w": r.standard_normal(8)}
    dy = r.standard_normal((4, 8))
    f = lambda: (layer.gated_norm(**a, gate=gate, eps=1e-3) * dy).sum()  # noqa: E731
    dx, dz, dw = layer.gated_norm_backward(**a, gate=gate, eps=1e-3, dy=dy)
    np.testing.assert_allclose(dx, _differences(f, a["x"]), rtol=0, atol=1e-7)
    np.testing.assert_allclose(dw.sum(0), _differences(f, a["w"]), rtol=0, atol=1e-7)
    if gate != "none":
        np.testing.assert_allclose(dz, _differences(f, a["z"]), rtol=0, atol=1e-7)
