"""The training oracle's gradients against central differences of its forward forms."""
import numpy as np
import pytest

from oracle import training_oracle as O


def differences(f, x, step=1e-6):
    g = np.empty_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


def close(a, b):
    # second-order error of the differences and their cancellation: far below any wrong term
    np.testing.assert_allclose(a, b, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(residual):
    g = np.random.default_rng(0)
    x, w, dy = g.standard_normal((3, 8)), g.standard_normal(8), g.standard_normal((3, 8))
    dres = g.standard_normal((3, 8)) if residual else None

    def f(x, w):
        h, y = O.rms_norm(x, None, w, 1e-3)
        return (y * dy).sum() + (0 if dres is None else (h * dres).sum())

    dh, mag, dw, dwmag = O.rms_norm_backward(dy, x, w, dres, 1e-3)
    close(dh, differences(lambda v: f(v, w), x))
    close(dw, differences(lambda v: f(x, v), w))
    assert np.all(mag >= np.abs(dh) - 1e-12) and np.all(dwmag >= np.abs(dw) - 1e-12)
    h, y = O.rms_norm(x, 2 * x, None, 0.0)
    np.testing.assert_allclose(h, 3 * x)
    np.testing.assert_allclose((y * y).mean(1), 1.0)


@pytest.mark.parametrize("linear_beta", [8.0, 0.0])
def test_situ(linear_beta):
    g = np.random.default_rng(1)
    gate, up, dy = (3 * g.standard_normal((4, 5)) for _ in range(3))

    def f(gate, up):
        a = 4.0 * np.tanh(gate / 4.0) / (1 + np.exp(-gate))
        return (dy * a * (8.0 * np.tanh(up / 8.0) if linear_beta else up)).sum()

    dg, mag, du = O.situ_backward(gate, up, dy, 4.0, linear_beta)
    close(dg, differences(lambda v: f(v, up), gate))
    close(du, differences(lambda v: f(gate, v), up))
    assert np.all(mag >= np.abs(dg) - 1e-12)


def test_grouped():
    g = np.random.default_rng(2)
    off = [1, 3, 3, 6]                             # the first and the last row belong to none
    x, w, dy = g.standard_normal((7, 4)), g.standard_normal((3, 5, 4)), g.standard_normal((7, 5))

    def f(x, w):
        return (O.grouped_linear(x, w, off, np.zeros((7, 5))) * dy).sum()

    close(O.grouped_linear_backward_x(dy, w, off, np.zeros((7, 4))), differences(lambda v: f(v, w), x))
    close(O.grouped_linear_backward_w(dy, x, off), differences(lambda v: f(x, v), w))
    add = g.standard_normal((3, 5, 4))
    np.testing.assert_allclose(O.grouped_linear_backward_w(dy, x, off, add), O.grouped_linear_backward_w(dy, x, off) + add)
    out = O.grouped_linear(x, w, [-5, 2, 99, 99], np.full((7, 5), 7.0))     # clamped
    np.testing.assert_allclose(out, np.concatenate([x[:2] @ w[0].T, x[2:] @ w[1].T]))
