"""Reference of the residual + RMSNorm, of the products grouped by expert, and of the
gradients of both and of SituGLU, in float64 NumPy (test infrastructure only), written
from the definitions.  Each gradient comes with the sum of the magnitudes of the terms it
is made of, which rounding errors are proportional to."""
from __future__ import annotations

import numpy as np


def rms_norm(x, residual, w, eps):
    """(h, y): the residual sum and its normalised rows."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else residual)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, y * (1.0 if w is None else w)


def rms_norm_backward(dy, h, w, dres, eps):
    """(dh, magnitude of dh's terms, dw, magnitude of dw's terms)."""
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    n = h * r
    g = dy * (1.0 if w is None else w)
    dh = r * (g - n * np.mean(g * n, axis=1, keepdims=True))
    mag = r * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), axis=1, keepdims=True))
    if dres is not None:
        dh, mag = dh + dres, mag + np.abs(dres)
    return dh, mag, (dy * n).sum(0), np.abs(dy * n).sum(0)


def situ_backward(g, u, dy, beta, linear_beta):
    """(grad_gate, its magnitude, grad_up) of out = beta tanh(g/beta) sigmoid(g) * up_out."""
    with np.errstate(over="ignore"):
        s, c = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
        sech2 = 1.0 / np.cosh(g / beta) ** 2
        if linear_beta > 0:
            b, db = linear_beta * np.tanh(u / linear_beta), 1.0 / np.cosh(u / linear_beta) ** 2
        else:
            b, db = u, 1.0
    a = beta * np.tanh(g / beta) * s
    one, two = sech2 * s, a * c
    return dy * b * (one + two), np.abs(dy * b) * (one + np.abs(two)), dy * a * db


def _groups(offsets, rows):
    for e in range(len(offsets) - 1):
        a = min(max(int(offsets[e]), 0), rows)
        yield e, a, min(max(int(offsets[e + 1]), a), rows)


def grouped_linear(x, w, offsets, out):
    """out[r] = W_e x[r] for the rows of each expert; other rows of `out` stay as they are."""
    for e, a, b in _groups(offsets, x.shape[0]):
        if b > a:
            out[a:b] = x[a:b] @ w[e].T
    return out


def grouped_linear_backward_x(dy, w, offsets, out):
    for e, a, b in _groups(offsets, dy.shape[0]):
        if b > a:
            out[a:b] = dy[a:b] @ w[e]
    return out


def grouped_linear_backward_w(dy, x, offsets, add=None):
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[1], x.shape[1])) if add is None else np.array(add, np.float64)
    for e, a, b in _groups(offsets, x.shape[0]):
        dw[e] += dy[a:b].T @ x[a:b]
    return dw
