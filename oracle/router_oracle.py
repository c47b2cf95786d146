"""Reference of the router's balance loss and of the gradient of its logits, in
float64 NumPy (test infrastructure only), written from the definitions."""
from __future__ import annotations

import numpy as np


def sigmoid(l):
    l = np.asarray(l, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-l))


def shares(l):
    """q = s / sum of s over the last axis; a row of -infinities has shares 0.
    (exp(l - m) / (1 + exp(l)) is proportional to s and cannot underflow as a row.)"""
    l = np.asarray(l, np.float64)
    m = np.minimum(l.max(axis=-1, keepdims=True, initial=-np.inf), 0.0)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        p = np.where(l > 0, sigmoid(l), np.exp(l - m) / (1.0 + np.exp(l)))
        p = np.where(np.isneginf(m), 0.0, p)
        return p / np.where(p.sum(-1, keepdims=True) == 0, 1.0, p.sum(-1, keepdims=True))


def ranges(T, seq):
    return [(0, T)] if seq is None else [(int(a), int(b)) for a, b in zip(seq[:-1], seq[1:])]


def counts(ids, E, seq=None, mask=None):
    """(c [S, E], n [S]): chosen experts and valid tokens of each sequence."""
    T = ids.shape[0]
    c, n = [], []
    for a, b in ranges(T, seq):
        keep = np.ones(b - a, bool) if mask is None else np.asarray(mask[a:b]) != 0
        chosen = ids[a:b][keep].ravel()
        c.append(np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E))
        n.append(int(keep.sum()))
    return np.array(c, np.int64).reshape(-1, E), np.array(n, np.int64)


def balance_loss(l, c, n, k, alpha, seq=None, mask=None):
    """alpha / S * sum over sequences of sum_e f P, with the counts c and n given."""
    T, E = l.shape
    total = 0.0
    R = ranges(T, seq)
    for s, (a, b) in enumerate(R):
        keep = np.ones(b - a, bool) if mask is None else np.asarray(mask[a:b]) != 0
        if n[s]:
            total += float((E / (k * n[s]) * c[s] * (shares(l[a:b][keep]).sum(0) / n[s])).sum())
    return alpha / len(R) * total


def route_weights(l, ids, renorm, rsf):
    """moe_route's weights of given (distinct) ids; dropped ids (< 0) weigh 0."""
    out = np.zeros(ids.shape)
    for t in range(ids.shape[0]):
        ok = (ids[t] >= 0) & (ids[t] < l.shape[1])
        ch = l[t, ids[t][ok]]
        out[t, ok] = rsf * (shares(ch) if renorm else sigmoid(ch))
    return out


def router_backward(l, ids, grad_w=None, renorm=1, rsf=1.0, grad_loss=None, c=None, n=None,
                    alpha=0.0, seq=None, mask=None):
    """(grad [T, E], bound [T, E]): the gradient, and the sum of the magnitudes that
    its terms are subtracted from, without the factor 1 - s."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    k = ids.shape[1]
    s = sigmoid(l)
    grad, mag = np.zeros((T, E)), np.zeros((T, E))
    if grad_w is not None:
        for t in range(T):
            ok = (ids[t] >= 0) & (ids[t] < E)
            i, g = ids[t][ok], np.asarray(grad_w[t][ok], np.float64)
            p = shares(l[t, i]) if renorm else s[t, i]
            mean = (g * p).sum() if renorm else 0.0
            amean = (np.abs(g) * p).sum() if renorm else 0.0
            grad[t, i] += rsf * (g - mean) * p * (1 - s[t, i])
            mag[t, i] += abs(rsf) * (np.abs(g) + amean) * p
    if grad_loss is not None:
        R = ranges(T, seq)
        q = shares(l)
        for b, (lo, hi) in enumerate(R):
            if not n[b]:
                continue
            f = E / (k * n[b]) * c[b]
            for t in range(lo, hi):
                if mask is None or mask[t]:
                    coef = grad_loss * alpha / (len(R) * n[b])
                    mean = (f * q[t]).sum()
                    grad[t] += coef * (f - mean) * q[t] * (1 - s[t])
                    mag[t] += abs(coef) * (f + mean) * q[t]
    return grad, mag
