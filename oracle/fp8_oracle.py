"""Reference of the block-scaled e4m3 operators in NumPy (test infrastructure only).

A matrix [rows, K] is e4m3 codes (uint8) and scales, one per block of `block_rows`
rows (1 for token rows, 128 for weights) and 128 columns; value = code * scale.
Products are formed in float64; the quantiser's own arithmetic is float32, as its
definition states, so its codes and scales are fixed to the bit.
"""
from __future__ import annotations

import numpy as np

from . import lmoe_oracle as O

BLOCK = 128
E4M3_MAX = np.float32(448.0)
TINY_AMAX = np.float32(2.0 ** -100)


def e4m3_value(code: np.ndarray) -> np.ndarray:
    """float64 value of e4m3 codes: sign, 4 exponent bits (bias 7, field 0
    subnormal), 3 mantissa bits; 0x7F and 0xFF are NaN, there is no infinity."""
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, np.ldexp(m / 8.0, -6), np.ldexp(1.0 + m / 8.0, e - 7))
    mag = np.where((c & 0x7F) == 0x7F, np.nan, mag)
    return np.where(c & 0x80, -mag, mag)


_POSITIVE = e4m3_value(np.arange(0x7F))            # 0 .. 448, ascending


def e4m3_code(v: np.ndarray) -> np.ndarray:
    """The nearest e4m3 code of each value (ties to the even code, magnitudes
    over 448 to 448, NaN to 0x7F)."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 448.0)
    hi = np.searchsorted(_POSITIVE, a, side="left").clip(0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    pick_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    code = np.where(pick_lo, lo, hi).astype(np.int64)
    code = np.where(np.isnan(v), 0x7F, code)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def spread(scales: np.ndarray, rows: int, cols: int, block_rows: int) -> np.ndarray:
    """One scale per element of a [rows, cols] matrix."""
    return np.repeat(np.repeat(scales, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]


def quantize_f32(x: np.ndarray, block_rows: int = 1):
    """(codes uint8, scales float32) of float32 x [rows, K]: per block, in float32,
    a = max(max |x|, 2^-100), scale = a / 448, code = e4m3(x * (448 / a))."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    p = np.zeros((-(-rows // block_rows) * block_rows, blocks(K) * BLOCK), np.float32)
    p[:rows, :K] = np.abs(x)
    a = p.reshape(p.shape[0] // block_rows, block_rows, blocks(K), BLOCK).max(axis=(1, 3))
    a = np.maximum(a, TINY_AMAX)
    with np.errstate(invalid="ignore"):
        scaled = x * spread(E4M3_MAX / a, rows, K, block_rows)
    return e4m3_code(scaled), a / E4M3_MAX


def quantize(x_bits: np.ndarray, block_rows: int = 1):
    """quantize_f32 of bf16 bits."""
    return quantize_f32(O.bf16_to_f64(x_bits).astype(np.float32), block_rows)


def dequantize(codes: np.ndarray, scales: np.ndarray, block_rows: int) -> np.ndarray:
    rows, K = codes.shape
    return e4m3_value(codes) * spread(np.asarray(scales, np.float64), rows, K, block_rows)


def linear(x, xs, w, ws, add=None):
    """(y, bound): the product in float64, and the sum of the magnitudes of its terms."""
    X, Wt = dequantize(x, xs, 1), dequantize(w, ws, BLOCK).T
    y, mag = X @ Wt, np.abs(X) @ np.abs(Wt)
    if add is not None:
        y, mag = y + add, mag + np.abs(add)
    return y, mag


def experts_h(x, xs, Q: dict, e: int):
    """(h, bound) of expert e's first product for its rows."""
    return linear(x, xs, Q["w13_q"][e], Q["w13_s"][e])


def experts(x, xs, offsets, Q: dict, inter: int, beta: float, linear_beta: float):
    """The routed experts on rows grouped by expert; returns y [rows, latent] and
    the activations' codes and scales, SituGLU in float64 before the quantiser.
    Rows that no expert owns are 0."""
    rows = x.shape[0]
    y = np.zeros(x.shape)
    act = np.zeros((rows, inter), np.uint8)
    act_s = np.zeros((rows, inter // BLOCK), np.float32)
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b <= a:
            continue
        h, _ = experts_h(x[a:b], xs[a:b], Q, e)
        act[a:b], act_s[a:b] = quantize_f32(O.situ(h[:, :inter], h[:, inter:], beta, linear_beta))
        y[a:b], _ = linear(act[a:b], act_s[a:b], Q["w2_q"][e], Q["w2_s"][e])
    return y, act, act_s
