"""The references of the e4m3 operators and of the router's training, checked on
the CPU against torch's own e4m3 conversion and against differences."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from oracle import lmoe_oracle as O
from oracle import router_oracle as R


def test_e4m3_values_and_rounding_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(F.e4m3_value(codes), t)
    g = np.random.default_rng(0)
    v = np.concatenate([g.standard_normal(20000) * 100, g.standard_normal(20000) * 0.01,
                        (F._POSITIVE[:-1] + F._POSITIVE[1:]) / 2, F._POSITIVE]).astype(np.float32)
    v = np.concatenate([v, -v])
    v = v[np.abs(v) <= 448]
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(F.e4m3_code(v), want)
    assert list(F.e4m3_code(np.array([1e9, -1e9, np.nan]))) == [0x7E, 0xFE, 0x7F]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 16), (5, 400), (130, 256)])
def test_quantize_error_is_half_a_step(rows, K, block_rows):
    g = np.random.default_rng(rows + K)
    x = O.f64_to_bf16_bits(g.standard_normal((rows, K)) * 3)
    v = O.bf16_to_f64(x)
    codes, scales = F.quantize(x, block_rows)
    assert scales.shape == (-(-rows // block_rows), F.blocks(K))
    s = F.spread(scales.astype(np.float64), rows, K, block_rows)
    # half a step of e4m3 (relative 2^-4, absolute 2^-10 of the scale in its
    # subnormals), and the two float32 roundings of 448 / a and the product
    assert np.all(np.abs(F.dequantize(codes, scales, block_rows) - v)
                  <= np.abs(v) * (2.0 ** -4 + 2.0 ** -22) + s * 2.0 ** -10 * (1 + 2.0 ** -20))


def test_quantize_zero_block_and_nonfinite():
    x = np.zeros((3, 256))
    x[1, 5], x[2, 200] = np.inf, np.nan
    x[:, 128] = 2.0
    codes, scales = F.quantize(O.f64_to_bf16_bits(x))
    assert np.all(codes[0, :128] == 0) and scales[0, 0] == np.float32(2.0 ** -100) / F.E4M3_MAX
    assert codes[0, 128] == 0x7E
    assert np.isinf(scales[1, 0]) and np.isnan(scales[2, 1])
    assert np.all(np.isnan(F.dequantize(codes, scales, 1)[1, :128]))


def _batch(T, E, k, S, seed, mask):
    g = np.random.default_rng(seed)
    l = g.standard_normal((T, E)) * 2
    ids = np.argsort(-l, axis=1)[:, :k].astype(np.int32)
    ids[g.random((T, k)) < 0.05] = -1
    seq = np.sort(np.concatenate([[0, T], g.integers(0, T + 1, S - 1)])).astype(np.int32)
    return l, ids, seq, (g.random(T) < 0.8).astype(np.uint8) if mask else None


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("T,E,k,S,mask", [(6, 9, 3, 2, True), (5, 16, 1, 1, False)])
def test_router_gradient_matches_differences(T, E, k, S, mask, renorm):
    l, ids, seq, m = _batch(T, E, k, S, 3 + T, mask)
    c, n = R.counts(ids, E, seq, m)
    gw = np.random.default_rng(1).standard_normal((T, k))
    alpha, gl, rsf = 0.7, 1.3, 2.5

    def value(x):
        w = R.route_weights(x, ids, renorm, rsf)
        return gl * R.balance_loss(x, c, n, k, alpha, seq, m) + (w * gw).sum()

    grad, mag = R.router_backward(l, ids, gw, renorm, rsf, gl, c, n, alpha, seq, m)
    assert np.all(np.abs(grad) <= mag * (1 + 1e-12))
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            # third derivatives are of the order of the value: h^2, and rounding 1e-16 / h
            assert abs((value(up) - value(down)) / (2 * h) - grad[t, e]) < 1e-8


def test_balance_loss_of_even_load_is_alpha():
    # every expert chosen equally often: f = 1, and the loss is alpha * sum P = alpha
    E, k = 8, 2
    ids = np.array([[2 * (t % 4), 2 * (t % 4) + 1] for t in range(8)], np.int32)
    l = np.random.default_rng(0).standard_normal((8, E))
    c, n = R.counts(ids, E)
    assert np.all(c == 2) and n[0] == 8
    assert abs(R.balance_loss(l, c, n, k, 0.5) - 0.5) < 1e-14


def test_shares_survive_underflow():
    q = R.shares(np.array([[-1000.0, -1001.0, -np.inf], [-np.inf] * 3, [5.0, -800.0, 0.0]]))
    assert abs(q[0, 0] - 1 / (1 + np.exp(-1))) < 1e-12 and q[0, 2] == 0
    assert np.all(q[1] == 0) and abs(q[2].sum() - 1) < 1e-12
