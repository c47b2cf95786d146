"""GPU parity of SituGLU's gradient against the float64 reference.

Tolerances.  The exponentials' arguments are rounded to 2^-23 relatively (a product with a
rounded constant and the hardware's scaling), so e^{-a} is off by a 2^-23; the hardware 2^x
and reciprocal by 2^-22 each; the hardware tanh by 2^-16.5 at the most (measured over every
fp32 input for the forward's bound).  All of it is far below bf16's 2^-8."""
import numpy as np
import pytest
import torch

from oracle import training_oracle as O

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def check(x, dy, beta, lbeta):
    d = x.shape[1] // 2
    buf = torch.full((x.numel() + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    dx = buf[:x.numel()].view(x.shape)
    lm.situ_and_mul_backward(x, dy, dx, beta, lbeta)
    assert bool((buf[-64:] == 3.0).all())
    g, u = f64(x)[:, :d], f64(x)[:, d:]
    dg, mag, du = O.situ_backward(g, u, f64(dy), beta, lbeta)
    far = np.minimum(np.abs(g) * (1 + 2 / beta), 300) + (np.minimum(np.abs(u) * 2 / lbeta, 300) if lbeta > 0 else 0)
    rel = 2.0 ** -16 + far * 2.0 ** -22
    # e^{-a} below 2^-126 is 0 (the hardware's flush), so is what bf16 cannot hold
    tiny = 2.0 ** -120 * np.abs(f64(dy)) * (1 + np.abs(u)) + 2.0 ** -133
    got = f64(dx)
    for v, ref, m in ((got[:, :d], dg, mag), (got[:, d:], du, np.abs(du))):
        err = np.abs(v - ref)
        bound = BF16 * np.abs(ref) * (1 + 2 ** -7) + rel * m + tiny
        assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:3])
    return dx


@pytest.mark.parametrize("lbeta", [8.0, 0.0])
@pytest.mark.parametrize("N,d", [(1, 8), (3, 24), (128, 512), (77, 1000), (1025, 64), (2, 8192), (5, 4104)])
def test_parity(N, d, lbeta):
    g = np.random.default_rng(N + d)
    x = 3 * g.standard_normal((N, 2 * d))
    x[g.random(x.shape) < 0.01] = 40.0
    x[g.random(x.shape) < 0.01] = -40.0
    x = bf16(x)
    dy = bf16(g.standard_normal((N, d)))
    dx = check(x, dy, 4.0, lbeta)
    lm.situ_and_mul_backward(x, dy, x, 4.0, lbeta)          # in place
    assert torch.equal(x, dx)


@pytest.mark.parametrize("beta,lbeta", [(4.0, 8.0), (0.25, 100.0), (50.0, 0.5), (1.0, 0.0)])
def test_every_magnitude(beta, lbeta):
    # all bf16 magnitudes of the gate beside ordinary ups, and the other way round
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    vals = torch.cat([bits, bits + 0x8000]).to(torch.int16).view(torch.bfloat16).float().numpy()
    vals = vals[: len(vals) // 8 * 8]
    g = np.random.default_rng(0)
    d = 510 * 8
    vals = np.resize(vals, (16, d))
    other = 2 * g.standard_normal((16, d))
    dy = bf16(g.standard_normal((16, d)))
    check(bf16(np.concatenate([vals, other], 1)), dy, beta, lbeta)
    if lbeta > 0:
        check(bf16(np.concatenate([other, vals], 1)), dy, beta, lbeta)


def test_specials():
    inf, nan = float("inf"), float("nan")
    gate = [inf, -inf, 1.0, 1.0, nan, 1.0, 0.0, -0.0]
    up = [1.0, 1.0, inf, -inf, 1.0, nan, 0.0, 2.0]
    x = torch.tensor([gate + up], device="cuda").to(torch.bfloat16)
    dy = torch.ones((1, 8), dtype=torch.bfloat16, device="cuda")
    dx = torch.empty_like(x)
    lm.situ_and_mul_backward(x, dy, dx, 4.0, 8.0)
    dg, _, du = O.situ_backward(f64(x)[:, :8], f64(x)[:, 8:], f64(dy), 4.0, 8.0)
    np.testing.assert_allclose(f64(dx), np.concatenate([dg, du], 1), rtol=2 ** -7, atol=1e-30)


def test_against_differences():
    # of the framework's own forward form: its float64 twin moved along directions
    g = np.random.default_rng(5)
    x, c = bf16(2 * g.standard_normal((4, 64))), bf16(g.standard_normal((4, 32)))
    dx = f64(check(x, c, 4.0, 8.0))

    def loss(v):
        gate, up = v[:, :32], v[:, 32:]
        return (f64(c) * 4 * np.tanh(gate / 4) / (1 + np.exp(-gate)) * 8 * np.tanh(up / 8)).sum()

    for _ in range(5):
        a = g.standard_normal(x.shape)
        diff = (loss(f64(x) + 1e-5 * a) - loss(f64(x) - 1e-5 * a)) / 2e-5
        assert abs((dx * a).sum() - diff) <= (2 * BF16 * np.abs(dx * a)).sum() + 1e-5
