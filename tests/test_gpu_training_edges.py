"""The training operators at the ends of their formats' ranges."""
import numpy as np
import pytest
import torch

from oracle import training_oracle as O
from tests.test_gpu_situ_backward import check

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


def f64(t):
    return t.detach().double().cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(torch.bfloat16)


@pytest.mark.parametrize("T,H", [(3, 64), (100, 96), (3, 256), (100, 512), (64, 1024), (100, 1024), (20, 2048), (9, 16384)])
def test_norm_gradient_of_subnormal_rows(T, H):
    # 1 / rms of these rows is 2^133 and outside fp32: a row without a gradient of its own still gets
    # grad_residual's, exactly, and adds nothing to grad_norm_w
    g = np.random.default_rng(0)
    h, dy, dres = bf16(g.standard_normal((T, H))), bf16(g.standard_normal((T, H))), bf16(g.standard_normal((T, H)))
    h[::2] = bf16(2.0 ** -133 * np.where(g.random((1, H)) < 0.5, -1.0, 1.0))
    dy[::2] = 0
    w = bf16(1 + 0.2 * g.standard_normal(H))
    ws = torch.empty(lm.lmoe_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    for residual in (dres, None):
        dh, dw = torch.empty_like(h), torch.empty(H, device="cuda")
        lm.lmoe_rms_norm_backward(dy, h, w, 0.0, dh, grad_norm_w=dw, grad_residual=residual, workspace=ws)
        assert torch.equal(dh[::2], torch.zeros_like(dh[::2]) if residual is None else residual[::2])
        # The other rows as ever (test_gpu_norm has the bounds: E = 40 * 2^-24, four times in dh; dw a sum
        # of T terms): not the bits of a call without the subnormal rows, which has fewer rows and may
        # take the kernel for few of them, whose sums have another order.
        ref, mag, dwr, dwmag = O.rms_norm_backward(f64(dy)[1::2], f64(h)[1::2], f64(w),
                                                   None if residual is None else f64(residual)[1::2], 0.0)
        assert np.all(np.abs(f64(dh)[1::2] - ref) <= BF16 * np.abs(ref) * (1 + 2 ** -7) + 160 * 2.0 ** -24 * mag)
        assert np.all(np.abs(f64(dw) - dwr) <= (40 + T + 64) * 2.0 ** -24 * dwmag)


@pytest.mark.parametrize("T,H", [(5, 64), (80, 512), (20, 2048)])
def test_norm_gradient_far_from_one(T, H):
    # rows whose squares leave fp32, with gradients that bring the result back into its range
    g = np.random.default_rng(1)
    n, d = g.standard_normal((T, H)), g.standard_normal((T, H))
    for of_h, of_dy in ((-47, 50), (-70, 50), (-120, -5), (-126, -3), (70, 50), (100, -10), (70, -60)):
        h, dy = bf16(n * 2.0 ** of_h), bf16(d * 2.0 ** of_dy)
        dh = torch.empty_like(h)
        lm.lmoe_rms_norm_backward(dy, h, None, 0.0, dh)
        ref, mag, _, _ = O.rms_norm_backward(f64(dy), f64(h), None, None, 0.0)
        assert np.abs(ref).max() < 2.0 ** 126 and np.abs(ref).max() > 2.0 ** -133
        # (bounds of test_gpu_norm; bf16 below 2^-126 rounds by 2^-134)
        bound = BF16 * np.abs(ref) * (1 + 2 ** -7) + 160 * 2.0 ** -24 * mag + 2.0 ** -134
        assert np.all(np.abs(f64(dh) - ref) <= bound), (of_h, of_dy)


@pytest.mark.parametrize("beta", [4.0, 1.0])
def test_situ_gradient_of_large_products(beta):
    # without a bound on up, grad_out * up may leave fp32 where the gate's small derivative brings the
    # result back: of a saturated gate, and NaN beside a derivative of 0
    g = np.random.default_rng(2)
    gate = np.array([40.0, -40.0, 20.0, -60.0, 300.0, 1000.0, -300.0, 6.0])
    up, dy = 2.0 ** np.array([100.0, 100, 110, 120, 127, 127, 127, 20]), 2.0 ** np.array([30.0, 30, 20, 10, 3, 3, 3, 100])
    x = np.concatenate([np.tile(gate, (4, 8)), np.tile(up, (4, 8)) * np.sign(g.standard_normal((4, 64)))], 1)
    dx = check(bf16(x), bf16(np.tile(dy, (4, 8))), beta, 0.0)
    assert bool(torch.isfinite(dx).all())
