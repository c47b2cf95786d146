"""The grouped products' kernel on pairs of SMs at sizes that never go to the kernel for few
rows, against float64 or the same bits.  Tolerances as in test_gpu_grouped."""
import numpy as np
import pytest
import torch

from oracle import training_oracle as O
from tests.test_gpu_grouped import BF16, f64, near, offsets, rand, slack, slack_w  # noqa: F401

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert lm.lmoe_device_error() == 0


@pytest.mark.parametrize("form", ["fp32", "bf16", "add"])
def test_weight_gradients_beside_experts_of_nan(form):
    # every rest of rows from 0 to 63 behind an expert's last full block of 64, each filled up with
    # zeros by both CTAs of a pair; the rows behind it, the next expert's, are NaN
    counts, N, K = [1 + (37 * i) % 130 for i in range(260)], 264, 136
    E, R = len(counts), sum(counts)
    assert {c % 64 for c in counts} == set(range(64))
    off = offsets(counts)
    x, dy = rand((R, K), 0), rand((R, N), 1)
    dt = torch.bfloat16 if form == "bf16" else torch.float32
    add = torch.randn((E, N, K), generator=torch.Generator().manual_seed(2)).to("cuda") if form == "add" else None
    want, got = (torch.empty((E, N, K), dtype=dt, device="cuda") for _ in range(2))
    lm.lmoe_grouped_linear_backward_w(dy, x, off, want, add=add)
    expert = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).to("cuda")
    for parity in (0, 1):
        xn, dn = x.clone(), dy.clone()
        xn[expert % 2 == parity] = NAN
        dn[expert % 2 == parity] = NAN
        for _ in range(25):
            got.fill_(7.0)
            lm.lmoe_grouped_linear_backward_w(dn, xn, off, got, add=add)
            assert torch.equal(got[1 - parity::2], want[1 - parity::2])
            assert bool(torch.isnan(got[parity::2]).all())


@pytest.mark.parametrize("rows", [200, 512, 1100])
@pytest.mark.parametrize("form", ["fp32", "bf16"])
def test_small_terms_behind_a_large_one(rows, form):
    # A first term of 1 and terms p, which the tensor cores cut: a step of 16 loses up to
    # 16 * 2^-25 and 2^-23 in its own sum (5 units of 2^-23 at the most) of the power of two below
    # the largest magnitude, here 1.  256 rows are summed so, and joined by additions that round: one
    # block loses what 16 steps do, the others nothing, as their terms are alike and less than 2^-16
    # of the sum.  (512 rows at once lose 127 units with p = 0.99 * 2^-25.)
    p = 0.9921875 * 2.0 ** torch.arange(-22, -30, -1, dtype=torch.float64)
    x = torch.ones((rows, 8), dtype=torch.bfloat16, device="cuda")
    dy = p.repeat(rows, 1)
    dy[0] = 1.0
    if form == "bf16":
        dy = dy - (dy == 1.0) * 1.0               # (the large term's own bits would hide them: p alone)
    dy = dy.to(torch.bfloat16).to("cuda")
    dw = torch.empty((1, 8, 8), dtype=torch.float32 if form == "fp32" else torch.bfloat16, device="cuda")
    lm.lmoe_grouped_linear_backward_w(dy, x, offsets([rows]), dw)
    ref = (dy.double().T @ x.double()).cpu().numpy()[None]
    joins = 2 + rows / 256
    if form == "fp32":
        bound = (16 * 5 + joins / 2) * 2.0 ** -23 * np.ones_like(ref)
    else:
        bound = (BF16 + (16 * 5 + joins / 2) * 2.0 ** -23) * np.abs(ref)
    assert np.all(np.abs(f64(dw) - ref) <= bound), (np.abs(f64(dw) - ref) / bound).max()
