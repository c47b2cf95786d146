"""The grouped products' kernel on pairs of SMs at sizes that never go to the kernel for few
rows, against float64 or the same bits.  Tolerances as in test_gpu_grouped."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import training_oracle as O
from tests.test_gpu_grouped import BF16, f64, near, offsets, rand, slack, slack_w  # noqa: F401

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
NAN = float("nan")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert lm.lmoe_device_error() == 0


def on_pairs(R, N, K):
    """That the forward and the rows' gradient run on pairs of SMs: the rule for few rows begins
    with the CTAs of the other kernel, one a row and 16 features or 32 columns."""
    with open(os.path.join(ROOT, "latent_mixture_experts_sigmoid_gb300", "csrc", "grouped.cu")) as f:
        most = int(re.search(r"if \(ctas > (\d+)\) return false;", f.read())[1])
    assert R * -(-N // 16) > most and R * -(-K // 32) > most


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


def outputs(R, E, N, K):
    return (torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((R, K), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((E, N, K), 7.0, device="cuda"))


def test_clamped_and_descending_offsets():
    # entries outside [0, rows] and descending ones lead nowhere outside the buffers
    R, N, K = 700, 128, 256
    on_pairs(R, N, K)
    x, dy, w = rand((R, K), 0), rand((R, N), 1), rand((3, N, K), 2)
    buf = torch.full((R * (N + K) + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    y, dx = buf[64:64 + R * N].view(R, N), buf[64 + R * N:64 + R * (N + K)].view(R, K)
    off = torch.tensor([-100, 300, 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    lm.lmoe_grouped_linear(x, w, off, y)
    lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
    for a, b, e in ((0, 100, 0), (300, 700, 2)):                     # rows 100 .. 299 are two experts'
        near(y[a:b], O.grouped_linear, x[a:b], w[e:e + 1], [0, b - a], K)
        near(dx[a:b], O.grouped_linear_backward_x, dy[a:b], w[e:e + 1], [0, b - a], N)
    dw = torch.full((3, N, K), 7.0, device="cuda")
    lm.lmoe_grouped_linear_backward_w(dy, x, off, dw)
    ref = O.grouped_linear_backward_w(f64(dy)[100:], f64(x)[100:], [0, 600])
    mag = O.grouped_linear_backward_w(np.abs(f64(dy))[100:], np.abs(f64(x))[100:], [0, 600])
    assert np.all(np.abs(f64(dw)[2:] - ref) <= 2.0 ** -24 * np.abs(ref) + slack_w(600) * mag) and not dw[1].any()
    # every row many experts': more tiles than rows, each of them within the buffers
    E = 1000
    w = rand((E, N, K), 3)
    off = torch.tensor([0, 2 ** 31 - 1] * (E // 2) + [-(2 ** 31)], dtype=torch.int32, device="cuda")
    lm.lmoe_grouped_linear(x, w, off, y)
    lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
    assert bool(torch.isfinite(buf.float()).all()) and bool((buf[:64] == 7.0).all()) and bool((buf[-64:] == 7.0).all())


@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
def test_specials_stay_with_their_rows(value):
    counts, N, K = [200, 700, 90, 330], 136, 200
    off, R = offsets(counts), sum(counts)
    on_pairs(R, N, K)
    x, dy, w = rand((R, K), 0), rand((R, N), 1), rand((4, N, K), 2)
    y, dx, dw = outputs(R, 4, N, K)

    def run():
        lm.lmoe_grouped_linear(x, w, off, y)
        lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
        lm.lmoe_grouped_linear_backward_w(dy, x, off, dw)
        return y.clone(), dx.clone(), dw.clone()

    want = run()
    for row in (899, 900):                     # the last of expert 1, the first of expert 2: in one's box of the other
        e = 1 if row == 899 else 2
        keep = torch.tensor([i for i in range(R) if i != row], device="cuda")
        xr, dr = x[row].clone(), dy[row].clone()
        x[row], dy[row] = value, value
        got = run()
        x[row], dy[row] = xr, dr
        others = [i for i in range(4) if i != e]
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
        assert torch.equal(got[2][others], want[2][others])
        assert not torch.isfinite(got[0][row].float()).any() and not torch.isfinite(got[2][e]).any()
    # weights: of one expert
    w[1] = value
    got = run()
    others = torch.tensor([i for i in range(R) if not 200 <= i < 900], device="cuda")
    assert torch.equal(got[0][others], want[0][others]) and torch.equal(got[1][others], want[1][others])


def test_first_call_of_a_process_inside_a_capture():
    # function attributes, occupancy queries and tensor maps of the first launch, inside a capture
    from tests.test_gpu_grouped import FIRST_IN_CAPTURE
    code = FIRST_IN_CAPTURE
    for a, b in (("(40, 1040)", "(700, 1040)"), ("(2, 64, 1040)", "(2, 128, 1040)"), ("[0, 30, 40]", "[0, 450, 700]"),
                 ("(40, 64)", "(700, 128)"), ("(40, 32)", "(700, 64)")):
        assert a in code
        code = code.replace(a, b)
    on_pairs(700, 128, 1040)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_against_differences():
    # the loss sum(c * y) along directions of x and w, as in test_gpu_grouped.  Rounding: each element
    # of dx to bf16, of dw to fp32 behind sums of 500 rows
    counts, N, K = [500, 0, 400], 72, 136
    off, R = offsets(counts), sum(counts)
    on_pairs(R, N, K)
    x, c, w = rand((R, K), 0), rand((R, N), 1), rand((3, N, K), 2)
    _, dx, dw = outputs(R, 3, N, K)
    lm.lmoe_grouped_linear_backward_x(c, w, off, dx)
    lm.lmoe_grouped_linear_backward_w(c, x, off, dw)
    g = np.random.default_rng(0)
    for _ in range(3):
        a, b = g.standard_normal((R, K)), g.standard_normal((3, N, K))

        def loss(t):
            return (f64(c) * O.grouped_linear(f64(x) + t * a, f64(w) + t * b, f64(off), np.zeros((R, N)))).sum()

        diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
        room = 2 * BF16 * np.abs(f64(dx) * a).sum() + 1e-4 * np.abs(f64(dw) * b).sum() + 1e-3
        assert abs((f64(dx) * a).sum() + (f64(dw) * b).sum() - diff) <= room


def test_weights_written_just_before():
    # in stream order: a call before this one may have written the weights and the offsets
    counts, N, K = [600, 4, 1000], 128, 256
    R = sum(counts)
    on_pairs(R, N, K)
    x, dy, w = rand((R, K), 0), rand((R, N), 1), rand((3, N, K), 2)
    off = offsets(counts)
    want, got = outputs(R, 3, N, K), outputs(R, 3, N, K)

    def run(o, w, off):
        lm.lmoe_grouped_linear(x, w, off, o[0])
        lm.lmoe_grouped_linear_backward_x(dy, w, off, o[1])
        lm.lmoe_grouped_linear_backward_w(dy, x, off, o[2])

    run(want, w, off)
    for _ in range(10):
        w2, off2 = torch.full_like(w, NAN), torch.zeros_like(off)
        w2.copy_(w)
        off2.copy_(off)
        run(got, w2, off2)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_most_experts_beside_the_largest_stages():
    # 1024 experts' table, token tiles of 256 rows
    E, N, K = 1024, 40, 64
    counts = [(37 * i) % 251 for i in range(E)]
    off, R = offsets(counts), sum(counts)
    assert R > 96 * E
    on_pairs(R, N, K)
    x, dy, w = rand((R, K), 0), rand((R, N), 1), rand((E, N, K), 2)
    y, dx, _ = outputs(R, 1, N, K)
    lm.lmoe_grouped_linear(x, w, off, y)
    near(y, O.grouped_linear, x, w, f64(off), K)
    lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
    near(dx, O.grouped_linear_backward_x, dy, w, f64(off), N)


def test_each_product_of_a_step_with_many_rows():
    # of a whole training step's own inputs, bf16 intermediates among them
    from tests.test_gpu_experts_training import Block
    T, H, E, d, k = 700, 256, 24, 128, 4
    on_pairs(T * k, 2 * d, H)
    on_pairs(T * k, H, d)
    b = Block(T, H, E, d, k, 7)
    r = b.step()
    off = f64(r["off"])
    near(r["g"], O.grouped_linear, r["a"], b.w13, off, H)
    near(r["y"], O.grouped_linear, r["act"], b.w2, off, d)
    near(r["dact"], O.grouped_linear_backward_x, r["dy"], b.w2, off, H)
    near(r["da"], O.grouped_linear_backward_x, r["dg"], b.w13, off, 2 * d)
    counts = np.diff(off)[:, None, None]
    for got, dy, x in ((r["dw2"], r["dy"], r["act"]), (r["dw13"], r["dg"], r["a"])):
        dy, x = f64(dy), f64(x)
        ref, mag = O.grouped_linear_backward_w(dy, x, off), O.grouped_linear_backward_w(np.abs(dy), np.abs(x), off)
        assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -24 * np.abs(ref) + slack_w(counts) * mag)


@pytest.mark.parametrize("R", [1, 16384])
@pytest.mark.parametrize("K", [16, 64, 256, 1024, 4096])
def test_sums_keep_the_documented_bound(R, K):
    # Terms 1, p, ..., p, -1: what the sums lose of the p is not hidden by the output's rounding.  Each
    # of K / 16 steps loses 5 units of 2^-23 of the largest magnitude, here a power of two up to twice
    # 1 + (K - 2) p; both kernels (few rows, pairs of SMs).
    p = 0.9921875 * 2.0 ** torch.arange(-16, -32, -1, dtype=torch.float64)
    w = p[:, None].repeat(1, K)
    w[:, 0], w[:, -1] = 1.0, -1.0
    w = w.to(torch.bfloat16).to("cuda")[None]
    if R > 1:
        on_pairs(R, 16, K)
    x = torch.ones((R, K), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((R, 16), dtype=torch.bfloat16, device="cuda")
    lm.lmoe_grouped_linear(x, w, offsets([R]), y)
    ref = f64(w)[0].sum(1)
    bound = K / 16 * 5 * 2.0 ** -23 * (1 + (K - 2) * p.numpy()) + BF16 * (1 + 2 ** -7) * np.abs(ref)
    assert np.all(np.abs(f64(y) - ref) <= bound), (np.abs(f64(y) - ref) / bound).max()


EDGES = """
import torch, latent_mixture_experts_sigmoid_gb300 as lm
lm.load_library()
# matrices that fill their pieces of device memory to the byte (2 MB ones), with short experts at both ends
R, N, K = 16384, 512, 1024
x, dy = (torch.empty((R, c), dtype=torch.bfloat16, device="cuda") for c in (K, N))
for t in (x, dy):
    t.normal_()
counts = [3, 5, 1, 17, 40, 0, 63, 64, 65, 1000]
tail = [90, 64, 31, 1, 0, 16, 7, 2]
counts += [R - sum(counts) - sum(tail)] + tail
E = len(counts)
off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
dw = torch.empty((E, N, K), device="cuda")
half, w, y, dx = torch.empty_like(dw, dtype=torch.bfloat16), torch.randn((E, N, K), device="cuda").bfloat16(), torch.empty_like(dy), torch.empty_like(x)
lm.lmoe_grouped_linear_backward_w(dy, x, off, dw)
lm.lmoe_grouped_linear_backward_w(dy, x, off, half)
lm.lmoe_grouped_linear(x, w, off, y)
lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
torch.cuda.synchronize()
assert lm.lmoe_device_error() == 0
a = 0
for e, n in enumerate(counts):
    d, v = dy[a:a + n].double(), x[a:a + n].double()
    a += n
    ref, mag = d.T @ v, d.abs().T @ v.abs()
    slack = ((min(n, 512) / 16 + 2) * 2.0 ** -23 + n / 512 * 2.0 ** -24) * mag
    assert bool(((dw[e].double() - ref).abs() <= 2.0 ** -24 * ref.abs() + slack).all()), e
    assert bool(((half[e].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + slack).all()), e
assert bool(torch.isfinite(y.float()).all()) and bool(torch.isfinite(dx.float()).all())
"""


def test_matrices_that_fill_their_memory():
    # in a process of its own, whose first large allocations they are: what is read or written ahead of
    # them or behind them is no memory
    r = subprocess.run([sys.executable, "-c", EDGES], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
