"""GPU parity of the products grouped by expert and of their gradients against float64.

Tolerance.  The tensor cores add up products in fp32: one rounding (of 2^-23 at most, the
hardware truncates) a step of 16 terms and one for the rows' own sums, so that a sum of n
terms is off by at most (n / 16 + 32) 2^-23 of the sum of their magnitudes; then one rounding
of the output: bf16 2^-8, fp32 2^-24 (twice with an addend)."""
import threading

import numpy as np
import pytest
import torch

from oracle import training_oracle as O

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
BF16 = torch.finfo(torch.bfloat16).eps / 2
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert lm.lmoe_device_error() == 0


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(torch.bfloat16).to("cuda")


def slack(n):
    return (n / 16 + 32) * 2.0 ** -23


def slack_w(n):
    """Of the weights' gradients: the tensor cores add up 512 rows at a time (32 steps), registers
    those sums, each addition rounded to 2^-24."""
    return (np.minimum(n, 512) / 16 + 2) * 2.0 ** -23 + n / 512 * 2.0 ** -24


def offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


LEAD, TRAIL = 3, 5          # rows before the first and behind the last expert's

# rows of each expert
COUNTS = {
    "one row": [1],
    "empty": [0, 0, 0],
    "borders": [0, 1, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 0],
    "more borders": [255, 256, 257, 0, 0, 1, 600],
    "many small": [(7 * i) % 5 for i in range(200)],
    "one of many": [0] * 99 + [90] + [0] * 100,
    "large": [1500],
}
DIMS = [(8, 8), (64, 64), (256, 128), (136, 200), (120, 264), (1024, 512), (384, 1032)]
FEW = [("borders", 256, 128), ("borders", 136, 200), ("more borders", 1032, 72), ("many small", 520, 136), ("large", 264, 520)]
CASES = [(c, n, k) for c in COUNTS for n, k in DIMS if COUNTS[c] != [1500] or n * k < 1 << 18]
# rows enough that tiles take the narrowest matrices, too; the widest ones, with few and with more rows
COUNTS |= {"long": [5000, 0, 37], "few": [1, 2], "some": [300, 0, 31]}
CASES += [("long", 8, 8), ("long", 24, 40), ("few", 16, 65536), ("some", 16, 65536), ("few", 65536, 16), ("some", 65536, 16)]


def make(name, N, K, seed=0):
    counts = COUNTS[name]
    R = sum(counts) + LEAD + TRAIL
    off = offsets(counts, LEAD)
    x, dy = rand((R, K), seed), rand((R, N), seed + 1, 1e-2)
    w = rand((len(counts), N, K), seed + 2, 0.05)
    # what belongs to nobody must not be looked at
    for t in (x, dy):
        t[:LEAD] = NAN
        t[R - TRAIL:] = NAN
    return off, x, dy, w, R


def owned(counts):
    return slice(LEAD, LEAD + sum(counts))


def check_rows(call, ref_fn, rows_in, w, off, counts, terms, out_dim):
    R = rows_in.shape[0]
    buf = torch.full((R * out_dim + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:R * out_dim].view(R, out_dim)
    call(rows_in, w, off, out)
    own = owned(counts)
    o, wi, xi = f64(off), f64(w), f64(rows_in)
    xi[:LEAD] = xi[R - TRAIL:] = 0
    ref = ref_fn(xi, wi, o, np.zeros((R, out_dim)))
    mag = ref_fn(np.abs(xi), np.abs(wi), o, np.zeros((R, out_dim)))
    err, bound = np.abs(f64(out) - ref)[own], (BF16 * np.abs(ref) + slack(terms) * mag)[own]
    assert np.all(err <= bound * (1 + 2 ** -7)), (float(np.nanmax(err / bound)), np.argwhere(~(err <= bound))[:5])
    assert bool((buf[-64:] == 7.0).all()) and bool((out[:LEAD] == 7.0).all()) and bool((out[R - TRAIL:] == 7.0).all())
    again = torch.full_like(out, 7.0)
    call(rows_in, w, off, again)
    assert torch.equal(again, out)


@pytest.mark.parametrize("name,N,K", CASES)
def test_forward(name, N, K):
    off, x, dy, w, R = make(name, N, K)
    check_rows(lm.lmoe_grouped_linear, O.grouped_linear, x, w, off, COUNTS[name], K, N)


@pytest.mark.parametrize("name,N,K", CASES)
def test_backward_x(name, N, K):
    off, x, dy, w, R = make(name, N, K)
    check_rows(lm.lmoe_grouped_linear_backward_x, O.grouped_linear_backward_x, dy, w, off, COUNTS[name], N, K)


# (the addend at a few sizes)
@pytest.mark.parametrize("name,N,K,form", [(*c, f) for c in CASES for f in ("fp32", "bf16")] +
                         [(*c, f) for c in FEW for f in ("add", "in place")])
def test_backward_w(name, N, K, form):
    off, x, dy, w, R = make(name, N, K)
    E, counts = w.shape[0], COUNTS[name]
    dt = torch.bfloat16 if form == "bf16" else torch.float32
    buf = torch.full((E * N * K + 64,), 7.0, dtype=dt, device="cuda")
    dw = buf[:E * N * K].view(E, N, K)
    add = None
    if form == "add":
        add = torch.randn((E, N, K), generator=torch.Generator().manual_seed(3)).to("cuda")
    elif form == "in place":
        dw.copy_(torch.randn((E, N, K), generator=torch.Generator().manual_seed(3)))
        add = dw
    before = None if add is None else f64(add)
    lm.lmoe_grouped_linear_backward_w(dy, x, off, dw, add=add)
    xi, di = f64(x), f64(dy)
    for a in (xi, di):
        a[:LEAD] = a[R - TRAIL:] = 0
    ref = O.grouped_linear_backward_w(di, xi, f64(off), before)
    mag = O.grouped_linear_backward_w(np.abs(di), np.abs(xi), f64(off))
    n = np.array(counts)[:, None, None]
    if form == "bf16":
        bound = BF16 * np.abs(ref) * (1 + 2 ** -7) + slack_w(n) * mag
    else:
        bound = 2.0 ** -23 * np.abs(ref) + slack_w(n) * mag + (0 if before is None else 2.0 ** -23 * np.abs(before))
    err = np.abs(f64(dw) - ref)
    assert np.all(err <= bound), (float(np.nanmax(err - bound)), np.argwhere(~(err <= bound))[:5])
    assert bool((buf[-64:] == 7.0).all())
    assert not f64(dw)[np.array(counts) == 0].any() or before is not None
    if form in ("fp32", "bf16"):
        again = torch.full_like(dw, 7.0)
        lm.lmoe_grouped_linear_backward_w(dy, x, off, again)
        assert torch.equal(again, dw)


@pytest.mark.parametrize("sign", [False, True])
def test_long_sums_keep_fp32(sign):
    # where the tensor cores' truncating sums alone would be 4e-5 (of one sign 2e-4) off
    counts, N, K = [30000, 513, 0, 1025], 64, 72
    off, R = offsets(counts), sum(counts)
    x, dy = rand((R, K), 0), rand((R, N), 1)
    if sign:
        x, dy = x.abs(), dy.abs()
    dw = torch.empty((4, N, K), device="cuda")
    lm.lmoe_grouped_linear_backward_w(dy, x, off, dw)
    ref = O.grouped_linear_backward_w(f64(dy), f64(x), f64(off))
    mag = O.grouped_linear_backward_w(np.abs(f64(dy)), np.abs(f64(x)), f64(off))
    assert np.all(np.abs(f64(dw) - ref) <= 2.0 ** -24 * np.abs(ref) + slack_w(np.array(counts)[:, None, None]) * mag)
    assert np.linalg.norm(f64(dw) - ref) <= 2e-6 * np.linalg.norm(ref)


def test_clamped_offsets():
    # entries outside [0, rows] and descending ones lead nowhere outside the buffers
    R, N, K = 40, 64, 64
    x, w = rand((R, K), 0), rand((3, N, K), 1)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([-100, 10, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    lm.lmoe_grouped_linear(x, w, off, out)
    ref = O.grouped_linear(f64(x)[5:], f64(w)[2:], [0, 35], np.zeros((35, N)))
    assert np.allclose(f64(out)[10:], ref[5:], rtol=2 ** -7, atol=1e-2)     # rows 5 .. 9 are two experts'
    ref = O.grouped_linear(f64(x)[:5], f64(w)[:1], [0, 5], np.zeros((5, N)))
    assert np.allclose(f64(out)[:5], ref, rtol=2 ** -7, atol=1e-2)
    dw = torch.full((3, N, K), 7.0, device="cuda")
    lm.lmoe_grouped_linear_backward_w(x, x, off, dw)
    assert bool(torch.isfinite(dw).all()) and not dw[1].any()


@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
def test_specials_stay_with_their_rows(value):
    counts, N, K = [20, 70, 9, 33], 136, 200
    off, R = offsets(counts), sum(counts)
    x, dy, w = rand((R, K), 0), rand((R, N), 1), rand((4, N, K), 2)
    y, dx, dw = (torch.empty(s, dtype=d, device="cuda") for s, d in
                 (((R, N), torch.bfloat16), ((R, K), torch.bfloat16), ((4, N, K), torch.float32)))

    def run():
        lm.lmoe_grouped_linear(x, w, off, y)
        lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
        lm.lmoe_grouped_linear_backward_w(dy, x, off, dw)
        return y.clone(), dx.clone(), dw.clone()

    want = run()
    row = 20 + 70 - 1                                  # the last of expert 1: next to expert 2's in a tile
    x[row] = value
    dy[row] = value
    got = run()
    keep = [i for i in range(R) if i != row]
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
    assert torch.equal(got[2][[0, 2, 3]], want[2][[0, 2, 3]])
    assert not torch.isfinite(got[0][row].float()).any() and not torch.isfinite(got[2][1]).any()
    # weights: of one expert
    x[row], dy[row] = 1.0, 1.0
    w[1] = value
    lm.lmoe_grouped_linear(x, w, off, y)
    lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
    others = [i for i in range(R) if not 20 <= i < 90]
    assert torch.equal(y[others], want[0][others]) and torch.equal(dx[others], want[1][others])


def near(got, fn, rows, w, off, terms):
    rows, w, shape = f64(rows), f64(w), tuple(got.shape)
    ref, mag = fn(rows, w, off, np.zeros(shape)), fn(np.abs(rows), np.abs(w), off, np.zeros(shape))
    assert np.all(np.abs(f64(got) - ref) <= BF16 * (1 + 2 ** -7) * np.abs(ref) + slack(terms) * mag)


def test_far_rows_and_experts():
    # element offsets past 2^31: the last rows of a long batch, the last of many experts
    K, N = 2048, 72
    R = 2 ** 20 + 100
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    tail = rand((200, K), 0)
    x[-200:] = tail
    off = torch.tensor([R - 190, R - 150, R - 3], dtype=torch.int32, device="cuda")
    rel, rows = [0, 40, 187], slice(R - 190, R - 3)
    w = rand((2, N, K), 1, 0.05)
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    lm.lmoe_grouped_linear(x, w, off, out)
    near(out[rows], O.grouped_linear, tail[10:197], w, rel, K)
    dy = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    dy[-200:] = rand((200, N), 2)
    dx, dw = torch.empty_like(x), torch.empty((2, N, K), device="cuda")
    lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
    near(dx[rows], O.grouped_linear_backward_x, dy[rows], w, rel, N)
    lm.lmoe_grouped_linear_backward_w(dy, x, off, dw)
    ref = O.grouped_linear_backward_w(f64(dy[rows]), f64(tail[10:197]), rel)
    mag = O.grouped_linear_backward_w(np.abs(f64(dy[rows])), np.abs(f64(tail[10:197])), rel)
    assert np.all(np.abs(f64(dw) - ref) <= 2.0 ** -24 * np.abs(ref) + slack_w(150) * mag)
    del x, dx, dy, out
    E, N, K = 1024, 1032, 2088                          # 2.2e9 weights
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[-2:] = rand((2, N, K), 3, 0.05)
    for counts in ([30, 40], [1, 1]):                   # a few rows more and fewer than tiles are worth
        R = sum(counts)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[-2], off[-1] = counts[0], R
        rel = [0, counts[0], R]
        x, dy = rand((R, K), 4), rand((R, N), 5)
        out, dx = torch.empty((R, N), dtype=torch.bfloat16, device="cuda"), torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
        lm.lmoe_grouped_linear(x, w, off, out)
        near(out, O.grouped_linear, x, w[-2:], rel, K)
        lm.lmoe_grouped_linear_backward_x(dy, w, off, dx)
        near(dx, O.grouped_linear_backward_x, dy, w[-2:], rel, N)
    dw = torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    lm.lmoe_grouped_linear_backward_w(dy, x, off, dw)
    ref = O.grouped_linear_backward_w(f64(dy), f64(x), rel)
    assert np.all(np.abs(f64(dw[-2:]) - ref) <= BF16 * (1 + 2 ** -7) * np.abs(ref) + 1e-30) and not dw[:-2].any()


def test_most_experts_in_large_tiles():
    # the largest table beside the largest stages
    E, N, K = 1024, 40, 64
    counts = [(37 * i) % 83 for i in range(E)]
    off, R = offsets(counts), sum(counts)
    assert R > 32 * E
    x, w = rand((R, K), 0), rand((E, N, K), 1)
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    lm.lmoe_grouped_linear(x, w, off, out)
    ref = O.grouped_linear(f64(x), f64(w), f64(off), np.zeros((R, N)))
    mag = O.grouped_linear(np.abs(f64(x)), np.abs(f64(w)), f64(off), np.zeros((R, N)))
    assert np.all(np.abs(f64(out) - ref) <= BF16 * (1 + 2 ** -7) * np.abs(ref) + slack(K) * mag)


FIRST_IN_CAPTURE = """
import torch, latent_mixture_experts_sigmoid_gb300 as lm
d, b, f = "cuda", torch.bfloat16, torch.float32
x, w = torch.randn((40, 1040), device=d).to(b), torch.randn((2, 64, 1040), device=d).to(b)
off = torch.tensor([0, 30, 40], dtype=torch.int32, device=d)
y, dx, dw = torch.zeros((40, 64), dtype=b, device=d), torch.zeros_like(x), torch.zeros((2, 64, 1040), device=d)
n, dh, ds = torch.zeros_like(x), torch.zeros_like(x), torch.zeros((40, 64), dtype=b, device=d)
g, dg = torch.zeros(1040, device=d), torch.randn((40, 32), device=d).to(b)
lm.load_library()
ws = torch.empty(lm.lmoe_rms_norm_backward_workspace_bytes(40, 1040), dtype=torch.uint8, device=d)
def run():
    lm.lmoe_rms_norm(x, None, 1e-6, out=n)
    lm.lmoe_grouped_linear(n, w, off, y)
    lm.situ_and_mul_backward(y, dg, ds, 4.0, 8.0)
    lm.lmoe_grouped_linear_backward_x(ds, w, off, dx)
    lm.lmoe_grouped_linear_backward_w(ds, n, off, dw)
    lm.lmoe_rms_norm_backward(dx, x, None, 1e-6, dh, grad_norm_w=g, workspace=ws)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, dx, dw, dh, g)]
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) and a.any() for a, b in zip(got, (y, dx, dw, dh, g)))
assert lm.lmoe_device_error() == 0
"""


def test_first_call_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_no_rows():
    w, off = rand((3, 64, 64), 0), torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    lm.lmoe_grouped_linear(e, w, off, e)
    lm.lmoe_grouped_linear_backward_x(e, w, off, e)
    for dt in (torch.float32, torch.bfloat16):
        dw = torch.full((3, 64, 64), 7.0, dtype=dt, device="cuda")
        lm.lmoe_grouped_linear_backward_w(e, e, off, dw)
        assert not dw.any()
    add = torch.randn((3, 64, 64), device="cuda")
    dw = torch.full((3, 64, 64), 7.0, device="cuda")
    lm.lmoe_grouped_linear_backward_w(e, e, off, dw, add=add)
    assert torch.equal(dw, add)


def test_against_differences():
    # the loss sum(c * y) along directions of x and w: y is bilinear, so its float64 twin's
    # difference is exact up to cancellation
    counts, N, K = [5, 0, 40], 64, 72
    off, R = offsets(counts), 45
    x, c, w = rand((R, K), 0), rand((R, N), 1), rand((3, N, K), 2)
    dx, dw = torch.empty_like(x), torch.empty((3, N, K), device="cuda")
    lm.lmoe_grouped_linear_backward_x(c, w, off, dx)
    lm.lmoe_grouped_linear_backward_w(c, x, off, dw)
    g = np.random.default_rng(0)
    for _ in range(4):
        a, b = g.standard_normal((R, K)), g.standard_normal((3, N, K))

        def loss(t):
            return (f64(c) * O.grouped_linear(f64(x) + t * a, f64(w) + t * b, f64(off), np.zeros((R, N)))).sum()

        diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
        room = 2 * BF16 * np.abs(f64(dx) * a).sum() + 1e-4 * np.abs(f64(dw) * b).sum() + 1e-3
        assert abs((f64(dx) * a).sum() + (f64(dw) * b).sum() - diff) <= room


def test_captured_replayed_and_beside_another_stream():
    counts, N, K = [30, 0, 300, 77, 5, 128], 256, 320
    off, R = offsets(counts), sum(counts)
    x, dy, w = rand((R, K), 0), rand((R, N), 1), rand((6, N, K), 2)

    def outputs():
        return (torch.empty((R, N), dtype=torch.bfloat16, device="cuda"),
                torch.empty((R, K), dtype=torch.bfloat16, device="cuda"), torch.empty((6, N, K), device="cuda"))

    def run(o, stream=None):
        lm.lmoe_grouped_linear(x, w, off, o[0], stream=stream)
        lm.lmoe_grouped_linear_backward_x(dy, w, off, o[1], stream=stream)
        lm.lmoe_grouped_linear_backward_w(dy, x, off, o[2], stream=stream)

    want, a, b = outputs(), outputs(), outputs()
    run(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run(a)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            run(a)
    for t in a:
        t.zero_()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(20):
        graph.replay()
        run(b, stream=other)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) and torch.equal(r, q) for p, q, r in zip(a, want, b))
    results = []

    def thread():
        s = torch.cuda.Stream()
        o = outputs()
        torch.cuda.synchronize()
        for _ in range(20):
            run(o, stream=s)
        s.synchronize()
        results.append(all(torch.equal(p, q) for p, q in zip(o, want)))

    ts = [threading.Thread(target=thread) for _ in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert results == [True, True]


def test_weights_written_just_before():
    # in stream order: a call before this one may have written the weights and the offsets
    counts, N, K = [60, 4, 100], 128, 256
    R = sum(counts)
    x, w = rand((R, K), 0), rand((3, N, K), 1)
    off = offsets(counts)
    want, got = (torch.empty((R, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lm.lmoe_grouped_linear(x, w, off, want)
    for _ in range(10):
        w2, off2 = torch.full_like(w, NAN), torch.zeros_like(off)
        w2.copy_(w)
        off2.copy_(off)
        lm.lmoe_grouped_linear(x, w2, off2, got)
        assert torch.equal(got, want)
