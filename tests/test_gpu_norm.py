"""GPU parity of residual + RMSNorm (bf16 and e4m3 outputs) and of its gradient against
the float64 reference.

Tolerances, u = 2^-24.  A thread sums at most 32 squares, then ten steps of trees; 1/sqrt
halves that relative error; sum, quotient, root, reciprocal and the products with r, w (and
a power of two) add a few u: a relative error of E = 40 u for y covers them.  bf16 rounds by
2^-8 at most, e4m3 by 2^-4 (below its normal range by half of its step 2^-9)."""
import numpy as np
import pytest
import torch

from oracle import training_oracle as O

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")

U = 2.0 ** -24
E = 40 * U
BF16 = torch.finfo(torch.bfloat16).eps / 2
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


def f64(t):
    return t.detach().double().cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(torch.bfloat16)


def guarded(shape, dtype, fill):
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), fill, dtype=torch.float32, device="cuda").to(dtype)
    return buf[:n].view(shape), buf


def intact(buf, fill):
    return bool((buf[-GUARD:].float() == fill).all())


def batch(T, H, seed=0, std=1.0):
    g = np.random.default_rng(seed)
    x = bf16(std * g.standard_normal((T, H)))
    res = bf16(std * g.standard_normal((T, H)) * np.exp(0.5 * g.standard_normal(H)))
    return x, res, bf16(1 + 0.2 * g.standard_normal(H))


def check_codes(codes, scales, y, bound):
    """codes * scales against y, whose own error is `bound`; the scales against the block maxima."""
    T, H = y.shape
    c, s = f64(codes.view(torch.float8_e4m3fn).float()), f64(scales)
    for b in range(s.shape[1]):
        cols = slice(128 * b, min(H, 128 * b + 128))
        top = np.abs(y[:, cols]).max(1)
        # the scale: its maximum's error and a quotient; the code: a quotient and a product more
        assert np.all(np.abs(s[:, b] - np.maximum(top, 2.0 ** -100) / 448) <= (bound[:, cols].max(1) / 448 + 2 * U * s[:, b]))
        v = c[:, cols] * s[:, b:b + 1]
        step = np.maximum(2.0 ** -4 * np.abs(y[:, cols]), 2.0 ** -10 * s[:, b:b + 1])
        err = np.abs(v - y[:, cols])
        # (a rounding border may lie within the value's own error)
        assert np.all(err <= step * (1 + 8 * U) + 2 * bound[:, cols]), float((err / step).max())


SHAPES = [(1, 8), (3, 16), (5, 48), (9, 256), (17, 264), (33, 512), (8, 1024), (7, 1032), (2, 2048), (305, 2064), (1, 7168),
          (13, 7168), (400, 7168), (3, 8192), (2, 8200), (310, 8208), (1, 16384), (306, 16384), (2500, 128), (700, 144), (70000, 16)]


@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H):
    x, res, w = batch(T, H, T + H)
    h, y = O.rms_norm(f64(x), f64(res), f64(w), 1e-6)
    out, obuf = guarded((T, H), torch.bfloat16, 3.0)
    ho, hbuf = guarded((T, H), torch.bfloat16, 3.0)
    kw, bufs = {}, [obuf, hbuf]
    if H % 16 == 0:
        codes, cbuf = guarded((T, H), torch.float8_e4m3fn, 3.0)
        scales, sbuf = guarded((T, -(-H // 128)), torch.float32, 3.0)
        kw, bufs = dict(codes=codes, scales=scales), bufs + [cbuf, sbuf]
    lm.lmoe_rms_norm(x, w, 1e-6, out=out, residual=res, residual_out=ho, **kw)
    assert all(intact(b, 3.0) for b in bufs)
    # the row's error with that of h, which enters y directly and through the squares
    bound = E * np.abs(y) + 2 * U * np.abs(y)
    assert np.all(np.abs(f64(ho) - h) <= (BF16 + 2 * U) * np.abs(h))
    assert np.all(np.abs(f64(out) - y) <= BF16 * np.abs(y) * (1 + 2 ** -7) + bound)
    if kw:
        check_codes(codes, scales, y, bound)
    # each output alone, and again: the same bits
    alone = torch.empty_like(out)
    lm.lmoe_rms_norm(x, w, 1e-6, out=alone, residual=res)
    assert torch.equal(alone.view(torch.int16), out.view(torch.int16))
    if kw:
        c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
        lm.lmoe_rms_norm(x, w, 1e-6, codes=c2, scales=s2, residual=res)
        assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scales)


@pytest.mark.parametrize("T,H", [(3, 64), (6, 2048), (320, 4096)])
def test_plain_norm_and_in_place(T, H):
    x, res, w = batch(T, H, 5)
    _, y = O.rms_norm(f64(x), None, None, 1e-5)
    out = torch.empty_like(x)
    lm.lmoe_rms_norm(x, None, 1e-5, out=out)
    assert np.all(np.abs(f64(out) - y) <= (BF16 * (1 + 2 ** -7) + E) * np.abs(y))
    want_h, want = torch.empty_like(x), torch.empty_like(x)
    lm.lmoe_rms_norm(x, w, 1e-5, out=want, residual=res, residual_out=want_h)
    a, b = x.clone(), res.clone()
    lm.lmoe_rms_norm(a, w, 1e-5, out=a, residual=b, residual_out=b)        # both in place
    assert torch.equal(a, want) and torch.equal(b, want_h)


def test_codes_feed_the_products():
    # the codes are those that the quantiser would give the exact fp32 rows: close to its own of bf16 ones
    T, H, N = 40, 512, 256
    x, res, w = batch(T, H, 9)
    wt = bf16(0.05 * np.random.default_rng(1).standard_normal((N, H)))
    wq, ws = torch.empty((N, H), dtype=torch.uint8, device="cuda"), torch.empty((2, 4), device="cuda")
    lm.lmoe_quantize_fp8(wt, wq, ws, block_rows=128)
    codes, scales = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, 4), device="cuda")
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    lm.lmoe_rms_norm(x, w, 1e-6, codes=codes, scales=scales, residual=res)
    lm.lmoe_linear_fp8(codes, scales, wq, ws, y)
    v = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)
    q = wq.view(torch.float8_e4m3fn).double() * ws.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    ref, mag = v @ q.T, v.abs() @ q.abs().T
    assert bool(((y.double() - ref).abs() <= BF16 * ref.abs() + 64 * U * mag).all())


@pytest.mark.parametrize("H", [64, 1024, 2048])
def test_range(H):
    # rows whose squares overflow fp32, underflow it, and zeros
    g = np.random.default_rng(3)
    n = g.standard_normal((6, H))
    x = bf16(n * np.array([1e25, 1e-25, 3e37, 1e-38, 1.0, 0.0])[:, None])
    out = torch.empty_like(x)
    lm.lmoe_rms_norm(x, None, 0.0, out=out)
    _, y = O.rms_norm(f64(x)[:5], None, None, 0.0)
    assert np.all(np.abs(f64(out)[:5] - y) <= (BF16 * (1 + 2 ** -7) + E) * np.abs(y))
    assert bool(torch.isnan(out[5]).all())                 # 0 / 0
    lm.lmoe_rms_norm(x, None, 1e-6, out=out)
    _, y = O.rms_norm(f64(x), None, None, 1e-6)            # (rows of 1e-38 are 1e-35, those of 0 stay 0)
    assert np.all(np.abs(f64(out) - y) <= (BF16 * (1 + 2 ** -7) + E) * np.abs(y) + 2.0 ** -134)
    dy = bf16(g.standard_normal((6, H)))
    dh = torch.empty_like(x)
    lm.lmoe_rms_norm_backward(dy, x, None, 0.0, dh)
    ref, mag, _, _ = O.rms_norm_backward(f64(dy)[:5], f64(x)[:5], None, None, 0.0)
    fits = mag < 3e38                                        # (of a row of 1e-38 the gradient may not be)
    bound = BF16 * np.abs(ref) * (1 + 2 ** -7) + 4 * E * mag + 2.0 ** -134
    assert np.all((np.abs(f64(dh)[:5] - ref) <= bound)[fits])


@pytest.mark.parametrize("H", [256, 4096])
def test_specials_stay_in_their_row(H):
    x, res, w = batch(12, H, 2)
    want = torch.empty_like(x)
    lm.lmoe_rms_norm(x, w, 1e-6, out=want, residual=res)
    bad = x.clone()
    bad[3, 17], bad[5, H - 1] = float("nan"), float("inf")
    out, codes = torch.empty_like(x), torch.empty((12, H), dtype=torch.uint8, device="cuda")
    scales = torch.empty((12, H // 128), device="cuda")
    lm.lmoe_rms_norm(bad, w, 1e-6, out=out, codes=codes, scales=scales, residual=res)
    keep = [i for i in range(12) if i not in (3, 5)]
    assert torch.equal(out[keep], want[keep]) and bool(torch.isfinite(scales[keep]).all())
    assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(scales[3]).all())
    assert bool(torch.isnan(out[5, H - 1])) and not out[5, :H - 1].any()


BACK = [(63, 24), (64, 512), (64, 1024), (65, 1024), (17, 768), (1, 1024), (1, 8), (2, 16), (9, 256), (40, 264), (100, 520), (1300, 1024), (3, 1032), (33, 2048), (700, 2056), (300, 4096), (1, 4104),
        (650, 7168), (5, 8192), (40, 8200), (1300, 16384), (5000, 64), (6000, 1024), (70000, 16)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", BACK)
def test_backward(T, H, residual):
    h, dres, w = batch(T, H, T + H)
    dy = bf16(1e-3 * np.random.default_rng(T).standard_normal((T, H)))
    dres = (1e-3 * dres).contiguous() if residual else None
    dh, hbuf = guarded((T, H), torch.bfloat16, 3.0)
    dw, wbuf = guarded((H,), torch.float32, 3.0)
    ws = torch.full((lm.lmoe_rms_norm_backward_workspace_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
    lm.lmoe_rms_norm_backward(dy, h, w, 1e-6, dh, grad_norm_w=dw, grad_residual=dres, workspace=ws)
    assert intact(hbuf, 3.0) and intact(wbuf, 3.0)
    ref, mag, dwr, dwmag = O.rms_norm_backward(f64(dy), f64(h), f64(w), None if dres is None else f64(dres), 1e-6)
    # r enters the term with the mean three times, its sum once: 4 E; a walker's sum over its rows
    # and the join's runs and warps: fewer terms than T + 64
    assert np.all(np.abs(f64(dh) - ref) <= BF16 * np.abs(ref) * (1 + 2 ** -7) + 4 * E * mag)
    assert np.all(np.abs(f64(dw) - dwr) <= (E + (T + 64) * U) * dwmag)
    again, dw2 = torch.empty_like(dh), torch.empty_like(dw)
    lm.lmoe_rms_norm_backward(dy, h, w, 1e-6, again, grad_norm_w=dw2, grad_residual=dres, workspace=ws)
    assert torch.equal(again, dh) and torch.equal(dw2, dw)
    lm.lmoe_rms_norm_backward(dy, h, w, 1e-6, dy, grad_residual=dres)      # in place, rows alone
    assert torch.equal(dy, dh)


def test_backward_against_differences():
    # the loss sum(c * out) moved along one direction of h and of w: the forward's bf16 outputs are
    # too coarse, so the forward is the oracle's, the gradient the kernel's
    T, H = 6, 128
    h, c, w = batch(T, H, 4)
    dh, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    ws = torch.empty(lm.lmoe_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    lm.lmoe_rms_norm_backward(c, h, w, 1e-6, dh, grad_norm_w=dw, workspace=ws)
    g = np.random.default_rng(0)
    for _ in range(5):
        a, b = g.standard_normal((T, H)), g.standard_normal(H)

        def loss(t):
            return (f64(c) * O.rms_norm(f64(h) + t * a, None, f64(w) + t * b, 1e-6)[1]).sum()

        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        ref, mag, _, dwmag = O.rms_norm_backward(f64(c), f64(h), f64(w), None, 1e-6)
        slack = ((BF16 * np.abs(ref) + 4 * E * mag) * np.abs(a)).sum() + (64 * U * dwmag * np.abs(b)).sum() + 1e-5
        assert abs((f64(dh) * a).sum() + (f64(dw) * b).sum() - diff) <= slack


def test_empty_batch():
    dw = torch.full((64,), 7.0, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    lm.lmoe_rms_norm(e, None, 1e-6, out=e)
    lm.lmoe_rms_norm_backward(e, e, None, 1e-6, e, grad_norm_w=dw)
    assert not dw.any()


@pytest.mark.parametrize("T,H", [(200, 2048), (20, 512), (300, 96)])
def test_captured_and_on_another_stream(T, H):
    h, res, w = batch(T, H, 1)
    dy = bf16(np.random.default_rng(0).standard_normal((T, H)))
    out, dh, dw = torch.empty_like(h), torch.empty_like(h), torch.empty(H, device="cuda")
    ws = torch.empty(lm.lmoe_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")

    def both():
        lm.lmoe_rms_norm(h, w, 1e-6, out=out, residual=res)
        lm.lmoe_rms_norm_backward(dy, h, w, 1e-6, dh, grad_norm_w=dw, workspace=ws)

    both()
    torch.cuda.synchronize()
    want = out.clone(), dh.clone(), dw.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        both()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            both()
    for t in (out, dh, dw):
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, dh, dw), want))
