"""GPU parity of the e4m3 operators against the float64 reference, at the sizes and
values where they can go wrong.

Tolerances.  A product's block sums are fp32 sums of at most 128 products on the
tensor cores, its scaled blocks an fp32 sum: at most 128 + blocks + 4 roundings of
the running magnitude, each counted as 2^-23 (a truncation) of the sum of the terms'
magnitudes; then one bf16 rounding, 2^-8 of the value.  The quantiser is exact."""
import dataclasses

import numpy as np
import pytest
import torch

import workloads as W
from oracle import fp8_oracle as F
from oracle import lmoe_oracle as O

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")

BETA, LBETA = 4.0, 8.0
GUARD = 64          # untouched elements behind every output


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


def dev(a):
    from tests.gpu_util import DEV
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def guarded(shape, dtype, fill):
    """A contiguous tensor of `shape` with GUARD elements of `fill` behind it."""
    from tests.gpu_util import DEV
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), fill, dtype=dtype, device=DEV)
    return buf[:n].view(shape), buf


def sum_tolerance(K):
    return (128 + F.blocks(K) + 4) * 2.0 ** -23


def assert_close(got, ref, mag, K):
    err = np.abs(got - ref)
    bound = 2.0 ** -8 * np.abs(ref) + sum_tolerance(K) * mag
    assert np.all(err <= bound), (float((err - bound).max()), np.argwhere(err > bound)[:3])


def codes_of(g, rows, K, block_rows, std=1.0):
    """e4m3 operands with scales that differ from block to block."""
    x = g.standard_normal((rows, K)) * std
    x *= np.exp(g.standard_normal((rows, 1)))
    return F.quantize(O.f64_to_bf16_bits(x), block_rows)


# --- quantiser --------------------------------------------------------------------


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (3, 112), (8, 7168), (129, 400), (256, 256),
                                    (1000, 144), (127, 2048)])
def test_quantize_is_exact(rows, K, block_rows):
    from tests.gpu_util import dev_bf16
    g = np.random.default_rng(rows * 31 + K)
    x = g.standard_normal((rows, K)) * np.exp(4 * g.standard_normal((rows, 1)))
    x[g.random((rows, K)) < 0.01] *= 100
    x[:, : min(K, 128)][g.random(rows) < 0.2] = 0.0
    bits = O.f64_to_bf16_bits(x)
    codes, cbuf = guarded((rows, K), torch.uint8, 0xA5)
    scales, sbuf = guarded((-(-rows // block_rows), F.blocks(K)), torch.float32, -7.0)
    lm.lmoe_quantize_fp8(dev_bf16(bits), codes, scales, block_rows=block_rows)
    want, ws = F.quantize(bits, block_rows)
    np.testing.assert_array_equal(scales.cpu().numpy(), ws)
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    assert bool((cbuf[-GUARD:] == 0xA5).all()) and bool((sbuf[-GUARD:] == -7.0).all())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_extreme_values(block_rows):
    from tests.gpu_util import dev_bf16
    x = np.zeros((130, 512))
    x[0, 3], x[1, 200], x[129, 300] = np.inf, np.nan, -np.inf
    x[2, :128] = 1e-38                     # under the floor of the block maximum
    x[3, 384:] = 3e38
    x[4, 0] = -448.0
    bits = O.f64_to_bf16_bits(x)
    codes, _ = guarded((130, 512), torch.uint8, 0)
    scales, _ = guarded((130 if block_rows == 1 else 2, 4), torch.float32, 0.0)
    lm.lmoe_quantize_fp8(dev_bf16(bits), codes, scales, block_rows=block_rows)
    want, ws = F.quantize(bits, block_rows)
    got_s, got = scales.cpu().numpy(), codes.cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got_s), np.isnan(ws))
    np.testing.assert_array_equal(got_s[~np.isnan(ws)], ws[~np.isnan(ws)])
    nan = (want & 0x7F) == 0x7F            # a NaN's sign is not fixed
    np.testing.assert_array_equal((got & 0x7F) == 0x7F, nan)
    np.testing.assert_array_equal(got[~nan], want[~nan])


# --- product ----------------------------------------------------------------------


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("T,N,K", [
    (1, 8, 16), (1, 128, 128), (1, 2048, 7168), (2, 136, 272), (5, 1000, 4112), (8, 8192, 1024),
    (9, 24, 7168), (15, 256, 144),
    (16, 264, 256), (17, 128, 512), (32, 1024, 2048), (33, 120, 640), (64, 1032, 128), (128, 256, 1024),
    (129, 392, 272), (255, 640, 400), (300, 512, 192), (513, 1000, 1168), (1024, 768, 512),
    (2050, 2056, 336), (1300, 4104, 1040), (2049, 2304, 2176), (300, 4104, 528), (500, 2560, 272)])
def test_linear_matches_float64(T, N, K, with_add):
    from tests.gpu_util import dev_bf16, host_bits
    g = np.random.default_rng(T * 7 + N + K)
    x, xs = codes_of(g, T, K, 1)
    w, ws = codes_of(g, N, K, 128, 0.02)
    add = O.f64_to_bf16_bits(g.standard_normal((T, N))) if with_add else None
    out, buf = guarded((T, N), torch.bfloat16, 7.0)
    lm.lmoe_linear_fp8(dev(x), dev(xs), dev(w), dev(ws), out, add=None if add is None else dev_bf16(add))
    ref, mag = F.linear(x, xs, w, ws, None if add is None else O.bf16_to_f64(add))
    got = O.bf16_to_f64(host_bits(out))
    assert lm.lmoe_device_error() == 0
    assert_close(got, ref, mag, K)
    assert bool((buf[-GUARD:] == 7.0).all())


@pytest.mark.parametrize("T,N,K", [(3, 48, 272), (40, 272, 400), (140, 1040, 384), (1300, 4112, 144)])
def test_linear_16_byte_alignment(T, N, K):
    # every operand 16 bytes past a 256-byte boundary: what the header asks for and no more
    from tests.gpu_util import dev_bf16, host_bits
    g = np.random.default_rng(T)
    x, xs = codes_of(g, T, K, 1)
    w, ws = codes_of(g, N, K, 128, 0.02)
    add = O.f64_to_bf16_bits(g.standard_normal((T, N)))

    def off(t):
        n = 16 // t.element_size()
        buf = torch.zeros(t.numel() + n, dtype=t.dtype, device="cuda")
        buf[n:].copy_(t.flatten())
        return buf[n:].view(t.shape)

    out = off(torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda"))
    assert out.data_ptr() % 32 == 16
    for a in (None, off(dev_bf16(add))):
        lm.lmoe_linear_fp8(off(dev(x)), off(dev(xs)), off(dev(w)), off(dev(ws)), out, add=a)
        ref, mag = F.linear(x, xs, w, ws, None if a is None else O.bf16_to_f64(add))
        assert_close(O.bf16_to_f64(host_bits(out)), ref, mag, K)
    codes, scales = off(torch.zeros((T, K), dtype=torch.uint8, device="cuda")), off(torch.zeros((T, F.blocks(K)), device="cuda"))
    bits = O.f64_to_bf16_bits(g.standard_normal((T, K)))
    lm.lmoe_quantize_fp8(off(dev_bf16(bits)), codes, scales)
    want, want_s = F.quantize(bits)
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)


@pytest.mark.parametrize("T", [1, 17])
def test_linear_most_features(T):
    # N = 2^31 - 8, the most that the argument holds: a stream and a tensor-core form; all of the
    # weights' rows but a few are zeros
    N, K = 2 ** 31 - 8, 16
    if torch.cuda.mem_get_info()[0] < 1.3 * (N * K + 2 * T * N) + (8 << 30):
        pytest.skip("needs %d GB" % (1.3 * (N * K + 2 * T * N) / 2 ** 30 + 8))
    from tests.gpu_util import host_bits
    g = np.random.default_rng(T)
    x, xs = codes_of(g, T, K, 1)
    rows = np.array([0, 1, 130, 12345678, N // 2, N - 300, N - 129, N - 8, N - 1])
    wr, _ = F.quantize(O.f64_to_bf16_bits(g.standard_normal((len(rows), K)) + 3), 1)
    at = dev(rows)
    w = torch.zeros((N, K), dtype=torch.uint8, device="cuda")
    w[at] = dev(wr)
    ws = torch.full((F.blocks(N), 1), 0.5, device="cuda")
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lm.lmoe_linear_fp8(dev(x), dev(xs), w, ws, out)
    got = O.bf16_to_f64(host_bits(out[:, at]))
    assert lm.lmoe_device_error() == 0
    ref, mag = F.linear(x, xs, wr, np.full((1, 1), 0.5, np.float32))
    assert_close(got, ref, mag, K)
    assert [int(torch.count_nonzero(o)) for o in out] == [int(np.count_nonzero(r)) for r in got]
    del w, ws, out
    torch.cuda.empty_cache()


def test_linear_every_code():
    # every finite e4m3 code as an operand, one product a row: exact but for the bf16 rounding
    from tests.gpu_util import host_bits
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    x = np.zeros((len(codes), 128), np.uint8)
    x[np.arange(len(codes)), np.arange(len(codes)) % 128] = codes
    w = np.zeros((128, 128), np.uint8)
    w[np.arange(128), np.arange(128)] = 0x38       # 1.0
    out = torch.empty((len(codes), 128), dtype=torch.bfloat16, device="cuda")
    lm.lmoe_linear_fp8(dev(x), dev(np.full((len(codes), 1), 0.5, np.float32)), dev(w),
                       dev(np.ones((1, 1), np.float32)), out)
    want = np.zeros((len(codes), 128))
    want[np.arange(len(codes)), np.arange(len(codes)) % 128] = 0.5 * F.e4m3_value(codes)
    np.testing.assert_array_equal(O.bf16_to_f64(host_bits(out)), want)


def test_linear_rows_with_nan_stay_apart():
    from tests.gpu_util import host_bits
    g = np.random.default_rng(5)
    x, xs = codes_of(g, 40, 256, 1)
    w, ws = codes_of(g, 136, 256, 128)
    x[7, 130], xs[21, 1] = 0x7F, np.inf
    out = torch.empty((40, 136), dtype=torch.bfloat16, device="cuda")
    lm.lmoe_linear_fp8(dev(x), dev(xs), dev(w), dev(ws), out)
    got = O.bf16_to_f64(host_bits(out))
    keep = [i for i in range(40) if i not in (7, 21)]
    assert np.all(np.isnan(got[7])) and not np.any(np.isfinite(got[21]))
    ref, mag = F.linear(x[keep], xs[keep], w, ws)
    assert_close(got[keep], ref, mag, 256)


def test_linear_chained_stream_graph_and_bits():
    # quantise -> product on a stream of its own (the weights quantised by the call
    # before), the same in a graph, and twice: the same bits
    from tests.gpu_util import dev_bf16, host_bits, DEV
    g = np.random.default_rng(9)
    T, N, K = 24, 520, 384
    xb, wb = O.f64_to_bf16_bits(g.standard_normal((T, K))), O.f64_to_bf16_bits(g.standard_normal((N, K)))
    x, w = dev_bf16(xb), dev_bf16(wb)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()

    def chain():
        lm.lmoe_quantize_fp8(w, wq, ws, block_rows=128, stream=s)
        lm.lmoe_quantize_fp8(x, xq, xs, stream=s)
        lm.lmoe_linear_fp8(xq, xs, wq, ws, out, stream=s)

    with torch.cuda.stream(s):
        wq = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=DEV)
        ws = torch.empty((F.blocks(N), F.blocks(K)), device=DEV)
        xq, xs = torch.empty((T, K), dtype=torch.uint8, device=DEV), torch.empty((T, F.blocks(K)), device=DEV)
        out = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
        chain()
    s.synchronize()
    first = host_bits(out)
    ref, mag = F.linear(*F.quantize(xb), *F.quantize(wb, 128))
    assert_close(O.bf16_to_f64(first), ref, mag, K)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        chain()
    for _ in range(3):
        for t in (wq.view(torch.uint8), xq, ws, xs, out):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(host_bits(out), first)


# --- experts ----------------------------------------------------------------------


def expert_weights(g, E, L, d):
    q = {}
    for name, rows, K in (("w13", 2 * d, L), ("w2", L, d)):
        c, s = codes_of(g, E * rows, K, 128, 0.05)
        q[name + "_q"] = c.reshape(E, rows, K)
        q[name + "_s"] = s.reshape(E, rows // 128, K // 128)
    return q


def check_experts(x, xs, off, Q, L, d, beta, lbeta, y):
    """y against float64.  The kernel's activations differ from the reference's by
    the first product's sum (through SituGLU's derivatives, |d gate_out| <= 1.1 and
    |d up_out| <= 1) and by 2^-9 (the hardware tanh, 2^-11, twice, the exponential and
    the reciprocal); their codes lie between those of the two ends of that range,
    and y may be off by what that makes of them."""
    for e in range(len(off) - 1):
        a, b = int(off[e]), int(off[e + 1])
        if b <= a:
            continue
        h, mag = F.experts_h(x[a:b], xs[a:b], Q, e)
        ref = O.situ(h[:, :d], h[:, d:], beta, lbeta)
        gate, up = h[:, :d], h[:, d:]
        up_out = lbeta * np.tanh(up / lbeta) if lbeta > 0 else up
        with np.errstate(over="ignore"):
            gate_out = beta * np.tanh(gate / beta) / (1 + np.exp(-gate))
        eh = sum_tolerance(L) * mag
        err = eh[:, :d] * 1.1 * np.abs(up_out) + eh[:, d:] * np.abs(gate_out) + 2.0 ** -9 * np.abs(ref)
        amax = np.maximum(np.abs(ref).reshape(b - a, -1, 128).max(-1), 2.0 ** -100)
        es = np.repeat(err.reshape(b - a, -1, 128).max(-1) / amax + 2.0 ** -22, 128, 1)
        S = np.repeat(amax / 448, 128, 1)
        t = ref / S
        delta = err / S + np.abs(t) * es
        q, lo, hi = (F.e4m3_value(F.e4m3_code(v)) for v in (t, t - delta, t + delta))
        D = np.maximum(hi - q, q - lo) * S + np.abs(q) * S * es
        W2 = F.dequantize(Q["w2_q"][e], Q["w2_s"][e], 128)
        yr, ym = (q * S) @ W2.T, (np.abs(q) * S) @ np.abs(W2).T
        off_by = D @ np.abs(W2).T + sum_tolerance(d) * ym
        bad = np.abs(y[a:b] - yr) > off_by + 2.0 ** -8 * (np.abs(yr) + off_by)
        assert not bad.any(), (e, np.argwhere(bad)[:3])


@pytest.mark.parametrize("E,L,d,counts,lbeta", [
    (1, 128, 128, [1], 8.0),
    (4, 128, 128, [3, 0, 16, 17], 8.0),
    (5, 256, 128, [0, 1, 128, 129, 300], 0.0),
    (3, 640, 384, [33, 500, 2], 8.0),
    (8, 1024, 256, [1, 1, 2, 0, 0, 15, 64, 1], -1.0),
    (64, 128, 256, [i % 7 for i in range(64)], 8.0),
    (1024, 128, 128, [int(i % 9 == 4) * 2 for i in range(1024)], 8.0),
    (2, 2048, 512, [260, 140], 8.0),
    (6, 512, 384, [8, 9, 16, 17, 0, 40], 8.0),       # passes of eight tokens
    (900, 256, 128, [i % 2 for i in range(900)], 8.0),
    (900, 128, 256, [int(i % 3 > 0) for i in range(900)], 8.0),    # over 512 rows, few each
    (200, 256, 128, [1, 33, 32, 0, 70] + [i % 2 for i in range(195)] , 8.0),   # light and heavy experts
    (300, 256, 128, [i % 2 for i in range(300)], 8.0),                         # ... none heavy
    (300, 128, 256, [0] * 7 + [290] + [0] * 292, 8.0),                         # ... none light
    (20, 256, 128, [120] + [0] * 18 + [8], 8.0),     # few rows, nearly all one expert's
    (700, 256, 128, [1, 33, 32, 0, 70] + [int(i % 4 == 1) for i in range(695)], 8.0),  # both kernels
    (700, 128, 256, [0] * 7 + [290] + [0] * 692, 8.0),                       # ... light one without work
    (1024, 128, 128, [int(i % 31 == 30) * 40 for i in range(1024)], 8.0),    # heavy, groups far apart
])
def test_experts_match_float64(E, L, d, counts, lbeta):
    from tests.gpu_util import host_bits
    g = np.random.default_rng(E + L + d)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1])
    x, xs = codes_of(g, R, L, 1)
    Q = expert_weights(g, E, L, d)
    y, buf = guarded((R, L), torch.bfloat16, 7.0)
    ws = torch.empty(lm.lmoe_experts_fp8_workspace_bytes(R, E, L, d), dtype=torch.uint8, device="cuda")
    lm.lmoe_experts_fp8({k: dev(v) for k, v in Q.items()}, dev(x), dev(xs), dev(off), y, ws, inter=d,
                        beta=BETA, linear_beta=lbeta)
    got = O.bf16_to_f64(host_bits(y))
    assert lm.lmoe_device_error() == 0
    check_experts(x, xs, off, Q, L, d, BETA, lbeta, got)
    assert bool((buf[-GUARD:] == 7.0).all())


def test_experts_rows_outside_stay_untouched():
    # rows before the first offset and behind the last belong to no expert; an
    # offset past the rows is clamped
    from tests.gpu_util import host_bits
    g = np.random.default_rng(2)
    L = d = 128
    x, xs = codes_of(g, 40, L, 1)
    Q = expert_weights(g, 3, L, d)
    qd = {k: dev(v) for k, v in Q.items()}
    ws = torch.empty(lm.lmoe_experts_fp8_workspace_bytes(40, 3, L, d), dtype=torch.uint8, device="cuda")
    for off, owned in (([4, 10, 10, 30], [(0, 4, 10), (2, 10, 30)]), ([0, 0, 0, 0], []),
                       ([0, 25, 99, 99], [(0, 0, 25), (1, 25, 40)])):
        y = torch.full((40, L), 7.0, dtype=torch.bfloat16, device="cuda")
        lm.lmoe_experts_fp8(qd, dev(x), dev(xs), dev(np.array(off, np.int32)), y, ws, inter=d, beta=BETA,
                            linear_beta=LBETA)
        got = O.bf16_to_f64(host_bits(y))
        want = np.full((40, L), 7.0)
        for e, a, b in owned:
            yr, _, _ = F.experts(x[a:b], xs[a:b], [0, b - a], {k: v[e:e + 1] for k, v in Q.items()}, d,
                                 BETA, LBETA)
            # a code of the activations may round the other way: a step of 2^-3 of one of
            # 128 terms, far under the difference between experts
            assert np.linalg.norm(got[a:b] - yr) <= 0.02 * np.linalg.norm(yr)
            want[a:b] = got[a:b]
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("E,sizes", [(300, (1000, 400, 151, 150, 129, 128, 40, 1)),
                                     (16, (400, 129, 128, 9, 8)), (2, (300, 17, 16, 8))])
def test_experts_in_the_workspace_of_a_larger_call(E, sizes):
    # one workspace, of the largest call, over the changes of kernel from call to call
    L = d = 128
    g = np.random.default_rng(E)
    Q = expert_weights(g, E, L, d)
    qd = {k: dev(v) for k, v in Q.items()}
    ws = torch.empty(lm.lmoe_experts_fp8_workspace_bytes(sizes[0], E, L, d), dtype=torch.uint8, device="cuda")
    for R in sizes:
        off = np.concatenate([[0], np.cumsum(np.bincount(g.integers(0, E, R), minlength=E))]).astype(np.int32)
        x, xs = codes_of(g, R, L, 1)
        got = []
        for w in (ws, torch.empty(lm.lmoe_experts_fp8_workspace_bytes(R, E, L, d), dtype=torch.uint8, device="cuda")):
            y, buf = guarded((R, L), torch.bfloat16, 7.0)
            lm.lmoe_experts_fp8(qd, dev(x), dev(xs), dev(off), y, w, inter=d, beta=BETA, linear_beta=LBETA)
            assert bool((buf[-GUARD:] == 7.0).all())
            got.append(y)
        assert torch.equal(got[0], got[1])
        yr, _, _ = F.experts(x, xs, off, Q, d, BETA, LBETA)
        y = got[0].double().cpu().numpy()
        # (a code of the activations may round the other way: a step of 2^-3 of one of 128 terms)
        assert np.linalg.norm(y - yr) <= 0.02 * np.linalg.norm(yr)


# --- the layer --------------------------------------------------------------------


def quantized_experts(wts):
    out = {}
    for name in ("w13", "w2"):
        E, rows, K = wts[name].shape
        c, s = F.quantize(wts[name].reshape(E * rows, K), 128)
        out[name + "_q"], out[name + "_s"] = c.reshape(E, rows, K), s.reshape(E, rows // 128, K // 128)
    return out


@pytest.mark.parametrize("T,E,topk,shared", [(1, 64, 4, True), (8, 64, 4, True), (100, 16, 4, True),
                                             (128, 64, 4, False), (40, 1024, 4, True), (129, 64, 4, True), (300, 64, 4, True),
                                             (257, 8, 8, False)])
def test_layer_forward(T, E, topk, shared):
    # Z (or the scattered rows) from the GPU -> quantised rows -> experts' Y, each
    # stage against the reference on the GPU's own inputs, then Y -> the output
    from tests.gpu_util import (DEV, weights_to_device, dev_bf16, dev_f32, host_bits, workspace_view,
                                assert_layer_close, assert_stage_close)
    d = dataclasses.replace(W.TINY, T=T, num_experts=E, topk=topk)
    wts = W.layer_weights(d, T)
    if not shared:
        wts["ws13"] = wts["ws2"] = None
    Q = quantized_experts(wts)
    wdev = weights_to_device(dict(wts, w13=None, w2=None))
    xb, lg = W.hidden_states(d, T), W.router_logits(T, E, T)
    out = torch.empty((T, d.hidden), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(lm.latent_moe_workspace_bytes_fp8(d), dtype=torch.uint8, device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    args = (d, wdev, {k: dev(v) for k, v in Q.items()}, dev_bf16(xb), dev_f32(lg), out, ws)
    lm.latent_moe_forward_fp8(*args, debug={"expert_offsets": off})
    first = host_bits(out)
    assert lm.lmoe_device_error() == 0
    lm.latent_moe_forward_fp8(*args)
    np.testing.assert_array_equal(host_bits(out), first)
    v = workspace_view(lm, d, ws)
    ids, w = O.route(lg, wts["bias"], topk, d.routed_scaling_factor, d.renormalize)
    _, offsets, row_of, tok_of_row = O.permute(ids, E)
    np.testing.assert_array_equal(off.cpu().numpy(), offsets)
    np.testing.assert_array_equal(v["row_of"], row_of)
    Zref = O.linear_bf16(O.bf16_to_f64(xb), wts["w_down"])
    rows = v["A"] if T <= 128 else v["Z"][tok_of_row]
    assert_stage_close(O.bf16_to_f64(rows), Zref[tok_of_row], "Z")
    x, xs = F.quantize(rows)
    # the bounds are test_experts_match_float64's: here a code may round the other way (2^-3
    # of a term), far under the difference between experts
    yr, _, _ = F.experts(x, xs, offsets, Q, d.inter, d.beta, d.linear_beta)
    Y = O.bf16_to_f64(v["Y"])
    assert np.linalg.norm(Y - yr) <= 0.01 * np.linalg.norm(yr)
    C = np.einsum("tk,tkl->tl", w, Y[row_of])
    N = O.round_bf16(O.rms_norm(C, O.bf16_to_f64(wts["norm_w"]), d.rms_eps))
    Sh = np.zeros((T, d.hidden))
    if shared:
        Gs = O.linear_bf16(O.bf16_to_f64(xb), wts["ws13"])
        ds = d.shared_inter
        Sh = O.linear_bf16(O.round_bf16(O.situ(Gs[:, :ds], Gs[:, ds:], d.beta, d.linear_beta)), wts["ws2"])
    NW = N @ O.bf16_to_f64(wts["w_up"]).T
    ref = O.round_bf16(NW + Sh)
    assert_layer_close(O.bf16_to_f64(first), ref, scale=np.maximum(np.abs(ref), np.maximum(np.abs(NW), np.abs(Sh))))


def test_layer_in_a_graph_and_launch_count():
    from tests.gpu_util import DEV, weights_to_device, dev_bf16, dev_f32, host_bits
    from tests.test_gpu_launch_count import _kernel_nodes
    for T in (8, 300):
        d = dataclasses.replace(W.TINY, T=T)
        wts = W.layer_weights(d, 2)
        q = {k: dev(v) for k, v in quantized_experts(wts).items()}
        wdev = weights_to_device(dict(wts, w13=None, w2=None))
        x, lg = dev_bf16(W.hidden_states(d, 2)), dev_f32(W.router_logits(T, d.num_experts, 2))
        out = torch.empty((T, d.hidden), dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(lm.latent_moe_workspace_bytes_fp8(d), dtype=torch.uint8, device=DEV)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        lm.latent_moe_forward_fp8(d, wdev, q, x, lg, out, ws, stream=s)
        s.synchronize()
        want = host_bits(out)
        try:
            g = torch.cuda.CUDAGraph(keep_graph=True)
        except TypeError:
            pytest.skip("this PyTorch cannot keep the captured graph")
        with torch.cuda.graph(g, stream=s):
            lm.latent_moe_forward_fp8(d, wdev, q, x, lg, out, ws, stream=s)
        assert _kernel_nodes(g) == lm.latent_moe_launch_count_fp8(d, True)
        g.instantiate()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(host_bits(out), want)


@pytest.mark.parametrize("E,topk", [(64, 4), (896, 4), (8, 8)])
def test_layer_in_the_workspace_of_a_larger_batch(E, topk):
    # one workspace, of the largest batch, against one of the batch's own size, over the changes
    # between the decode form, the streaming and the tensor-core kernels
    from tests.gpu_util import DEV, weights_to_device, dev_bf16, dev_f32
    base = dataclasses.replace(W.TINY, T=400, num_experts=E, topk=topk)
    wts = W.layer_weights(base, E)
    q = {k: dev(v) for k, v in quantized_experts(wts).items()}
    wdev = weights_to_device(dict(wts, w13=None, w2=None))
    ws = torch.full((lm.latent_moe_workspace_bytes_fp8(base),), 0xFF, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for T in (400, 129, 128, 112, 33, 32, 9, 1, 300):
        d = dataclasses.replace(base, T=T)
        x, lg = dev_bf16(W.hidden_states(d, T)), dev_f32(W.router_logits(T, E, T))
        got = []
        for w in (ws, torch.full((lm.latent_moe_workspace_bytes_fp8(d),), 0xFF, dtype=torch.uint8, device=DEV)):
            out, buf = guarded((T, d.hidden), torch.bfloat16, 7.0)
            n = w.numel()
            lm.latent_moe_forward_fp8(d, wdev, q, x, lg, out, w, workspace_bytes=n)
            assert bool((buf[-GUARD:] == 7.0).all())
            got.append(out)
        assert lm.lmoe_device_error() == 0
        assert torch.equal(got[0], got[1]) and bool(torch.isfinite(got[0].float()).all())
