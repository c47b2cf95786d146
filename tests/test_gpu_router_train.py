"""GPU parity of the router's balance loss, counts and logit gradient against the
float64 reference.

Tolerances.  A sigmoid's relative error: its argument's rounding, |l| 2^-24 (one
product with log2 e) for logits up to L, the hardware 2^x (2^-22), the sum and the
hardware reciprocal (2^-23 each): e_s = (L + 8) 2^-24.  Sums of n positive terms add
n 2^-24 relatively; Z and the dot product each have a lane's E/32 terms and five
steps of a tree."""
import numpy as np
import pytest
import torch

from oracle import router_oracle as R

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")

U = 2.0 ** -24
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def guarded(shape, dtype, fill):
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), fill, dtype=dtype, device="cuda")
    return buf[:n].view(shape), buf


def batch(T, E, k, S, seed, mask=False, drop=0.0, std=1.5):
    g = np.random.default_rng(seed)
    l = (g.standard_normal((T, E)) * std).astype(np.float32)
    ids = np.argsort(-l + g.standard_normal((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[g.random((T, k)) < drop] = -1
    seq = None
    if S > 1:
        seq = np.sort(np.concatenate([[0, T], g.integers(0, T + 1, S - 1)])).astype(np.int32)
    m = (g.random(T) < 0.7).astype(np.uint8) if mask else None
    return l, ids, seq, m


def run_loss(l, ids, seq, m, alpha, stream=None):
    T, E = l.shape
    S = 1 if seq is None else len(seq) - 1
    loss, lbuf = guarded((1,), torch.float32, -7.0)
    cnt, cbuf = guarded((S, E), torch.int32, -7)
    tok, tbuf = guarded((S,), torch.int32, -7)
    ws = torch.full((lm.moe_balance_loss_workspace_bytes(T, E, S),), 0xFF, dtype=torch.uint8, device="cuda")
    lm.moe_balance_loss(dev(l), dev(ids), alpha, loss, cnt, tok, ws, token_mask=dev(m), seq_offsets=dev(seq),
                        stream=stream)
    torch.cuda.synchronize()
    for b in (lbuf, cbuf, tbuf):
        assert bool((b[-GUARD:] == -7).all())
    return loss, cnt, tok


def loss_tolerance(l, E, T):
    L = float(np.abs(l[np.isfinite(l)]).max(initial=0.0))
    # sigmoids and sums of Z and the dot product; the sum over tokens (a warp's run, the CTA's
    # eight, the last CTA's); the factors
    return (2 * (L + 8 + E / 32 + 5 + 2) + T / 16 + 8 + 32 + 8) * U


CASES = [(1, 8, 1, 1, False), (2, 4, 4, 1, False), (16, 64, 4, 2, False), (33, 50, 3, 3, True),
         (100, 1, 1, 1, True), (257, 127, 8, 5, True), (300, 896, 16, 2, False), (512, 1024, 32, 4, True),
         (777, 1023, 16, 1, True), (64, 300, 5, 40, False), (5000, 129, 2, 3, True), (2500, 768, 8, 7, True),
         (3000, 640, 8, 1, False), (700, 384, 6, 2, False), (700, 512, 6, 2, True), (1200, 260, 6, 2, True),
         # every number of 128-expert chunks, odd sizes that end early in the last one
         (90, 257, 4, 2, True), (400, 259, 4, 1, False), (300, 385, 4, 2, True), (310, 513, 4, 2, False),
         (40, 641, 8, 3, True), (320, 642, 8, 3, True), (330, 769, 8, 1, True), (340, 897, 16, 2, False),
         # the largest batch of one launch, and over its limits of logits and of counts
         (256, 512, 8, 4, True), (256, 516, 8, 4, True), (17, 798, 2, 8, False)]


@pytest.mark.parametrize("T,E,k,S,mask", CASES)
def test_loss_and_counts(T, E, k, S, mask):
    l, ids, seq, m = batch(T, E, k, S, T + E, mask, drop=0.02)
    loss, cnt, tok = run_loss(l, ids, seq, m, 0.25)
    c, n = R.counts(ids, E, seq, m)
    np.testing.assert_array_equal(cnt.cpu().numpy(), c)
    np.testing.assert_array_equal(tok.cpu().numpy(), n)
    ref = R.balance_loss(l, c, n, k, 0.25, seq, m)
    assert abs(float(loss) - ref) <= loss_tolerance(l, E, T) * abs(ref)
    again, _, _ = run_loss(l, ids, seq, m, 0.25)
    assert torch.equal(loss, again)


def backward_tolerance(l, E, k):
    L = float(np.abs(l[np.isfinite(l)]).max(initial=0.0))
    # of the magnitudes: s, 1 - s, the share's quotient, mean and its sums, the factors
    return (4 * (L + 8) + 2 * (E / 32 + 5) + 2 * (k + 5) + 16) * U


def check_backward(l, ids, seq, m, gw, renorm, rsf, gl, alpha):
    T, E = l.shape
    S = 1 if seq is None else len(seq) - 1
    c, n = R.counts(ids, E, seq, m)
    grad, buf = guarded((T, E), torch.float32, 5.0)
    kw = {}
    if gl is not None:
        kw = dict(grad_loss=dev(np.array([gl], np.float32)), expert_counts=dev(c.astype(np.int32)),
                  seq_tokens=dev(n.astype(np.int32)), alpha=alpha)
    lm.moe_router_backward(dev(l), dev(ids), grad, grad_topk_weights=dev(gw), routed_scaling_factor=rsf,
                           renormalize=renorm, token_mask=dev(m), seq_offsets=dev(seq), **kw)
    got = grad.cpu().numpy().astype(np.float64)
    ref, mag = R.router_backward(l, ids, gw, renorm, rsf, gl, c, n, alpha, seq, m)
    err = np.abs(got - ref)
    bound = backward_tolerance(l, E, ids.shape[1]) * mag + 1e-37
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:3])
    assert bool((buf[-GUARD:] == 5.0).all())
    return got


@pytest.mark.parametrize("T,E,k,S,mask", CASES)
def test_backward(T, E, k, S, mask):
    l, ids, seq, m = batch(T, E, k, S, T + E + 1, mask, drop=0.02)
    gw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    check_backward(l, ids, seq, m, gw, 1, 2.5, 0.75, 0.5)


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("parts", ["weights", "loss", "both"])
@pytest.mark.parametrize("E", [96, 97])
def test_backward_parts(E, parts, renorm):
    l, ids, seq, m = batch(90, E, 6, 3, 11, True, drop=0.1)
    gw = np.random.default_rng(4).standard_normal((90, 6)).astype(np.float32)
    check_backward(l, ids, seq, m, gw if parts != "loss" else None, renorm, 2.5,
                   -1.5 if parts != "weights" else None, 0.5)


@pytest.mark.parametrize("E", [64, 33])
def test_extreme_logits(E):
    # rows whose sigmoids underflow, whose experts are partly or wholly masked by
    # -infinity, saturated rows, and one whose masked experts were chosen
    l, ids, _, _ = batch(12, E, 3, 1, 5)
    l[0] = -200.0 + np.arange(E) * 0.25
    l[1] = -np.inf
    l[2, ::2] = -np.inf
    l[3] = 60.0
    l[4] = -30.0
    l[5], l[5, 7] = -np.inf, -150.0
    l[6, ids[6, 0]] = -np.inf
    l[7] = np.float32(-3e38)
    loss, cnt, tok = run_loss(l, ids, None, None, 0.25)
    c, n = R.counts(ids, E)
    ref = R.balance_loss(l, c, n, 3, 0.25)
    small = np.where(np.abs(l) < 1000, l, 0)
    assert abs(float(loss) - ref) <= loss_tolerance(small, E, 12) * ref
    gw = np.random.default_rng(4).standard_normal((12, 3)).astype(np.float32)
    grad = torch.empty((12, E), device="cuda")
    lm.moe_router_backward(dev(l), dev(ids), grad, grad_topk_weights=dev(gw), routed_scaling_factor=2.5,
                           grad_loss=dev(np.ones(1, np.float32)), expert_counts=cnt, seq_tokens=tok, alpha=0.5)
    got = grad.cpu().numpy().astype(np.float64)
    refg, mag = R.router_backward(l, ids, gw, 1, 2.5, 1.0, c, n, 0.5)
    bound = backward_tolerance(small, E, 3) * mag + 1e-37
    assert np.all(np.abs(got - refg) <= bound), np.argwhere(np.abs(got - refg) > bound)[:5]
    assert np.all(got[1] == 0) and np.all(got[2, ::2][~np.isin(np.arange(0, E, 2), ids[2])] == 0)


def test_nothing_valid():
    l, ids, seq, _ = batch(20, 16, 2, 3, 1)
    m = np.zeros(20, np.uint8)
    loss, cnt, tok = run_loss(l, ids, seq, m, 0.25)
    assert float(loss) == 0.0 and int(cnt.abs().sum()) == 0 and int(tok.abs().sum()) == 0
    got = check_backward(l, ids, seq, m, None, 1, 2.5, 1.0, 0.25)
    assert np.all(got == 0)
    # NaN logits reach the loss
    l[3, 2] = np.nan
    loss, _, _ = run_loss(l, ids, None, None, 0.25)
    assert np.isnan(float(loss))


def test_gradient_against_differences():
    # the loss's change along a direction, by the kernel's own loss: step h, an error
    # of h^2 times the third derivative and of the loss's rounding over h
    l, ids, seq, m = batch(40, 32, 3, 2, 8, True)
    alpha, h = 1.0, 2.0 ** -5
    g = np.random.default_rng(3).standard_normal(l.shape).astype(np.float32)
    up, _, _ = run_loss(l + h * g, ids, seq, m, alpha)
    down, _, _ = run_loss(l - h * g, ids, seq, m, alpha)
    got = check_backward(l, ids, seq, m, None, 1, 1.0, 1.0, alpha)
    along = float((got * g).sum())
    diff = (float(up) - float(down)) / (2 * h)
    scale = float((np.abs(got) * np.abs(g)).sum())
    assert abs(diff - along) <= 4 * h * h * scale + loss_tolerance(l, 32, 40) * abs(float(up)) / h


def test_graph_replay_and_autograd_beside_it():
    # captured on a stream of its own, beside a live autograd graph of the same logits
    l, ids, seq, m = batch(200, 64, 4, 2, 6, True)
    logits = dev(l).requires_grad_()
    eager = torch.sigmoid(logits).sum()
    d_ids, d_seq, d_m = dev(ids), dev(seq), dev(m)
    loss, cnt = torch.empty(1, device="cuda"), torch.empty((2, 64), dtype=torch.int32, device="cuda")
    tok, grad = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty((200, 64), device="cuda")
    ws = torch.empty(lm.moe_balance_loss_workspace_bytes(200, 64, 2), dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    s = torch.cuda.Stream()

    def step():
        lm.moe_balance_loss(logits.detach(), d_ids, 0.5, loss, cnt, tok, ws, token_mask=d_m, seq_offsets=d_seq,
                            stream=s)
        lm.moe_router_backward(logits.detach(), d_ids, grad, grad_loss=one, expert_counts=cnt, seq_tokens=tok,
                               alpha=0.5, token_mask=d_m, seq_offsets=d_seq, stream=s)

    torch.cuda.synchronize()
    step()
    s.synchronize()
    want = (loss.clone(), grad.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for _ in range(3):
        loss.fill_(-1), grad.fill_(-1), cnt.fill_(-1), tok.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])
    eager.backward()
    assert logits.grad is not None


def test_largest_batch():
    # T * topk = 2^31 - 1: the ends of the last warps' and CTAs' runs, and the tokens that are
    # looked ahead for, lie past 2^31
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    T, tail = 2 ** 31 - 1, 1000
    gen = torch.Generator(device="cuda").manual_seed(1)
    l = torch.empty((T, 1), device="cuda").uniform_(-3, 3, generator=gen)
    gw = torch.empty((T, 1), device="cuda").uniform_(0.5, 1, generator=gen)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    m = torch.ones(T, dtype=torch.uint8, device="cuda")
    m[5::1 << 20] = 0
    m[-7:-3] = 0
    seq = dev(np.array([0, T - tail, T], np.int32))
    loss, cnt, tok = (torch.full(s, -7, dtype=t, device="cuda") for s, t in (
        ((1,), torch.float32), ((2, 1), torch.int32), ((2,), torch.int32)))
    ws = torch.empty(lm.moe_balance_loss_workspace_bytes(T, 1, 2), dtype=torch.uint8, device="cuda")
    lm.moe_balance_loss(l, ids, 0.5, loss, cnt, tok, ws, token_mask=m, seq_offsets=seq)
    n = [int(m[:T - tail].sum(dtype=torch.int64)), int(m[T - tail:].sum(dtype=torch.int64))]
    assert tok.tolist() == n and cnt.flatten().tolist() == n
    # one expert: each sequence's share of the loss is alpha / 2; a warp's run is summed up in fp32
    run = T / (16 * torch.cuda.get_device_properties(0).multi_processor_count)
    assert abs(float(loss) - 0.5) <= 0.5 * ((run + 100) * U + 2.0 ** -16)
    grad = torch.full((T + GUARD,), 5.0, device="cuda")
    lm.moe_router_backward(l, ids, grad[:T].view(T, 1), grad_topk_weights=gw, renormalize=0,
                           routed_scaling_factor=2.0, grad_loss=torch.ones(1, device="cuda"), expert_counts=cnt,
                           seq_tokens=tok, alpha=0.5, token_mask=m, seq_offsets=seq)
    for a in range(0, T, 1 << 28):
        b = min(a + (1 << 28), T)
        s = torch.sigmoid(l[a:b, 0].double())
        want = 2.0 * gw[a:b, 0] * s * (1 - s)
        # the weights' part; the balance loss of one expert has gradient 0 (f - mean f)
        bound = backward_tolerance(np.array([3.0]), 1, 1) * (2.0 * gw[a:b, 0] * s + 0.5 / tail)
        assert bool(((grad[a:b].double() - want).abs() <= bound).all()), a
        del s, want, bound
    assert bool((grad[T:] == 5.0).all())
    del l, gw, ids, m, grad
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,S", [(3 << 24, 1), ((1 << 25) + 77, 3)])
def test_loss_of_many_tokens(T, S):
    # one expert, chosen by every token: the loss is alpha exactly.  The bound has no term that
    # grows with T: the sigmoids, a term's factors, two roundings of a compensated sum, the
    # CTA's eight and the last CTA's sums (loss_tolerance's others)
    l = torch.empty((T, 1), device="cuda").uniform_(-3, 3)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    cuts = dev(np.array([0, T // 5, T // 2, T] if S == 3 else [0, T], np.int32))
    loss, cnt, tok = torch.empty(1, device="cuda"), *(torch.empty(S, dtype=torch.int32, device="cuda") for _ in "ab")
    ws = torch.empty(lm.moe_balance_loss_workspace_bytes(T, 1, S), dtype=torch.uint8, device="cuda")
    lm.moe_balance_loss(l, ids, 0.25, loss, cnt, tok, ws, seq_offsets=cuts)
    assert int(tok.sum()) == T and torch.equal(cnt, tok)
    assert abs(float(loss) - 0.25) <= 0.25 * (2 * (3 + 8 + 1 / 32 + 5 + 2) + 2 + 8 + 32 + 8) * U


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("parts", ["weights", "loss", "both"])
@pytest.mark.parametrize("E", [8, 96, 257, 896])
def test_gradient_of_confident_experts(E, parts, renorm):
    # logits of 6 to 40 beside ordinary ones: s (1 - s) is exp(-l) there, and the bound has the
    # factor 1 - s (1 / (1 + exp(l))) that the other tests' leaves out
    g = np.random.default_rng(E)
    T, k = 50, 4
    l, ids, seq, m = batch(T, E, k, 3, 17, True)
    high = g.random((T, E)) < 0.5
    l[high] = g.uniform(6, 40, int(high.sum())).astype(np.float32)
    l[:8] = np.linspace(6, 40, 8, dtype=np.float32)[:, None]          # whole rows of one logit
    gw = g.standard_normal((T, k)).astype(np.float32) if parts != "loss" else None
    gl = -1.5 if parts != "weights" else None
    got = check_backward(l, ids, seq, m, gw, renorm, 2.5, gl, 0.5)
    c, n = R.counts(ids, E, seq, m)
    ref, mag = R.router_backward(l, ids, gw, renorm, 2.5, gl, c, n, 0.5, seq, m)
    l64 = l.astype(np.float64)
    # (the reference's own 1 - s, a difference of float64s, is 2^-53 off and as much of mag)
    # backward_tolerance counts s, Z, the dot product and Z again; here 1 - s and the product too
    tol = backward_tolerance(l, E, k) + (float(l.max()) + 8 + 2) * U
    bound = (tol / (1.0 + np.exp(l64)) + 2.0 ** -52) * mag + 1e-37
    assert np.all(np.abs(got - ref) <= bound), (float((np.abs(got - ref) / bound).max()),
                                                np.argwhere(np.abs(got - ref) > bound)[:3])


@pytest.mark.parametrize("S", [1, 3])
def test_empty_batch(S):
    # no tokens: loss and counts are 0, not what an earlier batch left there, on the call's stream
    # and in a graph; the gradient has no element to write
    E = 40
    loss, lbuf = guarded((1,), torch.float32, -7.0)
    cnt, cbuf = guarded((S, E), torch.int32, -7)
    tok, tbuf = guarded((S,), torch.int32, -7)
    l, ids = torch.empty((0, E), device="cuda"), torch.empty((0, 4), dtype=torch.int32, device="cuda")
    seq = None if S == 1 else torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(lm.moe_balance_loss_workspace_bytes(0, E, S), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call():
        lm.moe_balance_loss(l, ids, 0.25, loss, cnt, tok, ws, seq_offsets=seq, stream=s)

    call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    for replay in (False, True):
        if replay:
            with torch.cuda.graph(g, stream=s):
                call()
            loss.fill_(-7), cnt.fill_(-7), tok.fill_(-7)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
        assert float(loss) == 0.0 and int(cnt.abs().sum()) == 0 and int(tok.abs().sum()) == 0
        for b in (lbuf, cbuf, tbuf):
            assert bool((b[-GUARD:] == -7).all())
    lm.moe_router_backward(l, ids, torch.empty((0, E), device="cuda"), grad_loss=torch.ones(1, device="cuda"),
                           expert_counts=cnt, seq_tokens=tok, alpha=0.25, seq_offsets=seq)


def test_workspace_of_a_larger_batch():
    # one workspace for a batch of 5000 tokens, then smaller ones with more CTAs and with fewer
    E, k, big = 96, 4, 5000
    ws = torch.empty(lm.moe_balance_loss_workspace_bytes(big, E, 1), dtype=torch.uint8, device="cuda")
    for T in (big, 4864, 3000, 2433, 2432, 300, 256, 5):
        l, ids, _, m = batch(T, E, k, 1, T, True)
        want, _, _ = run_loss(l, ids, None, m, 0.25)
        loss, cnt = torch.empty(1, device="cuda"), torch.empty((1, E), dtype=torch.int32, device="cuda")
        tok = torch.empty(1, dtype=torch.int32, device="cuda")
        lm.moe_balance_loss(dev(l), dev(ids), 0.25, loss, cnt, tok, ws, token_mask=dev(m))
        assert torch.equal(loss, want)
