"""The training operators together, as a training step of a pre-norm block of routed experts
uses them: residual + norm, routing, the experts' two products around SituGLU on rows grouped
by expert, the combine, and back to every input and weight.  Also the norm in front of the
layer's own forward.

Each operator's output is checked against float64 of the same inputs that the GPU had (so
that the bf16 roundings between them do not accumulate), and the whole step's gradients
against a float64 step: the roundings of its nine bf16 intermediates are 2^-8 of a value each
and nearly independent, so their norm is within a few 2^-8 of the gradient's; 0.05 is an
order of magnitude above that, and far below what a wrong term gives (about 1)."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import training_oracle as O

pytestmark = pytest.mark.gpu
lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
BF16 = torch.finfo(torch.bfloat16).eps / 2
EPS, BETA, LBETA, RSF = 1e-6, 4.0, 8.0, 2.5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    lm.load_library()


def f64(t):
    return t.detach().double().cpu().numpy()


class Block:
    """One block: H wide, E experts of d features, k of them a token."""

    def __init__(self, T, H, E, d, k, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, std=1.0: (std * torch.randn(s, generator=g)).to(torch.bfloat16).to("cuda")  # noqa: E731
        self.T, self.H, self.E, self.d, self.k = T, H, E, d, k
        self.x, self.res = r(T, H), r(T, H)
        self.gamma = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).to("cuda")
        self.w_router = r(E, H, std=H ** -0.5)
        self.w13, self.w2 = r(E, 2 * d, H, std=0.05), r(E, H, d, std=0.05)
        self.bias = torch.zeros(E, device="cuda")
        self.dout = r(T, H, std=0.1)

    def empty(self, *shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def step(self):
        T, H, E, d, k, R = self.T, self.H, self.E, self.d, self.k, self.T * self.k
        h, n = self.empty(T, H), self.empty(T, H)
        lm.lmoe_rms_norm(self.x, self.gamma, EPS, out=n, residual=self.res, residual_out=h)
        logits, ids, w = (self.empty(T, E, dtype=torch.float32), self.empty(T, k, dtype=torch.int32),
                          self.empty(T, k, dtype=torch.float32))
        ws = torch.empty(lm.lmoe_router_logits_workspace_bytes(T, E, H), dtype=torch.uint8, device="cuda")
        lm.lmoe_router_logits(n, self.w_router, logits, ws)
        lm.moe_route(logits, self.bias, k, RSF, ids, w)
        # rows grouped by expert
        order = torch.argsort(ids.flatten(), stable=True)
        token, place = order // k, torch.argsort(order)

        def of_tokens(rows):                       # the sum of each token's rows, always in the same order
            return rows[place].view(T, k, -1).sum(1)

        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = torch.bincount(ids.flatten(), minlength=E).cumsum(0)
        a = n[token]
        g, act, y = self.empty(R, 2 * d), self.empty(R, d), self.empty(R, H)
        lm.lmoe_grouped_linear(a, self.w13, off, g)
        lm.situ_and_mul(g, act, BETA, LBETA)
        lm.lmoe_grouped_linear(act, self.w2, off, y)
        wr = w.flatten()[order][:, None]
        out = h.float() + of_tokens(wr * y.float())
        # back: out's gradient is dout
        dy = (wr * self.dout.float()[token]).to(torch.bfloat16)
        dw_rows = (self.dout.float()[token] * y.float()).sum(1)
        dact, dg, da = self.empty(R, d), self.empty(R, 2 * d), self.empty(R, H)
        dw2, dw13 = self.empty(E, H, d, dtype=torch.float32), self.empty(E, 2 * d, H, dtype=torch.float32)
        lm.lmoe_grouped_linear_backward_x(dy, self.w2, off, dact)
        lm.lmoe_grouped_linear_backward_w(dy, act, off, dw2)
        lm.situ_and_mul_backward(g, dact, dg, BETA, LBETA)
        lm.lmoe_grouped_linear_backward_x(dg, self.w13, off, da)
        lm.lmoe_grouped_linear_backward_w(dg, a, off, dw13)
        dwt = torch.empty_like(w)
        dwt.view(-1)[order] = dw_rows
        dlogits = torch.empty_like(logits)
        lm.moe_router_backward(logits, ids, dlogits, grad_topk_weights=dwt, routed_scaling_factor=RSF)
        dn = of_tokens(da.float()) + dlogits @ self.w_router.float()
        dn = dn.to(torch.bfloat16)
        dh, dgamma = self.empty(T, H), self.empty(H, dtype=torch.float32)
        nws = torch.empty(lm.lmoe_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        lm.lmoe_rms_norm_backward(dn, h, self.gamma, EPS, dh, grad_norm_w=dgamma, grad_residual=self.dout, workspace=nws)
        assert lm.lmoe_device_error() == 0
        return dict(locals())


def reference(b, ids):
    """The step in float64 by autograd, the experts chosen as on the GPU."""
    t = {n: getattr(b, n).double().cpu().requires_grad_() for n in ("x", "res", "gamma", "w_router", "w13", "w2")}
    ids = ids.long().cpu()
    h = t["x"] + t["res"]
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * t["gamma"]
    s = torch.sigmoid(n @ t["w_router"].T).gather(1, ids)
    w = RSF * s / s.sum(1, keepdim=True)
    out = h
    for j in range(b.k):
        g = torch.einsum("th,tdh->td", n, t["w13"][ids[:, j]])
        gate, up = g[:, :b.d], g[:, b.d:]
        act = BETA * torch.tanh(gate / BETA) * torch.sigmoid(gate) * LBETA * torch.tanh(up / LBETA)
        out = out + w[:, j:j + 1] * torch.einsum("td,thd->th", act, t["w2"][ids[:, j]])
    (out * b.dout.double().cpu()).sum().backward()
    return out.detach(), {n: v.grad for n, v in t.items()}


@pytest.mark.parametrize("T,H,E,d,k", [(37, 128, 8, 64, 2), (150, 256, 24, 128, 4)])
def test_step_against_float64(T, H, E, d, k):
    b = Block(T, H, E, d, k, T)
    r = b.step()
    out, grad = reference(b, r["ids"])

    def near(got, ref, name):
        off = np.linalg.norm(f64(got) - ref.numpy()) / np.linalg.norm(ref.numpy())
        assert off <= 0.05, (name, off)

    near(r["out"], out, "out")
    for name, got in (("x", r["dh"]), ("res", r["dh"]), ("gamma", r["dgamma"]), ("w13", r["dw13"]), ("w2", r["dw2"]),
                      ("w_router", r["dlogits"].T @ r["n"].float())):
        near(got, grad[name], name)


def test_each_operator_on_the_step_s_own_inputs():
    b = Block(90, 192, 12, 64, 3, 5)
    r = b.step()
    off = f64(r["off"])

    def close(got, ref, mag, terms):
        err = np.abs(f64(got) - ref)
        assert np.all(err <= BF16 * (1 + 2 ** -7) * np.abs(ref) + (terms / 16 + 32) * 2.0 ** -23 * mag)

    for got, fn, rows, w in ((r["g"], O.grouped_linear, r["a"], b.w13), (r["y"], O.grouped_linear, r["act"], b.w2),
                             (r["dact"], O.grouped_linear_backward_x, r["dy"], b.w2),
                             (r["da"], O.grouped_linear_backward_x, r["dg"], b.w13)):
        rows, w, shape = f64(rows), f64(w), got.shape
        close(got, fn(rows, w, off, np.zeros(shape)), fn(np.abs(rows), np.abs(w), off, np.zeros(shape)), rows.shape[1])
    for got, dy, x in ((r["dw2"], r["dy"], r["act"]), (r["dw13"], r["dg"], r["a"])):
        dy, x = f64(dy), f64(x)
        ref, mag = O.grouped_linear_backward_w(dy, x, off), O.grouped_linear_backward_w(np.abs(dy), np.abs(x), off)
        assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -24 * np.abs(ref) + (32 + 2 + len(x) / 1024) * 2.0 ** -23 * mag)
    dgate, mag, dup = O.situ_backward(f64(r["g"])[:, :64], f64(r["g"])[:, 64:], f64(r["dact"]), BETA, LBETA)
    assert np.all(np.abs(f64(r["dg"])[:, :64] - dgate) <= BF16 * (1 + 2 ** -7) * np.abs(dgate) + 2.0 ** -14 * mag + 1e-37)
    assert np.all(np.abs(f64(r["dg"])[:, 64:] - dup) <= (BF16 * (1 + 2 ** -7) + 2.0 ** -14) * np.abs(dup) + 1e-37)


def test_step_in_a_graph_beside_eager_steps():
    # a captured step replayed while another block's step runs eagerly: the same bits as alone
    a, b = Block(64, 128, 8, 64, 2, 1), Block(80, 128, 8, 64, 2, 2)
    keep = ("out", "dh", "dgamma", "dw13", "dw2", "dlogits")
    want_a, want_b = ({n: r[n].clone() for n in keep} for r in (a.step(), b.step()))
    torch.cuda.synchronize()
    # (the routing's grouping through torch ops and the error word's read are not for a capture: the
    # operators are captured on the buffers of an eager step)
    r = a.step()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def operators():
        lm.lmoe_rms_norm(a.x, a.gamma, EPS, out=r["n"], residual=a.res, residual_out=r["h"])
        lm.lmoe_grouped_linear(r["a"], a.w13, r["off"], r["g"])
        lm.situ_and_mul(r["g"], r["act"], BETA, LBETA)
        lm.lmoe_grouped_linear(r["act"], a.w2, r["off"], r["y"])
        lm.lmoe_grouped_linear_backward_x(r["dy"], a.w2, r["off"], r["dact"])
        lm.lmoe_grouped_linear_backward_w(r["dy"], r["act"], r["off"], r["dw2"])
        lm.situ_and_mul_backward(r["g"], r["dact"], r["dg"], BETA, LBETA)
        lm.lmoe_grouped_linear_backward_x(r["dg"], a.w13, r["off"], r["da"])
        lm.lmoe_grouped_linear_backward_w(r["dg"], r["a"], r["off"], r["dw13"])
        lm.lmoe_rms_norm_backward(r["dn"], r["h"], a.gamma, EPS, r["dh"], grad_norm_w=r["dgamma"],
                                  grad_residual=a.dout, workspace=r["nws"])

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        operators()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            operators()
    for n in ("n", "h", "g", "act", "y", "dact", "dw2", "dg", "da", "dw13", "dh", "dgamma"):
        r[n].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        graph.replay()
        rb = b.step()
    torch.cuda.synchronize()
    for n in ("dh", "dgamma", "dw13", "dw2"):
        assert torch.equal(r[n], want_a[n]), n
    for n in keep:
        assert torch.equal(rb[n], want_b[n]), n


def test_norm_in_front_of_the_layer():
    # hidden states normalised on the way into the layer's forward, in bf16 and in e4m3: the codes are
    # those of the e4m3 products on the same rows
    d = W.TINY
    host = W.layer_weights(d, 0)
    dev = lambda a: torch.from_numpy(a.view(np.int16)).to("cuda").view(torch.bfloat16)  # noqa: E731
    wts = {n: (torch.from_numpy(v).to("cuda") if v.dtype == np.float32 else dev(v)) for n, v in host.items()}
    x = dev(W.hidden_states(d, 0))
    res = torch.roll(x, 1, 0).contiguous()
    h, n = torch.empty_like(x), torch.empty_like(x)
    codes, scales = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((d.T, d.hidden // 128), device="cuda")
    lm.lmoe_rms_norm(x, None, EPS, out=n, codes=codes, scales=scales, residual=res, residual_out=h)
    lg = torch.from_numpy(W.router_logits(d.T, d.num_experts, 0)).to("cuda")
    out, again = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(lm.latent_moe_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    lm.latent_moe_forward(d, wts, n, lg, out, ws)
    _, y = O.rms_norm(f64(x), f64(res), None, EPS)
    lm.latent_moe_forward(d, wts, torch.from_numpy(y).to("cuda").to(torch.bfloat16), lg, again, ws)
    # the inputs differ by a bf16 step in few places at the most
    assert float((out.float() - again.float()).norm() / again.float().norm()) <= 2 * BF16
    wq, wsc = torch.empty(wts["w_down"].shape, dtype=torch.uint8, device="cuda"), torch.empty((1, d.hidden // 128), device="cuda")
    lm.lmoe_quantize_fp8(wts["w_down"], wq, wsc, block_rows=128)
    z8, z16 = (torch.empty((d.T, d.latent), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lm.lmoe_linear_fp8(codes, scales, wq, wsc, z8)
    lm.lmoe_linear(n, wts["w_down"], z16)
    # e4m3 rounds by 2^-4 at most, 2^-5.8 in the mean square, on each of the two operands
    assert float((z8.float() - z16.float()).norm() / z16.float().norm()) <= 2.0 ** -4
