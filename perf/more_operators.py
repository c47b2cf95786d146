"""Cases that time and check the operators of training the routed experts and of the
normalisation in front of them: each case runs either in plain torch (own = False) or
through the framework's entry points (own = True) on the same inputs.

Kinds of case
  norm           residual addition, RMSNorm, bf16 and e4m3 outputs (lmoe_rms_norm)
  norm_backward  its gradient (lmoe_rms_norm_backward)
  forward        product of rows grouped by expert (lmoe_grouped_linear)
  grad_x         its gradient to the rows (lmoe_grouped_linear_backward_x)
  grad_w         its gradient to the experts' weights (lmoe_grouped_linear_backward_w)
  situ_backward  gradient of SituGLU (situ_and_mul_backward)
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3_MAX = 448.0
TINY_AMAX = 2.0 ** -100     # smallest block maximum that the quantiser scales by
BETA, LINEAR_BETA = 4.0, 8.0
EPS = 1e-6


def listed():
    return [
        # one decoded token in front of the layer: latency
        {"name": "norm_token", "kind": "norm", "T": 1, "H": 7168, "residual": True, "out": "both"},
        # a prefill batch: bf16 for the router, codes for the 8-bit products
        {"name": "norm_prefill", "kind": "norm", "T": 4096, "H": 7168, "residual": True, "out": "both"},
        # a short ragged batch in the latent width
        {"name": "norm_backward_short", "kind": "norm_backward", "T": 300, "H": 2048, "residual": False},
        # a training batch, with the gradient that comes down the residual path
        {"name": "norm_backward_train", "kind": "norm_backward", "T": 16384, "H": 7168, "residual": True},
        # a decode step of the 896-expert layer: 128 rows over about 120 experts, weights stream from memory
        {"name": "forward_decode", "kind": "forward", "T": 8, "topk": 16, "E": 896, "N": 1024, "K": 2048, "skew": 0.0},
        # gate and up products of a batch: 65536 rows over 896 unevenly loaded experts
        {"name": "forward_train", "kind": "forward", "T": 4096, "topk": 16, "E": 896, "N": 1024, "K": 2048, "skew": 0.15},
        # the smallest layer of the tests, ragged
        {"name": "grad_x_tiny", "kind": "grad_x", "T": 75, "topk": 4, "E": 64, "N": 256, "K": 128, "skew": 0.2},
        # down product of 128 experts: tensor cores
        {"name": "grad_x_train", "kind": "grad_x", "T": 4096, "topk": 16, "E": 128, "N": 2048, "K": 512, "skew": 0.15},
        # the smallest layer again, gradients in bf16, experts without rows among them
        {"name": "grad_w_tiny", "kind": "grad_w", "T": 75, "topk": 4, "E": 64, "N": 256, "K": 128, "skew": 0.5, "dtype": "bf16",
         "add": False},
        # gate and up weights of 128 experts in fp32, over the gradient of an earlier micro-batch
        {"name": "grad_w_train", "kind": "grad_w", "T": 4096, "topk": 16, "E": 128, "N": 1024, "K": 2048, "skew": 0.15,
         "dtype": "fp32", "add": True},
        # the rows of a decode-sized batch
        {"name": "situ_backward_short", "kind": "situ_backward", "rows": 128, "d": 512, "linear": True},
        # the rows of a training batch
        {"name": "situ_backward_train", "kind": "situ_backward", "rows": 65536, "d": 512, "linear": True},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_backward", "forward", "forward", "grad_x", "grad_x", "grad_w", "grad_w", "situ_backward"])
    if kind == "norm":
        return {"kind": kind, "T": _log_int(rng, 1, 4096), "H": 16 * _log_int(rng, 4, 448), "residual": rng.random() < 0.7,
                "out": rng.choice(["both", "both", "bf16", "codes"])}
    if kind == "norm_backward":
        return {"kind": kind, "T": _log_int(rng, 1, 16384), "H": 8 * _log_int(rng, 8, 896), "residual": rng.random() < 0.7}
    if kind == "situ_backward":
        return {"kind": kind, "rows": _log_int(rng, 1, 65536), "d": 8 * _log_int(rng, 4, 64), "linear": rng.random() < 0.7}
    E = _log_int(rng, 4, 128 if kind == "grad_w" else 896)
    N = 8 * _log_int(rng, 8, 256)
    case = {"kind": kind, "T": _log_int(rng, 1, 4096), "topk": rng.randint(1, min(16, E)), "E": E, "N": N,
            "K": 8 * _log_int(rng, 8, min(256, (1 << 18) // N)), "skew": rng.choice([0.0, 0.1, 0.2])}
    if kind == "grad_w":
        case["dtype"] = rng.choice(["fp32", "bf16"])
        case["add"] = case["dtype"] == "fp32" and rng.random() < 0.5
    return case


# --- inputs ---------------------------------------------------------------------


def _normal(g, *shape, std=1.0):
    return (std * torch.randn(shape, generator=g, device=DEV)).to(torch.bfloat16)


def _groups(g, case):
    """Rows of each expert: the choices of T tokens by unevenly offset scores, sorted by expert."""
    T, E = case["T"], case["E"]
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1.0
    score = torch.randn((T, E), generator=g, device=DEV) - case["skew"] * torch.log(rank)
    counts = torch.bincount(torch.topk(score, case["topk"], dim=1).indices.flatten(), minlength=E)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32), counts


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    kind = case["kind"]
    st = {"case": case}
    if kind in ("norm", "norm_backward"):
        T, H = case["T"], case["H"]
        # a residual stream: a few columns much larger than the others
        spread = torch.exp(0.5 * torch.randn(H, generator=g, device=DEV))
        st["w"] = (1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
        if kind == "norm":
            st["x"] = _normal(g, T, H)
            st["residual"] = (spread * torch.randn((T, H), generator=g, device=DEV)).to(torch.bfloat16) if case["residual"] else None
            st["h"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV) if case["residual"] else None
            if case["out"] != "codes":
                st["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            if case["out"] != "bf16":
                st["codes"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
                st["scales"] = torch.empty((T, -(-H // BLOCK)), device=DEV)
        else:
            st["h"] = (spread * torch.randn((T, H), generator=g, device=DEV)).to(torch.bfloat16)
            st["dy"] = _normal(g, T, H, std=1e-3)
            st["dres"] = _normal(g, T, H, std=1e-3) if case["residual"] else None
            st["dh"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            st["dw"] = torch.empty(H, device=DEV)
        return st
    if kind == "situ_backward":
        rows, d = case["rows"], case["d"]
        x = 3.0 * torch.randn((rows, 2 * d), generator=g, device=DEV)
        far = torch.rand((rows, 2 * d), generator=g, device=DEV) < 0.01        # saturated
        st["x"] = torch.where(far, torch.sign(x) * 40.0, x).to(torch.bfloat16)
        st["dy"] = _normal(g, rows, d, std=1e-3)
        st["dx"] = torch.empty((rows, 2 * d), dtype=torch.bfloat16, device=DEV)
        return st
    E, N, K, R = case["E"], case["N"], case["K"], case["T"] * case["topk"]
    st["offsets"], counts = _groups(g, case)
    st["used"] = counts.nonzero().flatten()      # experts with rows, and the most rows of one:
    st["most"] = int(counts.max())               # what a host-planned batched product goes by
    if kind != "grad_x":
        st["x"] = _normal(g, R, K)
    if kind != "forward":
        st["dy"] = _normal(g, R, N, std=1e-3)
    if kind == "grad_w":
        st["before"] = 1e-2 * torch.randn((E, N, K), generator=g, device=DEV) if case["add"] else None
        st["dw"] = torch.empty((E, N, K), dtype=torch.float32 if case["dtype"] == "fp32" else torch.bfloat16, device=DEV)
    else:
        st["w"] = _normal(g, E, N, K, std=0.02)
        st["out"] = torch.empty((R, N if kind == "forward" else K), dtype=torch.bfloat16, device=DEV)
    return st


# --- the plain forms ------------------------------------------------------------


def _quantize(y):
    """e4m3 codes and fp32 scales of a [rows, cols] fp32 tensor, one scale per row and 128 columns."""
    rows, cols = y.shape
    p = torch.nn.functional.pad(y, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    amax = p.abs().amax(2, keepdim=True).clamp_min(TINY_AMAX)
    codes = (p * (E4M3_MAX / amax)).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return codes.contiguous(), (amax / E4M3_MAX).squeeze(2)


def _places(st, rows):
    """Place of every row in a [used experts, most rows] table, and the rows of that table
    (the first row stands where an expert has none left)."""
    off, used = st["offsets"].long(), st["used"]
    row = torch.arange(rows, device=DEV)
    slot = torch.searchsorted(off[1:][used].contiguous(), row, right=True)
    return (slot, row - off[used][slot]), used


def _table(rows, at, shape):
    """The rows grouped by expert, those of each padded with zeros."""
    t = torch.zeros((*shape, rows.shape[1]), device=DEV)
    t[at] = rows.float()
    return t


def _plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "norm":
        h = st["x"].float()
        if st["residual"] is not None:
            h = h + st["residual"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["w"].float()
        res = {}
        if st["residual"] is not None:
            res["h"] = h.to(torch.bfloat16)
        if case["out"] != "codes":
            res["out"] = y.to(torch.bfloat16)
        if case["out"] != "bf16":
            res["codes"], res["scales"] = _quantize(y)
        return res
    if kind == "norm_backward":
        h, dy, w = st["h"].float(), st["dy"].float(), st["w"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        n = h * r
        g = dy * w
        dh = r * (g - n * (g * n).mean(1, keepdim=True))
        if st["dres"] is not None:
            dh = dh + st["dres"].float()
        return {"dh": dh.to(torch.bfloat16), "dw": (dy * n).sum(0)}
    if kind == "situ_backward":
        d = case["d"]
        gate, up, dy = st["x"][:, :d].float(), st["x"][:, d:].float(), st["dy"].float()
        s, t = torch.sigmoid(gate), torch.tanh(gate / BETA)
        sech2 = 1.0 / torch.cosh(gate / BETA) ** 2
        lin, dlin = up, 1.0
        if case["linear"]:
            lin = LINEAR_BETA * torch.tanh(up / LINEAR_BETA)
            dlin = 1.0 / torch.cosh(up / LINEAR_BETA) ** 2
        dgate = dy * lin * (sech2 * s + BETA * t * s * torch.sigmoid(-gate))
        return {"dx": torch.cat([dgate, dy * (BETA * t * s) * dlin], 1).to(torch.bfloat16)}
    at, used = _places(st, case["T"] * case["topk"])
    shape = (used.numel(), st["most"])
    if kind == "grad_w":
        dw = torch.zeros(st["dw"].shape, device=DEV)
        dw[used] = torch.bmm(_table(st["dy"], at, shape).transpose(1, 2), _table(st["x"], at, shape))
        if case["add"]:
            dw = st["before"] + dw
        return {"dw": dw.to(st["dw"].dtype)}
    w = st["w"][used].float()
    if kind == "forward":
        y = torch.bmm(_table(st["x"], at, shape), w.transpose(1, 2))
    else:
        y = torch.bmm(_table(st["dy"], at, shape), w)
    return {"out": y[at].to(torch.bfloat16)}


# --- the framework's entry points -----------------------------------------------


def _own(st):
    import latent_mixture_experts_sigmoid_gb300 as lm
    case = st["case"]
    kind = case["kind"]
    if kind == "norm":
        lm.lmoe_rms_norm(st["x"], st["w"], EPS, out=st.get("out"), codes=st.get("codes"), scales=st.get("scales"),
                         residual=st["residual"], residual_out=st["h"])
        return {k: st[k] for k in ("h", "out", "codes", "scales") if st.get(k) is not None}
    if kind == "norm_backward":
        if "workspace" not in st:
            n = lm.lmoe_rms_norm_backward_workspace_bytes(case["T"], case["H"])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        lm.lmoe_rms_norm_backward(st["dy"], st["h"], st["w"], EPS, st["dh"], grad_norm_w=st["dw"], grad_residual=st["dres"],
                                  workspace=st["workspace"])
        return {"dh": st["dh"], "dw": st["dw"]}
    if kind == "situ_backward":
        lm.situ_and_mul_backward(st["x"], st["dy"], st["dx"], BETA, LINEAR_BETA if case["linear"] else 0.0)
        return {"dx": st["dx"]}
    if kind == "forward":
        lm.lmoe_grouped_linear(st["x"], st["w"], st["offsets"], st["out"])
        return {"out": st["out"]}
    if kind == "grad_x":
        lm.lmoe_grouped_linear_backward_x(st["dy"], st["w"], st["offsets"], st["out"])
        return {"out": st["out"]}
    lm.lmoe_grouped_linear_backward_w(st["dy"], st["x"], st["offsets"], st["dw"], add=st["before"])
    return {"dw": st["dw"]}


def run(state):
    return _own(state) if own else _plain(state)


# --- the work of one pass -------------------------------------------------------


def work(case):
    kind = case["kind"]
    if kind == "norm":
        T, H = case["T"], case["H"]
        each = 2 + (4 if case["residual"] else 0) + (2 if case["out"] != "codes" else 0) + (1 + 4 / BLOCK if case["out"] != "bf16" else 0)
        return {"bytes": int(T * H * each) + 2 * H, "flops": 8 * T * H}
    if kind == "norm_backward":
        T, H = case["T"], case["H"]
        return {"bytes": T * H * (8 if case["residual"] else 6) + 6 * H, "flops": 12 * T * H}
    if kind == "situ_backward":
        return {"bytes": 10 * case["rows"] * case["d"], "flops": 25 * case["rows"] * case["d"]}
    E, N, K, R = case["E"], case["N"], case["K"], case["T"] * case["topk"]
    if kind == "grad_w":
        each = (4 if case["dtype"] == "fp32" else 2) * (2 if case["add"] else 1)
        return {"bytes": E * N * K * each + 2 * R * (N + K) + 4 * (E + 1), "flops": 2 * R * N * K}
    used = E * (1.0 - (1.0 - case["topk"] / E) ** case["T"])     # experts with rows, evenly loaded
    return {"bytes": int(2 * used * N * K) + 2 * R * (N + K) + 4 * (E + 1), "flops": 2 * R * N * K}


# --- the definition in 64 bits --------------------------------------------------


def _e4m3(v):
    """v (64 bits, |v| <= 448 but for rounding) to the nearest e4m3 value, ties to the even one."""
    exponent = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))).clamp(-6, 8)
    step = torch.exp2(exponent - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(st, case):
    x = st["x"].double()
    if st["residual"] is not None:
        x += st["residual"].double()
    res = {} if st["residual"] is None else {"h": x.clone()}
    x /= torch.sqrt((x ** 2).sum(1) / case["H"] + EPS)[:, None]
    x *= st["w"].double()
    if case["out"] != "codes":
        res["out"] = x.clone()
    if case["out"] != "bf16":
        res["codes"], res["scales"] = torch.empty_like(x), torch.empty(st["scales"].shape, dtype=torch.float64, device=DEV)
        for b in range(res["scales"].shape[1]):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            s = part.abs().amax(1).clamp_min(TINY_AMAX) / E4M3_MAX
            res["scales"][:, b] = s
            res["codes"][:, b * BLOCK:(b + 1) * BLOCK] = _e4m3(part / s[:, None])
    return res


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        return _exact_norm(st, case)
    if kind == "norm_backward":
        h, dy, H = st["h"].double(), st["dy"].double(), case["H"]
        ms = (h ** 2).sum(1, keepdim=True) / H + EPS
        # d(h ms^-1/2)/dh by the product rule
        dot = (dy * st["w"].double() * h).sum(1, keepdim=True)
        dh = dy * st["w"].double() * ms ** -0.5 - h * dot * ms ** -1.5 / H
        if st["dres"] is not None:
            dh += st["dres"].double()
        return {"dh": dh, "dw": torch.einsum("th,th,t->h", dy, h, ms[:, 0] ** -0.5)}
    if kind == "situ_backward":
        d, out = case["d"], torch.empty(st["dx"].shape, dtype=torch.float64, device=DEV)
        for a in range(0, case["rows"], 8192):
            x, dy = st["x"][a:a + 8192].double(), st["dy"][a:a + 8192].double()
            g, u = x[:, :d], x[:, d:]
            e = torch.exp(-g)                     # sigmoid 1 / (1 + e), its derivative e / (1 + e)^2
            f = BETA * torch.tanh(g / BETA)
            k, dk = (LINEAR_BETA * torch.tanh(u / LINEAR_BETA), torch.cosh(u / LINEAR_BETA) ** -2) if case["linear"] else (u, 1.0)
            out[a:a + 8192, :d] = dy * k * (torch.cosh(g / BETA) ** -2 / (1 + e) + f * e / (1 + e) ** 2)
            out[a:a + 8192, d:] = dy * f / (1 + e) * dk
        return {"dx": out}
    off = st["offsets"].tolist()
    if kind == "grad_w":
        dw = st["before"].double() if case["add"] else torch.zeros(st["dw"].shape, dtype=torch.float64, device=DEV)
        for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if b > a:
                dw[e] += st["dy"][a:b].double().T @ st["x"][a:b].double()
        return {"dw": dw}
    out = torch.empty(st["out"].shape, dtype=torch.float64, device=DEV)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if b > a:
            w = st["w"][e].double()
            out[a:b] = st["x"][a:b].double() @ w.T if kind == "forward" else st["dy"][a:b].double() @ w
    return {"out": out}
