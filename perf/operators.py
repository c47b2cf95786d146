"""Cases that time and check the 8-bit expert products and the router's training
operators: each case runs either in plain torch (own = False) or through the
framework's entry points (own = True) on the same inputs.

Kinds of case
  quantize   bf16 -> e4m3 codes with an fp32 scale per 128 elements (lmoe_quantize_fp8)
  linear     block-scaled e4m3 matrix product (lmoe_linear_fp8)
  experts    the routed experts' two products around SituGLU (lmoe_experts_fp8)
  balance    the router's balance loss and per-expert counts (moe_balance_loss)
  backward   the gradient of the router logits (moe_router_backward)
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3_MAX = 448.0
TINY_AMAX = 2.0 ** -100     # smallest block maximum that the quantiser scales by
BETA, LINEAR_BETA = 4.0, 8.0
ALPHA = 1e-3
RSF = 2.5


def listed():
    return [
        # hidden states of a decode step of the 896-expert layer, quantised for its products
        {"name": "quantize_decode", "kind": "quantize", "rows": 8, "K": 7168, "block_rows": 1},
        # a prefill batch's hidden states
        {"name": "quantize_prefill", "kind": "quantize", "rows": 4096, "K": 7168, "block_rows": 1},
        # the down-projection of a single decoded token: latency
        {"name": "linear_one_token", "kind": "linear", "T": 1, "N": 2048, "K": 7168, "add": False},
        # the up-projection of a ragged middle-sized batch, the shared expert's output added
        {"name": "linear_ragged", "kind": "linear", "T": 300, "N": 7168, "K": 2048, "add": True},
        # the shared expert's first product at prefill: tensor cores
        {"name": "linear_prefill", "kind": "linear", "T": 4096, "N": 8192, "K": 7168, "add": False},
        # the smallest layer of the tests
        {"name": "experts_tiny", "kind": "experts", "T": 8, "topk": 4, "E": 64, "latent": 128, "inter": 128, "skew": 0.0},
        # a decode step: about 120 experts with one or two tokens each, weights stream from memory
        {"name": "experts_decode", "kind": "experts", "T": 8, "topk": 16, "E": 896, "latent": 2048, "inter": 512, "skew": 0.0},
        # a prefill batch: 65536 rows over 896 unevenly loaded experts
        {"name": "experts_prefill", "kind": "experts", "T": 4096, "topk": 16, "E": 896, "latent": 2048, "inter": 512, "skew": 0.15},
        # one short training batch of the tiny layer's router
        {"name": "balance_small", "kind": "balance", "T": 256, "E": 64, "topk": 4, "S": 2, "mask": False},
        # a training batch of four ragged sequences with padding
        {"name": "balance_large", "kind": "balance", "T": 16384, "E": 896, "topk": 16, "S": 4, "mask": True},
        {"name": "backward_small", "kind": "backward", "T": 256, "E": 64, "topk": 4, "S": 2, "mask": False, "weights": True},
        {"name": "backward_large", "kind": "backward", "T": 16384, "E": 896, "topk": 16, "S": 4, "mask": True, "weights": True},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["quantize", "linear", "linear", "experts", "experts", "balance", "backward"])
    if kind == "quantize":
        block_rows = rng.choice([1, 1, BLOCK])
        return {"kind": kind, "rows": _log_int(rng, 1, 4096), "K": 16 * _log_int(rng, 4, 448), "block_rows": block_rows}
    if kind == "linear":
        return {"kind": kind, "T": _log_int(rng, 1, 4096), "N": 8 * _log_int(rng, 16, 1024), "K": 16 * _log_int(rng, 8, 448),
                "add": rng.random() < 0.5}
    if kind == "experts":
        E = _log_int(rng, 8, 896)
        return {"kind": kind, "T": _log_int(rng, 1, 4096), "topk": rng.randint(1, min(16, E)), "E": E,
                "latent": 128 * rng.randint(1, 16), "inter": 128 * rng.randint(1, 4), "skew": rng.choice([0.0, 0.1, 0.2])}
    E = _log_int(rng, 8, 896)
    case = {"kind": kind, "T": _log_int(rng, 16, 16384), "E": E, "topk": rng.randint(1, min(16, E)), "S": rng.randint(1, 8),
            "mask": rng.random() < 0.5}
    if kind == "backward":
        case["weights"] = rng.random() < 0.7
    return case


# --- inputs ---------------------------------------------------------------------


def _blocks(n):
    return -(-n // BLOCK)


def _spread(scales, rows, cols, block_rows):
    """One scale per element: `scales` [..., row blocks, column blocks] over [..., rows, cols]."""
    s = scales.repeat_interleave(BLOCK, -1)[..., :cols]
    return s if block_rows == 1 else s.repeat_interleave(block_rows, -2)[..., :rows, :]


def _quantize(x, block_rows):
    """e4m3 codes and fp32 scales of a [..., rows, cols] tensor, in fp32."""
    rows, cols = x.shape[-2:]
    x = x.float()
    pad = (0, _blocks(cols) * BLOCK - cols, 0, -rows % block_rows)
    p = torch.nn.functional.pad(x, pad)
    p = p.reshape(*x.shape[:-2], p.shape[-2] // block_rows, block_rows, _blocks(cols), BLOCK)
    amax = p.abs().amax(dim=(-3, -1)).clamp_min(TINY_AMAX)
    codes = (x * _spread(E4M3_MAX / amax, rows, cols, block_rows)).to(torch.float8_e4m3fn)
    return codes, amax / E4M3_MAX


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _route(g, case):
    """Router logits and the experts that the biased sigmoid scores choose."""
    T, E = case["T"], case["E"]
    logits = _normal(g, T, E)
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1.0
    logits = logits - case.get("skew", 0.2) * torch.log(rank)
    bias = 0.1 * _normal(g, E)
    ids = torch.topk(torch.sigmoid(logits) + bias, case["topk"], dim=1).indices.to(torch.int32)
    return logits.contiguous(), ids.contiguous()


def prepare(case, seed):
    g = _generator(seed)
    kind = case["kind"]
    st = {"case": case}
    if kind == "quantize":
        rows, K, b = case["rows"], case["K"], case["block_rows"]
        x = _normal(g, rows, K)
        x = torch.where(torch.rand((rows, K), generator=g, device=DEV) < 0.001, 20.0 * x, x)
        st["x"] = x.to(torch.bfloat16)
        st["codes"] = torch.empty((rows, K), dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty((-(-rows // b), _blocks(K)), device=DEV)
    elif kind == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        st["x"], st["xs"] = _quantize(_normal(g, T, K), 1)
        st["w"], st["ws"] = _quantize(0.02 * _normal(g, N, K), BLOCK)
        st["add"] = _normal(g, T, N).to(torch.bfloat16) if case["add"] else None
        st["out"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    elif kind == "experts":
        E, L, d = case["E"], case["latent"], case["inter"]
        _, ids = _route(g, case)
        counts = torch.bincount(ids.flatten().long(), minlength=E)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["used"] = counts.nonzero().flatten()      # experts with rows, and the most rows of one:
        st["most"] = int(counts.max())               # what a host-planned batched product goes by
        st["x"], st["xs"] = _quantize(_normal(g, case["T"] * case["topk"], L), 1)
        st["w13"], st["w13s"] = _quantize(0.02 * _normal(g, E, 2 * d, L), BLOCK)
        st["w2"], st["w2s"] = _quantize(0.02 * _normal(g, E, L, d), BLOCK)
        st["out"] = torch.empty((case["T"] * case["topk"], L), dtype=torch.bfloat16, device=DEV)
    else:
        T, E, k, S = case["T"], case["E"], case["topk"], case["S"]
        st["logits"], st["ids"] = _route(g, case)
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device=DEV).sort().values
        st["seq"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
        st["mask"] = (torch.rand(T, generator=g, device=DEV) < 0.9).to(torch.uint8) if case["mask"] else None
        st["loss"] = torch.empty(1, device=DEV)
        st["counts"] = torch.empty((S, E), dtype=torch.int32, device=DEV)
        st["tokens"] = torch.empty(S, dtype=torch.int32, device=DEV)
        if kind == "backward":
            # saved by the forward
            c, n = _counts(st)
            st["counts"].copy_(c)
            st["tokens"].copy_(n)
            st["grad_loss"] = torch.full((1,), 0.5, device=DEV)
            st["grad_w"] = _normal(g, T, k) * (1.0 / T) if case["weights"] else None
            st["grad"] = torch.empty((T, E), device=DEV)
    return st


# --- the plain forms ------------------------------------------------------------


def _widen(codes, scales, block_rows):
    return codes.float() * _spread(scales, codes.shape[-2], codes.shape[-1], block_rows)


def _rows_at(codes, index):
    """codes[index] (indexing goes by bytes: not every e4m3 operation exists in torch)."""
    return codes.view(torch.uint8)[index].view(torch.float8_e4m3fn)


def _situ(gate, up):
    return BETA * torch.tanh(gate / BETA) * torch.sigmoid(gate) * (LINEAR_BETA * torch.tanh(up / LINEAR_BETA))


def _sequence_of(st):
    """Sequence of each token."""
    T = st["logits"].shape[0]
    return torch.searchsorted(st["seq"][1:-1].contiguous(), torch.arange(T, device=DEV, dtype=torch.int32), right=True)


def _counts(st):
    """Chosen experts and valid tokens of each sequence, as whole numbers."""
    T, E = st["logits"].shape
    S = st["seq"].numel() - 1
    valid = torch.ones(T, dtype=torch.int32, device=DEV) if st["mask"] is None else st["mask"].to(torch.int32)
    seq = _sequence_of(st)
    tokens = torch.zeros(S, dtype=torch.int32, device=DEV).index_add_(0, seq, valid)
    at = seq[:, None] * E + st["ids"].long()
    counts = torch.zeros(S * E, dtype=torch.int32, device=DEV).index_add_(0, at.flatten(), valid[:, None].expand_as(at).flatten())
    return counts.view(S, E), tokens


def _share(counts, tokens, E, k):
    """f[s, e]: how many times its even share of the tokens expert e got."""
    return counts * (E / (k * tokens.clamp_min(1).to(counts.dtype)))[:, None]


def _plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "quantize":
        return dict(zip(("codes", "scales"), _quantize(st["x"], case["block_rows"])))
    if kind == "linear":
        y = _widen(st["x"], st["xs"], 1) @ _widen(st["w"], st["ws"], BLOCK).T
        if st["add"] is not None:
            y = y + st["add"].float()
        return {"out": y.to(torch.bfloat16)}
    if kind == "experts":
        d, R = case["inter"], st["x"].shape[0]
        off, used = st["offsets"].long(), st["used"]
        row = torch.arange(R, device=DEV)
        expert = torch.searchsorted(off[1:].contiguous(), row, right=True)
        slot = torch.zeros(case["E"], dtype=torch.long, device=DEV)
        slot[used] = torch.arange(used.numel(), device=DEV)
        at = (off[used][:, None] + torch.arange(st["most"], device=DEV)).clamp_max(R - 1)
        x = _widen(st["x"], st["xs"], 1)[at]
        g = torch.bmm(x, _widen(_rows_at(st["w13"], used), st["w13s"][used], BLOCK).transpose(1, 2))
        act = _widen(*_quantize(_situ(g[..., :d], g[..., d:]), 1), 1)
        y = torch.bmm(act, _widen(_rows_at(st["w2"], used), st["w2s"][used], BLOCK).transpose(1, 2))
        return {"out": y[slot[expert], row - off[expert]].to(torch.bfloat16)}
    E, k, S = case["E"], case["topk"], case["S"]
    counts, tokens = _counts(st) if kind == "balance" else (st["counts"], st["tokens"])
    f = _share(counts.float(), tokens, E, k)
    seq = _sequence_of(st)
    valid = 1.0 if st["mask"] is None else st["mask"].float()
    part = valid / (S * tokens.clamp_min(1).float()[seq])         # a token's part of the mean over sequences
    s = torch.sigmoid(st["logits"])
    z = s.sum(1)
    dot = (s * f[seq]).sum(1) / z
    if kind == "balance":
        return {"loss": (ALPHA * (part.double() * dot.double()).sum()).float().view(1), "counts": counts, "tokens": tokens}
    ds = (st["grad_loss"] * ALPHA * part / z)[:, None] * (f[seq] - dot[:, None])
    if st["grad_w"] is not None:
        ids = st["ids"].long()
        chosen = s.gather(1, ids)
        total = chosen.sum(1, keepdim=True)
        mean = (st["grad_w"] * chosen).sum(1, keepdim=True) / total
        ds = ds.scatter_add(1, ids, RSF / total * (st["grad_w"] - mean))
    return {"grad": ds * s * (1.0 - s)}


# --- the framework's entry points -----------------------------------------------


def _own(st):
    import latent_mixture_experts_sigmoid_gb300 as lm
    case = st["case"]
    kind = case["kind"]
    if kind == "quantize":
        lm.lmoe_quantize_fp8(st["x"], st["codes"], st["scales"], block_rows=case["block_rows"])
        return {"codes": st["codes"].view(torch.float8_e4m3fn), "scales": st["scales"]}
    if kind == "linear":
        lm.lmoe_linear_fp8(st["x"], st["xs"], st["w"], st["ws"], st["out"], add=st["add"])
        return {"out": st["out"]}
    if kind == "experts":
        if "workspace" not in st:
            R, E, L, d = st["x"].shape[0], case["E"], case["latent"], case["inter"]
            st["workspace"] = torch.empty(lm.lmoe_experts_fp8_workspace_bytes(R, E, L, d), dtype=torch.uint8, device=DEV)
            st["experts"] = lm.make_fp8_experts({"w13_q": st["w13"], "w13_s": st["w13s"], "w2_q": st["w2"], "w2_s": st["w2s"]},
                                                E=E, latent=L, inter=d)
        lm.lmoe_experts_fp8(st["experts"], st["x"], st["xs"], st["offsets"], st["out"], st["workspace"], inter=case["inter"],
                            beta=BETA, linear_beta=LINEAR_BETA)
        return {"out": st["out"]}
    if kind == "balance":
        if "workspace" not in st:
            n = lm.moe_balance_loss_workspace_bytes(case["T"], case["E"], case["S"])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        lm.moe_balance_loss(st["logits"], st["ids"], ALPHA, st["loss"], st["counts"], st["tokens"], st["workspace"],
                            token_mask=st["mask"], seq_offsets=st["seq"])
        return {"loss": st["loss"], "counts": st["counts"], "tokens": st["tokens"]}
    lm.moe_router_backward(st["logits"], st["ids"], st["grad"], grad_topk_weights=st["grad_w"], routed_scaling_factor=RSF,
                           grad_loss=st["grad_loss"], expert_counts=st["counts"], seq_tokens=st["tokens"], alpha=ALPHA,
                           token_mask=st["mask"], seq_offsets=st["seq"])
    return {"grad": st["grad"]}


def run(state):
    return _own(state) if own else _plain(state)


# --- the work of one pass -------------------------------------------------------


def work(case):
    kind = case["kind"]
    if kind == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": 3 * n + 4 * -(-case["rows"] // case["block_rows"]) * _blocks(case["K"]), "flops": 3 * n}
    if kind == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        scales = 4 * _blocks(K) * (T + _blocks(N))
        return {"bytes": (T + N) * K + scales + 2 * T * N * (2 if case["add"] else 1), "flops": 2 * T * N * K}
    if kind == "experts":
        E, L, d, R = case["E"], case["latent"], case["inter"], case["T"] * case["topk"]
        used = E * (1.0 - (1.0 - case["topk"] / E) ** case["T"])     # experts with rows, evenly loaded
        weights = used * 3 * d * L * (1 + 4 / BLOCK ** 2)
        return {"bytes": weights + R * L * (1 + 4 / BLOCK) + 2 * R * L + 4 * (E + 1), "flops": 2 * R * 3 * d * L}
    T, E, k, S = case["T"], case["E"], case["topk"], case["S"]
    small = 4 * S * E + 8 * S + (T if case["mask"] else 0)
    if kind == "balance":
        return {"bytes": 4 * T * E + 4 * T * k + small, "flops": 8 * T * E}
    return {"bytes": 8 * T * E + (8 * T * k if case["weights"] else 0) + small, "flops": 12 * T * E}


# --- the definition in 64 bits --------------------------------------------------


def _e4m3(v):
    """v (64 bits, |v| <= 448 but for rounding) to the nearest e4m3 value, ties to the even one."""
    exponent = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))).clamp(-6, 8)
    step = torch.exp2(exponent - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _quantize64(x):
    """Codes (as values) and scales of 1 x 128 blocks of a [..., n * 128] tensor of 64-bit numbers."""
    b = x.view(*x.shape[:-1], -1, BLOCK)
    scale = b.abs().amax(-1, keepdim=True).clamp_min(TINY_AMAX) / E4M3_MAX
    return (_e4m3(b / scale)).view(x.shape), scale.squeeze(-1)


def _expand64(codes, scales, block_rows):
    rows, cols = codes.shape
    r = torch.arange(rows, device=codes.device) // block_rows
    c = torch.arange(cols, device=codes.device) // BLOCK
    return codes.double() * scales.double()[r][:, c]


def _exact_experts(st, case):
    d = case["inter"]
    off = st["offsets"].cpu().numpy().astype(np.int64)
    y = torch.empty(st["out"].shape, dtype=torch.float64, device=DEV)
    for e in np.nonzero(np.diff(off))[0]:
        a, b = int(off[e]), int(off[e + 1])
        x = _expand64(st["x"][a:b], st["xs"][a:b], 1)
        g = x @ _expand64(st["w13"][e], st["w13s"][e], BLOCK).T
        gate, up = g[:, :d], g[:, d:]
        act = BETA * torch.tanh(gate / BETA) / (1 + torch.exp(-gate)) * LINEAR_BETA * torch.tanh(up / LINEAR_BETA)
        q, s = _quantize64(act)
        y[a:b] = _expand64(q, s, 1) @ _expand64(st["w2"][e], st["w2s"][e], BLOCK).T
    return {"out": y}


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        x, b = st["x"].double(), case["block_rows"]
        rows, K = x.shape
        scales = torch.empty(st["scales"].shape, dtype=torch.float64, device=DEV)
        codes = torch.empty_like(x)
        for j in range(_blocks(K)):
            cols = slice(j * BLOCK, min(K, (j + 1) * BLOCK))
            m = x[:, cols].abs().amax(1)
            m = torch.stack([p.amax() for p in m.split(b)]) if b > 1 else m
            scales[:, j] = m.clamp_min(TINY_AMAX) / E4M3_MAX
            codes[:, cols] = _e4m3(x[:, cols] / scales[:, j].repeat_interleave(b)[:rows, None])
        return {"codes": codes, "scales": scales}
    if kind == "linear":
        y = _expand64(st["x"], st["xs"], 1) @ _expand64(st["w"], st["ws"], BLOCK).T
        return {"out": y if st["add"] is None else y + st["add"].double()}
    if kind == "experts":
        return _exact_experts(st, case)
    E, k, S = case["E"], case["topk"], case["S"]
    cut = st["seq"].cpu().tolist()
    l, ids = st["logits"].double(), st["ids"].long()
    loss, counts, tokens = 0.0, [], []
    grad = torch.zeros_like(l)
    s = 1.0 / (1.0 + torch.exp(-l))
    for a, b in zip(cut[:-1], cut[1:]):
        keep = torch.ones(b - a, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"][a:b].bool()
        n = int(keep.sum())
        c = torch.bincount(ids[a:b][keep].flatten(), minlength=E)
        counts.append(c)
        tokens.append(n)
        if n == 0:
            continue
        f = c.double() * E / (k * n)
        z = s[a:b].sum(1, keepdim=True)
        q = s[a:b] / z
        loss += ALPHA / S * float((f * q[keep].mean(0)).sum())
        if kind == "backward":
            # d q[e] / d s[j] = (delta - q[e]) / z
            d = ALPHA * float(st["grad_loss"]) / (S * n) * (f - (f * q).sum(1, keepdim=True)) / z
            grad[a:b] = d * keep[:, None].double()
    if kind == "balance":
        return {"loss": np.array([loss]), "counts": torch.stack(counts).to(torch.int32), "tokens": np.array(tokens, dtype=np.int32)}
    if st["grad_w"] is not None:
        chosen, g = torch.gather(s, 1, ids), st["grad_w"].double()
        total = chosen.sum(1, keepdim=True)
        grad.scatter_add_(1, ids, RSF * (g * total - (g * chosen).sum(1, keepdim=True)) / total ** 2)
    return {"grad": grad * s * (1 - s)}
