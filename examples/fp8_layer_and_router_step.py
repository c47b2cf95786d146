"""The e4m3 operators and the router's training operators together.

A small latent-MoE layer whose experts are quantised on the GPU runs forward on e4m3
experts, and its router is trained for some steps: the routing weights follow a gradient
from outside (here: a fixed utility of each expert for each token) while the balance loss
holds the experts' load together.

    python examples/fp8_layer_and_router_step.py [--steps N]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import latent_mixture_experts_sigmoid_gb300 as lm
import workloads as W

DEV = "cuda"
BLOCK = 128


def to_device(bits: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(bits.view(np.int16)).to(DEV).view(torch.bfloat16)


def quantize(x: torch.Tensor, block_rows: int):
    """e4m3 codes and scales of a [..., rows, K] bf16 tensor (rows % block_rows == 0)."""
    K = x.shape[-1]
    rows = x.numel() // K
    codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(*x.shape[:-2], -(-x.shape[-2] // block_rows), -(-K // BLOCK), device=DEV)
    lm.lmoe_quantize_fp8(x, codes, scales, block_rows=block_rows, rows=rows, K=K)
    return codes, scales


def main(steps: int = 20, alpha: float = 0.2, lr: float = 0.5):
    d = W.LayerDims(T=192, hidden=256, latent=128, num_experts=32, topk=4, inter=128, shared_inter=128)
    T, E, k = d.T, d.num_experts, d.topk
    host = W.layer_weights(d, 0)
    weights = {n: (torch.from_numpy(v).to(DEV) if v.dtype == np.float32 else to_device(v))
               for n, v in host.items()}
    # the experts in e4m3: what a checkpoint would hold; the bf16 ones are not needed again
    experts = {}
    for name in ("w13", "w2"):
        experts[name + "_q"], experts[name + "_s"] = quantize(weights.pop(name), BLOCK)
    hidden = to_device(W.hidden_states(d, 0))
    w_router = to_device(W.w_router(d, 0)).float()

    # the layer's first dense product in e4m3 beside the bf16 one
    xq, xs = quantize(hidden, 1)
    wq, ws = quantize(weights["w_down"], BLOCK)
    z8 = torch.empty((T, d.latent), dtype=torch.bfloat16, device=DEV)
    z16 = torch.empty_like(z8)
    lm.lmoe_linear_fp8(xq, xs, wq, ws, z8)
    lm.lmoe_linear(hidden, weights["w_down"], z16)
    off = float((z8.float() - z16.float()).norm() / z16.float().norm())

    # three sequences of unequal length, the last tokens of each padding
    seq = torch.tensor([0, 64, 160, T], dtype=torch.int32, device=DEV)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[60:64] = mask[150:160] = mask[T - 5:] = 0
    g = torch.Generator(device=DEV).manual_seed(0)
    utility = torch.randn((T, E), generator=g, device=DEV) + torch.linspace(1, -1, E, device=DEV)

    logits = torch.empty((T, E), device=DEV)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    topw = torch.empty((T, k), device=DEV)
    out = torch.empty((T, d.hidden), dtype=torch.bfloat16, device=DEV)
    layer_ws = torch.empty(lm.latent_moe_workspace_bytes_fp8(d), dtype=torch.uint8, device=DEV)
    router_ws = torch.empty(lm.lmoe_router_logits_workspace_bytes(T, E, d.hidden), dtype=torch.uint8, device=DEV)
    loss_ws = torch.empty(lm.moe_balance_loss_workspace_bytes(T, E, 3), dtype=torch.uint8, device=DEV)
    loss, grad_loss = torch.empty(1, device=DEV), torch.ones(1, device=DEV)
    counts = torch.empty((3, E), dtype=torch.int32, device=DEV)
    tokens = torch.empty(3, dtype=torch.int32, device=DEV)
    grad = torch.empty((T, E), device=DEV)
    history = []
    for _ in range(steps):
        router = w_router.bfloat16()
        torch.cuda.synchronize()          # a weight is complete before a call that reads it starts
        lm.lmoe_router_logits(hidden, router, logits, router_ws)
        lm.moe_route(logits, weights["bias"], k, d.routed_scaling_factor, ids, topw)
        lm.latent_moe_forward_fp8(d, weights, experts, hidden, logits, out, layer_ws)
        lm.moe_balance_loss(logits, ids, alpha, loss, counts, tokens, loss_ws, token_mask=mask, seq_offsets=seq)
        chosen = utility.gather(1, ids.long()) * mask[:, None]
        grad_w = (-chosen / T).contiguous()
        lm.moe_router_backward(logits, ids, grad, grad_topk_weights=grad_w,
                               routed_scaling_factor=d.routed_scaling_factor, grad_loss=grad_loss,
                               expert_counts=counts, seq_tokens=tokens, alpha=alpha, token_mask=mask,
                               seq_offsets=seq)
        w_router -= lr * (grad.T @ hidden.float())
        value = float((topw * chosen).sum() / T)
        history.append((value, float(loss), int(counts.sum(0).max())))
    assert lm.lmoe_device_error() == 0
    return history, off, out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    hist, off, out = main(ap.parse_args().steps)
    print(f"e4m3 down-projection against bf16: {off:.4f} of its norm; layer output finite: "
          f"{bool(torch.isfinite(out.float()).all())}")
    for i, (value, loss, most) in enumerate(hist):
        print(f"step {i:3d}  routed utility {value:7.4f}  balance loss {loss:7.4f}  most loaded expert {most}")
