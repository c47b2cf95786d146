"""Refusals of the e4m3 and router-training entry points: host-side checks, before
any device access (addresses are never followed)."""
import ctypes
import dataclasses

import pytest
import torch

import workloads as W

lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
p = ctypes.c_void_p(256)
odd = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    from latent_mixture_experts_sigmoid_gb300 import build
    build.build()
    return lm.load_library()


def test_quantize(lib):
    f = lib.lmoe_quantize_fp8
    assert f(p, p, p, 4, 24, 1, None) == -2            # K % 16
    assert f(p, p, p, 4, 0, 1, None) == -2
    assert f(p, p, p, -1, 128, 1, None) == -2
    assert f(p, p, p, 4, 128, 64, None) == -2          # block_rows
    assert f(p, p, p, 1 << 31, 128, 1, None) == -2     # blocks past 2^31 - 1
    assert f(p, p, p, 1 << 30, 256, 128, None) == -2
    assert f(None, p, p, 4, 128, 1, None) == -1
    assert f(p, None, p, 4, 128, 1, None) == -1
    assert f(p, p, None, 4, 128, 1, None) == -1
    assert f(p, odd, p, 4, 128, 1, None) == -7
    assert f(None, None, None, 0, 128, 1, None) == 0
    assert f(p, p, p, 4, 128, 1, None) == -8           # no device memory


def test_linear(lib):
    f = lib.lmoe_linear_fp8
    assert f(p, p, p, p, None, p, 4, 12, 128, None) == -2       # N % 8
    assert f(p, p, p, p, None, p, 4, 128, 120, None) == -2      # K % 16
    assert f(p, p, p, p, None, p, -1, 128, 128, None) == -2
    assert f(p, p, p, p, None, p, 4, 0, 128, None) == -2
    big = 2147483640
    assert f(p, p, p, p, None, p, big, big, 128, None) == -2    # tiles past 2^31 - 1
    for i in (0, 1, 2, 3, 5):
        a = [p, p, p, p, None, p]
        a[i] = None
        assert f(*a, 4, 128, 128, None) == -1
        a[i] = odd
        assert f(*a, 4, 128, 128, None) == -7
    assert f(p, p, p, p, odd, p, 4, 128, 128, None) == -7
    assert f(None, None, None, None, None, None, 0, 128, 128, None) == 0
    assert f(p, p, p, p, None, p, 4, 128, 128, None) == -8


def test_experts(lib):
    n = lib.lmoe_experts_fp8_workspace_bytes
    assert n(100, 4, 256, 128) >= 100 * 128 + 100 * 4
    assert n(0, 4, 256, 128) > 0
    for bad in ((-1, 4, 256, 128), (100, 0, 256, 128), (100, 1025, 256, 128), (100, 4, 192, 128),
                (100, 4, 256, 64), (100, 4, 8320, 128), (100, 4, 256, 8320), ((1 << 27) + 1, 4, 256, 128)):
        assert n(*bad) == 0
    q = lm.LmoeFp8Experts(256, 256, 256, 256)
    need = n(100, 4, 256, 128)

    def f(q=q, x=p, xs=p, off=p, y=p, rows=100, E=4, L=256, d=128, beta=4.0, lb=8.0, ws=p, nb=need):
        return lib.lmoe_experts_fp8(ctypes.byref(q) if q else None, x, xs, off, y, rows, E, L, d, beta, lb, ws,
                                    nb, None)

    assert f(L=192) == -2 and f(d=64) == -2 and f(E=2000) == -2 and f(rows=-5) == -2
    assert f(beta=0.0) == -4 and f(beta=float("nan")) == -4 and f(lb=float("inf")) == -2
    assert f(q=None) == -1 and f(x=None) == -1 and f(xs=None) == -1 and f(off=None) == -1 and f(y=None) == -1
    assert f(q=lm.LmoeFp8Experts(256, None, 256, 256)) == -1
    assert f(q=lm.LmoeFp8Experts(264, 256, 256, 256)) == -7
    assert f(x=odd) == -7 and f(off=odd) == -7
    assert f(ws=None) == -5 and f(ws=odd) == -5 and f(nb=need - 1) == -5
    assert f(rows=0, x=None, xs=None, off=None, y=None, ws=None, nb=0) == 0
    assert f() == -8


def test_layer(lib):
    d = lm.make_dims(W.TINY)
    nb = lib.latent_moe_workspace_bytes_fp8(ctypes.byref(d))
    assert nb > lib.latent_moe_workspace_bytes(ctypes.byref(d))
    w = lm.LmoeWeights(256, None, None, None, None, None, 256, None)       # w13 / w2 unused
    q = lm.LmoeFp8Experts(256, 256, 256, 256)
    f = lib.latent_moe_forward_fp8
    B = ctypes.byref
    assert f(B(d), B(w), None, p, p, p, p, nb, None, None) == -1
    assert f(B(d), B(w), B(q), p, None, p, p, nb, None, None) == -1
    assert f(B(d), B(w), B(lm.LmoeFp8Experts(256, 256, None, 256)), p, p, p, p, nb, None, None) == -1
    assert f(B(d), B(w), B(lm.LmoeFp8Experts(256, 256, 264, 256)), p, p, p, p, nb, None, None) == -7
    assert f(B(d), B(w), B(q), p, p, p, ctypes.c_void_p(272), nb, None, None) == -5
    assert f(B(d), B(w), B(q), p, p, p, p, nb - 256, None, None) == -5
    assert f(B(d), B(w), B(q), p, p, p, p, nb, None, None) == -8
    half = lm.make_dims(dataclasses.replace(W.TINY, inter=192))             # inter % 128
    assert lib.latent_moe_workspace_bytes_fp8(B(half)) == 0
    assert f(B(half), B(w), B(q), p, p, p, p, nb, None, None) == -2
    assert lib.latent_moe_launch_count_fp8(B(half), 1) == 0
    # the quantisation of the scattered rows at decode sizes; a second kernel per product
    # for experts with more than 32 rows where the mean expert has one at the most
    for T, more in ((8, 1), (128, 1), (129, 0), (300, 0)):
        dt = lm.make_dims(dataclasses.replace(W.TINY, T=T))
        assert lib.latent_moe_launch_count_fp8(B(dt), 1) == lib.latent_moe_launch_count(B(dt), 1) + more
    many = lm.make_dims(dataclasses.replace(W.TINY, T=40, num_experts=1024))
    assert lib.latent_moe_launch_count_fp8(B(many), 1) == lib.latent_moe_launch_count(B(many), 1) + 3


def test_balance_loss(lib):
    n = lib.moe_balance_loss_workspace_bytes
    assert n(100, 64, 1) > 0 and n(-1, 64, 1) == 0 and n(100, 1025, 1) == 0 and n(100, 64, 0) == 0
    need = n(100, 64, 2)

    def f(lg=p, ids=p, mask=None, seq=p, T=100, E=64, k=4, S=2, alpha=0.1, loss=p, cnt=p, tok=p, ws=p, nb=need):
        return lib.moe_balance_loss(lg, ids, mask, seq, T, E, k, S, alpha, loss, cnt, tok, ws, nb, None)

    assert f(T=-1) == -2 and f(E=0) == -2 and f(E=1025) == -2 and f(k=0) == -2 and f(k=65) == -2
    assert f(E=64, k=33) == -2 and f(S=0) == -2 and f(S=65537) == -2 and f(alpha=float("nan")) == -2
    assert f(T=1 << 30, k=4) == -2
    for name in ("lg", "ids", "loss", "cnt", "tok", "seq"):
        assert f(**{name: None}) == -1, name
    for name in ("lg", "ids", "loss", "cnt", "tok", "seq", "mask"):
        assert f(**{name: odd}) == -7, name
    assert f(ws=None) == -5 and f(ws=odd) == -5 and f(nb=need - 256) == -5
    assert f(T=0, lg=None, ids=None) == 0
    assert f(seq=None, S=1) == -8 and f() == -8


def test_router_backward(lib):
    def f(lg=p, ids=p, gw=p, renorm=1, rsf=2.5, gl=p, cnt=p, tok=p, alpha=0.1, mask=None, seq=p, T=100, E=64, k=4,
          S=2, grad=p):
        return lib.moe_router_backward(lg, ids, gw, renorm, rsf, gl, cnt, tok, alpha, mask, seq, T, E, k, S, grad,
                                       None)

    assert f(T=-1) == -2 and f(E=1025) == -2 and f(k=65) == -2 and f(S=0) == -2
    assert f(rsf=float("inf")) == -2 and f(alpha=float("inf")) == -2
    for name in ("lg", "ids", "cnt", "tok", "seq", "grad"):
        assert f(**{name: None}) == -1, name
    assert f(gw=None, gl=None) == -1
    assert f(gw=None, ids=None) == -8                   # the loss's part needs no ids
    assert f(gl=None, cnt=None, tok=None) == -8         # the weights' part no counts
    for name in ("lg", "ids", "gw", "gl", "cnt", "tok", "mask", "seq", "grad"):
        assert f(**{name: odd}) == -7, name
    assert f(T=0, lg=None, grad=None) == 0
    assert f() == -8


def test_binding_refuses_host_tensors():
    lm.load_library()
    x, s = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((4, 1))
    q = torch.zeros((4, 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        lm.lmoe_quantize_fp8(x, q, s)
    with pytest.raises(ValueError, match="CUDA"):
        lm.lmoe_linear_fp8(q, s, q, s, x)
    with pytest.raises(ValueError, match="CUDA"):
        lm.lmoe_experts_fp8({"w13_q": q}, q, s, torch.zeros(2, dtype=torch.int32), x, q, inter=128, beta=4.0,
                            linear_beta=8.0)
    with pytest.raises(ValueError, match="CUDA"):
        lm.moe_balance_loss(torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), 0.1, s, q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        lm.moe_router_backward(torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 8)))
