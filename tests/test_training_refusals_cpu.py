"""Refusals of the norm's, SituGLU gradient's and grouped products' entry points: host-side
checks, before any device access (addresses are never followed)."""
import ctypes

import pytest
import torch

lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
p = ctypes.c_void_p(256)
odd = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    from latent_mixture_experts_sigmoid_gb300 import build
    build.build()
    return lm.load_library()


def test_rms_norm(lib):
    def f(x=p, res=p, w=p, eps=1e-6, h=p, out=p, codes=p, scales=p, T=4, H=256):
        return lib.lmoe_rms_norm(x, res, w, eps, h, out, codes, scales, T, H, None)

    assert f(T=-1) == -2 and f(H=0) == -2 and f(H=4) == -2 and f(H=12) == -2 and f(H=16392) == -2
    assert f(H=24) == -2                                     # codes: H % 16
    assert f(eps=-1e-6) == -2 and f(eps=float("nan")) == -2 and f(eps=float("inf")) == -2
    assert f(x=None) == -1 and f(out=None, codes=None, scales=None) == -1
    assert f(codes=None) == -1 and f(scales=None) == -1      # both or neither
    for name in ("x", "res", "w", "h", "out", "codes", "scales"):
        assert f(**{name: odd}) == -7, name
    assert f(T=0, x=None, out=None, codes=None, scales=None) == 0
    assert f() == -8
    assert f(res=None, w=None, h=None, codes=None, scales=None, H=24) == -8


def test_rms_norm_backward(lib):
    n = lib.lmoe_rms_norm_backward_workspace_bytes
    assert n(-1, 256) == 0 and n(4, 12) == 0 and n(4, 16392) == 0
    for H in (8, 256, 1024, 1032, 7168, 16384):
        sizes = [n(T, H) for T in (1, 2, 7, 8, 9, 100, 607, 608, 609, 5000, 1 << 20, (1 << 31) - 1)]
        assert sizes == sorted(sizes) and sizes[0] >= 4 * H, H
    need = n(4, 256)

    def f(dy=p, h=p, w=p, dres=p, eps=1e-6, dh=p, dw=p, T=4, H=256, ws=p, nb=need):
        return lib.lmoe_rms_norm_backward(dy, h, w, dres, eps, dh, dw, T, H, ws, nb, None)

    assert f(T=-1) == -2 and f(H=20) == -2 and f(H=1 << 20) == -2 and f(eps=-1.0) == -2
    for name in ("dy", "h", "dh"):
        assert f(**{name: None}) == -1, name
    for name in ("dy", "h", "w", "dres", "dh", "dw"):
        assert f(**{name: odd}) == -7, name
    assert f(ws=None) == -5 and f(ws=odd) == -5 and f(nb=need - 1) == -5
    assert f(dw=None, ws=None, nb=0) == -8                   # no workspace without grad_norm_w
    assert f(T=0, dy=None, h=None, dh=None, dw=None, ws=None, nb=0) == 0
    assert f() == -8


def test_situ_backward(lib):
    f = lib.situ_and_mul_backward
    assert f(p, p, p, 4, 8, 0.0, 8.0, None) == -4 and f(p, p, p, 4, 8, float("nan"), 8.0, None) == -4
    assert f(p, p, p, 4, (1 << 26) + 8, 4.0, 8.0, None) == -2
    assert f(p, p, p, 4, 12, 4.0, 8.0, None) == -2 and f(p, p, p, -4, 8, 4.0, 8.0, None) == -2
    assert f(p, p, p, 4, 8, 4.0, float("inf"), None) == -2 and f(p, p, p, (1 << 40) // 8 + 1, 8, 4.0, 8.0, None) == -2
    for i in range(3):
        a = [p, p, p]
        a[i] = None
        assert f(*a, 4, 8, 4.0, 8.0, None) == -1
        a[i] = odd
        assert f(*a, 4, 8, 4.0, 8.0, None) == -7
    assert f(None, None, None, 0, 8, 4.0, 8.0, None) == 0
    assert f(p, p, p, 4, 8, 4.0, 8.0, None) == -8


SIZES = [dict(rows=-1), dict(rows=(1 << 27) + 1), dict(E=0), dict(E=1025), dict(N=0), dict(N=12), dict(K=20), dict(K=4),
         dict(N=65544), dict(K=65544)]


@pytest.mark.parametrize("name", ["lmoe_grouped_linear", "lmoe_grouped_linear_backward_x"])
def test_grouped_rows(lib, name):
    def f(x=p, w=p, off=p, out=p, rows=10, E=4, N=64, K=128):
        return getattr(lib, name)(x, w, off, out, rows, E, N, K, None)

    for bad in SIZES:
        assert f(**bad) == -2, bad
    for a in ("x", "w", "off", "out"):
        assert f(**{a: None}) == -1, a
        assert f(**{a: odd}) == -7, a
    assert f(rows=0, x=None, w=None, off=None, out=None) == 0
    assert f() == -8


def test_grouped_weights(lib):
    def f(dy=p, x=p, off=p, add=None, dw=p, dwh=None, rows=10, E=4, N=64, K=128):
        return lib.lmoe_grouped_linear_backward_w(dy, x, off, add, dw, dwh, rows, E, N, K, None)

    for bad in SIZES:
        assert f(**bad) == -2, bad
    for a in ("dy", "x", "off"):
        assert f(**{a: None}) == -1, a
    assert f(dw=None) == -1 and f(dwh=p) == -1               # one of the two
    assert f(dw=None, dwh=p, add=p) == -1                    # the addend is fp32's
    for a in ("dy", "x", "off", "add", "dw"):
        assert f(**{a: odd}) == -7, a
    assert f(dw=None, dwh=odd) == -7
    assert f() == -8 and f(add=p) == -8 and f(dw=None, dwh=p) == -8
    assert f(rows=0, dy=None, x=None, off=None) == -8        # the gradient is written, too


def test_binding_refuses_host_tensors():
    lm.load_library()
    b, f = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((4, 1))
    off = torch.zeros(3, dtype=torch.int32)
    w = torch.zeros((2, 128, 128), dtype=torch.bfloat16)
    for call in (lambda: lm.lmoe_grouped_linear(b[:, :64], w, off, b),            # widths that do not fit
                 lambda: lm.lmoe_grouped_linear_backward_x(b[:, :64], w, off, b),
                 lambda: lm.lmoe_grouped_linear_backward_w(b[:2], b, off, w)):
        with pytest.raises(ValueError, match="rows of 64|grad_out"):
            call()
    for call in (lambda: lm.lmoe_rms_norm(b, None, 1e-6, out=b),
                 lambda: lm.lmoe_rms_norm_backward(b, b, None, 1e-6, b),
                 lambda: lm.situ_and_mul_backward(b, b, b, 4.0, 8.0),
                 lambda: lm.lmoe_grouped_linear(b, w, off, b),
                 lambda: lm.lmoe_grouped_linear_backward_x(b, w, off, b),
                 lambda: lm.lmoe_grouped_linear_backward_w(b, b, off, w),
                 lambda: lm.lmoe_grouped_linear_backward_w(b, b, off, w.float(), add=f)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
