"""More refusals of the training operators' entry points: host-side checks, before any device
access (addresses are never followed)."""
import ctypes

import pytest

lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
p = ctypes.c_void_p(256)
odd = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    from latent_mixture_experts_sigmoid_gb300 import build
    build.build()
    return lm.load_library()


def test_norm_gradient_of_an_empty_batch(lib):
    # grad_norm_w is written, so it has to be memory that the call can write
    def f(dw):
        return lib.lmoe_rms_norm_backward(None, None, None, None, 1e-6, None, dw, 0, 256, None, 0, None)

    assert f(None) == 0
    assert f(odd) == -7
    assert f(p) == -8                     # of no device


def test_sizes_past_the_abi_s_32_bits(lib):
    # ctypes would cut them: 2^32 rows became none, 2^32 + 8 columns eight
    big = 1 << 32
    for call in (lambda: lm.lmoe_rms_norm(256, None, 1e-6, out=256, T=big, H=8),
                 lambda: lm.lmoe_rms_norm(256, None, 1e-6, out=256, T=0, H=big + 8),
                 lambda: lm.lmoe_rms_norm_backward(256, 256, None, 1e-6, 256, T=big, H=8),
                 lambda: lm.lmoe_rms_norm_backward(256, 256, None, 1e-6, 256, T=0, H=big + 8),
                 lambda: lm.lmoe_rms_norm_backward_workspace_bytes(big + 1, 64),
                 lambda: lm.lmoe_rms_norm_backward_workspace_bytes(1, big + 64),
                 lambda: lm.situ_and_mul_backward(256, 256, 256, 4.0, 8.0, N=0, d=big + 8),
                 lambda: lm.lmoe_grouped_linear(256, 256, 256, 256, shape=(0, big + 1, 64, 64)),
                 lambda: lm.lmoe_grouped_linear(256, 256, 256, 256, shape=(0, 1, big + 64, 64)),
                 lambda: lm.lmoe_grouped_linear_backward_x(256, 256, 256, 256, shape=(0, 1, 64, big + 64)),
                 lambda: lm.lmoe_grouped_linear_backward_w(256, 256, 256, 256, shape=(10, big + 1, 64, 64))):
        with pytest.raises(ValueError, match="32 bits"):
            call()
