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
