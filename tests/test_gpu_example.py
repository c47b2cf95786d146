"""The example that runs the e4m3 layer and the router's training step together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
pytest.importorskip("latent_mixture_experts_sigmoid_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _main(**kw):
    spec = importlib.util.spec_from_file_location(
        "fp8_example", os.path.join(ROOT, "examples", "fp8_layer_and_router_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.main(**kw)


def test_example_trains_the_router(cuda_ok):
    history, off, out = _main(steps=12)
    # e4m3 operands: each rounded by at most 2^-4, about 2^-5 in the mean square
    assert 0 < off < 2.0 ** -4
    assert bool(torch.isfinite(out.float()).all())
    values, losses = [h[0] for h in history], [h[1] for h in history]
    assert values[-1] > values[0]
    # alpha is the loss of an even load; without its gradient the load drifts apart
    free, _, _ = _main(steps=12, alpha=0.0)
    assert history[-1][2] <= free[-1][2] and losses[0] > 0


def test_example_balances_the_load(cuda_ok):
    # the loss over alpha is 1 for an even load and more for any other.  A run whose alpha is too
    # small to act measures the same loss: its load drifts apart, while the balance gradient's
    # does not.  Without that gradient both runs would be the same but for rounding.
    small = 2.0 ** -20
    held, free = _main(steps=12, alpha=0.2)[0], _main(steps=12, alpha=small)[0]
    first, last, drifted = held[0][1] / 0.2 - 1, held[-1][1] / 0.2 - 1, free[-1][1] / small - 1
    assert abs(first - (free[0][1] / small - 1)) <= 2.0 ** -20      # the same first step
    assert drifted > 1.2 * first > 0
    assert last < 0.8 * drifted
    assert held[-1][2] < free[-1][2]
