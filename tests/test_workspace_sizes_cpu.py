"""Workspace sizes never fall as a batch grows: a buffer for the largest batch serves every
smaller one."""
import dataclasses

import pytest

import workloads as W

lm = pytest.importorskip("latent_mixture_experts_sigmoid_gb300")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from latent_mixture_experts_sigmoid_gb300 import build
    build.build()
    lm.load_library()


def assert_rising(sizes):
    falls = [(n, a, b) for (_, a), (n, b) in zip(sizes[:-1], sizes[1:]) if b < a]
    assert not falls, falls[:5]


LARGE = [3000, 4096, 9999, 16384, 65536, 1 << 20, 1 << 24]


@pytest.mark.parametrize("E,S", [(1, 1), (64, 4), (896, 40)])
def test_balance_loss(E, S):
    assert_rising([(T, lm.moe_balance_loss_workspace_bytes(T, E, S)) for T in [*range(0, 8000), *LARGE]])


@pytest.mark.parametrize("inter", [128, 512])
@pytest.mark.parametrize("E", [1, 2, 7, 8, 15, 16, 17, 64, 255, 256, 257, 300, 896, 1024])
def test_experts_fp8(E, inter):
    counts = sorted({*range(0, 2500), 8 * E, 8 * E + 1, *LARGE, 1 << 27})
    assert_rising([(n, lm.lmoe_experts_fp8_workspace_bytes(n, E, 256, inter)) for n in counts])


@pytest.mark.parametrize("E,topk", [(64, 4), (896, 16), (896, 1), (8, 8), (1024, 4)])
def test_layer_fp8(E, topk):
    sizes = []
    for T in [*range(0, 1200), 2048, 4096, 8192]:
        d = dataclasses.replace(W.TINY, T=T, num_experts=E, topk=topk)
        sizes.append((T, lm.latent_moe_workspace_bytes_fp8(d)))
        # above decode sizes the e4m3 rows and activations have the room of the bf16 ones
        if T > 128:
            assert sizes[-1][1] == max(lm.latent_moe_workspace_bytes(d), sizes[128][1])
    assert_rising(sizes)
