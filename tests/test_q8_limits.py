"""Sizes that the 8-bit operators cannot take are refused before anything is enqueued (no GPU)."""

import os

import pytest

from ffn_block_gb300 import binding as B

P, UNS, WS = 0x1000, B.RMX_ERR_UNSUPPORTED, B.RMX_ERR_WORKSPACE   # an aligned address, never followed


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from ffn_block_gb300 import build
        build.build()
    return B.lib()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K,N", [(1 << 20, 1 << 20), (1 << 20, 1 << 19), ((1 << 20) - 31, (1 << 19) - 7)])
def test_weights_past_a_tensor_map(lib, dt, K, N):
    l = B.make_layer(4, 1, K, N, dt)
    before = B.rmx_launch_count()
    assert B.rmx_linear_q8(l, P, P, P, P, None, None, P) == UNS
    assert B.rmx_weight_q8(l, P, P, P) == UNS
    assert B.rmx_ckpt8_wgrad_workspace_bytes(l) == 0
    assert B.rmx_ckpt8_wgrad(l, P, P, P, P, P, P, 1 << 62) == UNS
    assert B.rmx_launch_count() == before


@pytest.mark.parametrize("M,G,K,N", [(1 << 30, 1, 8, 1 << 20), (1 << 28, 1, 1 << 18, 1 << 20)])
def test_products_past_the_kernels_counters(lib, M, G, K, N):
    before = B.rmx_launch_count()
    assert B.rmx_linear_q8(B.make_layer(M, G, K, N, "bf16"), P, P, P, P, None, None, P) == UNS
    assert B.rmx_launch_count() == before


def test_the_largest_weights_are_not_refused(lib):
    """One channel and one input fewer: the first thing that is wrong with this call is its workspace."""
    l = B.make_layer(4, 1, 1 << 20, (1 << 19) - 8, "bf16")
    assert B.rmx_ckpt8_wgrad_workspace_bytes(l) > 0
    assert B.rmx_ckpt8_wgrad(l, P, P, P, P, P, P, 0) == WS
