"""Sizes that calls reject: their workspace functions give 0 there, and the
limits are where the headers put them (no GPU needed)."""
import ctypes
import os

import pytest

from mixture_experts_layer_fp32_amd import _binding as B

P = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails its checks


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):  # build only when nothing is built yet
        from mixture_experts_layer_fp32_amd import build
        build.build()
    return B.load_library()


@pytest.mark.parametrize("inter", [64, 192, 1024, 65536])
def test_ffn_fp8_rows_limit(lib, inter):
    """(cap_rows + 16) * inter up to 2^34."""
    r = ctypes.byref(B.make_desc(T=64, D=128, E=8, top_k=2, I=192))
    most = 2 ** 34 // inter - 16
    need = lib.moe_ffn_fp8_workspace_size(r, inter, most)
    assert need >= 3 * most * inter
    for rows in (most + 1, 2 ** 31 - 1):
        assert lib.moe_ffn_fp8_workspace_size(r, inter, rows) == 0
        assert lib.moe_expert_ffn_fp8(r, 1, inter, rows, P, P, P, P, P, P, P, P, P, 2 ** 63,
                                      None) == B.MOE_ERR_UNSUPPORTED
    # the last size that is taken fails for its workspace alone
    assert lib.moe_expert_ffn_fp8(r, 1, inter, most, P, P, P, P, P, P, P, P, P, need - 1,
                                  None) == B.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("D", [64, 192, 7168, 262144])
def test_router_dense_tokens_limit(lib, D):
    """ceil(T / 64) * (D / 64) below 2^23."""
    most = min((2 ** 23 - 1) // (D // 64) * 64, 2 ** 31 - 1)
    size, f = lib.moe_router_backward_dense_workspace_size, lib.moe_router_backward_dense
    need = size(most, 8, D)
    if need:  # (262144 columns are 2048 tiles of dW, which need no parts)
        assert f(most, 8, D, 0, P, P, P, 0, P, P, P, need - 1, None) == B.MOE_ERR_WORKSPACE
    else:
        assert D == 262144
    if most < 2 ** 31 - 1:
        assert size(most + 1, 8, D) == 0
        assert f(most + 1, 8, D, 0, P, P, P, 0, P, P, P, 2 ** 63,
                 None) == B.MOE_ERR_UNSUPPORTED
