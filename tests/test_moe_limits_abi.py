"""Sizes at the ends of what the layer norm's and the experts' row operators'
entry points take: what the kernels could not count is refused on the host."""
import ctypes as ct
import os

import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding

P = ct.c_void_p(0x10000)      # 16-byte aligned, never dereferenced
SHAPE = -2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from moe_grouped_gemm_scaled_amd import build
        build.build()
    return binding.lib()


@pytest.mark.parametrize("top_k", [(1 << 31) - 1, (1 << 31) - 63, (1 << 30) + 1])
def test_more_choices_than_a_kernel_counts(lib, top_k):
    """One token: its pairs stay below 2^31, but the step past its last choice would not."""
    T, K, R = 1, 128, 128
    assert lib.dg_moe_dispatch_quantize_e4m3_contiguous(P, 0, K, P, P, P, P, P, P, P, P, T, top_k, K, R, None) == SHAPE
    assert lib.dg_moe_dispatch_quantize_e4m3_masked(P, 0, K, P, P, P, P, P, T, top_k, K, 1, R, None) == SHAPE
    assert lib.dg_moe_combine_backward_quantize_e4m3_contiguous(P, 0, K, P, P, P, P, P, P, P, P, P, P, T, top_k, K, R,
                                                                None) == SHAPE
    assert lib.dg_moe_dispatch_e4m3_contiguous(P, P, 4, P, P, P, T, top_k, K, R, None) == SHAPE
    assert lib.dg_moe_dispatch_e4m3_masked(P, P, 4, P, P, P, T, top_k, K, 1, R, None) == SHAPE
    assert lib.dg_moe_combine(P, P, P, P, P, 0, T, top_k, K, R, None) == SHAPE
