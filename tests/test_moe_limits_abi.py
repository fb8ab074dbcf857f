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


def past_32_bits():
    """(call, arguments, the argument that its message names): low 32 bits that would make a valid call, and negative
    sizes that would."""
    def meta(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device="meta")

    bf16, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    for low in (128, 256):
        for n in ((1 << 32) + low, (1 << 33) + low, -(1 << 32) + low):
            ids, rows, x = meta(4, 2), meta(4, 2), meta(4, 256, dtype=bf16)
            yield binding.moe_sort_contiguous, (ids, n, 512), {}, "G"
            yield binding.moe_sort_contiguous, (ids, 4, n), dict(rows=rows, m_indices=meta(128)), "M_total"
            yield binding.moe_sort_masked, (ids, 4, n), dict(rows=rows, masked_m=meta(4)), "M_cap"
            yield binding.moe_sort_masked, (ids, n, 4), dict(rows=rows, masked_m=meta(4)), "G"
            yield binding.moe_dispatch_quantize_e4m3_masked, (x, rows, n, 4), {}, "G"
            yield binding.moe_dispatch_quantize_e4m3_masked, (x, rows, 4, n), {}, "rows"
            yield binding.moe_dispatch_quantize_e4m3_contiguous, (x, rows, n), {}, "rows"
            yield binding.moe_dispatch_e4m3_masked, (x.to(u8), meta(2, 4, dtype=f32), rows, n, 4), {}, "G"
            yield binding.moe_dispatch_e4m3_contiguous, (x.to(u8), meta(2, 4, dtype=f32), rows, n), {}, "rows"
            yield binding.layernorm_quantize_e4m3_1x128, (x,), dict(ld_sf=n), "ld_sf"
            yield binding.get_moe_rows, (n, 2, 8), {}, "T"
            yield binding.get_moe_rows, (4, n, 8), {}, "top_k"
            yield binding.get_moe_rows, (4, 2, n), {}, "G"
            yield binding.get_moe_sort_workspace_size, (n, 2, 8), {}, "T"
            yield binding.get_moe_sort_workspace_size, (4, n, 8), {}, "top_k"
            yield binding.get_moe_sort_workspace_size, (4, 2, n), {}, "G"
            yield binding.get_layernorm_backward_workspace_size, (n, 256), {}, "rows"
            yield binding.get_layernorm_backward_workspace_size, (4, n), {}, "K"
            if n > 0:
                wide = meta(4, n, dtype=bf16)
                yield binding.layernorm_quantize_e4m3_1x128, (wide,), {}, "K"
                yield binding.layernorm_quantize_e4m3_1x128, (x,), dict(sf=meta(2, n, dtype=f32)), "ld_sf"
                yield binding.layernorm_backward, (wide, wide), {}, "K"
                yield binding.moe_dispatch_quantize_e4m3_contiguous, (wide, rows, 512), {}, "K"
                yield binding.moe_dispatch_e4m3_contiguous, (wide.to(u8), meta(n // 128, 4, dtype=f32), rows, 512), {}, "K"
                yield binding.moe_combine_backward_quantize_e4m3_contiguous, (wide, wide, rows), {}, "K"


def test_sizes_past_32_bits_of_every_argument(lib):
    wrong = []
    for f, args, kw, name in past_32_bits():
        try:
            got = f(*args, **kw)
        except ValueError as e:
            got = str(e)
        except binding.DGError as e:
            got = str(e)
        if not (isinstance(got, str) and "32 bits" in got and f"{name}: " in got):
            wrong.append((f.__name__, name, [a for a in args if isinstance(a, int)], got))
    assert not wrong, wrong
