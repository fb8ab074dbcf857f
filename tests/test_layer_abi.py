"""Refusals of the feed-forward layer's entry points that need no GPU: every
invalid argument is found on the host before any HIP call, and calls without
rows succeed without one."""
import ctypes as ct
import math
import os

import numpy as np
import pytest

from moe_grouped_gemm_scaled_amd import binding

import layer_helpers

P = ct.c_void_p(0x10000)      # 16-byte aligned, never dereferenced
MIS = ct.c_void_p(0x10004)
ODD = ct.c_void_p(0x10002)
OK, NULL, SHAPE, ALIGN, ARG = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from moe_grouped_gemm_scaled_amd import build
        build.build()
    return binding.lib()


class Call:
    """An entry point with valid arguments by name; calling it replaces some."""

    def __init__(self, f, **args):
        self.f, self.args = f, args

    def __call__(self, **kw):
        assert set(kw) <= set(self.args), set(kw) - set(self.args)
        return self.f(*{**self.args, **kw}.values())


def refused(call, status, **kw):
    got = call(**kw)
    assert got == status, (kw, got)


@pytest.mark.parametrize("suffix", ["", "_ue8m0", "_ue8m0_packed"])
def test_rmsnorm_refusals(lib, suffix):
    c = Call(getattr(lib, "dg_rmsnorm_quantize_e4m3_1x128" + suffix), x=P, x_type=0, ld_x=256, residual=P, residual_type=0,
             weight=P, weight_type=0, eps=1e-6, residual_out=P, y=P, q=P, sf=P, ld_sf=8, rows=5, K=256, stream=None)
    for name in ("x", "weight", "sf"):
        refused(c, NULL, **{name: None})
    refused(c, NULL, y=None, q=None)
    for kw in (dict(rows=-1), dict(K=0), dict(K=64), dict(K=200), dict(K=16512, ld_x=16512)):
        refused(c, SHAPE, **kw)
    for kw in (dict(x_type=2), dict(residual_type=-1), dict(weight_type=7), dict(eps=-1.0), dict(eps=math.nan),
               dict(residual=None)):
        refused(c, ARG, **kw)
    for name in ("x", "residual", "weight", "residual_out", "y", "q", "sf"):
        refused(c, ALIGN, **{name: MIS})
    for kw in (dict(ld_x=255), dict(ld_x=260), dict(ld_x=258, x_type=1), dict(ld_sf=4), dict(ld_sf=7)):
        refused(c, ALIGN, **kw)
    refused(c, OK, rows=0, x=None, residual=None, residual_out=None, weight=None, y=None, q=None, sf=None)


def test_rmsnorm_backward_refusals(lib):
    c = Call(lib.dg_rmsnorm_backward, dy=P, dy_type=0, h=P, h_type=1, weight=P, weight_type=0, eps=1e-6, dres=P, dx=P, dw=P,
             rows=5, K=256, workspace=P, workspace_bytes=1 << 30, stream=None)
    for name in ("dy", "h", "weight", "dx", "dw"):
        refused(c, NULL, **{name: None})
    for kw in (dict(rows=-1), dict(K=100), dict(K=0), dict(K=32768)):
        refused(c, SHAPE, **kw)
    for kw in (dict(dy_type=2), dict(h_type=-1), dict(weight_type=3), dict(eps=-1e-9), dict(eps=math.nan)):
        refused(c, ARG, **kw)
    for name in ("dy", "h", "weight", "dres", "dx", "dw", "workspace"):
        refused(c, ALIGN, **{name: MIS})
    f = lib.dg_get_rmsnorm_backward_workspace_size
    assert f(-1, 256) == SHAPE and f(4, 100) == SHAPE and f(4, 16512) == SHAPE


def common_gated(c, rows_name):
    for name in ("a", "sfa", "b", "sfb", "sf"):
        refused(c, NULL, **{name: None})
    refused(c, NULL, h=None, q=None)
    for kw in ({rows_name: -128}, dict(I=0), dict(K=0), dict(K=64), dict(K=200), dict(I=200), dict(I=1 << 20, K=1024)):
        refused(c, SHAPE, **kw)
    for kw in (dict(act=2), dict(act=-1)):
        refused(c, ARG, **kw)
    for name in ("a", "sfa", "b", "sfb", "gu", "h", "q", "sf"):
        refused(c, ALIGN, **{name: MIS})


@pytest.mark.parametrize("suffix", ["", "_ue8m0_packed"])
def test_gated_refusals(lib, suffix):
    c = Call(getattr(lib, "dg_fp8_gated_gemm_nt" + suffix), a=P, sfa=P, ld_sfa=128, b=P, sfb=P, act=0, gu=P, h=P, q=P, sf=P,
             ld_sf=128, M=128, I=256, K=256, workspace=None, workspace_bytes=0, stream=None)
    common_gated(c, "M")
    for kw in (dict(ld_sfa=124), dict(ld_sfa=130), dict(ld_sf=124), dict(ld_sf=129), dict(workspace=MIS)):
        refused(c, ALIGN, **kw)
    refused(c, SHAPE, ld_sfa=1 << 29)                     # the scales' bytes reach 2^31
    refused(c, OK, M=0, a=None, sfa=None, b=None, sfb=None, h=None, q=None, sf=None, gu=None)

    c = Call(getattr(lib, "dg_m_grouped_fp8_gated_gemm_nt_contiguous" + suffix), a=P, sfa=P, b=P, sfb=P, act=0, gu=P, h=P,
             q=P, sf=P, m_indices=P, M_total=128, I=256, K=256, G=2, stream=None)
    common_gated(c, "M_total")
    for kw in (dict(M_total=100), dict(G=0)):
        refused(c, SHAPE, **kw)
    refused(c, NULL, m_indices=None)
    refused(c, ALIGN, m_indices=MIS)
    refused(c, OK, M_total=0, a=None, sfa=None, b=None, sfb=None, h=None, q=None, sf=None, gu=None, m_indices=None)

    c = Call(getattr(lib, "dg_m_grouped_fp8_gated_gemm_nt_masked" + suffix), a=P, sfa=P, b=P, sfb=P, act=0, gu=P, h=P, q=P,
             sf=P, masked_m=P, G=2, M_cap=64, I=256, K=256, expected_m=0, stream=None)
    common_gated(c, "M_cap")
    for kw in (dict(M_cap=0), dict(G=0)):
        refused(c, SHAPE, **kw)
    refused(c, NULL, masked_m=None)
    refused(c, ALIGN, masked_m=ODD)


def test_gated_workspace_size_refusals(lib):
    f = lib.dg_get_gated_workspace_size
    assert f(-1, 128, 128) == SHAPE and f(1, 0, 128) == SHAPE and f(1, 128, 100) == SHAPE
    assert f(1, 1 << 20, 1024) == SHAPE


@pytest.mark.parametrize("suffix", ["", "_ue8m0"])
def test_gated_backward_refusals(lib, suffix):
    c = Call(getattr(lib, "dg_gated_backward_quantize_e4m3" + suffix), gu=P, dh=P, act=0, m_indices=P, dgu=P, q=P, sf=P,
             ld_sf=8, qt=P, sft=P, ht=P, sfht=P, rows=5, I=256, stream=None)
    for name in ("gu", "dh", "sf", "sft", "sfht"):
        refused(c, NULL, **{name: None})
    refused(c, NULL, dgu=None, q=None, qt=None, ht=None)
    for kw in (dict(rows=-1), dict(I=0), dict(I=200), dict(I=64)):
        refused(c, SHAPE, **kw)
    for kw in (dict(act=5), dict(act=-2)):
        refused(c, ARG, **kw)
    for name in ("gu", "dh", "dgu", "q", "sf", "qt", "sft", "ht", "sfht"):
        refused(c, ALIGN, **{name: MIS})
    for kw in (dict(m_indices=ODD), dict(ld_sf=4), dict(ld_sf=6)):
        refused(c, ALIGN, **kw)
    refused(c, OK, rows=0, gu=None, dh=None, m_indices=None, dgu=None, q=None, sf=None, qt=None, sft=None, ht=None, sfht=None)


def test_binding_refusals():
    """The binding names the argument and raises before the library is called (host tensors are refused too)."""
    import torch
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x"):
        binding.rmsnorm_quantize_e4m3_1x128(x, w)
    with pytest.raises(ValueError, match="scales"):
        binding.rmsnorm_quantize_e4m3_1x128(x, w, scales="fp16")
    with pytest.raises(ValueError, match="act"):
        binding._act_of("relu")
    with pytest.raises(TypeError, match="w"):
        binding._type_of(w.half(), "w")
    with pytest.raises(ValueError, match="a\\[M, K\\]"):
        binding.fp8_gated_gemm_nt(x[0], w, x, w)
    with pytest.raises(ValueError, match="dh"):
        binding.gated_backward_quantize_e4m3(x, w)
    with pytest.raises(ValueError, match="workspace"):
        binding.rmsnorm_backward(x, x, w, workspace="none")
    with pytest.raises(TypeError, match="dy"):
        binding._raw(x, torch.float32, x.shape, "dy")


def test_reference_activations():
    """The tests' reference of the tanh form of GELU is 0.5 g (1 + tanh z), and both derivatives are the differences'."""
    g = np.linspace(-6, 6, 4001)
    z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    assert np.max(np.abs(layer_helpers.act(g, "gelu") - 0.5 * g * (1 + np.tanh(z)))) < 1e-14
    for kind in ("silu", "gelu"):
        d = (layer_helpers.act(g + 1e-6, kind) - layer_helpers.act(g - 1e-6, kind)) / 2e-6
        assert np.max(np.abs(d - layer_helpers.act_grad(g, kind))) < 1e-8


def test_limits_of_32_bit_offsets(lib):
    """Sizes whose offsets inside a tile would pass 32 bits."""
    K = 1 << 23
    assert lib.dg_get_gated_workspace_size(1, 1, K) == SHAPE
    c = Call(lib.dg_fp8_gated_gemm_nt, a=P, sfa=P, ld_sfa=4, b=P, sfb=P, act=0, gu=None, h=P, q=None, sf=None, ld_sf=4,
             M=1, I=1, K=K, workspace=None, workspace_bytes=0, stream=None)
    refused(c, SHAPE)
    c = Call(lib.dg_gated_backward_quantize_e4m3, gu=P, dh=P, act=0, m_indices=None, dgu=P, q=None, sf=None, ld_sf=4,
             qt=None, sft=None, ht=None, sfht=None, rows=1, I=1 << 22, stream=None)
    refused(c, SHAPE)
