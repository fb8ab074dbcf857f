"""GPU tests of the contiguous grouped GEMM where an expert owns several
segments: what the layout asks for is that an aligned 128-row block holds rows
of one expert, so blocks of the experts may come in any order."""
import sys

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_gemm_scaled_amd import binding as dg
from moe_grouped_gemm_scaled_amd import synth

from helpers import SENTINEL, Guarded, check_close, dev, dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    dg.set_kernel_family("auto")
    torch.cuda.synchronize()


def problem(blocks, G, N, K, ue8m0, seed):
    """Operands for blocks of these experts (-1: no data); every third block holds only its first rows."""
    rows = np.full(len(blocks), 128)
    rows[::3] = 1 + (np.arange(len(blocks)) * 37 % 128)[::3]
    idx = np.full((len(blocks), 128), -1, np.int32)
    for b, e in enumerate(blocks):
        idx[b, :rows[b]] = e
    idx = idx.reshape(-1)
    a, sfa = oracle.quantize_1x128(synth.normal_f32(seed, 0, (idx.size, K)), ue8m0=ue8m0)
    b, sfb = oracle.quantize_128x128(synth.normal_f32(seed, 1, (G, N, K)), ue8m0=ue8m0)
    return a, sfa, b, sfb, synth.normal_bf16_bits(seed, 2, (idx.size, N)), idx


UNITS, BLOCKS = "tile=256x256x128", "tile=128x256x128"      # of which the short K of many blocks takes the second
LAYOUTS = {
    "alternating": [0, 1] * 9,
    "shuffled": [0, 0, 0, 2, 1, 1, 0, 2, 2, 2, 2, 0, 1, 0, 1, 1, 1, 2, 0, 0, 1, 2, 0, 2, 1, 0, 1, 2, 2, 0, 1, 1],
    "gaps": [0, -1, 0, 1, -1, -1, 1, 0, 0, -1, 1, 1, 1, 0, -1, 0, 1, 0, 1, 0, -1, 0, 1, 0, 1, 0, 1],
    "bad ids": [0, 7, 1, 7, 0, 1 << 30, 0, 0, 7, 1, 1, 9, 0, 7, 1, 0, 1, 0, 7, 0, 1, 0],
    "many": [0, 1, 2] * 100,
    "more": [0, 1, 2, 2, 1, 0, 0] * 60,
}


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("scales", ["fp32", "ue8m0", "packed"])
def test_repeated_segments(name, scales):
    blocks, G, K = LAYOUTS[name], 3, 256
    N = {"many": 136, "more": 520}.get(name, 264)
    a, sfa, b, sfb, c, idx = problem(blocks, G, N, K, scales != "fp32", 40 + len(blocks))
    valid = (idx >= 0) & (idx < G)
    ref = oracle.m_grouped_contiguous(a, sfa, b, sfb, c, np.where(valid, idx, -1).astype(np.int32))
    for family in ("auto", "persist") if scales == "fp32" else ("auto",):
        print(f"\n[case] contiguous segments {name} {scales} {family}", file=sys.stderr, flush=True)
        dg.set_kernel_family(family)
        out = Guarded((idx.size, N))
        if scales == "packed":
            dg.m_grouped_fp8_gemm_nt_contiguous_ue8m0_packed(
                dev(a), dev(oracle.pack_ue8m0(sfa, k_axis=-2).view(np.int32)), dev(b),
                dev(oracle.pack_ue8m0(sfb, k_axis=-1).view(np.int32)), out.t, dev(idx), c=dev_bf16(c))
        else:
            dg.m_grouped_fp8_gemm_nt_contiguous(dev(a), dev(sfa), dev(b), dev(sfb), out.t, dev(idx), c=dev_bf16(c),
                                                ue8m0=scales == "ue8m0")
        torch.cuda.synchronize()
        if family == "auto":
            assert "family=pipe mode=1 " + (BLOCKS if name == "more" else UNITS) in dg.last_config()
        assert out.guards_intact()
        got = out.bits()
        assert np.all(got[~valid] == SENTINEL)
        check_close(got[valid], ref[valid], f"{name} {scales} {dg.last_config()}")
