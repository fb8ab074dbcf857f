"""GPU tests of the gated GEMM's contiguous layout where an expert owns several
segments: what the layout asks for is that an aligned 128-row block holds rows
of one expert, so blocks of the experts may come in any order."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

from helpers import dev
from test_gpu_gated import (QSENT, SENT, Outputs, announce, check_rows, few_cus, operands, problem,  # noqa: F401
                            projections, scales_of)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    torch.cuda.synchronize()


def indices(blocks, partial):
    """m_indices of blocks of these experts (-1: no data): full, or (some) with their first rows only."""
    rows = np.full(len(blocks), 128)
    if partial:
        rows[::3] = 1 + (np.arange(len(blocks)) * 37 % 128)[::3]
    idx = np.full((len(blocks), 128), -1, np.int32)
    for b, e in enumerate(blocks):
        idx[b, :rows[b]] = e
    return idx.reshape(-1)


ALTERNATING = [0, 1] * 20
SHUFFLED = [0, 0, 0, 2, 1, 1, 0, 2, 2, 2, 2, 0, 1, 0, 1, 1, 1, 2, 0, 0, 1, 2, 0, 2, 1, 0, 1, 2, 2, 0, 1, 1]
WITH_GAPS = [0, -1, 0, 1, -1, -1, 1, 0, 0, -1, 1, 1, 1, 0, -1, 0, 1, 0, 1, 0, -1, 0, 1, 0, 1, 0, 1]
WITH_BAD_IDS = [0, 7, 1, 7, 0, 1 << 30, 0, 0, 7, 1, 1, 9, 0, 7, 1, 0, 1, 0, 7, 0, 1, 0]
ONE_EXPERT = [0, -1] * 12


@pytest.mark.parametrize("blocks", [ALTERNATING, SHUFFLED, WITH_GAPS, WITH_BAD_IDS, ONE_EXPERT],
                         ids=["alternating", "shuffled", "gaps", "bad ids", "one expert"])
@pytest.mark.parametrize("I", [128, 384])
@pytest.mark.parametrize("partial,packed", [(False, False), (True, True)])
def test_repeated_segments(blocks, I, partial, packed, few_cus):  # noqa: F811
    announce(f"gated contiguous segments {blocks} I={I} partial={partial} packed={packed}")
    K, G = 256, 3
    idx = indices(blocks, partial)
    M = idx.size
    p = problem((), M, I, K, 7 + M, packed, (G,))
    valid = (idx >= 0) & (idx < G)
    a, sfa, b, sfb = (x.copy() for x in p)
    a[~valid] = 0x7F
    if not packed:
        sfa[:, ~valid] = np.nan
    ops = operands((a, sfa, b, sfb), packed)
    o = Outputs((), M, I, M, packed, True)
    dg.m_grouped_fp8_gated_gemm_nt_contiguous(*ops, dev(idx), act="silu", h=o.h, q=o.q, sf=o.sf, gu=o.gu)
    torch.cuda.synchronize()
    assert "rest: tile=128x256x128" in dg.last_config()              # 256-row units
    o.guards()
    pad = torch.from_numpy(~valid).cuda()
    assert torch.all(o.h.view(torch.int16)[pad] == SENT) and torch.all(o.gu.view(torch.int16)[pad] == SENT)
    assert torch.all(o.q[pad] == QSENT) and torch.all(o.sf[:, pad] == (0x5A5A5A5A if packed else -5.0))
    for e in range(G):
        at = np.flatnonzero(idx == e)
        if at.size == 0:
            continue
        t = torch.from_numpy(at).cuda()
        gate, up = projections(p[0][at], p[1][:, at], p[2][e], p[3][e])
        check_rows(f"expert {e}", o.gu[t], o.h[t], o.q[t], scales_of(o.sf[:, t], packed, I // 128).T, I, gate, up, "silu",
                   packed)


def test_many_repeated_segments():
    """More blocks than one round of the index walk (256), on all CUs: each block as the block alone comes out."""
    announce("gated contiguous, 600 alternating blocks")
    I, K, n = 256, 128, 600
    p = problem((), 256, I, K, 3, False, (2,))
    a, sfa, b, sfb = operands(p, False)
    idx = torch.arange(n, device="cuda", dtype=torch.int32).remainder(2).repeat_interleave(128)
    h, q, sf, _ = dg.m_grouped_fp8_gated_gemm_nt_contiguous(a.repeat(n // 2, 1), sfa.repeat(1, n // 2), b, sfb, idx, h=True, q=True)
    torch.cuda.synchronize()
    assert "rest: tile=128x256x128" in dg.last_config()
    for e in range(2):
        at = slice(128 * e, 128 * e + 128)
        gate, up = projections(p[0][at], p[1][:, at], p[2][e], p[3][e])
        check_rows(f"block {e}", None, h[at], q[at], scales_of(sf[:, at], False, I // 128).T, I, gate, up, "silu", False)
    h, q, sf = h.view(n // 2, 256, I), q.view(n // 2, 256, I), sf.view(I // 128, n // 2, 256)
    assert torch.equal(h, h[:1].expand_as(h)) and torch.equal(q, q[:1].expand_as(q)) and torch.equal(sf, sf[:, :1].expand_as(sf))
