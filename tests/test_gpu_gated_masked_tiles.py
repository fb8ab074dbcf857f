"""GPU tests of the gated GEMM's masked layout in every tile shape, the
quantised output among the outputs: its row maxima, scales and codes in groups
whose rows end inside a tile."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

from helpers import dev  # noqa: F401
from test_gpu_gated import (QSENT, SENT, Outputs, announce, check_rows, cu_caps, operands, problem,  # noqa: F401
                            projections, scales_of, tiles_of)

pytestmark = pytest.mark.gpu

WIDE = {"256x256x128", "128x256x128", "64x256x128"}
NARROW = {"128x128x128", "64x128x128", "64x64x128"}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("cap,I,mm", [(300, 256, [129, 300, -1, 0, 257]), (256, 640, [256, 1, 128, 255, 64]),
                                      (300, 268, [129, 300, -1, 0, 257])])
@pytest.mark.parametrize("packed", [False, True])
def test_every_tile(cap, I, mm, packed, cu_caps):  # noqa: F811
    """Widths of whole blocks with all outputs and with the quantised one alone, and another width in bf16."""
    K, G, quant = 640, len(mm), I % 128 == 0
    p = problem((G,), cap, I, K, cap + I, packed, (G,))
    a, sfa, b, sfb = (x.copy() for x in p)
    rows = [min(max(m, 0), cap) for m in mm]
    for g in range(G):
        a[g, rows[g]:] = 0x7F
        if not packed:
            sfa[g, :, rows[g]:] = np.nan
    ops = operands((a, sfa, b, sfb), packed)
    counts = torch.tensor(mm, dtype=torch.int32, device="cuda")
    want = [projections(p[0][g, :rows[g]], p[1][g][:, :rows[g]], p[2][g], p[3][g]) if rows[g] else None for g in range(G)]
    seen = set()
    for cus in cu_caps:
        dg.set_num_cus(cus)
        for every in (True, False) if quant else (True,):
            announce(f"gated masked tiles cap={cap} I={I} {mm} packed={packed} cus={cus} every output={every}")
            o = Outputs((G,), cap, I, (cap + 3) // 4 * 4, packed, quant)
            dg.m_grouped_fp8_gated_gemm_nt_masked(*ops, counts, act="silu", q=o.q, sf=o.sf,
                                                  **(dict(h=o.h, gu=o.gu) if every else {}))
            torch.cuda.synchronize()
            o.guards()
            seen |= tiles_of(dg.last_config())
            for g in range(G):
                n = rows[g] if every else 0
                assert torch.all(o.h[g, n:].contiguous().view(torch.int16) == SENT)
                assert torch.all(o.gu[g, n:].contiguous().view(torch.int16) == SENT)
                n = rows[g]
                if quant:
                    assert torch.all(o.q[g, n:] == QSENT)
                    assert torch.all(o.sf[g, :, n:] == (0x5A5A5A5A if packed else -5.0))
                if n:
                    check_rows(f"group {g} cus={cus} {dg.last_config()}", o.gu[g, :n] if every else None,
                               o.h[g, :n] if every else None, o.q[g, :n] if quant else None,
                               scales_of(o.sf[g][:, :n], packed, I // 128).T if quant else None, I, *want[g], "silu", packed)
    if quant:
        assert WIDE <= seen
    else:
        assert {"256x256x128", "128x256x128"} <= seen and seen & NARROW
