"""GPU test of the gated activation's gradient at gates whose square passes the
range of fp32: act' is 0 or 1 there, not NaN."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

from layer_helpers import act, act_grad, bf16, check_bf16, f64, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [40, 5000])
def test_gates_of_any_size(kind, rows):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"\n[case] gated_bwd, gates up to 3e38, {kind} rows={rows}", file=sys.stderr, flush=True)
    I = 128
    far = np.array([1e10, 9e18, 1.7e19, 2e19, 1e25, 3e38, 0.5, 2.0], np.float32)
    g = np.tile(np.concatenate([far, -far]), (rows, I // 16))
    gu = bf16(np.concatenate([g, 0.1 * normal(1, (rows, I))], 1)).cuda()
    dh = bf16(0.1 * normal(2, (rows, I))).cuda()
    dgu, q, sf, qt, sft, ht, sfht = dg.gated_backward_quantize_e4m3(gu, dh, kind, dgu=True, q=True, qt=True, ht=True)
    gn, un, dn = f64(gu)[:, :I], f64(gu)[:, I:], f64(dh)
    for k, ref in enumerate((dn * un * act_grad(gn, kind), dn * act(gn, kind))):
        # fp32 arithmetic in front of the rounding: 2^-18 of the value and, near act' = 0, of its terms (|act'| terms <= 2)
        extra = 2.0 ** -18 * (np.abs(ref) + 2 * np.abs(dn * un)) + 2.0 ** -130
        check_bf16(dgu[:, k * I:(k + 1) * I], ref, extra, f"{kind} {k}")
    for codes, scales in ((q, sf), (qt, sft), (ht, sfht)):
        assert torch.all((codes & 0x7F) != 0x7F) and torch.all(torch.isfinite(scales))
