"""GPU test of the gated gradient's column-scaled codes as both operands of the
K-grouped GEMM: codes stored [K][M] with one scale per column and 128 rows, the
K axis being the rows of the contiguous layout, expert by expert.  The other
operand has one nonzero code in every column and 128-row block, so each sum has
one product per block and no rounding but the sum's over the blocks: with one
block per expert it is exact, and the layouts are what is tested."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg
from moe_grouped_gemm_scaled_amd import synth

from layer_helpers import bf16, check, f64, normal

pytestmark = pytest.mark.gpu
ONE = 0x38                # 1 in E4M3


@pytest.mark.parametrize("counts", [[128], [5, 0, 300], [130, 256, 1, 0, 127]])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_operands_of_the_k_grouped_gemm(counts, ue8m0):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"\n[case] gated_bwd into the K-grouped GEMM {counts} ue8m0={ue8m0}", file=sys.stderr, flush=True)
    idx = synth.contiguous_m_indices(counts)
    rows, I = idx.size, 256
    gu, dh = bf16(normal(1, (rows, 2 * I))).cuda(), bf16(normal(2, (rows, I))).cuda()
    gu[torch.from_numpy(idx < 0).cuda()] = float("nan")
    _, _, _, qt, sft, ht, sfht = dg.gated_backward_quantize_e4m3(gu, dh, m_indices=torch.from_numpy(idx).cuda(), qt=True,
                                                                 ht=True, ue8m0=ue8m0)
    ks = [(c + 127) // 128 * 128 for c in counts]
    sizes = torch.tensor(ks, dtype=torch.int32, device="cuda")
    # column n of the other operand picks row (37 n + 11 block) mod 128 of every block
    N = 128
    pick = np.zeros((rows, N), np.uint8)
    for b in range(rows // 128):
        pick[128 * b + (37 * np.arange(N) + 11 * b) % 128, np.arange(N)] = ONE
    scale = np.exp2(synth.randint(3, 1, rows // 128 * N, -3, 3).astype(np.float32)).reshape(-1, N)
    other, other_sf = torch.from_numpy(pick).cuda(), torch.from_numpy(scale).cuda()
    y = f64(other) * np.repeat(f64(other_sf), 128, 0)
    for name, q, s in (("qt", qt, sft), ("ht", ht, sfht)):
        x = f64(q) * np.repeat(f64(s), 128, 0)
        M = x.shape[1]
        first = torch.full((len(ks), M, N), float("nan"), device="cuda")
        dg.k_grouped_fp8_gemm_tn_contiguous(q, s, other, other_sf, sizes, first, ue8m0=ue8m0)
        second = torch.full((len(ks), N, M), float("nan"), device="cuda")
        dg.k_grouped_fp8_gemm_tn_contiguous(other, other_sf, q, s, sizes, second, ue8m0=ue8m0)
        torch.cuda.synchronize()
        at = 0
        for g, k in enumerate(ks):
            blocks = x[at:at + k].reshape(-1, 128, M), y[at:at + k].reshape(-1, 128, N)
            ref = sum((a.T @ b for a, b in zip(*blocks)), np.zeros((M, N)))
            size = sum((np.abs(a).T @ np.abs(b) for a, b in zip(*blocks)), np.zeros((M, N)))
            # a product of two codes is exact; its scales' product and each block's addition round once in fp32
            tol = 2.0 ** -24 * (2 + k // 128) * size if k > 128 or not ue8m0 else 0.0
            check(f64(first[g]), ref, tol, f"{name} as A, expert {g}")
            check(f64(second[g]), ref.T, tol.T if np.ndim(tol) else tol, f"{name} as B, expert {g}")
            at += k
        assert np.abs(x).max() > 0
