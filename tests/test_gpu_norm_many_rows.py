"""GPU tests of the RMS norm with more rows than one launch takes workgroups
for (a grid may not reach 2^32 threads): one block of rows repeated, whose
every repeat has to come out as the block alone does."""
import sys

import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
BLOCK = 1 << 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# one wave a row (four rows per workgroup), four and sixteen: past 2^32 threads each
@pytest.mark.parametrize("rows,K", [((1 << 26) + 5, 128), ((1 << 24) + 3, 1152), ((1 << 22) + 1, 8320)])
def test_more_rows_than_a_grid(rows, K):
    if torch.cuda.mem_get_info()[0] < 4 * rows * K:
        pytest.skip("needs more device memory")
    print(f"\n[case] norm of {rows} x {K}", file=sys.stderr, flush=True)
    g = torch.Generator(device="cuda").manual_seed(K)
    block = torch.randn(BLOCK, K, generator=g, device="cuda").to(BF16)
    w = torch.randn(K, generator=g, device="cuda")
    want_q, want_sf, _, _ = dg.rmsnorm_quantize_e4m3_1x128(block, w)
    x = torch.empty((rows, K), dtype=BF16, device="cuda")
    for r in range(0, rows, BLOCK):
        x[r:r + BLOCK] = block[:rows - r]
    q, sf, _, _ = dg.rmsnorm_quantize_e4m3_1x128(x, w)
    torch.cuda.synchronize()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for r in range(0, rows, BLOCK):
        n = min(BLOCK, rows - r)
        differ += (q[r:r + n] != want_q[:n]).any() | (sf[:, r:r + n] != want_sf[:, :n]).any()
    assert int(differ) == 0
    assert not sf[:, rows:].any()
