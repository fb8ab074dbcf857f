"""GPU tests of sizes whose grid would reach 2^32 threads, which HIP takes
modulo 2^32 without an error: a larger tile takes them where there is one, and
the call fails where there is none."""
import sys

import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

pytestmark = pytest.mark.gpu


def announce(msg):
    print(f"\n[case] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 128 << 30:
        pytest.skip("needs 128 GiB of device memory")
    dg.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_gated_masked_of_few_columns():
    """8 columns and a hint of 64 rows: the 64-row tile serves them best, 2^23 + 2 of them here."""
    G, cap, I, K = (1 << 22) + 1, 128, 8, 128
    announce(f"gated masked of {G} x {cap} x {I} x {K}")
    g = torch.Generator(device="cuda").manual_seed(5)
    a, sfa = dg.quantize_e4m3_1x128(torch.randn(cap, K, generator=g, device="cuda"))
    w, sfw = dg.quantize_e4m3_128x128(torch.randn(2, I, K, generator=g, device="cuda"))
    big, sf = torch.zeros((G, cap, K), dtype=torch.uint8, device="cuda"), torch.zeros((G, 1, cap), device="cuda")
    b, sfb = torch.zeros((G, 2, I, K), dtype=torch.uint8, device="cuda"), torch.zeros((G, 2, 1, 1), device="cuda")
    counts = torch.zeros(G, dtype=torch.int32, device="cuda")
    groups = (0, 1, G // 2, G - 1)
    for e in groups:
        big[e], sf[e], b[e], sfb[e], counts[e] = a, sfa, w, sfw.view(2, 1, 1), cap - 3
    h = torch.zeros((G, cap, I), dtype=torch.bfloat16, device="cuda")
    dg.m_grouped_fp8_gated_gemm_nt_masked(big, sf, b, sfb, counts, expected_m=64, h=h)
    torch.cuda.synchronize()
    want = dg.fp8_gated_gemm_nt(a, sfa, w, sfw.view(2, 1, 1))[0]
    torch.cuda.synchronize()
    assert want.any()
    for e in groups:
        assert torch.equal(h[e, :cap - 3], want[:cap - 3]), f"group {e}"
        h[e, :cap - 3] = 0
    assert not h.any()


def test_gated_masked_of_many_groups_is_refused():
    """Every group takes a tile of each shape; no group has rows, so no operand is read."""
    cap, I, K = 4, 8, 128
    small = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    p = small.data_ptr()
    for G, status in (((1 << 23) + 1, -6), (1 << 23, -6), ((1 << 23) - 1, 0)):
        announce(f"gated masked of {G} groups")
        counts = torch.zeros(G, dtype=torch.int32, device="cuda")
        assert dg.lib().dg_m_grouped_fp8_gated_gemm_nt_masked(p, p, p, p, 0, None, p, None, None, counts.data_ptr(), G, cap, I,
                                                               K, 0, None) == status
        torch.cuda.synchronize()
    assert not small.any()


def test_quantiser_refuses_it():
    announce("128x128 quantiser of 2^24 groups and more")
    x = torch.ones(((1 << 24) + 1, 1, 128), device="cuda")
    for n in ((1 << 24) + 1, 1 << 24):
        with pytest.raises(dg.DGError, match="HIP"):
            dg.quantize_e4m3_128x128(x[:n])
    q, sf = dg.quantize_e4m3_128x128(x[2:])
    torch.cuda.synchronize()
    assert torch.all(q == 0x7E) and torch.all(sf == sf.view(-1)[0])   # 1 over 1/448 is the largest code
