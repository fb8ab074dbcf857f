"""GPU tests of the feed-forward layer where offsets pass 32 bits: tensors of
more than 2^31 elements, made of one block of rows repeated, whose every repeat
has to come out as the block alone does."""
import sys

import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def announce(msg):
    print(f"\n[case] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of device memory")
    dg.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture
def rand():
    g = torch.Generator(device="cuda").manual_seed(11)
    yield lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def same_repeats(big, small, n):
    """big = n copies of small along the first dimension, bit for bit."""
    big = big.view(n, *small.shape)
    for k in range(n):
        assert torch.equal(big[k], small), f"repeat {k} of {n}"


def test_norm(rand):
    rows, K, n = 1024, 7168, 300                       # 2.2e9 elements
    announce(f"norm of {n * rows} x {K}")
    x, w = rand(rows, K).to(BF16), rand(K).to(BF16)
    want_q, want_sf, want_h, _ = dg.rmsnorm_quantize_e4m3_1x128(x, w, residual=x)
    q, sf, h, _ = dg.rmsnorm_quantize_e4m3_1x128(x.repeat(n, 1), w, residual=x.repeat(n, 1))
    torch.cuda.synchronize()
    assert h.numel() > 1 << 31
    same_repeats(q, want_q, n)
    same_repeats(h, want_h, n)
    same_repeats(sf.t().contiguous(), want_sf.t().contiguous(), n)


def test_norm_backward(rand):
    rows, K, n = 1024, 7168, 300
    announce(f"norm backward of {n * rows} x {K}")
    h, dy, w = rand(rows, K).to(BF16), rand(rows, K).to(BF16), rand(K)
    want, _ = dg.rmsnorm_backward(dy, h, w)
    dx, dw = dg.rmsnorm_backward(dy.repeat(n, 1), h.repeat(n, 1), w)
    torch.cuda.synchronize()
    same_repeats(dx, want, n)
    hd = h.double()
    terms = dy.double() * hd * torch.rsqrt(hd.pow(2).mean(1, keepdim=True) + 1e-6)
    # sums of 600 rows a workgroup, 32 workgroups a wave and 16 waves, each term and the rows' factors within 8 ulp
    bar = (600 + 32 + 16 + 8) * 2.0 ** -24 * n * terms.abs().sum(0)
    assert torch.all((dw.double() - n * terms.sum(0)).abs() <= bar)


def operands(rand, rows, I, K, G=None):
    a, sfa = dg.quantize_e4m3_1x128(rand(rows, K))
    b, sfb = dg.quantize_e4m3_128x128(rand((G or 1) * 2, I, K) * K ** -0.5)
    return (a, sfa, b, sfb) if G is None else (a, sfa, b.view(G, 2, I, K), sfb.view(G, 2, *sfb.shape[1:]))


@pytest.mark.parametrize("I,K,n", [(128, 7168, 150), (3584, 128, 150)])
def test_gated_dense(rand, I, K, n):
    """A, or the outputs, of more than 2^31 elements."""
    rows = 2048
    announce(f"gated of {n * rows} x {I} x {K}")
    a, sfa, b, sfb = operands(rand, rows, I, K)
    want = dg.fp8_gated_gemm_nt(a, sfa, b, sfb, h=True, gu=True)
    h, _, _, gu = dg.fp8_gated_gemm_nt(a.repeat(n, 1), sfa.repeat(1, n), b, sfb, h=True, gu=True)
    torch.cuda.synchronize()
    assert max(n * rows * K, gu.numel()) > 1 << 31
    same_repeats(h, want[0], n)
    same_repeats(gu, want[3], n)


def test_gated_contiguous(rand):
    I, K, M = 128, 4224, 1 << 19
    announce(f"gated contiguous of {M} x {I} x {K}")
    a, sfa, b, sfb = operands(rand, 512, I, K, G=2)
    big = a.repeat(M // 512, 1)
    idx = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    idx[:100] = 0
    idx[-384:] = 1                                     # rows past 2^31 bytes of A
    h, _, _, _ = dg.m_grouped_fp8_gated_gemm_nt_contiguous(big, sfa.repeat(1, M // 512), b, sfb, idx)
    torch.cuda.synchronize()
    assert big.numel() > 1 << 31
    want = [dg.fp8_gated_gemm_nt(a, sfa, b[e], sfb[e].clone())[0] for e in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(h[:100], want[0][:100]) and torch.equal(h[-384:], want[1][-384:])
    assert not h[100:-384].any()


def test_gated_masked(rand):
    I, K, cap, G = 128, 4224, 8192, 64
    announce(f"gated masked of {G} x {cap} x {I} x {K}")
    a, sfa, b, sfb = operands(rand, cap, I, K, G=G)
    big = a.repeat(G, 1).view(G, cap, K)
    counts = torch.zeros(G, dtype=torch.int32, device="cuda")
    counts[0], counts[-1] = 3, 700
    h, _, _, _ = dg.m_grouped_fp8_gated_gemm_nt_masked(big, sfa.repeat(G, 1).view(G, *sfa.shape), b, sfb, counts, expected_m=200)
    torch.cuda.synchronize()
    assert big.numel() > 1 << 31
    for g, n in ((0, 3), (G - 1, 700)):
        want = dg.fp8_gated_gemm_nt(a, sfa, b[g], sfb[g].clone())[0]
        torch.cuda.synchronize()
        assert torch.equal(h[g, :n], want[:n]) and not h[g, n:].any()


def test_gated_backward(rand):
    rows, I, n = 2048, 3584, 150
    announce(f"gated backward of {n * rows} x {I}")
    gu, dh = rand(rows, 2 * I).to(BF16), rand(rows, I).to(BF16)
    want = dg.gated_backward_quantize_e4m3(gu, dh, q=True, qt=True, ht=True)
    _, q, sf, qt, sft, ht, sfht = dg.gated_backward_quantize_e4m3(gu.repeat(n, 1), dh.repeat(n, 1), q=True, qt=True, ht=True)
    torch.cuda.synchronize()
    assert q.numel() > 1 << 31
    same_repeats(q, want[1], n)
    same_repeats(sf.t().contiguous(), want[2].t().contiguous(), n)
    for big, small in ((qt, want[3]), (sft, want[4]), (ht, want[5]), (sfht, want[6])):
        same_repeats(big, small, n)
