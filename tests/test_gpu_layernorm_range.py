"""GPU tests of the layer norm at the ends of fp32's range."""
import sys

import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def announce(msg):
    print(f"\n[case] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("K", [512, 1024, 2048, 7168, 16384])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_rows_whose_sums_pass_fp32(K, xt):
    """Row 0: the sum of finite values is infinite: NaN throughout, as with an infinity.  Row 1: its squares are, its sum
    is not: the bias.  Row 2: an ordinary row beside them.  The gradient of row 1 is what arrives at h itself."""
    announce(f"ln sums past fp32 K={K} {xt}")
    x = torch.zeros((3, K), device="cuda")
    x[0] = 3e38
    x[1, ::2], x[1, 1::2] = 2.0 ** 100, -2.0 ** 100
    x[2, ::2], x[2, 1::2] = 2.0, -2.0
    x = x.to(xt)
    w, b = torch.full((K,), 2.0, dtype=BF16, device="cuda"), torch.full((K,), 0.5, dtype=BF16, device="cuda")
    q, sf, _, y = dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, y=True)
    assert bool(y[0].isnan().all()) and bool((q[0] == 0x7F).all())
    assert bool((y[1] == 0.5).all()) and bool((q[1] == 0x7E).all())     # 0.5 over 0.5 / 448
    # 2 / sqrt(4 + 1e-5) = 1 - 1.25e-6: bf16 of 2.5 and -1.5, each off by far less than half a step
    assert bool((y[2, ::2] == 2.5).all()) and bool((y[2, 1::2] == -1.5).all())
    dres = torch.randn(3, K, device="cuda").to(xt)
    dx, dw, db = dg.layernorm_backward(torch.ones((3, K), dtype=BF16, device="cuda"), x, w, EPS, dres=dres)
    assert bool(dx[0].isnan().all()) and torch.equal(dx[1], dres[1])
    assert bool((db == 3).all())


@pytest.mark.parametrize("K", [8, 520, 2048])
def test_equal_values_without_eps(K):
    announce(f"ln of equal values, eps = 0, K={K}")
    x = torch.full((2, K), 1.5, dtype=BF16, device="cuda")
    x[1, 0] = -1.5
    y = dg.layernorm_quantize_e4m3_1x128(x, eps=0.0, y=True, q=False)[3]
    assert bool(y[0].isnan().all()) and bool(y[1].isfinite().all())
