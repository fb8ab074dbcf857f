"""GPU tests of the experts' row operators at the ends of their sizes."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def announce(msg):
    print(f"\n[case] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def needs(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("G,cap", [(2, (1 << 30) - 1), (1, (1 << 31) - 1), (3, 715827882)])
def test_masked_sort_into_the_most_rows(G, cap):
    """G * M_cap just below 2^31: src holds the pairs and -1 elsewhere, and nothing is written around it."""
    needs(16)
    announce(f"masked sort into {G} x {cap} rows")
    T, k, pad = 50, 3, 64
    ids = np.random.default_rng(G).integers(-1, G + 1, (T, k)).astype(np.int32)
    flat = torch.full((G * cap + 2 * pad,), 77, dtype=I32, device="cuda")
    src = flat[pad:-pad].view(G, cap)
    rows, got, masked_m = dg.moe_sort_masked(torch.from_numpy(ids).cuda(), G, cap, src=src)
    torch.cuda.synchronize()
    want_rows = np.full(T * k, -1, np.int64)
    for e in range(G):
        pairs = np.flatnonzero(ids.reshape(-1) == e)
        want_rows[pairs] = e * cap + np.arange(pairs.size)
        assert int(masked_m[e]) == pairs.size
        assert np.array_equal(src[e, :pairs.size].cpu().numpy(), pairs)
        assert bool((src[e, pairs.size:] == -1).all())
    assert np.array_equal(rows.cpu().numpy().reshape(-1), want_rows)
    assert bool((flat[:pad] == 77).all()) and bool((flat[-pad:] == 77).all())


@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_of_a_token_with_many_choices(weighted):
    """One token with 2^24 choices, dealt to as many workgroups as there are CUs: every row holds it, and every weight has
    its gradient."""
    needs(24)
    k, K = (1 << 24) + 5, 128
    announce(f"dispatch of one token with {k} choices weighted={weighted}")
    x = torch.linspace(-3, 3, K, device="cuda").to(BF16).view(1, K)
    R = (k + 127) // 128 * 128
    # backwards, so that a choice's row tells its place
    rows = torch.arange(k - 1, -1, -1, dtype=I32, device="cuda").view(1, k)
    w = (1 + (torch.arange(k, device="cuda") % 7)).view(1, k).float() if weighted else None
    q, sf, _, _, _ = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, weights=w)
    values = x.float() * (torch.arange(1, 8, device="cuda").view(7, 1) if weighted else torch.ones(7, 1, device="cuda"))
    wq, wsf = dg.quantize_e4m3_1x128(values.contiguous())
    at = (k - 1 - torch.arange(k, device="cuda")) % 7                  # of the choice in each row
    for lo in range(0, k, 1 << 20):
        part = at[lo:lo + (1 << 20)]
        assert torch.equal(q[lo:lo + part.numel()], wq[part])
        assert torch.equal(sf[0, lo:lo + part.numel()], wsf[0, part])
    assert not q[k:].any() and not sf[0, k:].any()
    del q, sf
    ye = torch.zeros((R, K), dtype=BF16, device="cuda")
    ye[:k, 0] = (1 + torch.arange(k, device="cuda") % 5).to(BF16)      # exact products: -3 * 1 .. 5
    dw, *_ = dg.moe_combine_backward_quantize_e4m3_contiguous(x, ye, rows, w, dw=True)
    assert torch.equal(dw.view(-1), x[0, 0].float() * ye[:k, 0].float().flip(0))


@pytest.mark.parametrize("K", [(1 << 31) - 8, (1 << 31) - 512, 1 << 30])
def test_combine_of_the_widest_rows(K):
    """Rows of up to 2^31 - 8 columns: the last columns come out as the first, and nothing is written past them."""
    needs(24)
    announce(f"combine K={K}")
    flat = torch.full((K + 128,), 7.0, dtype=BF16, device="cuda")
    out, y = flat[64:-64].view(1, K), torch.empty((1, K), dtype=BF16, device="cuda")
    y.view(-1, 8).copy_(torch.arange(8, device="cuda").to(BF16))
    y[0, -8:] += 8
    rows = torch.tensor([[0, -1]], dtype=I32, device="cuda")
    dg.moe_combine(y, rows, weights=torch.tensor([[2.0, 5.0]], device="cuda"), out=out)
    torch.cuda.synchronize()
    y.mul_(2)
    assert torch.equal(out, y)
    assert bool((flat[:64] == 7).all()) and bool((flat[-64:] == 7).all())
