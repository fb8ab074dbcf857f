"""GPU tests of the RMS norm with residual and E4M3 output, and of its
gradient, against 64-bit references (bars: layer_helpers)."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

from layer_helpers import SLACK, check, check_bf16, check_quantised, f64, normal, ulp_bf16, unpack_words

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


def device(x, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(dtype)


def scale_values(sf, scales, blocks, rows):
    s = unpack_words(sf, blocks) if scales == "ue8m0_packed" else f64(sf)
    return s[:, :rows].T                                             # [rows, blocks]


def check_forward(x, res, w, out, scales, where, eps=EPS):
    q, sf, ro, y = out
    rows, K = x.shape
    h = f64(x) + (f64(res) if res is not None else 0.0)
    ref = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * f64(w)
    extra = SLACK * np.abs(ref) + 2.0 ** -149
    if res is not None:
        h32 = x.float() + res.float()
        assert torch.equal(ro, h32.to(res.dtype)), f"{where}: residual_out is not the rounded fp32 sum"
        # cancellation in x + residual: the fp32 sum is off by up to U of it, which is inside SLACK of h
    if y is not None:
        check_bf16(y, ref, extra, where + " y")
    if q is not None:
        s = scale_values(sf, scales, K // 128, rows)
        check_quantised(f64(q).reshape(rows, K // 128, 128), s, ref.reshape(rows, K // 128, 128),
                        extra.reshape(rows, K // 128, 128), scales != "fp32", where)


# rows and widths on both sides of every change of waves per row and chunks per lane
SIZES = [(1, 128), (1, 7168), (3, 2048), (5, 2176), (64, 7168), (333, 1536), (511, 4224), (515, 8192), (7, 8320),
         (2, 16384), (2049, 512), (2051, 1152), (2050, 2048), (2053, 4096), (2048, 6144), (2055, 8192)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("scales", ["fp32", "ue8m0_packed"])
def test_forward_sizes(rows, K, scales):
    announce(f"norm rows={rows} K={K} {scales}")
    x, res = device(normal(rows + K, (rows, K)), BF16), device(3 * normal(rows + K, (rows, K), 1), BF16)
    w = device(1 + 0.3 * normal(K, (K,), 2), BF16)
    out = dg.rmsnorm_quantize_e4m3_1x128(x, w, EPS, residual=res, y=True, scales=scales)
    check_forward(x, res, w, out, scales, f"rows={rows} K={K}")


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("rt", [None, BF16, F32])
@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("rows", [6, 2049])
def test_forward_types(xt, rt, wt, rows):
    K = 640
    announce(f"norm types {xt} {rt} {wt} rows={rows}")
    x = device(normal(5, (rows, K)), xt)
    res = None if rt is None else device(normal(6, (rows, K)), rt)
    w = device(normal(7, (K,)), wt)
    out = dg.rmsnorm_quantize_e4m3_1x128(x, w, EPS, residual=res, y=True, scales="ue8m0")
    check_forward(x, res, w, out, "ue8m0", "types")


@pytest.mark.parametrize("rows", [1, 9, 2100])
def test_forward_column_range_of_a_wider_matrix(rows):
    announce(f"norm pitch rows={rows}")
    full = device(normal(8, (rows, 2112)), BF16)
    w = device(normal(9, (512,)), BF16)
    x = full[:, 1536:2048]
    out = dg.rmsnorm_quantize_e4m3_1x128(x, w, EPS, y=True)
    check_forward(x, None, w, out, "fp32", "column range")


@pytest.mark.parametrize("rows,K", [(4, 7168), (600, 2048), (2500, 1024)])
def test_forward_in_place_and_guards(rows, K):
    """residual_out over the residual; nothing is written outside the outputs, and scales past the rows stay."""
    announce(f"norm in place rows={rows} K={K}")
    x, w = device(normal(10, (rows, K)), BF16), device(normal(11, (K,)), BF16)
    pad = 64
    flat = torch.full((rows * K + 2 * pad,), 7.0, dtype=BF16, device="cuda")
    res = flat[pad:pad + rows * K].view(rows, K)
    res.copy_(device(normal(12, (rows, K)), BF16))
    before = res.clone()
    qflat = torch.full((rows * K + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    q = qflat[pad:pad + rows * K].view(rows, K)
    ld = (rows + 3) // 4 * 4 + 8
    sf = torch.full((K // 128 + 1, ld), -5.0, dtype=F32, device="cuda")
    out = dg.rmsnorm_quantize_e4m3_1x128(x, w, EPS, residual=res, residual_out=res, q=q, sf=sf[:-1])
    check_forward(x, before, w, out, "fp32", "in place")
    assert torch.all(flat[:pad] == 7) and torch.all(flat[-pad:] == 7)
    assert torch.all(qflat[:pad] == 0xA5) and torch.all(qflat[-pad:] == 0xA5)
    assert torch.all(sf[:, rows:] == -5) and torch.all(sf[-1] == -5)


def test_forward_zero_rows_and_special_values():
    announce("norm special values")
    K = 512
    w = torch.ones(K, dtype=BF16, device="cuda")
    empty = torch.empty((0, K), dtype=BF16, device="cuda")
    q, sf, ro, y = dg.rmsnorm_quantize_e4m3_1x128(empty, w, EPS, residual=empty, y=True)
    assert q.shape == (0, K) and y.shape == (0, K)
    x = torch.zeros((6, K), dtype=F32, device="cuda")
    x[1] = 1e-30                                        # far below eps
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4, 200] = -1.0                                    # one value: |y| = sqrt(K) there
    x[5] = 1e15
    q, sf, _, y = dg.rmsnorm_quantize_e4m3_1x128(x, w, EPS, y=True)
    q, sf, y = q.cpu().numpy(), f64(sf), f64(y)
    floor = np.float64(np.float32(1e-4) / np.float32(448))
    assert np.all(q[0] == 0) and np.all(sf[:, 0] == floor) and np.all(y[0] == 0)
    assert np.all(q[1] == 0) and np.all(sf[:, 1] == floor)
    # inf: mean(h^2) = inf, 1/sqrt = 0, inf * 0 = NaN at its place, 0 elsewhere; the NaN is left out of the scale
    assert q[2, 5] == 0x7F and np.all(np.delete(q[2], 5) == 0) and np.all(sf[:, 2] == floor)
    assert np.all(q[3] == 0x7F) and np.all(np.isnan(y[3]))
    assert abs(y[4, 200] + np.sqrt(K)) <= 0.5 * ulp_bf16(np.sqrt(K)) + 1e-3 and np.count_nonzero(y[4]) == 1
    assert np.all(np.abs(y[5] - 1) <= 2.0 ** -8)


def test_forward_is_the_quantiser_on_its_values():
    """With unit weight and mean(h^2) = 1, eps = 0, the codes and scales are bit for bit those of the 1x128 quantiser."""
    announce("norm against the quantiser")
    rows, K = 300, 1024
    x = device(np.sign(normal(13, (rows, K))) * 1.0, F32)
    x[:, ::2] *= 0.0
    x[:, 1::4] *= float(np.sqrt(3.0))                    # h^2 averages (3 + 1) / 4 = 1 up to rounding: r may be 1 - 2^-24
    w = torch.ones(K, dtype=F32, device="cuda")
    q, sf, _, _ = dg.rmsnorm_quantize_e4m3_1x128(x, w, 0.0)
    h = f64(x)
    ref = h / np.sqrt((h * h).mean(1, keepdims=True))
    check_quantised(f64(q).reshape(rows, -1, 128), f64(sf)[:, :rows].T, ref.reshape(rows, -1, 128),
                    SLACK * np.abs(ref).reshape(rows, -1, 128), False, "unit rows")
    q2, sf2 = dg.quantize_e4m3_1x128(x)
    assert torch.equal(q, q2)
    assert torch.allclose(sf, sf2, rtol=2.0 ** -21, atol=0)


def test_forward_on_another_stream():
    announce("norm on a side stream")
    rows, K = 700, 2048
    w = torch.ones(K, dtype=BF16, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = device(normal(14, (rows, K)), BF16)
        res = device(normal(15, (rows, K)), BF16)
        out = dg.rmsnorm_quantize_e4m3_1x128(x, w, EPS, residual=res, y=True)
    s.synchronize()
    check_forward(x, res, w, out, "fp32", "stream")


# ---------------------------------------------------------------- backward

def reference_backward(dy, h, w, dres, eps=EPS):
    K = h.shape[1]
    v = (h * h).mean(1, keepdims=True) + eps
    g = dy * w
    dot = (g * h).mean(1, keepdims=True)
    dx = g / np.sqrt(v) - h * dot / (v * np.sqrt(v))
    size = np.abs(g) / np.sqrt(v) + np.abs(h) * np.abs(g * h).mean(1, keepdims=True) / (v * np.sqrt(v))
    if dres is not None:
        dx = dx + dres
        size = size + np.abs(dres)
    n = h / np.sqrt(v)
    return dx, size, (dy * n).sum(0), np.abs(dy * n).sum(0)


def check_backward(dy, h, w, dres, dx, dw, where, eps=EPS):
    """dx: SLACK of the terms it is made of; dw: sums of up to some hundred terms in sequence per workgroup and as
    many partial sums after, 2^-16 of the terms' magnitudes."""
    rdx, size, rdw, wsize = reference_backward(f64(dy), f64(h), f64(w), None if dres is None else f64(dres), eps)
    extra = SLACK * size + 2.0 ** -149
    if dx.dtype == BF16:
        check_bf16(dx, rdx, extra, where + " dx")
    else:
        check(f64(dx), rdx, extra, where + " dx")
    check(f64(dw), rdw, 2.0 ** -16 * wsize + 2.0 ** -149, where + " dw")


BWD = [(1, 128), (2, 512), (5, 640), (37, 1024), (333, 2048), (100, 2176), (65, 4096), (9, 7168), (1030, 1536),
       (2100, 896), (3, 8192), (17, 16384), (6, 8320), (4099, 256)]


@pytest.mark.parametrize("rows,K", BWD)
@pytest.mark.parametrize("ht", [BF16, F32])
def test_backward_sizes(rows, K, ht):
    announce(f"norm_bwd rows={rows} K={K} {ht}")
    dy, h = device(normal(20, (rows, K)), BF16), device(2 * normal(21, (rows, K)), ht)
    w, dres = device(1 + 0.3 * normal(22, (K,)), BF16), device(normal(23, (rows, K)), ht)
    dx, dw = dg.rmsnorm_backward(dy, h, w, EPS, dres=dres)
    check_backward(dy, h, w, dres, dx, dw, f"rows={rows} K={K}")
    dx2, dw2 = dg.rmsnorm_backward(dy, h, w, EPS, dres=dres)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2), "another run gives other bits"


@pytest.mark.parametrize("ht", [BF16, F32])
@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("K", [384, 2304])
def test_backward_types_without_dres(ht, yt, wt, K):
    announce(f"norm_bwd types {ht} {yt} {wt} K={K}")
    rows = 50
    dy, h, w = device(normal(24, (rows, K)), yt), device(normal(25, (rows, K)), ht), device(normal(26, (K,)), wt)
    dx, dw = dg.rmsnorm_backward(dy, h, w, EPS)
    check_backward(dy, h, w, None, dx, dw, "types")


@pytest.mark.parametrize("over", ["dres", "h"])
def test_backward_in_place(over):
    announce(f"norm_bwd in place over {over}")
    rows, K = 700, 1280
    dy, h = device(normal(27, (rows, K)), BF16), device(normal(28, (rows, K)), BF16)
    w, dres = device(normal(29, (K,)), F32), device(normal(30, (rows, K)), BF16)
    h0, dres0 = h.clone(), dres.clone()
    dx, dw = dg.rmsnorm_backward(dy, h, w, EPS, dres=dres, dx=dres if over == "dres" else h)
    check_backward(dy, h0, w, dres0, dx, dw, "in place")


def test_backward_no_rows_and_zero_rows_of_h():
    announce("norm_bwd no rows")
    K = 256
    w = torch.ones(K, dtype=BF16, device="cuda")
    e = torch.empty((0, K), dtype=BF16, device="cuda")
    dw = torch.full((K,), 3.0, device="cuda")
    dg.rmsnorm_backward(e, e, w, EPS, dw=dw)
    assert torch.all(dw == 0)
    h = torch.zeros((8, K), dtype=BF16, device="cuda")
    dy = device(normal(31, (8, K)), BF16)
    dx, dw = dg.rmsnorm_backward(dy, h, w, EPS)
    check_backward(dy, h, w, None, dx, dw, "zero rows")


@pytest.mark.parametrize("K", [256, 2048])
def test_backward_against_differences(K):
    """<dx, v> and <dw, u> against central differences of the 64-bit forward pass along random directions."""
    announce(f"norm_bwd differences K={K}")
    rows = 12
    dy, h, w = device(normal(32, (rows, K)), F32), device(normal(33, (rows, K)), F32), device(normal(34, (K,)), F32)
    dx, dw = dg.rmsnorm_backward(dy, h, w, EPS)
    dyn, hn, wn = f64(dy), f64(h), f64(w)

    def loss(hv, wv):
        return float((dyn * (hv / np.sqrt((hv * hv).mean(1, keepdims=True) + EPS) * wv)).sum())

    t = 1e-5                          # truncation ~ t^2, rounding ~ 1e-16 |loss| / t: both below 1e-8 of the sum of terms
    for seed in range(3):
        v, u = normal(40 + seed, (rows, K)).astype(np.float64), normal(50 + seed, (K,)).astype(np.float64)
        num = (loss(hn + t * v, wn) - loss(hn - t * v, wn)) / (2 * t)
        terms = np.abs(f64(dx) * v).sum()
        assert abs(num - (f64(dx) * v).sum()) <= 2.0 ** -16 * terms
        num = (loss(hn, wn + t * u) - loss(hn, wn - t * u)) / (2 * t)
        assert abs(num - (f64(dw) * u).sum()) <= 2.0 ** -16 * np.abs(f64(dw) * u).sum() + 2.0 ** -16
