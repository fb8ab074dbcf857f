"""GPU tests of the layer norm with residual and E4M3 output, and of its
gradient, against 64-bit references (bars: layer_helpers, and below)."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

from layer_helpers import SLACK, check, check_bf16, check_quantised, f64, normal, unpack_words

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
U = 2.0 ** -24


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


def reference(h, w, b, eps=EPS):
    """y, and the size of the terms that it is made of: an fp32 mean is off by SLACK of mean |h| at most (sums of 32
    terms in a lane and 10 steps across lanes and waves), h itself by U."""
    m = h.mean(1, keepdims=True)
    v = ((h - m) ** 2).mean(1, keepdims=True)
    r = 1 / np.sqrt(v + eps)
    y = (h - m) * r * w + b
    size = np.abs(w) * r * (np.abs(h) + np.abs(h).mean(1, keepdims=True)) + np.abs(b)
    return y, size


def check_forward(x, res, w, b, out, scales, where, eps=EPS):
    q, sf, ro, y = out
    rows, K = x.shape
    h = f64(x) + (f64(res) if res is not None else 0.0)
    ref, size = reference(h, 1.0 if w is None else f64(w), 0.0 if b is None else f64(b), eps)
    extra = SLACK * size + 2.0 ** -149
    if res is not None:
        assert torch.equal(ro, (x.float() + res.float()).to(res.dtype)), f"{where}: residual_out is not the rounded sum"
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
    announce(f"ln rows={rows} K={K} {scales}")
    x, res = device(normal(rows + K, (rows, K)), BF16), device(3 * normal(rows + K, (rows, K), 1) + 1, BF16)
    w, b = device(1 + 0.3 * normal(K, (K,), 2), BF16), device(0.5 * normal(K, (K,), 3), BF16)
    out = dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, residual=res, y=True, scales=scales)
    check_forward(x, res, w, b, out, scales, f"rows={rows} K={K}")


@pytest.mark.parametrize("K", [8, 16, 72, 504, 520, 1000, 1032, 2040, 2056, 4104, 8184, 8200, 16376])
@pytest.mark.parametrize("rows", [1, 6, 600])
def test_forward_widths_off_the_block(K, rows):
    """Without codes a row is any multiple of 8 wide; nothing is written past it."""
    announce(f"ln rows={rows} K={K} without codes")
    x, w, b = device(normal(K, (rows, K)), BF16), device(normal(K, (K,), 2), F32), device(normal(K, (K,), 3), F32)
    flat = torch.full((rows * K + 64,), 7.0, dtype=BF16, device="cuda")
    y = flat[32:32 + rows * K].view(rows, K)
    out = dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, y=y, q=False)
    check_forward(x, None, w, b, out, "fp32", f"K={K}")
    assert torch.all(flat[:32] == 7) and torch.all(flat[-32:] == 7)


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("rt", [None, BF16, F32])
@pytest.mark.parametrize("wt", [None, BF16, F32])
@pytest.mark.parametrize("rows", [6, 2049])
def test_forward_types(xt, rt, wt, rows):
    K = 640
    announce(f"ln types {xt} {rt} {wt} rows={rows}")
    x = device(normal(5, (rows, K)), xt)
    res = None if rt is None else device(normal(6, (rows, K)), rt)
    w = None if wt is None else device(normal(7, (K,)), wt)
    b = None if wt is None else device(normal(8, (K,)), wt)
    out = dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, residual=res, y=True, scales="ue8m0")
    check_forward(x, res, w, b, out, "ue8m0", "types")


@pytest.mark.parametrize("which", ["weight", "bias"])
def test_forward_one_of_weight_and_bias(which):
    announce(f"ln with {which} alone")
    x, v = device(normal(5, (9, 384)), BF16), device(normal(7, (384,)), BF16)
    w, b = (v, None) if which == "weight" else (None, v)
    check_forward(x, None, w, b, dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, y=True), "fp32", which)


@pytest.mark.parametrize("rows", [1, 9, 2100])
def test_forward_column_range_of_a_wider_matrix(rows):
    announce(f"ln pitch rows={rows}")
    full = device(normal(8, (rows, 2112)), BF16)
    w, b = device(normal(9, (512,)), BF16), device(normal(10, (512,)), BF16)
    x = full[:, 1536:2048]
    out = dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, y=True)
    check_forward(x, None, w, b, out, "fp32", "column range")


@pytest.mark.parametrize("rows,K", [(4, 7168), (600, 2048), (2500, 1024)])
def test_forward_in_place_and_guards(rows, K):
    """residual_out over the residual; nothing is written outside the outputs, and scales past the rows stay."""
    announce(f"ln in place rows={rows} K={K}")
    x, w, b = device(normal(10, (rows, K)), BF16), device(normal(11, (K,)), BF16), device(normal(13, (K,)), BF16)
    pad = 64
    flat = torch.full((rows * K + 2 * pad,), 7.0, dtype=BF16, device="cuda")
    res = flat[pad:pad + rows * K].view(rows, K)
    res.copy_(device(normal(12, (rows, K)), BF16))
    before = res.clone()
    qflat = torch.full((rows * K + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    q = qflat[pad:pad + rows * K].view(rows, K)
    ld = (rows + 3) // 4 * 4 + 8
    sf = torch.full((K // 128 + 1, ld), -5.0, dtype=F32, device="cuda")
    out = dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, residual=res, residual_out=res, q=q, sf=sf[:-1])
    check_forward(x, before, w, b, out, "fp32", "in place")
    assert torch.all(flat[:pad] == 7) and torch.all(flat[-pad:] == 7)
    assert torch.all(qflat[:pad] == 0xA5) and torch.all(qflat[-pad:] == 0xA5)
    assert torch.all(sf[:, rows:] == -5) and torch.all(sf[-1] == -5)


@pytest.mark.parametrize("K", [512, 2048, 7168, 16384])
@pytest.mark.parametrize("mean", [1e3, -3e4])
def test_forward_mean_far_from_zero(K, mean):
    """A mean of a thousand spreads and more: fp32 rows, whose values hold the spread to 2^-24 |mean|.  mean(h^2) -
    mean(h)^2 would lose all of it; the squared differences do not."""
    announce(f"ln mean={mean} K={K}")
    x = device(normal(17, (20, K)) + mean, F32)
    out = dg.layernorm_quantize_e4m3_1x128(x, None, None, EPS, y=True)
    # the mean: K equal terms in 32 additions of a lane and 10 across, each within U of the running sum: 42 U |mean|
    # at the outside, a quarter of SLACK |mean|; size holds 2 |mean| r
    check_forward(x, None, None, None, out, "fp32", "mean")


def test_forward_zero_rows_and_special_values():
    announce("ln special values")
    K = 512
    w, b = torch.ones(K, dtype=BF16, device="cuda"), torch.full((K,), 0.5, dtype=BF16, device="cuda")
    empty = torch.empty((0, K), dtype=BF16, device="cuda")
    q, sf, ro, y = dg.layernorm_quantize_e4m3_1x128(empty, w, b, EPS, residual=empty, y=True)
    assert q.shape == (0, K) and y.shape == (0, K)
    x = torch.full((5, K), 3.25, dtype=F32, device="cuda")
    x[1] = 1e-30
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4, 200] = 4.25
    q, sf, _, y = dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, y=True)
    q, sf, y = q.cpu().numpy(), f64(sf), f64(y)
    # equal values: no spread, the bias alone (codes of 0.5 over 0.5 / 448 are 448)
    for row in (0, 1):
        assert np.all(y[row] == 0.5) and np.all(q[row] == 0x7E)
    # a mean that is infinite or no number takes the row with it: inf - inf, and NaN is left out of the block's maximum
    for row in (2, 3):
        assert np.all(np.isnan(y[row])) and np.all(q[row] == 0x7F)
        assert np.all(sf[:, row] == np.float64(np.float32(1e-4) / np.float32(448)))
    want = (np.where(np.arange(K) == 200, 1.0, 0.0) - 1 / K) / np.sqrt((1 / K) * (1 - 1 / K) + EPS) + 0.5
    assert np.all(np.abs(y[4] - want) <= 2.0 ** -8 * np.abs(want))


def test_forward_on_another_stream():
    announce("ln on a side stream")
    rows, K = 700, 2048
    w = torch.ones(K, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = device(normal(14, (rows, K)), BF16)
        res = device(normal(15, (rows, K)), BF16)
        out = dg.layernorm_quantize_e4m3_1x128(x, w, w, EPS, residual=res, y=True)
        dx, dw, db = dg.layernorm_backward(x, out[2], w, EPS)
    s.synchronize()
    check_forward(x, res, w, w, out, "fp32", "stream")
    check_backward(x, out[2], w, None, dx, dw, db, "stream")


# one wave a row (four rows per workgroup), four and sixteen: past 2^32 threads each
@pytest.mark.parametrize("rows,K", [((1 << 26) + 5, 8), ((1 << 24) + 3, 1032), ((1 << 22) + 1, 8200)])
def test_more_rows_than_a_grid(rows, K):
    if torch.cuda.mem_get_info()[0] < 5 * rows * K + (1 << 30):
        pytest.skip("needs more device memory")
    announce(f"ln of {rows} x {K}")
    block = device(normal(K, (1 << 12, K)), BF16)
    _, _, _, want = dg.layernorm_quantize_e4m3_1x128(block, y=True, q=False)
    x = torch.empty((rows, K), dtype=BF16, device="cuda")
    whole = rows >> 12 << 12
    x[:whole].view(-1, 1 << 12, K).copy_(block.expand(whole >> 12, 1 << 12, K))
    x[whole:] = block[:rows - whole]
    y = dg.layernorm_quantize_e4m3_1x128(x, y=True, q=False)[3]
    del x
    torch.cuda.synchronize()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for r in range(0, rows, 1 << 20):
        part = y[r:r + (1 << 20)]
        n = part.shape[0] >> 12
        differ += (part[:n << 12].view(n, 1 << 12, K) != want).any()
        differ += (part[n << 12:] != want[:part.shape[0] - (n << 12)]).any()
    assert int(differ) == 0
    del y
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- backward

def reference_backward(dy, h, w, dres, eps=EPS):
    """dx, dw, db and what the fp32 arithmetic may be off: m by SLACK mean |h|, so n = (h - m) r by en, and each mean and
    product by SLACK of its terms; dw and db are sums over the rows in a fixed order, (rows + 64) U of their terms."""
    rows, K = h.shape
    m = h.mean(1, keepdims=True)
    d = h - m
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    n = d * r
    g = dy * w
    mean = lambda a: a.mean(1, keepdims=True)
    dx = r * (g - mean(g) - n * mean(g * n))
    en = SLACK * (np.abs(n) + r * (np.abs(h) + mean(np.abs(h))))
    gc = np.abs(g) + mean(np.abs(g))
    edx = r * (SLACK * (gc + np.abs(n) * mean(gc * np.abs(n))) + en * mean(gc * np.abs(n)) + np.abs(n) * mean(gc * en))
    if dres is not None:
        dx = dx + dres
        edx = edx + SLACK * np.abs(dres)
    deep = (rows + 64) * U
    edw = deep * np.abs(dy * n).sum(0) + (np.abs(dy) * en).sum(0)
    return dx, edx, (dy * n).sum(0), edw, dy.sum(0), deep * np.abs(dy).sum(0)


def check_backward(dy, h, w, dres, dx, dw, db, where, eps=EPS):
    ref = reference_backward(f64(dy), f64(h), 1.0 if w is None else f64(w), None if dres is None else f64(dres), eps)
    tiny = 2.0 ** -149
    if dx.dtype == BF16:
        check_bf16(dx, ref[0], ref[1] + tiny, where + " dx")
    else:
        check(f64(dx), ref[0], ref[1] + tiny, where + " dx")
    if dw is not None:
        check(f64(dw), ref[2], ref[3] + tiny, where + " dw")
    if db is not None:
        check(f64(db), ref[4], ref[5] + tiny, where + " db")


BWD = [(1, 8), (1, 128), (2, 512), (5, 640), (37, 1024), (333, 2048), (100, 2176), (65, 4096), (9, 7168), (1030, 1536),
       (2100, 896), (3, 8192), (17, 16384), (6, 8320), (4099, 256), (300, 504), (70, 1000), (1, 2040), (11, 8200), (9, 16376)]


@pytest.mark.parametrize("rows,K", BWD)
@pytest.mark.parametrize("ht", [BF16, F32])
def test_backward_sizes(rows, K, ht):
    announce(f"ln_bwd rows={rows} K={K} {ht}")
    dy, h = device(normal(20, (rows, K)), BF16), device(2 * normal(21, (rows, K)) + 1, ht)
    w, dres = device(1 + 0.3 * normal(22, (K,)), BF16), device(normal(23, (rows, K)), ht)
    guard = torch.full((2, K + 64), 9.0, device="cuda")
    dw, db = guard[0, 32:32 + K], guard[1, 32:32 + K]
    dx, _, _ = dg.layernorm_backward(dy, h, w, EPS, dres=dres, dw=dw, db=db)
    check_backward(dy, h, w, dres, dx, dw, db, f"rows={rows} K={K}")
    assert torch.all(guard[:, :32] == 9) and torch.all(guard[:, 32 + K:] == 9)
    dx2, dw2, db2 = dg.layernorm_backward(dy, h, w, EPS, dres=dres)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2), "another run gives other bits"


@pytest.mark.parametrize("ht", [BF16, F32])
@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("wt", [None, BF16, F32])
@pytest.mark.parametrize("K", [384, 2304, 8192])
def test_backward_types_without_dres(ht, yt, wt, K):
    announce(f"ln_bwd types {ht} {yt} {wt} K={K}")
    rows = 50
    dy, h = device(normal(24, (rows, K)), yt), device(normal(25, (rows, K)), ht)
    w = None if wt is None else device(normal(26, (K,)), wt)
    check_backward(dy, h, w, None, *dg.layernorm_backward(dy, h, w, EPS), "types")


@pytest.mark.parametrize("rows,K", [(3, 256), (300, 1024)])
def test_backward_optional_outputs(rows, K):
    announce(f"ln_bwd optional outputs rows={rows}")
    dy, h, w = device(normal(27, (rows, K)), BF16), device(normal(28, (rows, K)), BF16), device(normal(29, (K,)), F32)
    want = dg.layernorm_backward(dy, h, w, EPS)
    for dw in (None, False):
        for db in (None, False):
            got = dg.layernorm_backward(dy, h, w, EPS, dw=dw, db=db)
            assert torch.equal(got[0], want[0])
            assert got[1] is None if dw is False else torch.equal(got[1], want[1])
            assert got[2] is None if db is False else torch.equal(got[2], want[2])
    # neither: no workspace is needed
    assert torch.equal(dg.layernorm_backward(dy, h, w, EPS, dw=False, db=False, workspace=None)[0], want[0])


@pytest.mark.parametrize("cus", [1, 3])
@pytest.mark.parametrize("rows,K", [(50, 512), (41, 1032), (37, 2048), (30, 4096), (23, 7168), (9, 16384)])
def test_backward_many_rows_per_workgroup(rows, K, cus):
    """A workgroup's run of rows: even and odd numbers of them, more than it takes side by side."""
    announce(f"ln_bwd rows={rows} K={K} on {cus} CUs")
    dy, h = device(normal(20, (rows, K)), BF16), device(2 * normal(21, (rows, K)) + 1, F32)
    w = device(1 + 0.3 * normal(22, (K,)), BF16)
    try:
        dg.set_num_cus(cus)
        out = dg.layernorm_backward(dy, h, w, EPS)
        torch.cuda.synchronize()
    finally:
        dg.set_num_cus(0)
    check_backward(dy, h, w, None, *out, "few CUs")


@pytest.mark.parametrize("over", ["dres", "h"])
def test_backward_in_place(over):
    announce(f"ln_bwd in place over {over}")
    rows, K = 700, 1280
    dy, h = device(normal(27, (rows, K)), BF16), device(normal(28, (rows, K)), BF16)
    w, dres = device(normal(29, (K,)), F32), device(normal(30, (rows, K)), BF16)
    h0, dres0 = h.clone(), dres.clone()
    out = dg.layernorm_backward(dy, h, w, EPS, dres=dres, dx=dres if over == "dres" else h)
    check_backward(dy, h0, w, dres0, *out, "in place")


def test_backward_no_rows_and_equal_values():
    announce("ln_bwd no rows")
    K = 264
    w = torch.ones(K, dtype=BF16, device="cuda")
    e = torch.empty((0, K), dtype=BF16, device="cuda")
    dw, db = torch.full((K,), 3.0, device="cuda"), torch.full((K,), 3.0, device="cuda")
    dg.layernorm_backward(e, e, w, EPS, dw=dw, db=db)
    assert torch.all(dw == 0) and torch.all(db == 0)
    h = torch.full((8, K), 2.5, dtype=BF16, device="cuda")
    dy = device(normal(31, (8, K)), BF16)
    check_backward(dy, h, w, None, *dg.layernorm_backward(dy, h, w, EPS), "equal values")


@pytest.mark.parametrize("K", [256, 2048])
def test_backward_against_differences(K):
    """<dx, v>, <dw, u> and <db, u> against central differences of the 64-bit forward pass along random directions."""
    announce(f"ln_bwd differences K={K}")
    rows = 12
    dy, h, w = device(normal(32, (rows, K)), F32), device(normal(33, (rows, K)), F32), device(normal(34, (K,)), F32)
    dx, dw, db = dg.layernorm_backward(dy, h, w, EPS)
    dyn, hn, wn, zero = f64(dy), f64(h), f64(w), np.zeros(K)

    def loss(hv, wv, bv):
        return float((dyn * reference(hv, wv, bv)[0]).sum())

    t = 1e-5                          # truncation ~ t^2, rounding ~ 1e-16 |loss| / t: both below 1e-8 of the sum of terms
    for seed in range(3):
        v, u = normal(40 + seed, (rows, K)).astype(np.float64), normal(50 + seed, (K,)).astype(np.float64)
        for got, up, down in ((f64(dx) * v, (hn + t * v, wn, zero), (hn - t * v, wn, zero)),
                              (f64(dw) * u, (hn, wn + t * u, zero), (hn, wn - t * u, zero)),
                              (f64(db) * u, (hn, wn, t * u), (hn, wn, -t * u))):
            num = (loss(*up) - loss(*down)) / (2 * t)
            assert abs(num - got.sum()) <= 2.0 ** -16 * np.abs(got).sum()


@pytest.mark.parametrize("rows", [3, 700])
def test_captured_in_a_graph(rows):
    """Forward and backward replayed with new inputs, between eager calls of other sizes."""
    announce(f"ln in a graph rows={rows}")
    K = 1536
    x, res = torch.zeros((rows, K), dtype=BF16, device="cuda"), torch.zeros((rows, K), dtype=BF16, device="cuda")
    w, b = device(normal(60, (K,)), BF16), device(normal(61, (K,)), BF16)
    ws = torch.empty(max(1, dg.get_layernorm_backward_workspace_size(rows, K)), dtype=torch.uint8, device="cuda")
    outs = {"q": torch.zeros((rows, K), dtype=torch.uint8, device="cuda"), "y": torch.zeros_like(x),
            "sf": torch.zeros((K // 128, (rows + 3) // 4 * 4), device="cuda"), "residual_out": torch.zeros_like(x)}
    dx, dw, db = torch.zeros_like(x), torch.zeros(K, device="cuda"), torch.zeros(K, device="cuda")

    def step():
        dg.layernorm_quantize_e4m3_1x128(x, w, b, EPS, residual=res, **outs)
        dg.layernorm_backward(outs["y"], outs["residual_out"], w, EPS, dx=dx, dw=dw, db=db, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.copy_(device(normal(62 + k, (rows, K))))
        res.copy_(device(normal(70 + k, (rows, K))))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*outs.values(), dx, dw, db)]
        dg.layernorm_backward(x, x, w, EPS)            # eager work of its own between the replays
        step()
        torch.cuda.synchronize()
        for a, c in zip(got, (*outs.values(), dx, dw, db)):
            assert torch.equal(a, c)
