"""GPU tests of the tokens' way to the experts' rows and back: the sort against
a loop over the pairs, dispatch bit for bit against the oracle's quantisers,
combine and the gradients against 64-bit sums."""
import sys

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_gemm_scaled_amd import binding as dg

from layer_helpers import SLACK, check, check_bf16, f64, normal

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
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
    torch.cuda.empty_cache()


def device(x, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(dtype)


def random_ids(seed, T, k, G, drop=0.1, skew=1.0):
    """Ids with popular experts, some outside [0, G) in every way; an expert may come twice in a token."""
    g = np.random.default_rng(seed)
    p = np.exp(skew * g.standard_normal(G))
    ids = g.choice(G, size=(T, k), p=p / p.sum()).astype(np.int64)
    out = np.array([-1, G, G + 7, -2 ** 31, 2 ** 31 - 1])
    return np.where(g.random((T, k)) < drop, out[g.integers(0, 5, (T, k))], ids).astype(np.int32)


def plan(ids, G, R, cap=0):
    """rows, src, expert, counts, ks of the definition, pair by pair."""
    flat = ids.reshape(-1)
    lists = [np.flatnonzero(flat == e) for e in range(G)]
    rows, src, expert = np.full(flat.size, -1), np.full(R, -1), np.full(R, -1)
    counts, ks, lo = [], [], 0
    for e, pairs in enumerate(lists):
        if cap:
            lo = e * cap
        room = cap or max(0, R - lo)
        kept = pairs[:room]
        rows[kept] = lo + np.arange(kept.size)
        src[lo:lo + kept.size] = kept
        expert[lo:lo + kept.size] = e
        full = -(-pairs.size // 128) * 128
        counts.append(kept.size)
        ks.append(min(full, room))
        lo += full
    return rows.reshape(ids.shape), src, expert, np.array(counts), np.array(ks)


def same(t, want, where):
    assert np.array_equal(t.cpu().numpy().reshape(np.shape(want)), want), where


def sort(ids, G, R=None, cap=0, src=True):
    """The sort on the device: (rows, src)."""
    t = torch.from_numpy(ids).cuda()
    if cap:
        rows, s, _ = dg.moe_sort_masked(t, G, cap, src=src)
    else:
        rows, s, _, _, _ = dg.moe_sort_contiguous(t, G, R, src=src)
    return rows, s


# ---------------------------------------------------------------- sort

# pairs on both sides of a wave, a workgroup's chunk, and the second launch; experts on both sides of a wave and at the most
SORTS = [(0, 1, 3), (1, 1, 1), (1, 8, 64), (7, 9, 5), (63, 1, 2), (64, 1, 2), (65, 1, 65), (511, 2, 64), (512, 2, 1),
         (513, 2, 257), (333, 6, 32), (1000, 3, 1000), (4096, 1, 1024), (2049, 5, 63), (4096, 8, 256), (4097, 8, 128),
         (16384, 8, 64), (9001, 31, 1023)]


@pytest.mark.parametrize("T,k,G", SORTS)
@pytest.mark.parametrize("skew", [0.0, 3.0])
def test_sort(T, k, G, skew):
    announce(f"sort T={T} k={k} G={G} skew={skew}")
    ids = random_ids(T + k + G, T, k, G, skew=skew)
    R = dg.get_moe_rows(T, k, G)
    t = torch.from_numpy(ids).cuda()
    want = plan(ids, G, R)
    got = dg.moe_sort_contiguous(t, G, src=True, counts=True, ks=True)
    for name, a, w in zip(("rows", "src", "m_indices", "counts", "ks"), got, want):
        same(a, w, f"contiguous {name}")
    # too small a workspace, or none: the same plan
    for ws in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):
        again = dg.moe_sort_contiguous(t, G, src=True, counts=True, ks=True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
    for cap in {1, T * k // G + 1, T * k // (2 * G) + 3}:
        w = plan(ids, G, G * cap, cap)
        rows, src, counts = dg.moe_sort_masked(t, G, cap, src=True)
        for name, a, b in zip(("rows", "src", "masked_m"), (rows, src, counts), (w[0], w[1], w[3])):
            same(a, b, f"masked {cap} {name}")


@pytest.mark.parametrize("R", [0, 128, 256, 640, 1024])
def test_sort_into_fewer_rows(R):
    announce(f"sort into {R} rows")
    ids = random_ids(3, 200, 4, 6)
    got = dg.moe_sort_contiguous(torch.from_numpy(ids).cuda(), 6, R, src=True, counts=True, ks=True)
    for a, w in zip(got, plan(ids, 6, R)):
        same(a, w, f"R={R}")


def test_sort_of_no_expert_and_one():
    announce("sort with all pairs dropped, and all of one expert")
    for value in (-1, 5, 0):
        ids = np.full((300, 5), value, np.int32)
        R = dg.get_moe_rows(300, 5, 7)
        got = dg.moe_sort_contiguous(torch.from_numpy(ids).cuda(), 7, src=True, counts=True, ks=True)
        for a, w in zip(got, plan(ids, 7, R)):
            same(a, w, f"value {value}")


def test_sort_writes_its_outputs_only():
    announce("sort guards")
    ids = random_ids(9, 700, 3, 20)
    R = dg.get_moe_rows(700, 3, 20)
    sizes = {"rows": (700, 3), "src": (R,), "m_indices": (R,), "counts": (20,), "ks": (20,)}
    flat = {n: torch.full((int(np.prod(s)) + 8,), 77, dtype=I32, device="cuda") for n, s in sizes.items()}
    out = {n: flat[n][4:-4].view(s) for n, s in sizes.items()}
    dg.moe_sort_contiguous(torch.from_numpy(ids).cuda(), 20, R, **out)
    for (n, t), w in zip(out.items(), plan(ids, 20, R)):
        same(t, w, n)
        assert torch.all(flat[n][:4] == 77) and torch.all(flat[n][-4:] == 77), n


# ---------------------------------------------------------------- dispatch

def quantised(v, scales):
    """Codes [n, K] and scales [n, K/128] of the oracle's 1x128 quantiser (fp32 input)."""
    if v.shape[0] == 0:
        return np.zeros(v.shape, np.uint8), np.zeros((0, v.shape[1] // 128), np.float32)
    q, sf = oracle.quantize_1x128(np.ascontiguousarray(v, np.float32), ue8m0=scales != "fp32")
    return q, sf[:, :v.shape[0]].T


def scales_of(sf, scales, blocks):
    """[.., blocks (words), ld] -> fp32 scales [.., ld, blocks]; the unused bytes of filled words have to be zero."""
    a = sf.cpu().numpy()
    if scales != "ue8m0_packed":
        return np.swapaxes(a, -1, -2)
    w = a.view(np.uint32)
    e = np.stack([(w >> np.uint32(8 * j)) & np.uint32(0xFF) for j in range(4)], -2).reshape(*w.shape[:-2], -1, w.shape[-1])
    assert not e[..., blocks:, :].any()
    return np.swapaxes((e[..., :blocks, :] << np.uint32(23)).view(np.float32), -1, -2)


SENTINEL = {"q": 0xA5, "y": 7.0}


def check_rows(src, pairs_v, q, sf, y, scales, cap, where):
    """pairs_v [N, K] fp32: each pair's values.  Filled rows hold them; the others what the buffers held."""
    K = pairs_v.shape[1]
    live = src >= 0
    v = pairs_v[src[live]]
    if q is not None:
        wq, ws = quantised(v, scales)
        g = q.cpu().numpy().reshape(-1, K)
        assert np.array_equal(g[live], wq), f"{where}: codes"
        assert np.all(g[~live] == SENTINEL["q"]), f"{where}: a row without a pair was written"
        s = scales_of(sf, scales, K // 128)
        s = s[..., :cap, :].reshape(-1, K // 128) if cap else s
        assert np.array_equal(s[live], ws), f"{where}: scales"
        assert not s[~live].any(), f"{where}: a scale without a pair was written"
    if y is not None:
        g = y.view(-1, K)
        lt = torch.from_numpy(live)
        assert torch.equal(g[lt.cuda()].cpu(), torch.from_numpy(v).to(BF16)), f"{where}: bf16 rows"
        assert torch.all(g[~lt.cuda()] == SENTINEL["y"]), f"{where}: a bf16 row without a pair was written"


def check_cols(src, pairs_v, qt, sft, scales, where):
    R, K = qt.shape
    v = np.zeros((R, K), np.float32)
    v[src >= 0] = pairs_v[src[src >= 0]]
    for b in range(R // 128):
        wq, ws = quantised(v[128 * b:128 * b + 128].T, scales)
        assert np.array_equal(qt[128 * b:128 * b + 128].cpu().numpy().T, wq), f"{where}: column codes, block {b}"
        assert np.array_equal(sft[b].cpu().numpy(), ws[:, 0]), f"{where}: column scales, block {b}"


def pair_values(x, w, k):
    """fp32 values of every pair: weight times token, each product rounded once."""
    v = np.repeat(x.float().cpu().numpy(), k, axis=0)
    return v if w is None else (w.cpu().numpy().reshape(-1, 1) * v).astype(np.float32)


def buffers(lead, per, K, scales, y=True):
    ld = (per + 3) // 4 * 4
    words = (K // 128 + 3) // 4 if scales == "ue8m0_packed" else K // 128
    q = torch.full((*lead, per, K), SENTINEL["q"], dtype=torch.uint8, device="cuda")
    sf = torch.zeros((*lead, words, ld), dtype=I32 if scales == "ue8m0_packed" else F32, device="cuda")
    return q, sf, torch.full((*lead, per, K), SENTINEL["y"], dtype=BF16, device="cuda") if y else None


# tokens and widths on both sides of every change of waves per token and chunks per lane
SIZES = [(1, 8, 64, 7168), (1, 1, 1, 128), (5, 2, 3, 640), (130, 4, 8, 1024), (33, 3, 4, 1152), (70, 2, 9, 2176),
         (513, 2, 8, 2176), (520, 3, 5, 4224), (600, 2, 4, 7168), (9, 2, 4, 8320), (3, 2, 2, 16384)]


@pytest.mark.parametrize("T,k,G,K", SIZES)
@pytest.mark.parametrize("scales", ["fp32", "ue8m0", "ue8m0_packed"])
def test_dispatch(T, k, G, K, scales):
    announce(f"dispatch T={T} k={k} G={G} K={K} {scales}")
    ids = random_ids(T + K, T, k, G)
    x = device(normal(T, (T, K)), BF16)
    v = pair_values(x, None, k)
    R = dg.get_moe_rows(T, k, G)
    rows, src = sort(ids, G)
    s = src.cpu().numpy()
    q, sf, y = buffers((), R, K, scales)
    dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, q=q, sf=sf, y=y, scales=scales)
    check_rows(s, v, q, sf, y, scales, 0, "contiguous")
    # by tile, with column scales
    q, sf, y = buffers((), R, K, scales)
    _, _, qt, sft, _ = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, q=q, sf=sf, y=y, qt=True, scales=scales)
    check_rows(s, v, q, sf, y, scales, 0, "contiguous by tile")
    check_cols(s, v, qt, sft, scales, "contiguous")
    cap = T * k // G // 2 + 3                          # odd and even, some pairs without a row
    rows, src = sort(ids, G, cap=cap)
    q, sf, y = buffers((G,), cap, K, scales)
    dg.moe_dispatch_quantize_e4m3_masked(x, rows, G, cap, q=q, sf=sf, y=y, scales=scales)
    check_rows(src.cpu().numpy().reshape(-1), v, q, sf, y, scales, cap, "masked")


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("scales", ["fp32", "ue8m0_packed"])
@pytest.mark.parametrize("T,K", [(37, 384), (40, 1536), (530, 2560), (21, 16384)])
def test_dispatch_with_weights(xt, scales, T, K):
    """Weights of both signs, zero and large among them; strided tokens."""
    announce(f"dispatch with weights {xt} {scales} T={T} K={K}")
    k, G = 3, 5
    ids = random_ids(T, T, k, G)
    full = device(normal(T, (T, K + 64)), xt)
    x = full[:, 64:]
    w = normal(7, (T, k))
    w[::5, 0], w[1::7, 1], w[2::9, 2] = 0.0, 1e30, -1e-30
    w = device(w)
    v = pair_values(x, w, k)
    R = dg.get_moe_rows(T, k, G)
    rows, src = sort(ids, G)
    s = src.cpu().numpy()
    q, sf, y = buffers((), R, K, scales)
    dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, weights=w, q=q, sf=sf, y=y, scales=scales)
    check_rows(s, v, q, sf, y, scales, 0, "by token")
    q, sf, y = buffers((), R, K, scales)
    _, _, qt, sft, _ = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, weights=w, q=q, sf=sf, y=y, qt=True,
                                                                scales=scales)
    check_rows(s, v, q, sf, y, scales, 0, "by tile")
    check_cols(s, v, qt, sft, scales, "by tile")


@pytest.mark.parametrize("xt", [BF16, F32])
def test_dispatch_special_values(xt):
    """NaN, infinities and zeros, in tokens that are dropped and in others, with weights that are such themselves: codes
    and scales as the quantiser's on the fp32 products, by token and by tile."""
    announce("dispatch special values")
    T, k, G, K = 24, 2, 3, 256
    ids = random_ids(5, T, k, G, drop=0.2)
    x = normal(5, (T, K))
    x[0, 3], x[1, 130], x[2], x[3, :128], x[4, 5] = np.nan, np.inf, 0.0, np.nan, -np.inf
    x = device(x, xt)
    w = normal(6, (T, k))
    w[5, 0], w[6, 1], w[1, 0], w[2, 1], w[7] = np.nan, np.inf, 0.0, np.inf, 0.0
    w = device(w)
    rows, src = sort(ids, G)
    R = src.numel()
    for weights in (None, w):
        with np.errstate(invalid="ignore", over="ignore"):
            v = device(pair_values(x, weights, k))
        want_q, want_sf = dg.quantize_e4m3_1x128(v)    # its NaN and infinity rules are tested by themselves
        want_q, want_sf = want_q.cpu().numpy(), want_sf.cpu().numpy().T
        s = src.cpu().numpy()
        live = s >= 0
        for cols in (None, True):
            q, sf, _ = buffers((), R, K, "fp32")
            dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, weights=weights, q=q, sf=sf, qt=cols)
            assert np.array_equal(q.cpu().numpy()[live], want_q[s[live]])
            assert np.array_equal(sf.cpu().numpy().T[live], want_sf[s[live]])
            assert np.all(q.cpu().numpy()[~live] == SENTINEL["q"])
            if cols:                                   # the columns of each 128 rows, through the same quantiser
                full = torch.zeros((R, K), device="cuda")
                full[torch.from_numpy(live).cuda()] = v[torch.from_numpy(s[live]).cuda().long()]
                _, _, qt, sft, _ = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, weights=weights, q=False, qt=True)
                for b in range(R // 128):
                    cq, csf = dg.quantize_e4m3_1x128(full[128 * b:128 * b + 128].t().contiguous())
                    assert torch.equal(qt[128 * b:128 * b + 128].t(), cq) and torch.equal(sft[b], csf[0, :K])


def test_dispatch_column_codes_alone_and_empty():
    announce("dispatch of columns alone, of no tokens, of no rows")
    T, k, G, K = 50, 2, 4, 512
    ids = random_ids(8, T, k, G)
    x = device(normal(8, (T, K)), BF16)
    rows, src = sort(ids, G)
    R = src.numel()
    q, sf, qt, sft, y = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, q=False, qt=True)
    assert q is None and sf is None and y is None
    check_cols(src.cpu().numpy(), pair_values(x, None, k), qt, sft, "fp32", "alone")
    # no tokens: the columns are zeros of the floor's scale
    none, nrows = x[:0], rows[:0]
    nsrc = torch.full((256,), -1, dtype=I32, device="cuda")
    qt = torch.full((256, K), 1, dtype=torch.uint8, device="cuda")
    _, _, qt, sft, _ = dg.moe_dispatch_quantize_e4m3_contiguous(none, nrows, 256, src=nsrc, q=False, qt=qt)
    assert not qt.any() and torch.all(sft == sft[0, 0]) and float(sft[0, 0]) == np.float32(1e-4) / np.float32(448)
    # no rows at all
    dropped = torch.full((T, k), -1, dtype=I32, device="cuda")
    q, sf, _, _, _ = dg.moe_dispatch_quantize_e4m3_contiguous(x, dropped, 0)
    assert q.shape == (0, K)
    dw, *_ = dg.moe_combine_backward_quantize_e4m3_contiguous(x, torch.empty((0, K), dtype=BF16, device="cuda"), dropped,
                                                              dw=torch.full((T, k), 5.0, device="cuda"))
    assert not dw.any()


def test_dispatch_ignores_rows_and_pairs_outside():
    """Row indices at or past the layout, and src of other sizes, count as none (nothing is read or written there)."""
    announce("dispatch of rows outside")
    T, k, K, R = 6, 2, 256, 128
    x = device(normal(9, (T, K)), BF16)
    rows = torch.tensor([[0, 128], [1, -1], [2, 2 ** 31 - 1], [-2 ** 31, 3], [129, 1000], [127, -5]], dtype=I32, device="cuda")
    want = {0: 0, 1: 1, 2: 2, 3: 3, 127: 5}
    q, sf, y = buffers((), R, K, "fp32")
    dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, q=q, sf=sf, y=y)
    src = np.full(R, -1)
    for r, t in want.items():
        src[r] = t * k
    check_rows(src, pair_values(x, None, k), q, sf, y, "fp32", 0, "outside")
    bad = torch.from_numpy(src.astype(np.int32)).cuda()
    bad[5], bad[6], bad[7] = T * k, 2 ** 31 - 1, -7
    _, _, qt, sft, _ = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=bad, q=False, qt=True)
    check_cols(src, pair_values(x, None, k), qt, sft, "fp32", "outside")
    yy = device(normal(10, (R, K)), BF16)
    out = dg.moe_combine(yy, rows)
    ref = np.zeros((T, K))
    for r, t in want.items():
        ref[t] += f64(yy)[r]
    check_bf16(out, ref, 0.0, "combine")


@pytest.mark.parametrize("scales", ["fp32", "ue8m0_packed"])
@pytest.mark.parametrize("T,k,G,K", [(1, 8, 64, 7168), (333, 6, 32, 2048), (5, 1, 2, 128), (70, 3, 4, 4224), (9, 2, 3, 20480)])
def test_dispatch_of_codes(T, k, G, K, scales):
    announce(f"dispatch codes T={T} k={k} G={G} K={K} {scales}")
    ids = random_ids(T + 1, T, k, G)
    x = device(normal(T + 2, (T, K)))
    if scales == "fp32":
        q_in, sf_in = dg.quantize_e4m3_1x128(x)
    else:
        q_in, sf_in = dg.quantize_e4m3_1x128(x, ue8m0=True)
        sf_in = dg.pack_sf_ue8m0(sf_in, -2)
    R = dg.get_moe_rows(T, k, G)
    rows, src = sort(ids, G)
    q, sf, _ = buffers((), R, K, scales, y=False)
    dg.moe_dispatch_e4m3_contiguous(q_in, sf_in, rows, R, q=q, sf=sf)
    v = pair_values(x, None, k)
    check_rows(src.cpu().numpy(), v, q, sf, None, scales, 0, "contiguous")
    cap = T * k // G + 5
    rows, src = sort(ids, G, cap=cap)
    q, sf, _ = buffers((G,), cap, K, scales, y=False)
    dg.moe_dispatch_e4m3_masked(q_in.view(torch.float8_e4m3fn), sf_in, rows, G, cap, q=q, sf=sf)
    check_rows(src.cpu().numpy().reshape(-1), v, q, sf, None, scales, cap, "masked")


# ---------------------------------------------------------------- combine

def combined(y, rows, w, res):
    """out and the sum of the terms' magnitudes in 64 bits."""
    rows = rows.cpu().numpy()
    T, k = rows.shape
    yv = f64(y).reshape(-1, y.shape[-1])
    out = np.zeros((T, yv.shape[1])) if res is None else f64(res).copy()
    size = np.abs(out)
    for j in range(k):
        live = (rows[:, j] >= 0) & (rows[:, j] < yv.shape[0])
        v = yv[rows[live, j]] * (1.0 if w is None else f64(w)[live, j:j + 1])
        out[live] += v
        size[live] += np.abs(v)
    return out, size


@pytest.mark.parametrize("T,k,G,K", [(1, 8, 64, 7168), (1, 1, 1, 8), (64, 8, 64, 7168), (333, 2, 8, 1000), (50, 9, 16, 520),
                                     (1025, 4, 8, 2048), (7, 17, 20, 504), (3, 2, 2, 20480)])
@pytest.mark.parametrize("ot", [BF16, F32])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("res", [False, True])
def test_combine(T, k, G, K, ot, weighted, res):
    announce(f"combine T={T} k={k} G={G} K={K} {ot} weights={weighted} residual={res}")
    ids = random_ids(T + k, T, k, G)
    rows, src = sort(ids, G)
    y = device(normal(T, (src.numel(), K)), BF16)
    y[src < 0] = float("nan")                          # rows that hold no pair are not read into a result
    w = device(normal(3, (T, k))) if weighted else None
    if weighted:
        w[rows < 0] = float("nan")
    r = device(normal(4, (T, K)), ot) if res else None
    flat = torch.full((T * K + 64,), 7.0, dtype=ot, device="cuda")
    out = flat[32:-32].view(T, K)
    ref, size = combined(torch.where((src < 0).unsqueeze(1), 0, y), rows, w, r)
    dg.moe_combine(y, rows, weights=w, residual=r, out=out)
    extra = (k + 2) * U * size + 2.0 ** -149           # k fused or separate additions in sequence
    if ot is BF16:
        check_bf16(out, ref, extra, "out")
    else:
        check(f64(out), ref, extra, "out")
    assert torch.all(flat[:32] == 7) and torch.all(flat[-32:] == 7)
    if res:                                            # in place
        got = dg.moe_combine(y, rows, weights=w, residual=r, out=r)
        assert got is r and torch.equal(r, out)


def test_combine_special_values():
    announce("combine special values")
    y = torch.zeros((128, 8), dtype=BF16, device="cuda")
    y[0], y[1] = float("inf"), 2.0
    rows = torch.tensor([[0, 1], [1, 1], [-1, -1], [1, -1]], dtype=I32, device="cuda")
    w = torch.tensor([[1.0, 1.0], [3.0, -1.0], [5.0, 5.0], [0.5, float("nan")]], device="cuda")
    out = f64(dg.moe_combine(y, rows, weights=w))
    assert np.all(out[0] == np.inf) and np.all(out[1] == 4) and np.all(out[2] == 0) and np.all(out[3] == 1)
    empty = torch.empty((0, 8), dtype=BF16, device="cuda")
    assert dg.moe_combine(y, rows[:0], weights=w[:0]).shape == (0, 8)
    assert not dg.moe_combine(empty, rows).any()
    assert torch.all(dg.moe_combine(empty, rows, residual=torch.ones((4, 8), device="cuda")) == 1)


# ---------------------------------------------------------------- combine's gradient

@pytest.mark.parametrize("T,k,G,K", [(1, 8, 64, 7168), (5, 2, 3, 128), (130, 4, 8, 1024), (333, 2, 8, 2048), (40, 9, 16, 1152),
                                     (513, 3, 8, 2176), (600, 2, 4, 7168), (9, 17, 20, 8320)])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("cols", [False, True])
def test_combine_backward(T, k, G, K, dt, cols):
    announce(f"combine_bwd T={T} k={k} G={G} K={K} {dt} columns={cols}")
    scales = "ue8m0" if T % 2 else "fp32"
    ids = random_ids(T, T, k, G)
    rows, src = sort(ids, G)
    R = src.numel()
    ye = device(normal(T, (R, K)), BF16)
    ye[src < 0] = float("nan")
    w = device(normal(5, (T, k)))
    dout = device(normal(6, (T, K)), dt)
    q, sf, dy = buffers((), R, K, scales)
    flat = torch.full((T * k + 8,), 9.0, device="cuda")
    dw = flat[4:-4].view(T, k)
    got = dg.moe_combine_backward_quantize_e4m3_contiguous(dout, ye, rows, w, src=src if cols else None, dw=dw, dy=dy, q=q,
                                                           sf=sf, qt=True if cols else None, scales=scales)
    s = src.cpu().numpy()
    v = pair_values(dout, w, k)
    check_rows(s, v, q, sf, dy, scales, 0, "rows")
    if cols:
        check_cols(s, v, got[4], got[5], scales, "columns")
    r = rows.cpu().numpy()
    d, e = f64(dout), f64(torch.where((src < 0).unsqueeze(1), 0, ye))
    term = d[:, None, :] * e[np.maximum(r, 0)] * (r >= 0)[:, :, None]
    # 32 fused steps in a lane, 6 across the wave, 16 across waves: below SLACK of the terms
    check(f64(dw), term.sum(2), SLACK * np.abs(term).sum(2), "dw")
    assert np.all(f64(dw)[r < 0] == 0) and torch.all(flat[:4] == 9) and torch.all(flat[-4:] == 9)
    again = dg.moe_combine_backward_quantize_e4m3_contiguous(dout, ye, rows, w, dw=True)
    assert torch.equal(again[0], dw) and again[1] is None and again[2] is None


def test_combine_backward_against_differences():
    """The gradients of <g, combine(y, w, res)> along random directions, in 64 bits (combine is linear in each of its
    inputs: a difference of any length is exact up to rounding)."""
    announce("combine_bwd differences")
    T, k, G, K = 40, 3, 5, 256
    ids = random_ids(2, T, k, G)
    rows, src = sort(ids, G)
    live = (src >= 0).unsqueeze(1)
    y = torch.where(live, device(normal(1, (src.numel(), K)), BF16), 0)
    w, g = device(normal(2, (T, k))), device(normal(3, (T, K)))
    dw, dy, *_ = dg.moe_combine_backward_quantize_e4m3_contiguous(g, y, rows, w, dw=True, dy=True)
    gn = f64(g)
    u, v = device(normal(4, (T, k))), device(normal(5, (src.numel(), K)), BF16)
    base = (gn * combined(y, rows, w, None)[0]).sum()
    terms = np.abs(f64(dw) * f64(u)).sum()
    assert abs((gn * combined(y, rows, w + u, None)[0]).sum() - base - (f64(dw) * f64(u)).sum()) <= 2.0 ** -16 * terms
    step = (gn * combined(v, rows, w, None)[0]).sum()
    # dy is bf16: half a step, 2^-9 of each term
    assert abs(step - (f64(dy) * f64(v)).sum()) <= 2.0 ** -8 * np.abs(f64(dy) * f64(v)).sum()


def test_dispatch_gradient_is_combine():
    """<dispatch(x), d> = <x, combine(d)> with and without weights (exact in 64 bits but for the roundings of each)."""
    announce("dispatch's gradient")
    T, k, G, K = 60, 4, 6, 384
    ids = random_ids(12, T, k, G)
    rows, src = sort(ids, G)
    x, d = device(normal(1, (T, K)), BF16), device(normal(2, (src.numel(), K)), BF16)
    d = torch.where((src >= 0).unsqueeze(1), d, 0)
    for w in (None, device(normal(3, (T, k)))):
        y = torch.zeros((src.numel(), K), dtype=BF16, device="cuda")
        dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, src.numel(), weights=w, y=y)
        dx = dg.moe_combine(d, rows, weights=w, out=torch.empty((T, K), device="cuda"))
        left, right = f64(y) * f64(d), f64(x) * f64(dx)
        assert abs(left.sum() - right.sum()) <= 2.0 ** -8 * np.abs(left).sum() + 2.0 ** -20 * np.abs(right).sum()


# ---------------------------------------------------------------- many choices, few CUs, limits

def test_more_choices_than_lanes():
    """A token with more choices than a wave has lanes, and than a batch of loads holds, in every operator."""
    announce("70 choices")
    T, k, G, K = 5, 70, 100, 384
    ids = random_ids(4, T, k, G)
    rows, src = sort(ids, G)
    same(rows, plan(ids, G, src.numel())[0], "rows")
    s, R = src.cpu().numpy(), src.numel()
    x, w = device(normal(1, (T, K)), BF16), device(normal(2, (T, k)))
    for weights in (None, w):
        v = pair_values(x, weights, k)
        q, sf, y = buffers((), R, K, "fp32")
        dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, weights=weights, q=q, sf=sf, y=y)
        check_rows(s, v, q, sf, y, "fp32", 0, "by token")
    q_in, sf_in = dg.quantize_e4m3_1x128(x.float())
    q, sf, _ = buffers((), R, K, "fp32", y=False)
    dg.moe_dispatch_e4m3_contiguous(q_in, sf_in, rows, R, q=q, sf=sf)
    check_rows(s, pair_values(x, None, k), q, sf, None, "fp32", 0, "codes")
    ye = device(normal(3, (R, K)), BF16)
    ref, size = combined(ye, rows, w, x)
    check_bf16(dg.moe_combine(ye, rows, weights=w, residual=x), ref, (k + 2) * U * size, "combine")
    for cols in (None, True):
        dw, _, _, _, qt, sft = dg.moe_combine_backward_quantize_e4m3_contiguous(x, ye, rows, w, src=src, dw=True, q=False,
                                                                                qt=cols)
        r = rows.cpu().numpy()
        term = f64(x)[:, None, :] * f64(ye)[np.maximum(r, 0)] * (r >= 0)[:, :, None]
        check(f64(dw), term.sum(2), SLACK * np.abs(term).sum(2), "dw")
        if cols:
            check_cols(s, pair_values(x, w, k), qt, sft, "fp32", "columns")


@pytest.mark.parametrize("cus", [1, 5])
def test_few_compute_units(cus):
    """The number of workgroups that a token's choices are dealt to changes no result."""
    announce(f"{cus} CUs")
    T, k, G, K = 9, 8, 12, 2304
    ids = random_ids(6, T, k, G)
    rows, src = sort(ids, G)
    x, w, R = device(normal(1, (T, K)), BF16), device(normal(2, (T, k))), src.numel()
    ye = device(normal(3, (R, K)), BF16)
    want = dg.moe_combine_backward_quantize_e4m3_contiguous(x, ye, rows, w, dw=True, q=True, dy=True)
    try:
        dg.set_num_cus(cus)
        got = dg.moe_combine_backward_quantize_e4m3_contiguous(x, ye, rows, w, dw=True, q=True, dy=True)
        torch.cuda.synchronize()
    finally:
        dg.set_num_cus(0)
    for a, b in zip(got, want):
        assert a is b is None or torch.equal(a, b)


def test_grid_limit():
    """A grid that would reach 2^32 threads is refused; the one below it runs."""
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB of device memory")
    announce("grid limit")
    T = 1 << 26
    y = torch.arange(1, 129, device="cuda").to(BF16).repeat_interleave(8).view(128, 8)
    rows = torch.zeros((T, 1), dtype=I32, device="cuda")
    rows[-5:, 0] = torch.arange(5, dtype=I32, device="cuda")
    with pytest.raises(dg.DGError, match="HIP"):
        dg.moe_combine(y, rows)
    out = dg.moe_combine(y, rows[4:])
    torch.cuda.synchronize()
    assert torch.equal(out[-5:], y[:5]) and bool((out[:-5] == 1).all())
    assert dg.moe_combine(y[:0], rows, out=torch.full((T, 8), 3.0, dtype=BF16, device="cuda")).count_nonzero() == 0


# ---------------------------------------------------------------- streams, graphs, sizes

def run_all(ids, x, w, G, bufs):
    dg.moe_sort_contiguous(ids, G, bufs["R"], rows=bufs["rows"], src=bufs["src"], m_indices=bufs["m"], ks=bufs["ks"],
                           counts=bufs["counts"], workspace=bufs["ws"])
    dg.moe_dispatch_quantize_e4m3_contiguous(x, bufs["rows"], bufs["R"], src=bufs["src"], q=bufs["q"], sf=bufs["sf"],
                                             y=bufs["y"], qt=bufs["qt"], sft=bufs["sft"])
    dg.moe_combine(bufs["y"], bufs["rows"], weights=w, residual=x, out=bufs["out"])
    dg.moe_combine_backward_quantize_e4m3_contiguous(bufs["out"], bufs["y"], bufs["rows"], w, src=bufs["src"], dw=bufs["dw"],
                                                     q=bufs["q2"], sf=bufs["sf2"], qt=bufs["qt2"], sft=bufs["sft2"])


def new_bufs(T, k, G, K):
    R = dg.get_moe_rows(T, k, G)
    z = lambda *s, t=F32: torch.zeros(s, dtype=t, device="cuda")
    u8 = torch.uint8
    return {"R": R, "rows": z(T, k, t=I32), "src": z(R, t=I32), "m": z(R, t=I32), "ks": z(G, t=I32), "counts": z(G, t=I32),
            "ws": z(max(16, dg.get_moe_sort_workspace_size(T, k, G)), t=u8), "q": z(R, K, t=u8), "sf": z(K // 128, R),
            "y": z(R, K, t=BF16), "qt": z(R, K, t=u8), "sft": z(R // 128, K), "out": z(T, K, t=BF16), "dw": z(T, k),
            "q2": z(R, K, t=u8), "sf2": z(K // 128, R), "qt2": z(R, K, t=u8), "sft2": z(R // 128, K)}


@pytest.mark.parametrize("T,k,G,K", [(3, 2, 4, 256), (700, 4, 16, 640), (9000, 4, 8, 128)])
def test_captured_in_a_graph(T, k, G, K):
    """All calls in one graph, replayed with new tokens and ids, between eager calls with buffers of their own."""
    announce(f"graph T={T}")
    ids, x, w = torch.zeros((T, k), dtype=I32, device="cuda"), torch.zeros((T, K), dtype=BF16, device="cuda"), torch.zeros(
        (T, k), device="cuda")
    a, b = new_bufs(T, k, G, K), new_bufs(T, k, G, K)
    run_all(ids, x, w, G, a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_all(ids, x, w, G, a)
    for n in range(3):
        ids.copy_(torch.from_numpy(random_ids(n, T, k, G)))
        x.copy_(device(normal(n, (T, K))))
        w.copy_(device(normal(n + 9, (T, k))))
        for bufs in (a, b):                            # rows without a pair keep what they held: the same in both
            for t in bufs.values():
                if torch.is_tensor(t):
                    t.zero_()
        graph.replay()
        run_all(ids, x, w, G, b)
        torch.cuda.synchronize()
        for name in a:
            if torch.is_tensor(a[name]) and name != "ws":
                assert torch.equal(a[name], b[name]), (n, name)
        same(a["rows"], plan(ids.cpu().numpy(), G, a["R"])[0], "rows")


def test_two_streams_at_once():
    announce("two streams")
    T, k, G, K = 2000, 4, 8, 512
    want, got, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    inputs = []
    for n in range(2):
        ids, x, w = torch.from_numpy(random_ids(n, T, k, G)).cuda(), device(normal(n, (T, K)), BF16), device(normal(n + 5, (T, k)))
        inputs.append((ids, x, w))
        want.append(new_bufs(T, k, G, K))
        got.append(new_bufs(T, k, G, K))
        run_all(ids, x, w, G, want[n])
    torch.cuda.synchronize()
    for _ in range(5):
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                run_all(*inputs[n], G, got[n])
    torch.cuda.synchronize()
    for n in range(2):
        for name in want[n]:
            if torch.is_tensor(want[n][name]) and name != "ws":
                assert torch.equal(want[n][name], got[n][name]), (n, name)


def test_rows_past_31_bits_of_offset():
    """Tensors of more than 2^31 elements and bytes: the last tokens and rows come out as the first."""
    T, k, G, K = 1 << 18, 1, 3, 8320
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    announce("rows past 2^31 elements")
    block = device(normal(1, (128, K)), BF16)
    x = block.repeat(T // 128, 1)
    ids = torch.zeros((T, k), dtype=I32, device="cuda")
    ids[T // 2:] = 2
    rows, src, m, counts, ks = dg.moe_sort_contiguous(ids, G, src=True, counts=True, ks=True)
    assert counts.tolist() == [T // 2, 0, T // 2] and torch.equal(rows.view(-1), torch.arange(T, dtype=I32, device="cuda"))
    R = m.numel()
    q, sf, qt, sft, y = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, q=True, y=True, qt=True)
    wq, wsf = dg.quantize_e4m3_1x128(block.float())
    q1, sf1, _, _, _ = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R)
    assert torch.equal(q, q1) and torch.equal(sf, sf1)
    del q1, sf1
    for lo in (0, T // 2, T - 128):
        assert torch.equal(q[lo:lo + 128], wq) and torch.equal(sf[:, lo:lo + 128], wsf) and torch.equal(y[lo:lo + 128], block)
        assert torch.equal(qt[lo:lo + 128], qt[:128]) and torch.equal(sft[lo // 128], sft[0])
    assert not qt[T:].any()
    codes, csf = dg.moe_dispatch_e4m3_contiguous(q[:T].contiguous(), sf[:, :T].contiguous(), rows, R)
    assert torch.equal(codes[:T], q[:T]) and torch.equal(csf[:, :T], sf[:, :T])
    del q, qt, codes
    w = torch.full((T, k), 2.0, device="cuda")
    out = dg.moe_combine(y, rows, weights=w)
    dw, *_ = dg.moe_combine_backward_quantize_e4m3_contiguous(x, y, rows, w, dw=True)
    for lo in (0, T // 2, T - 128):
        assert torch.equal(out[lo:lo + 128], (2 * block.float()).to(BF16)) and torch.equal(dw[lo:lo + 128], dw[:128])


def test_sort_of_most_pairs():
    """2^26 pairs, the most that the sort takes: every pair once, in order within its expert, behind the segment's start."""
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB of device memory")
    T, k, G = 1 << 23, 8, 37
    announce("sort of 2^26 pairs")
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-1, G, (T, k), generator=g, device="cuda", dtype=I32)
    rows, src, m, counts, ks = dg.moe_sort_contiguous(ids, G, src=True, counts=True, ks=True)
    want = torch.zeros(G, dtype=torch.int64, device="cuda").index_add_(0, ids.view(-1).clamp_min(0).long(),
                                                                       (ids.view(-1) >= 0).long())
    assert torch.equal(counts.long(), want) and torch.equal(ks.long(), (want + 127) // 128 * 128)
    flat, live = rows.view(-1), ids.view(-1) >= 0
    assert torch.equal(flat >= 0, live)
    pair = live.nonzero().flatten()
    at = flat[pair].long()
    assert torch.equal(src[at].long(), pair) and torch.equal(m[at], ids.view(-1)[pair])
    assert int((src >= 0).sum()) == pair.numel() and torch.equal(src >= 0, m >= 0)
    start = (ks.long().cumsum(0) - ks)[ids.view(-1)[pair].long()]
    assert bool((at >= start).all()) and bool((at - start < want[ids.view(-1)[pair].long()]).all())
    for e in range(G):                                 # in pair order
        s = src[m == e]
        assert bool((s[1:] > s[:-1]).all())


# ---------------------------------------------------------------- the binding's refusals

@pytest.fixture(params=["native", "python"])
def checks(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(dg, "_native_addresses", lambda *_: None)
    else:
        assert dg._native_addresses.__name__ == "addresses", "the native checks are not built"


def refused(error, match, f, *args, **kw):
    with pytest.raises(error, match=match):
        f(*args, **kw)


def test_refusals_of_device_tensors(checks):
    announce("binding refusals")
    x = torch.zeros((4, 256), dtype=BF16, device="cuda")
    ids = torch.zeros((4, 2), dtype=I32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    f = dg.moe_sort_contiguous
    rows, src, *_ = f(ids, 3, src=True)
    R = src.numel()
    refused(TypeError, "ids", f, ids.long(), 3)
    refused(ValueError, "ids", f, ids.t(), 3)
    refused(ValueError, "rows", f, ids, 3, rows=rows[:2])
    refused(ValueError, "m_indices", f, ids, 3, m_indices=src[:128])
    refused(TypeError, "ks", f, ids, 3, ks=torch.zeros(3, device="cuda"))
    refused(ValueError, "src", f, ids, 3, src=src.cpu())
    refused(dg.DGError, "SHAPE", f, ids, 0)
    refused(dg.DGError, "SHAPE", f, ids, 3, 100)
    refused(dg.DGError, "SHAPE", dg.moe_sort_masked, ids, 3, 0)
    refused(ValueError, "masked_m", dg.moe_sort_masked, ids, 3, 4, masked_m=src)
    f = dg.moe_dispatch_quantize_e4m3_contiguous
    f(x, rows, R)
    refused(TypeError, "x", f, x.half(), rows, R)
    refused(ValueError, "rows", f, x, rows[:2], R)
    refused(TypeError, "weights", f, x, rows, R, weights=w.double())
    refused(ValueError, "sf", f, x, rows, R, q=True, sf=torch.zeros((2, 4), device="cuda"))
    refused(TypeError, "sf", f, x, rows, R, q=True, sf=torch.zeros((1, R), device="cuda"), scales="ue8m0_packed")
    refused(dg.DGError, "NULL", f, x, rows, R, qt=True)
    refused(dg.DGError, "SHAPE", f, x[:, :192], rows, R)
    refused(dg.DGError, "SHAPE", f, x, rows, 100)
    refused(dg.DGError, "ALIGN", f, torch.zeros((4, 257), dtype=BF16, device="cuda")[:, 1:], rows, R)
    f = dg.moe_dispatch_e4m3_contiguous
    codes, sf = torch.zeros((4, 256), dtype=torch.uint8, device="cuda"), torch.ones((2, 4), device="cuda")
    f(codes, sf, rows, R)
    refused(TypeError, "q_in", f, x, sf, rows, R)
    refused(ValueError, "sf_in", f, codes, sf[:1], rows, R)
    refused(ValueError, "sf_in", f, codes, torch.ones((2, 8), device="cuda")[:, ::2], rows, R)
    f = dg.moe_combine
    y = torch.zeros((R, 256), dtype=BF16, device="cuda")
    f(y, rows)
    refused(TypeError, "y", f, y.float(), rows)
    refused(ValueError, "weights", f, y, rows, weights=w[:, :1])
    refused(TypeError, "residual", f, y, rows, residual=x, out=torch.zeros((4, 256), device="cuda"))
    refused(TypeError, "out", f, y, rows, out=torch.zeros((4, 256), dtype=torch.float16, device="cuda"))
    refused(ValueError, "out", f, y, rows, out=x[:2])
    f = dg.moe_combine_backward_quantize_e4m3_contiguous
    f(x, y, rows, w, dw=True)
    refused(ValueError, "dw", f, x, y, rows, w, dw=torch.zeros(8, device="cuda"))
    refused(ValueError, "ye", f, x, y[:, :128].contiguous(), rows, w, dw=True)
    f = dg.layernorm_quantize_e4m3_1x128
    wn = torch.ones(256, dtype=BF16, device="cuda")
    f(x, wn, wn)
    refused(TypeError, "bias", f, x, wn, wn.float())
    refused(ValueError, "weight", f, x, wn[:128])
    refused(ValueError, "residual_out", f, x, wn, residual_out=x)
    refused(dg.DGError, "SHAPE", f, x[:, :192], wn[:192])
    f = dg.layernorm_backward
    f(x, x, wn)
    refused(ValueError, "db", f, x, x, wn, db=torch.zeros(128, device="cuda"))
    refused(TypeError, "dres", f, x, x, wn, dres=x.float())
    big = torch.zeros((64, 256), dtype=BF16, device="cuda")
    refused(dg.DGError, "NULL", f, big, big, wn, workspace=None)
    refused(dg.DGError, "ARG", f, big, big, wn, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
