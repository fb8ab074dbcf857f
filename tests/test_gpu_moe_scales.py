"""GPU tests of the scales that the dispatches and the layer norm write into
buffers that hold something already, and of blocks that hold infinities and
NaN in every scale format."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg

from layer_helpers import normal

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FILL = 0x5A5A5A5A             # as a word; as fp32 1.5e16, a scale that nothing here has
FORMS = ["fp32", "ue8m0", "ue8m0_packed"]


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


def quantise(v, scales):
    """The 1x128 quantiser's codes and scales [blocks (words), rows] as int32 words."""
    q, sf = dg.quantize_e4m3_1x128(v.contiguous(), ue8m0=scales != "fp32")
    if scales == "ue8m0_packed":
        sf = dg.pack_sf_ue8m0(sf, -2)
    return q, sf[:, :v.shape[0]].contiguous().view(I32)


def filled(scales, *shape):
    words = torch.full(shape, FILL, dtype=I32, device="cuda")
    return words if scales == "ue8m0_packed" else words.view(F32)


def sf_rows(scales, K):
    return (K // 128 + 3) // 4 if scales == "ue8m0_packed" else K // 128


def ids_of(seed, T, k, G):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.integers(-1, G + 1, (T, k)).astype(np.int32)).cuda()


def check_scales(sf, want, live, src, k, where):
    """sf [words, ld]: the words of held rows are the quantiser's (bytes of blocks past K among them: 0), all others as
    they were."""
    w = sf.view(I32)
    held = live.nonzero().flatten()
    assert torch.equal(w[:, held], want[:, (src[held] // k).long()]), f"{where}: a held row's scales"
    other = torch.ones(w.shape[1], dtype=torch.bool, device="cuda")
    other[held] = False
    assert bool((w[:, other] == FILL).all()), f"{where}: scales of a row without a pair were written"


# blocks of a row on both sides of a whole number of words, and of every change of waves per token
@pytest.mark.parametrize("T,K", [(5, 128), (37, 640), (70, 896), (9, 1024), (40, 1408), (33, 2304), (520, 4736), (6, 7168),
                                 (3, 8448), (2, 16384)])
@pytest.mark.parametrize("scales", FORMS)
def test_dispatch_into_used_scale_buffers(T, K, scales):
    announce(f"dispatch into used buffers T={T} K={K} {scales}")
    k, G = 3, 5
    ids = ids_of(T + K, T, k, G)
    x = device(normal(T, (T, K)), BF16)
    want_q, want = quantise(x.float(), scales)
    rows, src, *_ = dg.moe_sort_contiguous(ids, G, src=True)
    R, n = src.numel(), sf_rows(scales, K)
    for cols in (None, True):
        sf, q = filled(scales, n, R), torch.full((R, K), 0xA5, dtype=torch.uint8, device="cuda")
        dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, q=q, sf=sf, qt=cols, scales=scales)
        check_scales(sf, want, src >= 0, src, k, f"contiguous, columns {cols}")
        held = src >= 0
        assert torch.equal(q[held], want_q[(src[held] // k).long()]) and bool((q[~held] == 0xA5).all())
    sft = torch.full((R // 128, K), 7.0, device="cuda")
    dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, q=False, qt=True, sft=sft, scales=scales)
    assert not bool((sft == 7).any())                  # written entirely
    if scales != "ue8m0":                              # codes: the formats that a row of codes has
        padded = torch.zeros(n, (T + 3) // 4 * 4, dtype=I32, device="cuda")
        padded[:, :T] = want
        sf = filled(scales, n, R)
        dg.moe_dispatch_e4m3_contiguous(want_q, padded if scales == "ue8m0_packed" else padded.view(F32), rows, R, sf=sf)
        check_scales(sf, want, src >= 0, src, k, "codes")
    # masked: the columns between M_cap and the pitch belong to no row
    cap = T * k // G // 2 + 2
    cap += cap % 4 == 0
    ld = (cap + 3) // 4 * 4
    rows, src, _ = dg.moe_sort_masked(ids, G, cap, src=True)
    at = torch.full((G, ld), -1, dtype=I32, device="cuda")
    at[:, :cap] = src
    flat = at.view(-1)
    sf = filled(scales, G, n, ld)
    dg.moe_dispatch_quantize_e4m3_masked(x, rows, G, cap, sf=sf, q=torch.zeros((G, cap, K), dtype=torch.uint8, device="cuda"),
                                         scales=scales)
    check_scales(sf.transpose(0, 1).reshape(n, G * ld), want, flat >= 0, flat, k, "masked")
    if scales != "ue8m0":
        sf = filled(scales, G, n, ld)
        dg.moe_dispatch_e4m3_masked(want_q, padded if scales == "ue8m0_packed" else padded.view(F32), rows, G, cap, sf=sf)
        check_scales(sf.transpose(0, 1).reshape(n, G * ld), want, flat >= 0, flat, k, "masked codes")


@pytest.mark.parametrize("rows,K", [(1, 128), (5, 640), (37, 896), (9, 1408), (600, 2304), (6, 7168), (2, 16384)])
@pytest.mark.parametrize("scales", FORMS)
def test_layernorm_into_used_scale_buffers(rows, K, scales):
    announce(f"ln into used buffers rows={rows} K={K} {scales}")
    x = device(normal(rows, (rows, K)), F32)
    ld = (rows + 3) // 4 * 4 + 4
    clean = torch.zeros((sf_rows(scales, K), ld), dtype=I32 if scales == "ue8m0_packed" else F32, device="cuda")
    q0, *_ = dg.layernorm_quantize_e4m3_1x128(x, sf=clean, scales=scales)
    used = filled(scales, *clean.shape)
    q1, *_ = dg.layernorm_quantize_e4m3_1x128(x, sf=used, scales=scales)
    assert torch.equal(q0, q1)
    assert torch.equal(used.view(I32)[:, :rows], clean.view(I32)[:, :rows])
    assert bool((used.view(I32)[:, rows:] == FILL).all())


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("scales", FORMS)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("K", [256, 640, 2176])
def test_special_values_in_every_format(xt, scales, weighted, K):
    """NaN, infinities, zeros and numbers whose products overflow or vanish: codes and scales are the quantiser's on the
    fp32 products, by token and by tile, along rows and along columns."""
    announce(f"special values {xt} {scales} weighted={weighted} K={K}")
    T, k, G = 30, 2, 3
    ids = ids_of(5, T, k, G)
    x = normal(5, (T, K))
    x[0, 3], x[1, 130], x[2], x[3, :128], x[4, 5] = np.nan, np.inf, 0.0, np.nan, -np.inf
    x[8, ::2], x[9], x[10, 7], x[11] = 3e38, 1e-38, 3e38, -0.0
    x = device(x, xt)
    w = None
    if weighted:
        w = normal(6, (T, k))
        w[5, 0], w[6, 1], w[1, 0], w[2, 1], w[7], w[8, 0], w[9, 1], w[10] = np.nan, np.inf, 0.0, np.inf, 0.0, 5.0, 1e-30, -4.0
        w[12, 0], w[13, 1] = -np.inf, -0.0
        w = device(w)
    rows, src, *_ = dg.moe_sort_contiguous(ids, G, src=True)
    R, n = src.numel(), sf_rows(scales, K)
    v = x.float().repeat_interleave(k, 0)
    if weighted:
        v = v * w.view(-1, 1)
    want_q, want = quantise(v, scales)
    held = src >= 0
    pair = src[held].long()
    full = torch.zeros((R, K), device="cuda")
    full[held] = v[pair]
    for cols in (None, True):
        sf, q = filled(scales, n, R), torch.full((R, K), 0xA5, dtype=torch.uint8, device="cuda")
        _, _, qt, sft, _ = dg.moe_dispatch_quantize_e4m3_contiguous(x, rows, R, src=src, weights=w, q=q, sf=sf, qt=cols,
                                                                    scales=scales)
        assert torch.equal(q[held], want_q[pair]), f"codes, columns {cols}"
        assert torch.equal(sf.view(I32)[:, held], want[:, pair]), f"scales, columns {cols}"
        assert bool((q[~held] == 0xA5).all()) and bool((sf.view(I32)[:, ~held] == FILL).all())
    for b in range(R // 128):
        cq, csf = quantise(full[128 * b:128 * b + 128].t(), "fp32" if scales == "fp32" else "ue8m0")
        assert torch.equal(qt[128 * b:128 * b + 128].t(), cq), f"column codes of block {b}"
        assert torch.equal(sft[b].view(I32), csf[0]), f"column scales of block {b}"
