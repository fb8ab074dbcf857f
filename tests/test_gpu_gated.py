"""GPU tests of the gated GEMM (both projections, activation, product) in its
three row layouts, against the fp64 oracle's projections.

Bars: the projections to the GEMM bar (half a bf16 ulp, and E = 1e-4 max|.| for
the accumulation); h to what that E allows through act(g) u, |act'| <= 1.13,
plus half a bf16 ulp; quantised outputs as in layer_helpers with the same E."""
import sys

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_gemm_scaled_amd import binding as dg
from moe_grouped_gemm_scaled_amd import synth

from helpers import dev, dev_bf16
from layer_helpers import SLACK, act, check_bf16, check_quantised, f64, unpack_words

pytestmark = pytest.mark.gpu

SENT = 0x7FA5            # a bf16 NaN that rounding never produces
QSENT = 0xA5


def announce(msg):
    print(f"\n[case] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    torch.cuda.synchronize()


def problem(lead, rows, I, K, seed, packed, G=()):
    """Quantised operands: activations N(0,1), weights N(0,1)/sqrt(K) (both projections then are N(0,1))."""
    a, sfa = oracle.quantize_1x128(synth.normal_f32(seed, 0, (*lead, rows, K)), ue8m0=packed)
    w = synth.normal_f32(seed, 1, (*(G or (1,)), 2, I, K)) * np.float32(K ** -0.5)
    b, sfb = oracle.quantize_128x128(w.reshape(-1, I, K), ue8m0=packed)
    b, sfb = b.reshape(*G, 2, I, K), sfb.reshape(*G, 2, *sfb.shape[1:])
    return a, sfa, b, sfb


def operands(p, packed):
    a, sfa, b, sfb = p
    if packed:
        return (dev(a), dev(oracle.pack_ue8m0(sfa, k_axis=-2).view(np.int32)), dev(b),
                dev(oracle.pack_ue8m0(sfb, k_axis=-1).view(np.int32)))
    return dev(a), dev(sfa), dev(b), dev(sfb)


class Outputs:
    """gu, h, q, sf filled with sentinels, guard bands around each."""

    def __init__(self, lead, rows, I, ld, packed, quant):
        n = int(np.prod(lead, dtype=np.int64)) * rows * I
        self.flat = {}

        def make(name, count, shape, dtype, fill):
            t = torch.full((count + 128,), fill, dtype=dtype, device="cuda")
            self.flat[name] = (t, fill, count)
            return t[64:64 + count].view(shape)

        self.h = make("h", n, (*lead, rows, I), torch.int16, SENT).view(torch.bfloat16)
        self.gu = make("gu", 2 * n, (*lead, rows, 2 * I), torch.int16, SENT).view(torch.bfloat16)
        self.q = self.sf = None
        if quant:
            self.q = make("q", n, (*lead, rows, I), torch.uint8, QSENT)
            blocks = I // 128
            nb = (blocks + 3) // 4 if packed else blocks
            count = int(np.prod(lead, dtype=np.int64)) * nb * ld
            # the packed form may leave nothing of a word it writes; words of rows without data stay
            self.sf = make("sf", count, (*lead, nb, ld), torch.int32 if packed else torch.float32,
                           0x5A5A5A5A if packed else -5.0)

    def guards(self):
        for name, (t, fill, count) in self.flat.items():
            assert torch.all(t[:64] == fill) and torch.all(t[64 + count:] == fill), f"{name}: written outside"


def check_rows(where, gu, h, q, sf, I, gate, up, kind, packed):
    """Device outputs of some rows (sf: fp64 [rows, blocks]) against fp64 projections of these rows."""
    if gate.size == 0:
        return
    Eg, Eu = 1e-4 * np.abs(gate).max(), 1e-4 * np.abs(up).max()
    if gu is not None:
        check_bf16(gu[:, :I], gate, np.full(gate.shape, Eg), where + " gate")
        check_bf16(gu[:, I:], up, np.full(up.shape, Eu), where + " up")
    a = act(gate, kind)
    ref = a * up
    extra = 1.13 * Eg * (np.abs(up) + Eu) + np.abs(a) * Eu + SLACK * np.abs(ref)
    if h is not None:
        check_bf16(h, ref, extra, where + " h")
    if q is not None:
        n = gate.shape[0]
        check_quantised(f64(q).reshape(n, I // 128, 128), sf, ref.reshape(n, I // 128, 128),
                        extra.reshape(n, I // 128, 128), packed, where + " q")


def projections(a, sfa, b, sfb):
    """fp64 gate and up of one expert: a [n, K], sfa [K/128, ld], b [2, I, K], sfb [2, .., K/128]."""
    ld = sfa.shape[1]
    pad = (-ld) % 4
    if pad:
        sfa = np.concatenate([sfa, np.zeros((sfa.shape[0], pad), np.float32)], 1)
    sfa = np.ascontiguousarray(sfa)
    a = np.ascontiguousarray(a)
    return tuple(oracle.gemm_nt(a, sfa, np.ascontiguousarray(b[x]), np.ascontiguousarray(sfb[x])) for x in range(2))


def scales_of(sf, packed, blocks):
    return unpack_words(sf, blocks) if packed else f64(sf)


# rows on both sides of every tile and dispatch boundary, K of one, few and odd block counts, widths of whole and partial blocks
DENSE = [(1, 128, 128), (1, 2048, 1024), (2, 256, 512), (15, 128, 384), (16, 640, 1152), (17, 128, 256), (31, 384, 512),
         (33, 256, 640), (63, 128, 896), (64, 512, 2048), (65, 256, 512), (127, 128, 256), (128, 256, 512),
         (129, 128, 384), (200, 640, 256), (255, 128, 512), (256, 128, 128), (257, 384, 640), (300, 256, 1152),
         (513, 128, 256), (700, 512, 384)]


@pytest.mark.parametrize("M,I,K", DENSE)
@pytest.mark.parametrize("packed", [False, True])
def test_dense(M, I, K, packed):
    announce(f"gated dense M={M} I={I} K={K} packed={packed}")
    kind = "silu" if (M + I // 128) % 2 else "gelu"
    p = problem((), M, I, K, M + I + K, packed)
    ld = p[1].shape[1]
    ops = operands(p, packed)
    gate, up = projections(*p)
    for want in ("all", "h", "q"):
        o = Outputs((), M, I, ld, packed, want != "h")
        kw = dict(h=o.h, q=o.q, sf=o.sf, gu=o.gu) if want == "all" else dict(h=o.h) if want == "h" else dict(q=o.q, sf=o.sf)
        dg.fp8_gated_gemm_nt(*ops, act=kind, **kw)
        torch.cuda.synchronize()
        o.guards()
        sf = scales_of(o.sf[:, :M], packed, I // 128).T if want != "h" else None
        check_rows(f"M={M} I={I} K={K} {want} {dg.last_config()}", o.gu if want == "all" else None,
                   o.h if want != "q" else None, o.q, sf, I, gate, up, kind, packed)
        if o.sf is not None and ld > M:
            assert torch.all(o.sf[:, M:] == (0x5A5A5A5A if packed else -5.0)), "scales past the rows written"


@pytest.mark.parametrize("M,I,K", [(1, 1, 128), (3, 7, 256), (5, 8, 384), (1, 200, 512), (40, 136, 512), (130, 129, 256),
                                   (64, 1000, 512), (300, 196, 384), (260, 8, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_dense_any_width(M, I, K, packed):
    """Widths that are no multiple of a block, or not even of 8: the bf16 outputs."""
    announce(f"gated width M={M} I={I} K={K} packed={packed}")
    p = problem((), M, I, K, M + I + K, packed)
    ops = operands(p, packed)
    o = Outputs((), M, I, p[1].shape[1], packed, False)
    dg.fp8_gated_gemm_nt(*ops, h=o.h, gu=o.gu)
    torch.cuda.synchronize()
    o.guards()
    gate, up = projections(*p)
    check_rows(f"M={M} I={I} K={K}", o.gu, o.h, None, None, I, gate, up, "silu", packed)


@pytest.mark.parametrize("counts", [[1], [128, 128], [0, 5, 300, 128, 0, 257], [1000, 1], [129, 3, 130, 500], [0, 0, 7]])
@pytest.mark.parametrize("packed", [False, True])
def test_contiguous(counts, packed):
    check_contiguous(counts, 256, 640, packed)


def check_contiguous(counts, I, K, packed):
    announce(f"gated contiguous {counts} packed={packed}")
    idx = synth.contiguous_m_indices(counts)
    M, G = idx.size, len(counts)
    p = problem((), M, I, K, 77 + M, packed, (G,))
    a, sfa, b, sfb = (x.copy() for x in p)
    a[idx < 0] = 0x7F                                    # NaN codes and scales on the rows without data stay inert
    if not packed:
        sfa[:, idx < 0] = np.nan
    ops = operands((a, sfa, b, sfb), packed)
    o = Outputs((), M, I, M, packed, True)
    dg.m_grouped_fp8_gated_gemm_nt_contiguous(*ops, dev(idx), act="silu", h=o.h, q=o.q, sf=o.sf, gu=o.gu)
    torch.cuda.synchronize()
    o.guards()
    pad = torch.from_numpy(idx < 0).cuda()
    assert torch.all(o.h.view(torch.int16)[pad] == SENT) and torch.all(o.gu.view(torch.int16)[pad] == SENT)
    assert torch.all(o.q[pad] == QSENT) and torch.all(o.sf[:, pad] == (0x5A5A5A5A if packed else -5.0))
    for e in range(G):
        at = np.flatnonzero(idx == e)
        if at.size == 0:
            continue
        gate, up = projections(p[0][at], p[1][:, at], p[2][e], p[3][e])
        t = torch.from_numpy(at).cuda()
        check_rows(f"expert {e} of {counts}", o.gu[t], o.h[t], o.q[t], scales_of(o.sf[:, t], packed, I // 128).T, I, gate,
                   up, "silu", packed)


@pytest.fixture
def few_cus():
    """A cap of 4 CUs: small problems then take several rounds of tiles, as large ones do on all CUs."""
    dg.set_num_cus(4)
    yield
    dg.set_num_cus(0)


@pytest.mark.parametrize("M,I,K", [(512, 256, 256), (520, 256, 384), (700, 256, 256), (1030, 128, 256), (1100, 384, 128),
                                   (900, 1, 128), (1285, 136, 256), (2050, 128, 128), (64, 512, 256), (100, 640, 384)])
@pytest.mark.parametrize("packed", [False, True])
def test_dense_in_rounds(M, I, K, packed, few_cus):
    """Full rounds of large tiles, then the remaining rows in smaller ones."""
    announce(f"gated rounds M={M} I={I} K={K} packed={packed}")
    p = problem((), M, I, K, M + I + K, packed)
    ops = operands(p, packed)
    ld = p[1].shape[1]
    quant = I % 128 == 0
    o = Outputs((), M, I, ld, packed, quant)
    dg.fp8_gated_gemm_nt(*ops, h=o.h, q=o.q, sf=o.sf, gu=o.gu)
    torch.cuda.synchronize()
    o.guards()
    gate, up = projections(*p)
    sf = scales_of(o.sf[:, :M], packed, I // 128).T if quant else None
    check_rows(f"M={M} I={I} {dg.last_config()}", o.gu, o.h, o.q, sf, I, gate, up, "silu", packed)


@pytest.mark.parametrize("counts", [[600], [128, 900, 0, 130], [1, 1, 1, 1, 1, 1, 1], [300, 300, 300], [512, 512, 40], [1500, 128],
                                    [0, 0, 1300, 0, 257]])
@pytest.mark.parametrize("I", [128, 384])
@pytest.mark.parametrize("packed", [False, True])
def test_contiguous_in_rounds(counts, I, packed, few_cus):
    check_contiguous(counts, I, 256, packed)


def test_contiguous_nothing_and_bad_ids():
    announce("gated contiguous without valid rows")
    I, K, M = 128, 256, 384
    p = problem((), M, I, K, 5, False, (2,))
    ops = operands(p, False)
    for fill in (-1, 2, 1 << 30, -(1 << 31)):
        idx = torch.full((M,), fill, dtype=torch.int32, device="cuda")
        o = Outputs((), M, I, M, False, True)
        dg.m_grouped_fp8_gated_gemm_nt_contiguous(*ops, idx, h=o.h, q=o.q, sf=o.sf, gu=o.gu)
        torch.cuda.synchronize()
        o.guards()
        assert torch.all(o.h.view(torch.int16) == SENT) and torch.all(o.q == QSENT) and torch.all(o.sf == -5)


MASKED = [(3, 16, 128, 256, [0, 1, 16]), (5, 64, 256, 640, [64, 0, 33, -4, 99]), (4, 200, 384, 384, [200, 1, 128, 129]),
          (6, 256, 128, 1152, [256, 0, 7, 128, 255, 31]), (2, 300, 256, 256, [300, 0]), (2, 130, 128, 128, [0, 0]),
          (9, 128, 512, 256, [5, 0, 0, 128, 64, 65, 1, 17, 96])]


@pytest.mark.parametrize("G,cap,I,K,mm", MASKED)
@pytest.mark.parametrize("packed", [False, True])
def test_masked(G, cap, I, K, mm, packed):
    announce(f"gated masked G={G} cap={cap} I={I} K={K} {mm} packed={packed}")
    mm = (mm + [cap // 2] * G)[:G]
    p = problem((G,), cap, I, K, G + cap + I, packed, (G,))
    a, sfa, b, sfb = (x.copy() for x in p)
    rows = [min(max(m, 0), cap) for m in mm]
    for g in range(G):
        a[g, rows[g]:] = 0x7F
        if not packed:
            sfa[g, :, rows[g]:] = np.nan
    ops = operands((a, sfa, b, sfb), packed)
    ld = (cap + 3) // 4 * 4
    counts = torch.tensor(mm, dtype=torch.int32, device="cuda")
    for expected in (0, 20):
        o = Outputs((G,), cap, I, ld, packed, True)
        dg.m_grouped_fp8_gated_gemm_nt_masked(*ops, counts, expected_m=expected, act="gelu", h=o.h, q=o.q, sf=o.sf, gu=o.gu)
        torch.cuda.synchronize()
        o.guards()
        for g in range(G):
            n = rows[g]
            assert torch.all(o.h[g, n:].contiguous().view(torch.int16) == SENT)
            assert torch.all(o.gu[g, n:].contiguous().view(torch.int16) == SENT)
            assert torch.all(o.q[g, n:] == QSENT) and torch.all(o.sf[g, :, n:] == (0x5A5A5A5A if packed else -5.0))
            if n == 0:
                continue
            gate, up = projections(p[0][g, :n], p[1][g][:, :n], p[2][g], p[3][g])
            check_rows(f"group {g} rows {n}", o.gu[g, :n], o.h[g, :n], o.q[g, :n],
                       scales_of(o.sf[g][:, :n], packed, I // 128).T, I, gate, up, "gelu", packed)


def test_wide_values():
    """Scales spread over many binades and a gate far on both sides of zero: act saturates to 0 and to g."""
    announce("gated wide values")
    M, I, K = 48, 128, 256
    xa = synth.normal_f32(3, 0, (M, K)) * np.exp2(synth.randint(3, 5, M, -6, 6).astype(np.float32))[:, None]
    a, sfa = oracle.quantize_1x128(xa)
    w = synth.normal_f32(3, 1, (2, I, K))
    b, sfb = oracle.quantize_128x128(w)
    o = Outputs((), M, I, sfa.shape[1], False, True)
    dg.fp8_gated_gemm_nt(dev(a), dev(sfa), dev(b), dev(sfb), act="silu", h=o.h, q=o.q, sf=o.sf)
    torch.cuda.synchronize()
    gate, up = projections(a, sfa, b, sfb)
    assert gate.max() > 500 and gate.min() < -500
    for r in range(M):                                    # the bar follows each row's own magnitude
        check_rows(f"row {r}", None, o.h[r:r + 1], o.q[r:r + 1], f64(o.sf)[:, r:r + 1].T, I, gate[r:r + 1], up[r:r + 1],
                   "silu", False)


def test_no_rows():
    announce("gated without rows")
    I, K = 256, 256
    _, _, b, sfb = problem((), 4, I, K, 9, False)
    a = torch.empty((0, K), dtype=torch.uint8, device="cuda")
    sfa = torch.empty((K // 128, 0), dtype=torch.float32, device="cuda")
    h, q, sf, gu = dg.fp8_gated_gemm_nt(a, sfa, dev(b), dev(sfb), h=True, q=True, gu=True)
    assert h.shape == (0, I) and q.shape == (0, I) and gu.shape == (0, 2 * I)


def test_workspace_reuse_streams_and_graph():
    """One workspace for calls of several shapes in stream order, two streams with one each, and a captured graph that
    is replayed several times with eager calls between: the same bits as the first call."""
    announce("gated workspace, streams, graph")
    shapes = [(1, 2048, 2048, False), (64, 512, 2048, True), (16, 640, 1152, True), (33, 256, 640, False), (128, 256, 512, True)]
    cases = []
    for M, I, K, packed in shapes:
        p = problem((), M, I, K, M + K, packed)
        cases.append((operands(p, packed), M, I, K, packed, p))
    size = max(dg.get_gated_workspace_size(M, I, K) for _, M, I, K, _, _ in cases)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")      # NaN everywhere: any content will do
    ws2 = ws.clone()

    def call(c, w):
        ops, M, I, K, packed, _ = c
        return dg.fp8_gated_gemm_nt(*ops, q=True, h=True, workspace=w)

    first = [call(c, ws) for c in cases]
    torch.cuda.synchronize()
    for c, (h, q, sf, _) in zip(cases, first):
        gate, up = projections(*c[5])
        check_rows(f"M={c[1]}", None, h, q, scales_of(sf[:, :c[1]], c[4], c[2] // 128).T, c[2], gate, up, "silu", c[4])
    for _ in range(3):
        for c, f in zip(cases, first):
            h, q, sf, _ = call(c, ws)
            assert torch.equal(h, f[0]) and torch.equal(q, f[1]) and torch.equal(sf, f[2])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for c in cases * 2:
        with torch.cuda.stream(s1):
            x = call(c, ws)
        with torch.cuda.stream(s2):
            y = call(c, ws2)
        got.append((x, y))
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(got):
        f = first[i % len(cases)]
        assert torch.equal(x[0], f[0]) and torch.equal(y[0], f[0]) and torch.equal(x[1], f[1]) and torch.equal(y[1], f[1])
    c, f = cases[0], first[0]
    h, q = torch.empty_like(f[0]), torch.empty_like(f[1])
    sf = torch.zeros_like(f[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.fp8_gated_gemm_nt(*c[0], h=h, q=q, sf=sf, workspace=ws)
    for _ in range(4):
        h.zero_()
        q.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, f[0]) and torch.equal(q, f[1]) and torch.equal(sf, f[2])
        call(cases[1], ws)
        torch.cuda.synchronize()


@pytest.fixture
def cu_caps():
    """Caps of the CU count: the tile that fills the CUs best changes with it, so one problem meets them all."""
    yield (1, 3, 4, 8, 12, 16, 24, 40, 80, 200)
    dg.set_num_cus(0)


def tiles_of(config):
    return {part.split()[0] for part in config.split("tile=")[1:]}


@pytest.mark.parametrize("packed", [False, True])
def test_dense_every_tile(packed, cu_caps):
    """One problem in each tile shape, all outputs, with scratch for the quantised output and without it; and a width
    that is no multiple of a block."""
    seen = {}
    for M, I, K in ((300, 256, 4096), (301, 269, 640)):       # the second kernel pays where K is long
        p = problem((), M, I, K, M, packed)
        ld = p[1].shape[1]
        ops = operands(p, packed)
        gate, up = projections(*p)
        quant = I % 128 == 0
        for cus in cu_caps:
            dg.set_num_cus(cus)
            for ws in ("auto", None) if quant else ("auto",):
                announce(f"gated tiles M={M} I={I} packed={packed} cus={cus} workspace={ws}")
                o = Outputs((), M, I, ld, packed, quant)
                dg.fp8_gated_gemm_nt(*ops, act="gelu", h=o.h, q=o.q, sf=o.sf, gu=o.gu, workspace=ws)
                torch.cuda.synchronize()
                o.guards()
                sf = scales_of(o.sf[:, :M], packed, I // 128).T if quant else None
                check_rows(f"cus={cus} {dg.last_config()}", o.gu, o.h, o.q, sf, I, gate, up, "gelu", packed)
                seen.setdefault((I, ws), set()).update(tiles_of(dg.last_config()))
    wide = {"256x256x128", "128x256x128", "64x256x128"}
    narrow = {"128x128x128", "64x128x128", "64x64x128"}
    assert seen[256, None] == wide
    assert len(narrow & seen[256, "auto"]) >= 2 and narrow <= seen[269, "auto"] and wide <= seen[256, "auto"] | seen[269, "auto"]


@pytest.mark.parametrize("counts", [[100, 0, 257, 129], [1, 2, 3, 4], [640]])
@pytest.mark.parametrize("packed", [False, True])
def test_contiguous_every_tile(counts, packed, cu_caps):
    """The bf16 outputs of the contiguous layout, where narrow tiles serve too; NaN on the rows without data."""
    I, K = 268, 640
    idx = synth.contiguous_m_indices(counts)
    M, G = idx.size, len(counts)
    p = problem((), M, I, K, 70 + M, packed, (G,))
    a, sfa, b, sfb = (x.copy() for x in p)
    a[idx < 0] = 0x7F
    if not packed:
        sfa[:, idx < 0] = np.nan
    ops = operands((a, sfa, b, sfb), packed)
    pad = torch.from_numpy(idx < 0).cuda()
    want = {e: projections(p[0][idx == e], p[1][:, idx == e], p[2][e], p[3][e]) for e in range(G) if counts[e]}
    seen = set()
    for cus in cu_caps:
        dg.set_num_cus(cus)
        announce(f"gated contiguous tiles {counts} packed={packed} cus={cus}")
        o = Outputs((), M, I, M, packed, False)
        dg.m_grouped_fp8_gated_gemm_nt_contiguous(*ops, dev(idx), act="silu", h=o.h, gu=o.gu)
        torch.cuda.synchronize()
        o.guards()
        seen |= tiles_of(dg.last_config())
        assert torch.all(o.h.view(torch.int16)[pad] == SENT) and torch.all(o.gu.view(torch.int16)[pad] == SENT)
        for e, (gate, up) in want.items():
            t = torch.from_numpy(np.flatnonzero(idx == e)).cuda()
            check_rows(f"expert {e} cus={cus} {dg.last_config()}", o.gu[t], o.h[t], None, None, I, gate, up, "silu", packed)
    assert {"128x256x128", "128x128x128"} <= seen and seen & {"64x128x128", "64x64x128"}


@pytest.mark.parametrize("cap,mm", [(200, [200, 0, 77]), (300, [129, 300, -1]), (16, [1, 16, 9])])
@pytest.mark.parametrize("packed", [False, True])
def test_masked_every_tile(cap, mm, packed, cu_caps):
    I, K, G = 268, 640, len(mm)
    p = problem((G,), cap, I, K, cap, packed, (G,))
    a, sfa, b, sfb = (x.copy() for x in p)
    rows = [min(max(m, 0), cap) for m in mm]
    for g in range(G):
        a[g, rows[g]:] = 0x7F
        if not packed:
            sfa[g, :, rows[g]:] = np.nan
    ops = operands((a, sfa, b, sfb), packed)
    counts = torch.tensor(mm, dtype=torch.int32, device="cuda")
    want = [projections(p[0][g, :rows[g]], p[1][g][:, :rows[g]], p[2][g], p[3][g]) if rows[g] else None for g in range(G)]
    seen = set()
    for cus in cu_caps:
        dg.set_num_cus(cus)
        announce(f"gated masked tiles {mm} packed={packed} cus={cus}")
        o = Outputs((G,), cap, I, (cap + 3) // 4 * 4, packed, False)
        dg.m_grouped_fp8_gated_gemm_nt_masked(*ops, counts, act="silu", h=o.h, gu=o.gu)
        torch.cuda.synchronize()
        o.guards()
        seen |= tiles_of(dg.last_config())
        for g in range(G):
            assert torch.all(o.h[g, rows[g]:].contiguous().view(torch.int16) == SENT)
            assert torch.all(o.gu[g, rows[g]:].contiguous().view(torch.int16) == SENT)
            if rows[g]:
                check_rows(f"group {g} cus={cus} {dg.last_config()}", o.gu[g, :rows[g]], o.h[g, :rows[g]], None, None, I,
                           *want[g], "silu", packed)
    assert seen & {"128x128x128", "64x128x128", "64x64x128"}


# rows on both sides of every fragment count, few and many columns, K long enough that the sums go through scratch
SMALL_Q = [(1, 128, 1152), (15, 256, 2048), (17, 384, 1280), (32, 4224, 1152), (33, 256, 1408), (48, 4224, 1152), (64, 640, 1152),
           (65, 128, 3200), (100, 2048, 1152), (127, 256, 1280), (128, 4224, 1152)]


@pytest.mark.parametrize("M,I,K", SMALL_Q)
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("cus", [0, 24])
def test_dense_few_rows_quantised(M, I, K, packed, cus):
    announce(f"gated few rows M={M} I={I} K={K} packed={packed} cus={cus}")
    p = problem((), M, I, K, M + I + K, packed)
    ld = p[1].shape[1]
    ops = operands(p, packed)
    dg.set_num_cus(cus)
    try:
        assert dg.get_gated_workspace_size(M, I, K) > 0
        for all_outputs in (True, False):
            o = Outputs((), M, I, ld, packed, True)
            dg.fp8_gated_gemm_nt(*ops, act="gelu", q=o.q, sf=o.sf, **(dict(h=o.h, gu=o.gu) if all_outputs else {}))
            torch.cuda.synchronize()
            assert "family=gated_small" in dg.last_config()
            o.guards()
            gate, up = projections(*p)
            check_rows(f"M={M} I={I} K={K} {dg.last_config()}", o.gu if all_outputs else None, o.h if all_outputs else None, o.q,
                       scales_of(o.sf[:, :M], packed, I // 128).T, I, gate, up, "gelu", packed)
    finally:
        dg.set_num_cus(0)
