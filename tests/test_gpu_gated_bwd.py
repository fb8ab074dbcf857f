"""GPU tests of the gated activation's gradient and its quantised outputs,
against 64-bit references (bars: layer_helpers)."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg
from moe_grouped_gemm_scaled_amd import synth

from layer_helpers import SLACK, act, act_grad, bf16, check_bf16, check_quantised, f64, normal

pytestmark = pytest.mark.gpu


def announce(msg):
    print(f"\n[case] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    torch.cuda.synchronize()


def reference(gu, dh, kind, live=None):
    """d_gate | d_up, h, and the error their fp32 arithmetic may have (through the logistic function's argument)."""
    I = dh.shape[1]
    g, u = gu[:, :I], gu[:, I:]
    d = np.concatenate([dh * u * act_grad(g, kind), dh * act(g, kind)], 1)
    h = act(g, kind) * u
    # an error of e(1 + |v|) in 1 / (1 + exp(-v)), v = g or 1.6 g + 0.07 g^3: 2^-20 (2 + |g| + |g|^3) of the factors
    w = 2.0 ** -20 * (2 + 2 * np.abs(g) + 0.1 * np.abs(g) ** 3)
    de = np.concatenate([np.abs(dh * u) * w, np.abs(dh * act(g, kind)) * w], 1) + 2.0 ** -130
    he = np.abs(h) * w + 2.0 ** -130
    if live is not None:
        for x in (d, h, de, he):
            x[~live] = 0
    return d, h, de, he


def by_rows(x):
    return x.reshape(x.shape[0], -1, 128)


def by_columns(x):
    """[128 t, n] -> [t, n, 128]"""
    return x.reshape(-1, 128, x.shape[1]).transpose(0, 2, 1)


def pad128(x):
    return np.concatenate([x, np.zeros((-x.shape[0] % 128, x.shape[1]))], 0)


def check_all(out, gu, dh, kind, pow2, where, live=None):
    dgu, q, sf, qt, sft, ht, sfht = out
    rows = dh.shape[0]
    d, h, de, he = reference(f64(gu), f64(dh), kind, live)
    if dgu is not None:
        check_bf16(dgu, d, de, where + " dgu")
    if q is not None:
        check_quantised(by_rows(f64(q)), f64(sf)[:, :rows].T, by_rows(d), by_rows(de), pow2, where + " q")
    if qt is not None:
        check_quantised(by_columns(f64(qt)), f64(sft), by_columns(pad128(d)), by_columns(pad128(de)), pow2, where + " qt")
    if ht is not None:
        check_quantised(by_columns(f64(ht)), f64(sfht), by_columns(pad128(h)), by_columns(pad128(he)), pow2, where + " ht")


SIZES = [(1, 128), (5, 256), (127, 128), (128, 384), (129, 256), (200, 2048), (300, 640), (513, 128)]


@pytest.mark.parametrize("rows,I", SIZES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_all_outputs(rows, I, kind, ue8m0):
    announce(f"gated_bwd rows={rows} I={I} {kind} ue8m0={ue8m0}")
    gu = bf16(2 * normal(rows + I, (rows, 2 * I))).cuda()
    dh = bf16(0.1 * normal(rows + I, (rows, I), 1)).cuda()
    out = dg.gated_backward_quantize_e4m3(gu, dh, kind, dgu=True, q=True, qt=True, ht=True, ue8m0=ue8m0)
    check_all(out, gu, dh, kind, ue8m0, f"rows={rows} I={I}")


@pytest.mark.parametrize("want", [("dgu",), ("q",), ("qt",), ("ht",), ("q", "qt"), ("dgu", "ht")])
@pytest.mark.parametrize("rows", [3, 140])
def test_each_output_alone(want, rows):
    announce(f"gated_bwd {want} rows={rows}")
    I = 256
    gu, dh = bf16(normal(1, (rows, 2 * I))).cuda(), bf16(normal(2, (rows, I))).cuda()
    out = dg.gated_backward_quantize_e4m3(gu, dh, "silu", **{w: True for w in want})
    given = dict(zip(("dgu", "q", "sf", "qt", "sft", "ht", "sfht"), out))
    assert all((given[n] is not None) == (n in want) for n in ("dgu", "q", "qt", "ht"))
    check_all(out, gu, dh, "silu", False, str(want))


@pytest.mark.parametrize("counts", [[0, 5, 300], [128], [1, 1, 1, 129]])
def test_rows_without_data_count_as_zeros(counts):
    """NaN and infinities in the rows of the contiguous layout's padding reach no output."""
    announce(f"gated_bwd padding {counts}")
    idx = synth.contiguous_m_indices(counts)
    rows, I = idx.size, 256
    live = idx >= 0
    gu, dh = bf16(normal(3, (rows, 2 * I))).cuda(), bf16(normal(4, (rows, I))).cuda()
    pad = torch.from_numpy(~live).cuda()
    clean = gu.clone(), dh.clone()
    gu[pad] = float("nan")
    dh[pad] = float("inf")
    out = dg.gated_backward_quantize_e4m3(gu, dh, "gelu", m_indices=torch.from_numpy(idx).cuda(), dgu=True, q=True, qt=True,
                                          ht=True)
    check_all(out, clean[0], clean[1], "gelu", False, str(counts), live)
    assert torch.all(out[0][pad] == 0) and torch.all(out[1][pad] & 0x7F == 0)


def test_nothing_valid_and_no_rows():
    announce("gated_bwd without data")
    I = 128
    gu = torch.full((256, 2 * I), float("nan"), dtype=torch.bfloat16, device="cuda")
    dh = torch.ones((256, I), dtype=torch.bfloat16, device="cuda")
    idx = torch.full((256,), -1, dtype=torch.int32, device="cuda")
    dgu, q, sf, qt, sft, ht, sfht = dg.gated_backward_quantize_e4m3(gu, dh, m_indices=idx, dgu=True, q=True, qt=True, ht=True)
    for t in (dgu, q, qt, ht):
        assert torch.all(t == 0)
    floor = torch.tensor(1e-4) / 448
    assert torch.all(sf.cpu() == floor) and torch.all(sft.cpu() == floor) and torch.all(sfht.cpu() == floor)
    out = dg.gated_backward_quantize_e4m3(gu[:0], dh[:0], q=True, qt=True)
    assert out[1].shape == (0, 2 * I) and out[3].shape == (0, 2 * I)


def test_saturated_gates():
    """Gates far from zero: act' is 0 or 1 there, without NaN."""
    announce("gated_bwd saturated gates")
    rows, I = 40, 128
    g = np.tile(np.array([-200.0, -90.0, -30.0, -8.0, 0.0, 8.0, 30.0, 200.0], np.float32), (rows, I // 8))
    gu = bf16(np.concatenate([g, normal(5, (rows, I))], 1)).cuda()
    dh = bf16(normal(6, (rows, I))).cuda()
    for kind in ("silu", "gelu"):
        out = dg.gated_backward_quantize_e4m3(gu, dh, kind, dgu=True, q=True, qt=True, ht=True)
        assert all(torch.isfinite(t.float()).all() for t in (out[0], out[2], out[4], out[6]))
        gn, un, dn = f64(gu)[:, :I], f64(gu)[:, I:], f64(dh)
        with np.errstate(over="ignore"):
            ref = np.concatenate([dn * un * act_grad(gn, kind), dn * act(gn, kind)], 1)
        tol = 2.0 ** -8 * np.abs(ref) + 1e-6 * np.abs(np.concatenate([dn * un, dn], 1))
        assert np.all(np.abs(f64(out[0]) - ref) <= tol)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_against_differences(kind):
    """<dgu, v> against central differences of sum(dh * act(gate) * up) in 64 bits; dgu is rounded to bf16, so the bar is
    half an ulp of each of its terms."""
    announce(f"gated_bwd differences {kind}")
    rows, I = 30, 256
    gu, dh = bf16(normal(7, (rows, 2 * I))).cuda(), bf16(normal(8, (rows, I))).cuda()
    dgu = f64(dg.gated_backward_quantize_e4m3(gu, dh, kind, dgu=True)[0])
    gn, dn = f64(gu), f64(dh)

    def loss(x):
        return float((dn * act(x[:, :I], kind) * x[:, I:]).sum())

    t = 1e-5
    for seed in range(3):
        v = normal(60 + seed, (rows, 2 * I)).astype(np.float64)
        num = (loss(gn + t * v) - loss(gn - t * v)) / (2 * t)
        assert abs(num - (dgu * v).sum()) <= 2.0 ** -8 * np.sqrt((dgu * v) ** 2).sum() + 1e-6


def test_gradient_gemms_take_the_outputs():
    """The codes as operands of the weight-gradient GEMM (TN) and the input-gradient GEMM (NN): the products of the
    quantised values, to the GEMM bar."""
    announce("gated_bwd into the gradient GEMMs")
    rows, I, H = 256, 128, 256
    gu, dh = bf16(normal(9, (rows, 2 * I))).cuda(), bf16(normal(10, (rows, I))).cuda()
    _, q, sf, qt, sft, _, _ = dg.gated_backward_quantize_e4m3(gu, dh, q=True, qt=True)
    w, sfw = dg.quantize_e4m3_128x128(torch.from_numpy(normal(11, (2 * I, H))).cuda())
    x, sfx = dg.quantize_e4m3_128x128(torch.from_numpy(normal(12, (rows, H))).cuda())
    dx = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    dg.fp8_gemm("nn", q, sf, w, sfw.t().contiguous(), dx)
    dw = torch.empty((2 * I, H), dtype=torch.bfloat16, device="cuda")
    dg.fp8_gemm("tn", qt, sft, x, sfx.t().contiguous(), dw)
    rep = lambda s: np.repeat(np.repeat(f64(s), 128, 0), 128, 1)  # noqa: E731
    d_row = f64(q) * np.repeat(f64(sf).T[:rows], 128, 1)
    d_col = f64(qt) * np.repeat(f64(sft), 128, 0)
    ref = d_row @ (f64(w) * rep(sfw))
    check_bf16(dx, ref, np.full(ref.shape, 1e-4 * np.abs(ref).max()), "dx")
    ref = d_col.T @ (f64(x) * rep(sfx))
    check_bf16(dw, ref, np.full(ref.shape, 1e-4 * np.abs(ref).max()), "dw")
