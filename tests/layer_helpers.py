"""64-bit references and bars of the feed-forward layer's GPU tests, written
from the operators' definitions in numpy, apart from the library's code.

Bars (derived from the number formats; U = 2^-24, the fp32 unit roundoff):
 - a bf16 output: half a bf16 ulp for its rounding, plus what the fp32
   arithmetic in front of it may be off;
 - a quantised output: the scale within the relative error of the fp32
   arithmetic (a power of two: one of the values that such an error allows),
   and every code within half a step of E4M3 of value / scale, the scale being
   the one returned; so a value next to a rounding boundary may take either
   code, and nothing else passes.
"""
import math

import numpy as np
import torch

from moe_grouped_gemm_scaled_amd import synth

SLACK = 2.0 ** -18        # relative error of a chain of fp32 operations and short fp32 sums (64 U)

_CODES = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def ulp_bf16(x):
    ax = np.abs(np.asarray(x, dtype=np.float64))
    e = np.floor(np.log2(np.maximum(ax, 2.0 ** -126)))
    return np.where(ax >= 2.0 ** -126, np.ldexp(1.0, (e - 7).astype(np.int64)), 2.0 ** -133)


def f64(t):
    """Any device tensor of numbers as fp64 on the host (uint8: E4M3 codes)."""
    if t.dtype == torch.uint8:
        return _CODES[t.cpu().numpy()]
    return t.detach().double().cpu().numpy()


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def normal(seed, shape, stream=0):
    return synth.normal_f32(seed, stream, shape)


def check(got, ref, tol, where):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (where, got.shape, ref.shape)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    if np.any(bad):
        i = tuple(np.argwhere(bad)[0])
        t = np.broadcast_to(tol, got.shape)
        raise AssertionError(f"{where}: {int(bad.sum())} of {bad.size} outside; first {i}: got {got[i]!r}, "
                             f"ref {ref[i]!r}, tol {t[i]!r}")


def check_bf16(got, ref, extra, where):
    """got: bf16 tensor; extra: absolute error allowed before its rounding."""
    got = f64(got)
    check(got, ref, 0.5 * ulp_bf16(np.maximum(np.abs(ref) + extra, np.abs(got))) + extra, where)


def unpack_words(sf, blocks):
    """int32 words [.., ceil(blocks/4), n] -> fp64 scales [.., blocks, n]; bytes past the last block must be zero."""
    w = sf.cpu().numpy().view(np.uint32).astype(np.int64)
    e = np.stack([(w >> (8 * j)) & 0xFF for j in range(4)], axis=-2)          # [.., words, 4, n]
    e = e.reshape(*e.shape[:-3], -1, e.shape[-1])
    assert np.all(e[..., blocks:, :] == 0), "unused high bytes are not zero"
    return np.exp2(e[..., :blocks, :].astype(np.float64) - 127)


def pow2_up(s):
    return np.exp2(np.ceil(np.log2(s)))


def check_quantised(q, s, ref, extra, pow2, where):
    """q: fp64 code values [.., B], one block per row; s: fp64 scales [..]; ref: the values; extra: absolute error
    allowed on a value before quantisation (broadcast to ref)."""
    extra = np.broadcast_to(extra, ref.shape)
    amax = np.abs(ref).max(-1)
    lo = np.maximum((np.abs(ref) - extra).max(-1), 1e-4) / 448 * (1 - 2.0 ** -22)
    hi = np.maximum((np.abs(ref) + extra).max(-1), 1e-4) / 448 * (1 + 2.0 ** -22)
    if pow2:
        assert np.all(s == np.exp2(np.round(np.log2(s)))), f"{where}: a scale is no power of two"
        lo, hi = pow2_up(lo), pow2_up(hi)
    bad = ~((s >= lo) & (s <= hi))
    assert not np.any(bad), (f"{where}: {int(bad.sum())} scales outside, first at {np.argwhere(bad)[0].tolist()}: "
                             f"{s[bad][0]!r} not in [{lo[bad][0]!r}, {hi[bad][0]!r}], amax {amax[bad][0]!r}")
    v = np.abs(q)
    e = np.floor(np.log2(np.maximum(v, 2.0 ** -9)))
    half = np.exp2(np.maximum(e, -6) - 3) / 2                                  # half a step of E4M3 above |q|
    check(q * s[..., None], ref, half * s[..., None] * (1 + 2.0 ** -20) + extra, where)


def logistic(v):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-v))


# The tanh form of GELU is evaluated through (1 + tanh z) / 2 = logistic(2z): for z far below zero the left side
# cancels (its 64-bit value is 2^-53 off in absolute terms, as much as the value itself near z = -18).

def act(g, kind):
    if kind == "silu":
        return g * logistic(g)
    return g * logistic(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def act_grad(g, kind):
    if kind == "silu":
        s = logistic(g)
        return s * (1 + g * (1 - s))
    k = 2 * math.sqrt(2 / math.pi)
    s = logistic(k * (g + 0.044715 * g ** 3))
    return s + g * s * (1 - s) * k * (1 + 3 * 0.044715 * g ** 2)
