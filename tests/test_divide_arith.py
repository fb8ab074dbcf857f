"""The fp32 form of the quantisers' division (dg_quant.h, divide) is the IEEE
quotient: q0 = RN(x y), e = q0 s - x (one fma), q = RN(q0 - e y) (one fma) with
y = RN(1 / s), on random pairs, on quotients next to rounding boundaries of
fp32 and of E4M3, and on a block's largest value.  Each fma is formed exactly:
the product of two fp32 values in fp64 (48 bits), its sum with the addend in
80-bit arithmetic (64 bits; q0 s - x cancels, and q0 - e y is checked to need
no more bits than a correct rounding to fp32 can tell)."""
import numpy as np
import pytest

f32, f64, ld = np.float32, np.float64, np.longdouble


def divide(x, s):
    y = (f32(1) / s).astype(f32)
    q0 = (x * y).astype(f32)
    e = (q0.astype(f64) * s.astype(f64) - x.astype(ld)).astype(f32)
    return (-(e.astype(f64) * y.astype(f64)).astype(ld) + q0.astype(ld)).astype(f32)


def check(x, s):
    assert x.dtype == f32 and s.dtype == f32
    want = (x / s).astype(f32)
    got = divide(x, s)
    big = np.abs(want) >= 2.0 ** -10              # E4M3's smallest step is 2^-9: half of it and below encodes as zero
    assert np.array_equal(got[big], want[big])
    assert np.array_equal(np.signbit(got), np.signbit(want))
    assert np.all(np.abs(got[~big]) <= 2.0 ** -10 * (1 + 2.0 ** -20))


@pytest.mark.skipif(np.finfo(ld).nmant < 63, reason="needs 80-bit long double")
@pytest.mark.parametrize("seed", range(4))
def test_divide_is_the_ieee_quotient(seed):
    rng = np.random.default_rng(seed)
    n = 1 << 20
    s = (np.maximum(np.exp(rng.uniform(np.log(1e-4), np.log(1e6), n)), 1e-4).astype(f32) / f32(448)).astype(f32)
    check((rng.uniform(-448, 448, n).astype(f32) * s).astype(f32), s)
    # quotients near fp32 midpoints and near E4M3 rounding boundaries
    q = (rng.integers(8, 16, n) + 0.5) * np.exp2(rng.integers(-6, 5, n))
    for off in (0, 1, -1):
        check(np.nextafter((q * s.astype(f64)).astype(f32), f32(off * 1e30) if off else f32(0), dtype=f32) if off
              else (q * s.astype(f64)).astype(f32), s)
    m = rng.uniform(1, 2, n).astype(f32).astype(f64) + 2.0 ** -24
    check((m * s.astype(f64)).astype(f32), s)
    # the block's largest value over its own scale
    amax = np.exp(rng.uniform(np.log(1e-4), np.log(1e8), n)).astype(f32)
    check(amax, (amax / f32(448)).astype(f32))
    check(np.array([0.0, -0.0], f32), np.array([0.5, 0.5], f32))
