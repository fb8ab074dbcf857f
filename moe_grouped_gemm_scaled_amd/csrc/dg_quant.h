// dg_quant.h -- E4M3 quantisation of one block, shared by the kernels that
// write quantised tensors: the block scale sf = max(amax, 1e-4) / 448 (fp32,
// or rounded up to a power of two) and the codes of x / sf.
#pragma once

#include "dg_device.h"

namespace dg {

// Four quotients x / s, already rounded to fp32, to E4M3FN codes (byte i
// from element i) with gfx950's packed conversion.  For every finite |v| <
// 464 it gives the nearest E4M3FN value, ties to the even code, subnormals
// (steps of 2^-9 below 2^-6) included, which was checked against a software
// encoder over all 2^32 fp32 inputs.  Above 464 it does not saturate, but a
// block's values divided by its scale stay below 448 * (1 + 2^-23).  NaN keeps
// its sign through the conversion; NaN codes are made positive (0x7f) here,
// the quantisers' NaN code.
__device__ __forceinline__ uint32_t e4m3_encode4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    const uint32_t u = (uint32_t)w;
    const uint32_t nan = ((u & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // bytes whose low 7 bits are all ones
    return u & ~nan;
}

// x / s rounded to fp32 (IEEE division), for finite s > 0, from y = 1/s
// rounded to fp64: RN32(x * y) with the product rounded to fp64 first.  This
// is exact: a quotient of two fp32 values is never closer than 2^-49
// (relative) to a point halfway between two fp32 values, while the two fp64
// roundings move it by less than 2^-51, so both round to the same fp32.
// (x = +-inf or NaN gives NaN, as the division does; s = inf gives y = 0.)
__device__ __forceinline__ float div_by_scale(float x, double y) { return (float)((double)x * y); }

// The block's four quotients as codes.  Power-of-two scales: multiplying by
// the exact reciprocal is the division.
template <bool UE8M0>
__device__ __forceinline__ uint32_t encode_block4(const v4f &v, float inv, double y) {
    if constexpr (UE8M0) return e4m3_encode4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    return e4m3_encode4(div_by_scale(v.x, y), div_by_scale(v.y, y), div_by_scale(v.z, y), div_by_scale(v.w, y));
}

template <bool UE8M0>
__device__ __forceinline__ float block_scale(float amax) {
    const float s = fmaxf(amax, 1e-4f) / 448.0f;          // IEEE division (no fast-math)
    if constexpr (!UE8M0) return s;
    // s is a normal fp32 (>= 1e-4/448): clear the mantissa and, if it was not
    // zero, step the exponent up by one
    const uint32_t u = __float_as_uint(s);
    return __uint_as_float((u & 0x7fffffu) ? (u & 0x7f800000u) + 0x00800000u : u);
}

// Division by a block's scale in fp32 only, for kernels whose arithmetic shows
// beside their memory time: with y = RN(1 / s),
//     q0 = RN(x y),  e = RN(q0 s - x),  q = RN(q0 - e y)      (each line one rounding)
// q0 is within 1.5 ulp of z = x / s, and the relative errors of y and e, 2^-24
// each, leave what the last step rounds within 1.5 * 2^-23 ulp of z.  So q is
// the IEEE quotient or, next to a midpoint of fp32, its neighbour, which gives
// another E4M3 code only where one of the two is a boundary between codes.  The
// pairs x, s of 24 bits that come so close to a midpoint beside a boundary are
// few; all of them give the code of the IEEE quotient (tests).
// In this form e = +0 for x = +-0 leaves the sign of the zero.  Power-of-two
// scales: x y is exact.  An infinite scale (y = 0) counts as 0 in e, which keeps
// 0 for finite x and NaN for infinities.
struct BlockDivisor {
    float y, s;
};
template <bool UE8M0>
__device__ __forceinline__ BlockDivisor block_divisor(float s) {
    const float y = 1.0f / s;                             // IEEE division (no fast-math)
    return {y, y == 0.f ? 0.f : s};
}
template <bool UE8M0>
__device__ __forceinline__ float divide(float x, const BlockDivisor &d) {
    const float q0 = x * d.y;
    if constexpr (UE8M0) return q0;
    return __builtin_fmaf(-__builtin_fmaf(q0, d.s, -x), d.y, q0);
}
template <bool UE8M0>
__device__ __forceinline__ uint32_t encode4(const v4f &v, const BlockDivisor &d) {
    return e4m3_encode4(divide<UE8M0>(v.x, d), divide<UE8M0>(v.y, d), divide<UE8M0>(v.z, d), divide<UE8M0>(v.w, d));
}

// Scale of block nb (of nnb) of a row, in K-block-major scales of ld columns:
// fp32, or packed (PK): byte nb % 4 of the row's word, where the last block
// clears the bytes past it.
template <bool PK>
__device__ __forceinline__ void store_block_scale(uint32_t *sf, int ld, int64_t row, int nb, int nnb, float s) {
    if constexpr (PK) {
        uint8_t *w = reinterpret_cast<uint8_t *>(sf + (int64_t)(nb / 4) * ld + row);
        w[nb & 3] = (uint8_t)(__float_as_uint(s) >> 23);
        if (nb == nnb - 1)
            for (int e = (nb & 3) + 1; e < 4; ++e) w[e] = 0;
    } else {
        sf[(int64_t)nb * ld + row] = __float_as_uint(s);
    }
}

}  // namespace dg
