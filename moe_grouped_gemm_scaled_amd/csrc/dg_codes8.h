// dg_codes8.h -- 1x128 quantisation of eight consecutive columns per lane, 16
// lanes to a block, four blocks (one packed scale word) to a wave: how the layer
// norm writes its rows.
#pragma once

#include "dg_layer.h"
#include "dg_quant.h"
#include "dg_rows.h"

namespace dg {

// Largest magnitude of the lane's eight values; over the block with max16.
__device__ __forceinline__ float amax8(const float (&y)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
    return m;
}

// The block's scale s from its largest magnitude, and the lane's codes of y / s
// (`format`, an SfFormat, is uniform).
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float amax, int format, float &s) {
    const v4f lo = v4f{y[0], y[1], y[2], y[3]}, hi = v4f{y[4], y[5], y[6], y[7]};
    if (format == kSfFp32) {
        s = block_scale<false>(amax);
        const BlockDivisor d = block_divisor<false>(s);
        return uint2{encode4<false>(lo, d), encode4<false>(hi, d)};
    }
    s = block_scale<true>(amax);
    const BlockDivisor d = block_divisor<true>(s);
    return uint2{encode4<true>(lo, d), encode4<true>(hi, d)};
}

// The wave's four exponents as a packed word, 0 for blocks past K (`in` false).
__device__ __forceinline__ uint32_t scale_word(float s, bool in, int lane) {
    uint32_t e = in ? (__float_as_uint(s) >> 23) << (8 * (lane >> 4)) : 0u;
    e |= (uint32_t)__shfl_xor((int)e, 16);
    return e | (uint32_t)__shfl_xor((int)e, 32);
}

}  // namespace dg
