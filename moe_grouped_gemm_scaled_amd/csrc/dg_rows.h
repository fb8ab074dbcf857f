// dg_rows.h -- device helpers of the row-wise kernels (norm and gating):
// eight consecutive values per lane as one or two 16-byte accesses, and
// reductions over the 16 lanes that share a 128-column block and over a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_device.h"

namespace dg {

// Eight consecutive values as stored: bf16 (16 bytes) or fp32 (32 bytes).
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    v4i a;
};
template <>
struct Raw8<float> {
    v4f a, b;
};

template <bool NT = false>
__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t *p) {
    const v4i *q = reinterpret_cast<const v4i *>(p);
    return NT ? Raw8<uint16_t>{__builtin_nontemporal_load(q)} : Raw8<uint16_t>{*q};
}
template <bool NT = false>
__device__ __forceinline__ Raw8<float> load8(const float *p) {
    const v4f *q = reinterpret_cast<const v4f *>(p);
    return NT ? Raw8<float>{__builtin_nontemporal_load(q), __builtin_nontemporal_load(q + 1)} : Raw8<float>{q[0], q[1]};
}

// element i (a constant after unrolling) as fp32
__device__ __forceinline__ float get8(const Raw8<uint16_t> &r, int i) {
    const uint32_t u = (uint32_t)r.a[i >> 1];
    return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
}
__device__ __forceinline__ float get8(const Raw8<float> &r, int i) { return i < 4 ? r.a[i & 3] : r.b[i & 3]; }

// Eight fp32 values rounded to the stored type.
template <bool NT = false>
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8]) {
    const v4i w = v4i{(int)pack_bf16x2_rne(v[0], v[1]), (int)pack_bf16x2_rne(v[2], v[3]),
                      (int)pack_bf16x2_rne(v[4], v[5]), (int)pack_bf16x2_rne(v[6], v[7])};
    if (NT) __builtin_nontemporal_store(w, reinterpret_cast<v4i *>(p));
    else *reinterpret_cast<v4i *>(p) = w;
}
template <bool NT = false>
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    const v4f lo = v4f{v[0], v[1], v[2], v[3]}, hi = v4f{v[4], v[5], v[6], v[7]};
    v4f *q = reinterpret_cast<v4f *>(p);
    if (NT) {
        __builtin_nontemporal_store(lo, q);
        __builtin_nontemporal_store(hi, q + 1);
    } else {
        q[0] = lo;
        q[1] = hi;
    }
}

// The value of the lane `N` places further round the 16-lane row (DPP
// row_ror): reducing over N = 8, 4, 2, 1 leaves the row's result in every lane
// without LDS traffic.
template <int N>
__device__ __forceinline__ float ror16(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x120 + N, 0xf, 0xf, true));
}
// NaN operands are left out by fmaxf
__device__ __forceinline__ float max16(float x) {
    x = fmaxf(x, ror16<8>(x));
    x = fmaxf(x, ror16<4>(x));
    x = fmaxf(x, ror16<2>(x));
    return fmaxf(x, ror16<1>(x));
}
__device__ __forceinline__ float sum16(float x) {
    x += ror16<8>(x);
    x += ror16<4>(x);
    x += ror16<2>(x);
    return x + ror16<1>(x);
}
// sum over the wave, the same bits in every lane
__device__ __forceinline__ float sum64(float x) {
    x = sum16(x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

}  // namespace dg
