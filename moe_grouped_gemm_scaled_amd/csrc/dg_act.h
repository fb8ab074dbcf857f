// dg_act.h -- the gate's activation and its derivative.  Both kinds are
// act(g) = g * s(v) with the logistic function s: SiLU has v = g; the tanh
// form of GELU, 0.5 g (1 + tanh z) with z = sqrt(2/pi) (g + 0.044715 g^3), has
// v = 2z, since (1 + tanh z) / 2 = s(2z).  So
//     act'(g) = s + act(g) (1 - s) v'.
// act(g) (1 - s) is 0 long before g^2 in GELU's v' leaves the range of fp32; the
// square is bounded there, so that the product stays 0.
// s(v) = 1 / (1 + 2^(-v log2 e)) with the hardware exponential and reciprocal
// (about 1 ulp each), without cancellation for any v; v -> -inf gives 0.
#pragma once

#include "dg_device.h"

namespace dg {

constexpr int kActSilu = 0, kActGelu = 1;

template <int ACT>
__device__ __forceinline__ float act_sigmoid(float g) {
    float v = g;
    if constexpr (ACT == kActGelu) v = g * __builtin_fmaf(0.071354816f, g * g, 1.5957691f);   // 2 sqrt(2/pi) (0.044715 g^2 + 1)
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * v));
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    return g * act_sigmoid<ACT>(g);
}

template <int ACT>
__device__ __forceinline__ void act_and_grad(float g, float &a, float &da) {
    const float s = act_sigmoid<ACT>(g);
    a = g * s;
    float k = 1.0f;
    if constexpr (ACT == kActGelu) k = __builtin_fmaf(0.21406445f, fminf(g * g, 1e30f), 1.5957691f);
    da = __builtin_fmaf(a * (1.0f - s), k, s);
}

}  // namespace dg
