// dg_index.h -- index arithmetic of the experts' row operators that has to hold
// up to the ends of their sizes; plain C++, which the tests run on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

// f(i) for thread t's indices, every `step`th, of part `part` of [0, n) dealt to
// `parts` in order; n below 2^31.  Counted without a sign: the step past the
// last index may reach 2^31, where an int would wrap round and go on.
template <class F>
__host__ __device__ __forceinline__ void for_share(int n, int part, int parts, int t, int step, F &&f) {
    const uint32_t lo = (uint32_t)((int64_t)n * part / parts), hi = (uint32_t)((int64_t)n * (part + 1) / parts);
    for (uint32_t i = lo + (uint32_t)t; i < hi; i += (uint32_t)step) f((int)i);
}

// Part `part` of [0, n) dealt to `parts`: [lo, hi).  The first n % parts of them
// take one more; no product passes n.
struct Share {
    int lo, hi;
};
__host__ __device__ __forceinline__ Share share_of(int n, int part, int parts) {
    const int each = n / parts, more = n - each * parts;
    const int lo = each * part + (part < more ? part : more);
    return {lo, lo + each + (part < more ? 1 : 0)};
}

// Runs of `size` that cover n (n + size may pass 2^31).
__host__ __device__ __forceinline__ int runs_of(int n, int size) { return n / size + (n % size != 0); }

}  // namespace dg
