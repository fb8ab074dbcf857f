// dg_gated.h -- device helpers of the gated GEMM's kernels: small LDS-DMA
// loads, and the walk over the contiguous layout's expert segments.
#pragma once

#include "dg_pipeline.h"

namespace dg {

// One 4-byte-per-lane buffer load into LDS (256 B per wave at `dst`).
__device__ __forceinline__ void dma_lds4(__amdgpu_buffer_rsrc_t r, uint8_t *dst, int voffset, int soffset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, DG_LDS(dst), 4, voffset, soffset, 0, 0);
}

// Waits for this wave's LDS reads, so that a DMA may overwrite what they
// read; a stage that only one wave uses needs no barrier besides.
__device__ __forceinline__ void lds_reads_done() {
    __builtin_amdgcn_s_waitcnt(0xc07f);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Expert indices of blocks base + 64 q + lane (-1 past the end): one round of
// contig_scan, all loads in flight together.
struct ContigBlocks {
    int e[4];
};
__device__ __forceinline__ ContigBlocks contig_load(const int32_t *idx, int nblocks, int base) {
    ContigBlocks r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int b = base + 64 * q + (int)(threadIdx.x & 63);
        r.e[q] = b < nblocks ? idx[(int64_t)b * 128] : -1;
    }
    return r;
}

// Contiguous layout with 256-row tiles: a "unit" is every other 128-row block
// of an expert's segment (its first, its third, ..) with the block behind it,
// so it never mixes two experts' rows; the last one of a segment with an odd
// number of blocks holds 128 rows.  Returns the first block of unit u (-1 for
// none, or u < 0) to every lane and leaves the number of units in `units`.
// `first`: the first round's blocks, which two walks can share.
__device__ __forceinline__ int contig_scan(const int32_t *idx, int nblocks, const ContigBlocks &first, int u, int &units) {
    const int lane = threadIdx.x & 63;
    const uint64_t upto = ~0ull >> (63 - lane);   // this lane and those before it
    int prev_e = -1;     // expert of the block before this step (none: -1)
    int seg = -1;        // first block of the segment running into this step
    int count = 0, found = -1;
    for (int base = 0; base < nblocks; base += 256) {
        ContigBlocks r = first;
        if (base > 0) r = contig_load(idx, nblocks, base);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int e = r.e[q], b0 = base + 64 * q;
            int ep = __shfl_up(e, 1);
            if (lane == 0) ep = prev_e;
            const uint64_t starts = __ballot(e >= 0 && e != ep);
            const int sg = starts & upto ? b0 + 63 - __clzll((long long)(starts & upto)) : seg;
            const bool unit = e >= 0 && ((b0 + lane - sg) & 1) == 0;
            const uint64_t m = __ballot(unit);
            const int n = __popcll(m);
            if (u >= count && u < count + n) {
                const int rank = __popcll(m & (upto >> 1));
                const uint64_t hit = __ballot(unit && rank == u - count);
                found = b0 + __ffsll((unsigned long long)hit) - 1;
            }
            count += n;
            prev_e = __shfl(e, 63);
            seg = __shfl(sg, 63);
        }
    }
    units = count;
    return found;
}

}  // namespace dg
