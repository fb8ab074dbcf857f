// moe.hip -- tokens to the experts' rows and back, for gfx950.
//
// With T tokens, top_k choices each and G experts, a pair p = t * top_k + j is
// a token's j-th choice.  The sort gives every pair a row of the experts'
// layout (contiguous: segments of whole 128-row blocks, masked: M_cap rows per
// expert), in pair order within an expert:
//     rows[p] = start[e] + |{p' < p : ids[p'] = ids[p] = e}|
// dispatch:  row rows[t, j] of q, sf = quantise(w[t, j] * x[t])
// combine:   out[t] = residual[t] + sum_j w[t, j] * y[rows[t, j]]
// gradient of combine:  dw[t, j] = dout[t] . y[rows[t, j]],
//                       dy[rows[t, j]] = w[t, j] * dout[t]  (a dispatch)
// (and combine without weights is the gradient of dispatch).
//
// Everything but the sort is HBM-bound.
#include "dg_index.h"
#include "dg_layer.h"
#include "dg_quant.h"
#include "dg_rows.h"

namespace dg {

// Division of numbers below 2^31 by a number known to the host: n / d =
// (n * mul) >> (31 + l) with mul = ceil(2^(31 + l) / d) and 2^(l - 1) < d <= 2^l.
// mul is below 2^32, and d * mul at most d - 1 above 2^(31 + l), which moves the
// quotient of n < 2^31 by less than 1 / d, while its fraction is at most 1 - 1 / d.
struct Divisor {
    uint32_t mul = 0;
    int shift = 0;
    explicit Divisor(int d) {
        int l = 0;
        while (((int64_t)1 << l) < d) ++l;
        mul = (uint32_t)((((uint64_t)1 << (31 + l)) + (uint32_t)d - 1) / (uint32_t)d);
        shift = 31 + l;
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (uint32_t)(((uint64_t)n * mul) >> shift); }
};

// ---------------------------------------------------------------- sort

struct SortArgs {
    const int32_t *ids;
    int32_t *rows, *src, *expert, *counts, *ks;
    int32_t *hist;       // per workgroup and expert, from the counting kernel; NULL: counted here
    int n, G, cap, R, chunk, chunks;
};

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

// Counts of every chunk's ids, for sorts of so many pairs that each workgroup
// counting all of them would take longer than a second launch.
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(SortArgs p) {
    extern __shared__ int32_t bins[];
    for (int e = threadIdx.x; e < p.G; e += kSortThreads) bins[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.n);
    for (int i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const int e = p.ids[i];
        if ((unsigned)e < (unsigned)p.G) atomicAdd(&bins[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.G; e += kSortThreads) p.hist[(int64_t)blockIdx.x * p.G + e] = bins[e];
}

// Lanes of the wave that hold the same key (below 2^bits) as this one.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool one = (key >> b) & 1;
        const uint64_t v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
}

// A stable counting sort: workgroup b ranks the pairs of its chunk.  It needs
// the counts of the pairs before the chunk (ranks) and of all pairs (starts);
// within the chunk, wave w ranks a run of consecutive pairs, 64 at a time, from
// ballots over the bits of their keys, and the waves' counts are added up in
// order.  No result depends on the order in which anything runs: LDS atomics
// only count.  Bound by latency: some ten dependent steps, 2.8 us for 8 pairs, 5.5
// for 1998, 6.1 (and 4.7 for the counts) for 32768.
//
// LDS: before[G], total[G], start[G] (32 bits) and the waves' counts [16][G]
// (16 bits: a chunk is at most 2^13 pairs), whose place the counting of other
// chunks uses first, four copies of each bin by lane so that a popular expert
// holds a wave up a quarter as long.
__global__ void __launch_bounds__(kSortThreads) moe_sort_kernel(SortArgs p) {
    extern __shared__ __attribute__((aligned(16))) int32_t lds[];
    const int G = p.G, t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int32_t *bins = lds, *before = lds + 8 * G, *total = before + G, *start = total + G;
    uint16_t *hist = reinterpret_cast<uint16_t *>(lds);
    __shared__ int32_t scan[kSortWaves];
    // workgroups past the last chunk rank nothing: they fill rows
    const int lo = min((int)blockIdx.x * p.chunk, p.n), hi = min(lo + p.chunk, p.n);
    const bool alone = gridDim.x == 1;
    // the wave's run of pairs, on its way while the others are counted
    constexpr int kMostRounds = 8;                     // chunk <= 8192
    const int rounds = p.chunk / kSortThreads;
    int key[kMostRounds];
    static_for<kMostRounds>([&](auto rc) __attribute__((always_inline)) {
        constexpr int r = decltype(rc)::value;
        const int i = lo + (wave * rounds + r) * 64 + lane;
        key[r] = r < rounds && i < hi ? p.ids[i] : -1;
    });
    for (int e = t; e < 10 * G; e += kSortThreads) lds[e] = 0;
    __syncthreads();
    // ---- counts of the pairs before the chunk, and of those behind it
    if (p.hist) {
        const int parts = kSortThreads / G, part = t / G, e = t - part * G;      // G <= 1024
        if (part < parts) {
            int a = 0, b = 0;
#pragma unroll 8
            for (int c = part; c < p.chunks; c += parts) {
                const int v = p.hist[(int64_t)c * G + e];
                a += c < (int)blockIdx.x ? v : 0;
                b += c > (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&before[e], a);
            atomicAdd(&total[e], b);
        }
        __syncthreads();
    } else if (!alone) {
        constexpr int kLoads = 8;                      // in flight
        const int copy = lane & 3;
        for (int i0 = 0; i0 < p.n; i0 += kLoads * kSortThreads) {          // n <= 2^26
            int e[kLoads];
            static_for<kLoads>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const int i = i0 + u * kSortThreads + t;
                e[u] = i < p.n && (i < lo || i >= hi) ? p.ids[i] : -1;
            });
            static_for<kLoads>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value;
                const bool behind = i0 + u * kSortThreads >= hi;    // chunks are whole rows of threads
                if ((unsigned)e[u] < (unsigned)G) atomicAdd(&bins[(behind ? 4 * G : 0) + 4 * e[u] + copy], 1);
            });
        }
        __syncthreads();
        if (t < 2 * G) {
            const v4i c = *reinterpret_cast<const v4i *>(bins + 4 * t);
            before[t] = c.x + c.y + c.z + c.w;         // before[G], then total[G]
        }
        if (G > kSortThreads / 2 && t + kSortThreads < 2 * G) {
            const v4i c = *reinterpret_cast<const v4i *>(bins + 4 * (t + kSortThreads));
            before[t + kSortThreads] = c.x + c.y + c.z + c.w;
        }
        __syncthreads();
        for (int e = t; e < 8 * G; e += kSortThreads) bins[e] = 0;
        __syncthreads();
    }
    // ---- ranks within the wave's run
    const int bits = 32 - __clz(G);                    // keys 0 .. G, G: no expert
    uint16_t *mine = hist + wave * G;
    int rank[kMostRounds];
    static_for<kMostRounds>([&](auto rc) __attribute__((always_inline)) {
        constexpr int r = decltype(rc)::value;
        if (r < rounds) {                              // uniform
            key[r] = (unsigned)key[r] < (unsigned)G ? key[r] : G;
            const uint64_t m = same_key(key[r], bits);
            const int below = __popcll(m & ((1ull << lane) - 1));
            rank[r] = 0;
            if (key[r] < G) {
                // one wave's LDS accesses stay in order: all lanes read, then the first writes
                const int had = *reinterpret_cast<volatile uint16_t *>(&mine[key[r]]);
                __builtin_amdgcn_wave_barrier();
                rank[r] = had + below;
                if (below == 0) *reinterpret_cast<volatile uint16_t *>(&mine[key[r]]) = (uint16_t)(had + __popcll(m));
            }
        }
    });
    __syncthreads();
    // ---- the waves' counts become offsets; totals and padded sizes
    int32_t sum = 0;
    if (t < G) {
        int run = 0, c[kSortWaves];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) c[w] = hist[w * G + t];     // all before the first is written
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            hist[w * G + t] = (uint16_t)run;
            run += c[w];
        }
        total[t] += before[t] + run;
        sum = p.cap ? 0 : (total[t] + 127) & ~127;
    }
    // ---- starts: an exclusive scan of the padded sizes (G <= 1024 threads)
    if (p.cap) {
        if (t < G) start[t] = t * p.cap;
    } else {
        int inc = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(inc, d);
            if (lane >= d) inc += v;
        }
        if (lane == 63) scan[wave] = inc;
        __syncthreads();
        if (t < G) {
            int base = 0;
            for (int w = 0; w < wave; ++w) base += scan[w];
            start[t] = base + inc - sum;
        }
    }
    __syncthreads();
    auto room = [&](int e) __attribute__((always_inline)) { return p.cap ? p.cap : max(p.R - start[e], 0); };
    if (blockIdx.x == 0 && t < G) {
        if (p.counts) p.counts[t] = min(total[t], room(t));
        if (p.ks) p.ks[t] = min((total[t] + 127) & ~127, room(t));
    }
    static_for<kMostRounds>([&](auto rc) __attribute__((always_inline)) {
        constexpr int r = decltype(rc)::value;
        if (r < rounds) {
            const int i = lo + (wave * rounds + r) * 64 + lane;
            if (i < hi) {
                const int e = key[r];
                int row = -1;
                if (e < G) {
                    const int at = before[e] + hist[wave * G + e] + rank[r];
                    if (at < room(e)) row = start[e] + at;
                }
                p.rows[i] = row;
                if (p.src && row >= 0) p.src[row] = i;
            }
        }
    });
    // ---- this workgroup's share of the rows: the expert of each, and -1 where there is none
    if (p.cap) {
        if (!p.src) return;
        for_share(p.R, (int)blockIdx.x, (int)gridDim.x, t, kSortThreads, [&](int r) __attribute__((always_inline)) {
            const int e = r / p.cap;
            if (r - e * p.cap >= total[e]) p.src[r] = -1;
        });
        return;
    }
    if (!p.src && !p.expert) return;
    // a 128-row block per wave: all of it belongs to one segment, or to none
    const int blocks = p.R / 128, step = (int)gridDim.x * kSortWaves;
    for (int b = (int)blockIdx.x * kSortWaves + wave; b < blocks; b += step) {
        int e = 0, top = G;                            // the last expert that starts at or before the block
        while (top - e > 1) {
            const int m = (e + top) >> 1;
            if (start[m] <= 128 * b) e = m;
            else top = m;
        }
        const int held = total[e] - (128 * b - start[e]);
#pragma unroll
        for (int h = 0; h < 128; h += 64) {
            const bool in = h + lane < held;
            if (p.expert) p.expert[128 * b + h + lane] = in ? e : -1;
            if (p.src && !in) p.src[128 * b + h + lane] = -1;
        }
    }
}

// Pairs per workgroup: 1024, more only where that would be more than 64
// workgroups.
static int sort_chunk(int64_t n) {
    int chunk = kSortThreads;
    while (chunk < 8 * kSortThreads && n > (int64_t)64 * chunk) chunk *= 2;
    return chunk;
}

// Most pairs for which every workgroup counts all of them instead of a kernel
// before it (32768 pairs, 64 experts: 8.0 us with the kernel before it, 9.3 without;
// 16384 pairs: 7.1 without; each in a graph).  The table of counts has a row per
// chunk, and every workgroup reads all of it: chunks grow to 8192 pairs, and past
// 2^19 pairs the reads grow with the square of the pairs (in a graph, 64 experts:
// 2^19 pairs 22 us, 2^23 100, 2^26 1.9 ms; 1024 experts: 2^20 44 us, 2^23 454, 2^26
// 22 ms).
constexpr int64_t kSortOneLaunch = 16384;

// Workgroups: one per chunk, and one per 2048 rows of m_indices and src to
// fill (512 pairs on 256 experts, 33024 rows: 5.7 us, 15.9 with one
// workgroup; 1998 pairs on 32: 5.3, 6.6 with one).
constexpr int kSortFill = 2048;
static int64_t sort_groups(int64_t n, int64_t R) {
    const int chunk = sort_chunk(n);
    const int64_t by_pairs = (n + chunk - 1) / chunk, by_rows = (R + kSortFill - 1) / kSortFill;
    const int64_t g = by_rows < 64 ? by_rows : 64;
    return by_pairs > g ? by_pairs : g > 0 ? g : 1;
}

size_t moe_sort_workspace(int64_t n, int G) {
    if (n <= kSortOneLaunch) return 0;
    return (size_t)((n + sort_chunk(n) - 1) / sort_chunk(n)) * G * sizeof(int32_t);
}

hipError_t launch_moe_sort(const MoeSortProblem &p, hipStream_t stream) {
    const int chunk = sort_chunk(p.n);
    const int64_t chunks = ((int64_t)p.n + chunk - 1) / chunk;
    const int64_t groups = sort_groups(p.n, p.src || p.expert ? p.R : 0);
    if (!grid_fits(groups, kSortThreads)) return hipErrorInvalidValue;
    const size_t need = moe_sort_workspace(p.n, p.G);
    SortArgs a{p.ids, p.rows, p.src, p.expert, p.counts, p.ks, nullptr, p.n, p.G, p.cap, p.R, chunk, (int)chunks};
    if (need && p.ws && p.ws_bytes >= need) {
        a.hist = static_cast<int32_t *>(p.ws);
        hipLaunchKernelGGL(moe_count_kernel, dim3((unsigned)chunks), dim3(kSortThreads), p.G * sizeof(int32_t), stream, a);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(moe_sort_kernel, dim3((unsigned)groups), dim3(kSortThreads), 11 * p.G * sizeof(int32_t), stream, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- dispatch, by token

struct DispatchArgs {
    const void *x;
    const float *weights;         // [T][top_k] or NULL
    const int32_t *rows;          // [T][top_k]
    const uint16_t *ye;           // kDot: the experts' outputs [R][K]
    float *dw;                    // kDot: [T][top_k]
    uint16_t *y;
    uint8_t *q;
    void *sf;
    int64_t ld_x, sf_group;       // sf words of one group
    int T, top_k, K, R, cap, ld_sf, format;
};

// Sixteen consecutive values as stored.
template <typename T>
struct Raw16 {
    Raw8<T> lo, hi;
};
template <typename T>
__device__ __forceinline__ Raw16<T> load16(const T *p) {
    return {load8<true>(p), load8<true>(p + 8)};
}
template <typename T>
__device__ __forceinline__ float get16(const Raw16<T> &r, int i) {
    return i < 8 ? get8(r.lo, i) : get8(r.hi, i - 8);
}

// The maximum over each 8 lanes (of a 128-column block), in all of them; NaN is left out.
__device__ __forceinline__ float max_of_8_lanes(float x) {
    auto moved = [&](auto ctrl) __attribute__((always_inline)) {
        return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    x = fmaxf(x, moved(std::integral_constant<int, 0xb1>{}));     // quad_perm 1 0 3 2
    x = fmaxf(x, moved(std::integral_constant<int, 0x4e>{}));     // quad_perm 2 3 0 1
    return fmaxf(x, moved(std::integral_constant<int, 0x141>{})); // row_half_mirror
}

// A dot product over K columns is the sum, in order, of those over each run of
// 512 columns, 8 to a lane: the same bits whichever kernel computes it.
constexpr int kDotBatch = 4, kDotRuns = kNormMaxK / 512;
template <typename TX>
__device__ __forceinline__ float dot_of_run(const Raw8<TX> &x, const Raw8<uint16_t> &y, bool in) {
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) d = __builtin_fmaf(get8(x, i), get8(y, i), d);
    return sum64(in ? d : 0.f);
}
__device__ __forceinline__ float sum_of_runs(const float *d, int runs) {
    float s = d[0];
    for (int c = 1; c < runs; ++c) s += d[c];
    return s;
}

// A token's row is read once, quantised (once without weights) and written to
// each of its rows.  WPR waves share a token (WPR = 1: four tokens per
// workgroup); lane l of wave w holds the 16 columns from
// 16 * (64 * (WPR * c + w) + l), c < NCH, so 8 lanes hold a 128-column block and
// a store writes 1 KB of a row's codes.  The blocks' maxima meet in LDS, from
// where one store writes up to 64 scales of a row: each lies in a line of its
// own, and neighbouring tokens, which run on one XCD, have neighbouring rows in
// each expert, so that their scales fill these lines in one L2.
// With weights, the block's maximum is |w| max|x|: rounding is monotone, so
// that is the largest of the rounded products.
// blockIdx.y: a share of the choices, where there are few tokens.
// Bound by the stores: 4096 tokens of 7168 to 8 rows each 62 to 65 us, 3.8 TB/s of
// codes (76 with 8 columns per lane and every row and scale looked up and stored
// per chunk; 68 of those without the scales); one token to 8 rows 3.7 us, 5.5 from
// a single workgroup.  With weights a token is encoded once per choice: 79 us, and
// with the dot products, which read the experts' rows, 149 (5.2 TB/s in all).
// kDot: also dw[t, j] = x[t] . ye[rows[t, j]], added up in a fixed order.
template <typename TX, int WPR, int NCH, bool kW, bool kDot>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR)
moe_dispatch_kernel(DispatchArgs p) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blk = xcd_remap(blockIdx.x, gridDim.x);
    const int tok = WPR == 1 ? blk * 4 + wave : blk;
    const int w0 = WPR == 1 ? 0 : wave;
    const int K = p.K;
    if (WPR == 1 && tok >= p.T) return;
    const Share choices = share_of(p.top_k, (int)blockIdx.y, (int)gridDim.y);
    const int j_lo = choices.lo, j_hi = choices.hi;
    const int32_t *rows = p.rows + (int64_t)tok * p.top_k;
    const float *ws = kW ? p.weights + (int64_t)tok * p.top_k : nullptr;

    const TX *xr = static_cast<const TX *>(p.x) + (int64_t)tok * p.ld_x;
    // up to 64 choices' rows and weights in the lanes of a wave: one load, not one after the other
    auto row_of = [&](int j0) __attribute__((always_inline)) { return j0 + lane < j_hi ? rows[j0 + lane] : -1; };
    auto weight_of = [&](int j0) __attribute__((always_inline)) { return kW && j0 + lane < j_hi ? ws[j0 + lane] : 0.f; };
    int row64 = row_of(j_lo);
    if constexpr (kDot) {
        // 8 columns per lane here, so that a load reads 1 KB of a row of ye
        Raw8<TX> xd[2 * NCH];
        int cold[2 * NCH];
        static_for<2 * NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            cold[c] = 8 * (64 * (WPR * c + w0) + lane);
            xd[c] = load8(xr + min(cold[c], K - 8));
        });
        __shared__ float runs_of[WPR == 1 ? 4 : 1][kDotBatch][2 * WPR * NCH];
        float(&red)[kDotBatch][2 * WPR * NCH] = runs_of[WPR == 1 ? wave : 0];
        for (int j0 = j_lo; j0 < j_hi; j0 += kDotBatch) {
            const int rj = j0 == j_lo ? row64 : row_of(j0);
            static_for<kDotBatch>([&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                if (j0 + j < j_hi) {                   // uniform
                    const int r = __builtin_amdgcn_readlane(rj, j);
                    if ((unsigned)r < (unsigned)p.R) {
                        const uint16_t *yr = p.ye + (int64_t)r * K;
                        Raw8<uint16_t> yv[2 * NCH];
                        static_for<2 * NCH>([&](auto cc) __attribute__((always_inline)) {
                            constexpr int c = decltype(cc)::value;
                            yv[c] = load8<true>(yr + min(cold[c], K - 8));
                        });
                        static_for<2 * NCH>([&](auto cc) __attribute__((always_inline)) {
                            constexpr int c = decltype(cc)::value;
                            const float s = dot_of_run(xd[c], yv[c], cold[c] < K);
                            if (lane == 0) red[j][WPR * c + w0] = s;
                        });
                    }
                }
            });
            if constexpr (WPR > 1) __syncthreads();
            else __builtin_amdgcn_wave_barrier();      // one wave's LDS accesses stay in order
            const int j = WPR > 1 ? (int)threadIdx.x : lane;
            if (j < kDotBatch && j0 + j < j_hi) {
                const bool held = (unsigned)rows[j0 + j] < (unsigned)p.R;
                p.dw[(int64_t)tok * p.top_k + j0 + j] = held ? sum_of_runs(red[j], (K + 511) / 512) : 0.f;
            }
            if constexpr (WPR > 1) __syncthreads();
            else __builtin_amdgcn_wave_barrier();
        }
    }
    if (!p.q && !p.y) return;                          // uniform
    Raw16<TX> xv[NCH];
    int col[NCH];
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        col[c] = 16 * (64 * (WPR * c + w0) + lane);
        xv[c] = load16(xr + min(col[c], K - 16));
    });
    // ---- the blocks' maxima, in registers and LDS
    __shared__ float maxima[WPR == 1 ? 4 : 1][8 * WPR * NCH];
    float *bmax = maxima[WPR == 1 ? wave : 0];
    float amax[NCH];
    uint4 code[NCH];
    auto encode = [&](int c, float w, float m) __attribute__((always_inline)) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = kW ? w * get16(xv[c], i) : get16(xv[c], i);
        uint32_t o[4];
        auto four = [&](auto ue) __attribute__((always_inline)) {
            constexpr bool UE = decltype(ue)::value;
            const BlockDivisor d = block_divisor<UE>(block_scale<UE>(m));
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = encode4<UE>(v4f{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}, d);
        };
        if (p.format == kSfFp32) four(std::false_type{});
        else four(std::true_type{});
        return uint4{o[0], o[1], o[2], o[3]};
    };
    if (p.q) {
        static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(get16(xv[c], i)));
            amax[c] = max_of_8_lanes(m);
            if ((lane & 7) == 0) bmax[8 * (WPR * c + w0) + (lane >> 3)] = amax[c];
            if constexpr (!kW) code[c] = encode(c, 1.f, amax[c]);
        });
        if constexpr (WPR > 1) __syncthreads();
        else __builtin_amdgcn_wave_barrier();          // one wave's LDS accesses stay in order
    }
    const int blocks = K / kKBlock, words = p.format == kSfPacked ? (blocks + 3) / 4 : blocks;
    for (int j0 = j_lo; j0 < j_hi; j0 += 64) {
        if (j0 > j_lo) row64 = row_of(j0);
        const float weight64 = weight_of(j0);
        const int n = min(j_hi - j0, 64);
        // ---- the rows
        for (int j = 0; j < n; ++j) {
            const int r = __builtin_amdgcn_readlane(row64, j);
            if ((unsigned)r >= (unsigned)p.R) continue;
            const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight64), j));
            static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
                constexpr int c = decltype(cc)::value;
                if (p.q) {
                    if constexpr (kW) code[c] = encode(c, w, fabsf(w) * amax[c]);
                    if (col[c] < K)
                        __builtin_nontemporal_store(__builtin_bit_cast(v4i, code[c]),
                                                    reinterpret_cast<v4i *>(p.q + (int64_t)r * K + col[c]));
                }
                if (p.y && col[c] < K) {
                    float lo[8], hi[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        lo[i] = kW ? w * get16(xv[c], i) : get16(xv[c], i);
                        hi[i] = kW ? w * get16(xv[c], i + 8) : get16(xv[c], i + 8);
                    }
                    uint16_t *dst = p.y + (int64_t)r * K + col[c];
                    store8<true>(dst, lo);
                    store8<true>(dst + 8, hi);
                }
            });
        }
        if (!p.q) continue;
        // ---- their scales, a row per wave at a time
        for (int j = w0; j < n; j += WPR) {
            const int r = __builtin_amdgcn_readlane(row64, j);
            if ((unsigned)r >= (unsigned)p.R) continue;
            const float w = fabsf(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight64), j)));
            const int g = p.cap == p.R ? 0 : r / p.cap;
            uint32_t *sf = static_cast<uint32_t *>(p.sf) + g * p.sf_group + (r - g * p.cap);
            for (int b = lane; b < words; b += 64) {
                uint32_t word;
                if (p.format == kSfPacked) {
                    word = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * b + i < blocks)
                            word |= (__float_as_uint(block_scale<true>(kW ? w * bmax[4 * b + i] : bmax[4 * b + i])) >> 23) << (8 * i);
                } else {
                    const float m = kW ? w * bmax[b] : bmax[b];
                    word = __float_as_uint(p.format == kSfFp32 ? block_scale<false>(m) : block_scale<true>(m));
                }
                sf[(int64_t)b * p.ld_sf] = word;
            }
        }
    }
}

template <typename TX, int WPR, int NCH, bool kW, bool kDot>
static hipError_t launch_dispatch_t(const DispatchArgs &a, int num_cus, hipStream_t stream) {
    const int64_t groups = WPR == 1 ? ((int64_t)a.T + 3) / 4 : a.T;
    constexpr int kThreads = WPR == 1 ? 256 : 64 * WPR;
    // few tokens: the choices of one are dealt to several workgroups
    const int64_t share = groups < num_cus ? (num_cus / groups < a.top_k ? num_cus / groups : a.top_k) : 1;
    if (!grid_fits(groups * share, kThreads)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((moe_dispatch_kernel<TX, WPR, NCH, kW, kDot>), dim3((unsigned)groups, (unsigned)share), dim3(kThreads), 0,
                       stream, a);
    return hipGetLastError();
}

// Waves per token, 16 columns of each lane's where they reach; two runs of columns
// per lane from 4097 columns on, but eight waves for fewer than 512 tokens, where a
// token's latency shows and each wave encodes half as much per choice (in a graph,
// 8 choices, 7168 columns: 500 tokens 8.9 us, 9.7 with four waves, with weights 13.6
// and 14.6; 64 tokens with weights 4.7 and 5.4; 1024 tokens 16.8, 17.5 with eight, of
// 4224 columns 10.4 and 12.6).
template <typename TX, bool kW, bool kDot>
static hipError_t launch_dispatch_k(const DispatchArgs &a, int num_cus, hipStream_t stream) {
    const int n = (a.K + 1023) / 1024;                 // 1024-column chunks
    if (n <= 1) return launch_dispatch_t<TX, 1, 1, kW, kDot>(a, num_cus, stream);
    if (n <= 2) return launch_dispatch_t<TX, 2, 1, kW, kDot>(a, num_cus, stream);
    if (n <= 4) return launch_dispatch_t<TX, 4, 1, kW, kDot>(a, num_cus, stream);
    if (n <= 8 && a.T < 512) return launch_dispatch_t<TX, 8, 1, kW, kDot>(a, num_cus, stream);
    if (n <= 8) return launch_dispatch_t<TX, 4, 2, kW, kDot>(a, num_cus, stream);
    if (n <= 16) return launch_dispatch_t<TX, 8, 2, kW, kDot>(a, num_cus, stream);
    return hipErrorInvalidValue;
}

template <typename TX>
static hipError_t launch_dispatch_w(const DispatchArgs &a, int num_cus, hipStream_t stream) {
    if (a.dw)
        return a.weights ? launch_dispatch_k<TX, true, true>(a, num_cus, stream)
                         : launch_dispatch_k<TX, false, true>(a, num_cus, stream);
    return a.weights ? launch_dispatch_k<TX, true, false>(a, num_cus, stream)
                     : launch_dispatch_k<TX, false, false>(a, num_cus, stream);
}

// ---------------------------------------------------------------- dispatch, by 128 x 128 tile

struct TileArgs {
    const void *x;
    const float *weights;
    const int32_t *src;
    uint16_t *y;
    uint8_t *q;
    void *sf;
    uint8_t *qt;
    float *sft;
    int64_t ld_x;
    int pairs, K, R, tiles_m;
    Divisor by_top_k;
    // kDot: the first T workgroups' work
    const int32_t *rows;
    const uint16_t *ye;
    float *dw;
    int T, top_k;
};

// Magnitudes as integers, whose order is that of the numbers, with infinities
// and then NaN on top: no canonicalisation, no separate test for NaN.  bf16:
// two to a register.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
template <typename T>
struct Mag8;   // magnitudes of 8 values, elementwise maxima of them, and their largest as fp32 bits
template <>
struct Mag8<uint16_t> {
    uint32_t m[4];
    __device__ __forceinline__ explicit Mag8(const Raw8<uint16_t> &r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = (uint32_t)r.a[i] & 0x7fff7fffu;
    }
    __device__ __forceinline__ void max(const Mag8 &o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = max_u16x2(m[i], o.m[i]);
    }
    __device__ __forceinline__ uint32_t largest() const {
        const uint32_t v = max_u16x2(max_u16x2(m[0], m[1]), max_u16x2(m[2], m[3]));
        return ::max(v & 0xffff0000u, v << 16);
    }
};
template <>
struct Mag8<float> {
    uint32_t m[8];
    __device__ __forceinline__ explicit Mag8(const Raw8<float> &r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = __float_as_uint(get8(r, i)) & 0x7fffffffu;
    }
    __device__ __forceinline__ void max(const Mag8 &o) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = ::max(m[i], o.m[i]);
    }
    __device__ __forceinline__ uint32_t largest() const {
        return ::max(::max(::max(m[0], m[1]), ::max(m[2], m[3])), ::max(::max(m[4], m[5]), ::max(m[6], m[7])));
    }
};
template <int N>
__device__ __forceinline__ uint32_t ror16u(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x120 + N, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t max16u(uint32_t x) {
    x = max(x, ror16u<8>(x));
    x = max(x, ror16u<4>(x));
    x = max(x, ror16u<2>(x));
    return max(x, ror16u<1>(x));
}
// lane I of each four, in all of them
template <int I>
__device__ __forceinline__ float of_quad(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), I * 0x55, 0xf, 0xf, true));
}

typedef unsigned Codes __attribute__((ext_vector_type(2)));   // of eight values

// Four quotients as codes where none is NaN.
__device__ __forceinline__ uint32_t e4m3_encode4_numbers(float a, float b, float c, float d) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// dw[tok, j] = x[tok] . ye[rows[tok, j]] by a workgroup of 8 waves, each of which
// takes every 8th run of 512 columns; 4 choices at a time, whose loads are in
// flight together.  A choice without a row reads row 0 and counts as nothing.
// In the launch of the tiles, whose stores and arithmetic run beside these reads:
// 8192 tokens of 7168, 4 choices: 217 us, 5.0 TB/s in all, 226 in two launches; 333
// tokens of 2048, 2 choices: 6.2 against 8.4 us in a graph.
// `red`: kDotBatch * kDotRuns floats of LDS.
template <typename TX>
__device__ __forceinline__ void dot_of_token(const TileArgs &p, int tok, float *red) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t *rows = p.rows + (int64_t)tok * p.top_k;
    const TX *x = static_cast<const TX *>(p.x) + (int64_t)tok * p.ld_x;
    const int runs = (p.K + 511) / 512;
    for (int j0 = 0; j0 < p.top_k; j0 += kDotBatch) {
        const int mine = lane < kDotBatch && j0 + lane < p.top_k ? rows[j0 + lane] : -1;
        for (int c = wave; c < runs; c += 8) {
            const int col = 512 * c + 8 * lane, at = min(col, p.K - 8);
            const Raw8<TX> xv = load8(x + at);
            Raw8<uint16_t> yv[kDotBatch];
            static_for<kDotBatch>([&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                const int r = __builtin_amdgcn_readlane(mine, j);
                yv[j] = load8<true>(p.ye + (int64_t)((unsigned)r < (unsigned)p.R ? r : 0) * p.K + at);
            });
            static_for<kDotBatch>([&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                const float s = dot_of_run(xv, yv[j], col < p.K);
                if (lane == 0) red[kDotRuns * j + c] = s;
            });
        }
        __syncthreads();
        const int j = threadIdx.x;
        if (j < kDotBatch && j0 + j < p.top_k) {
            const bool held = (unsigned)rows[j0 + j] < (unsigned)p.R;
            p.dw[(int64_t)tok * p.top_k + j0 + j] = held ? sum_of_runs(red + kDotRuns * j, runs) : 0.f;
        }
        __syncthreads();
    }
}

// Both scale directions of a 128 x 128 tile of the experts' rows at once: 512
// threads, thread t holds columns 8 (t % 16) .. +7 of rows t / 16 + 32 i
// (i < 4), so 16 lanes hold a row's 128 columns (its scale is a reduction
// inside the DPP row); the column maxima go through LDS.  Rows that hold no
// pair are zeros; they are written in qt and left alone in q and y.
//
// A token's row is read once per choice.  The tiles of one column run one after
// the other on one XCD, so that all but the first read of a token's 128 columns
// find them in its L2 (8192 tokens: 2 MB of 4; 122 MB read of HBM for 117 MB of
// tokens, top_k = 4).
//
// Two codes per element are nearly as much arithmetic as the stores are time
// (34500 rows of 7168, 8192 tokens, bf16: the loads and stores alone 133 us, the
// arithmetic without the stores 80 us), so it is kept short: maxima of
// magnitudes as integers, two bf16 at a time; of a row's 16 lanes, lane i % 4
// works out row i's scale and divisor and hands them round by DPP; codes without
// the NaN rule, which can only matter to a wave that has seen an infinity or NaN
// (or a weight that makes one) and takes the general path.  Buffer stores keep
// the addresses in scalar registers, which leaves room for four workgroups on a
// CU (64 registers at most for bf16).  166 us, with weights 165; 192 and 203 with
// the general arithmetic and addresses throughout; a fixed grid that fetches the
// next tile ahead needs 80 to 97 registers and takes 190.
template <typename TX, int FMT, bool kW, bool kDot>
__global__ void __launch_bounds__(512, 4) moe_dispatch_tile_kernel(TileArgs p) {
    constexpr bool UE = FMT != kSfFp32;
    constexpr uint32_t kInf = 0x7f800000u;
    __shared__ __attribute__((aligned(16))) float wmax[32][128];
    const int tokens = kDot ? p.T : 0;
    if (kDot && (int)blockIdx.x < tokens) {
        dot_of_token<TX>(p, blockIdx.x, wmax[0]);
        return;
    }
    const int t = threadIdx.x;
    const int c8 = 8 * (t & 15), rg = t >> 4;
    const int tile = xcd_remap((int)blockIdx.x - tokens, (int)gridDim.x - tokens);
    const int tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
    const int K = p.K, n0 = tn * 128, m0 = tm * 128;
    __shared__ __attribute__((aligned(16))) float div_y[128], div_s[128];
    __shared__ int odd;                                // a wave has seen an infinity or NaN
    if (t == 0) odd = 0;
    uint32_t held = 0;                                 // bit i: row i holds a pair
    float w[4];
    Raw8<TX> raw[4];
    {
        int pair[4];
        static_for<4>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            pair[i] = p.src[m0 + rg + 32 * i];         // R is a multiple of 128
        });
        static_for<4>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            raw[i] = Raw8<TX>{};
            w[i] = 0.f;
            if ((unsigned)pair[i] < (unsigned)p.pairs) {
                held |= 1u << i;
                const int64_t tok = p.by_top_k.quotient((uint32_t)pair[i]);
                raw[i] = load8(static_cast<const TX *>(p.x) + tok * p.ld_x + n0 + c8);
                if constexpr (kW) w[i] = p.weights[pair[i]];
            }
        });
    }
    auto value = [&](int i, int e) __attribute__((always_inline)) {
        return kW ? w[i] * get8(raw[i], e) : get8(raw[i], e);
    };
    // ---- magnitudes: of the rows (over 16 lanes), and of the columns over the thread's four rows
    uint32_t top[4];
    bool strange = false;
    {
        Mag8<TX> cols(raw[0]);
        static_for<4>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            const Mag8<TX> m(raw[i]);
            top[i] = max16u(m.largest());
            strange = strange || top[i] >= kInf;
            if constexpr (kW) {
                // rounding is monotone: the largest product is that of the largest magnitude
                top[i] = __float_as_uint(fabsf(w[i]) * __uint_as_float(top[i]));
                strange = strange || top[i] >= kInf || !(fabsf(w[i]) < __builtin_inff());
            } else {
                if constexpr (i > 0) cols.max(m);
            }
        });
        strange = __any(strange);                      // uniform
        float m[8];
        if (kW || strange) {
#pragma unroll
            for (int e = 0; e < 8; ++e)                // fmaxf leaves NaN out
                m[e] = fmaxf(fmaxf(fabsf(value(0, e)), fabsf(value(1, e))), fmaxf(fabsf(value(2, e)), fabsf(value(3, e))));
        } else if constexpr (std::is_same<TX, float>::value) {
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = __uint_as_float(cols.m[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = __uint_as_float(e & 1 ? cols.m[e / 2] & 0xffff0000u : cols.m[e / 2] << 16);
        }
        store8(&wmax[rg][c8], m);
    }
    if (strange) {
        static_for<4>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(value(i, e)));
            top[i] = __float_as_uint(max16(m));
        });
    }
    auto codes = [&](int i, auto general, auto &&div) __attribute__((always_inline)) {
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = divide<UE>(value(i, e), div(e));
        if constexpr (decltype(general)::value)
            return Codes{e4m3_encode4(z[0], z[1], z[2], z[3]), e4m3_encode4(z[4], z[5], z[6], z[7])};
        return Codes{e4m3_encode4_numbers(z[0], z[1], z[2], z[3]), e4m3_encode4_numbers(z[4], z[5], z[6], z[7])};
    };
    // The tile's window of a row-major tensor; row i of the thread lies 32 * i * K
    // elements (a scalar) past its first, and an offset past the window drops
    // the store of a row without a pair.
    auto window = [&](const void *base, int size) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc((void *)((const char *)base + ((int64_t)m0 * K + n0) * size), (short)0,
                                                 128 * K * size, 0x00020000);
    };
    const int at = rg * K + c8;
    constexpr int kPast = 0x7ffffff0, kNt = 2;
    // ---- the rows
    if (p.y) {                                         // uniform
        const __amdgpu_buffer_rsrc_t r = window(p.y, 2);
        static_for<4>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            const v4i o = v4i{(int)pack_bf16x2_rne(value(i, 0), value(i, 1)), (int)pack_bf16x2_rne(value(i, 2), value(i, 3)),
                              (int)pack_bf16x2_rne(value(i, 4), value(i, 5)), (int)pack_bf16x2_rne(value(i, 6), value(i, 7))};
            // the offset in the vector register alone: with a scalar one beside it, gfx950 still reads the data of a
            // 16-byte store when the next instruction writes them over, and the compiler puts no wait between
            __builtin_amdgcn_raw_buffer_store_b128(o, r, held & (1u << i) ? 2 * at + 64 * i * K : kPast, 0, kNt);
        });
    }
    if (p.q) {                                         // uniform
        const __amdgpu_buffer_rsrc_t r = window(p.q, 1);
        const int mine = t & 3;
        const float amax = __uint_as_float(mine & 2 ? (mine & 1 ? top[3] : top[2]) : (mine & 1 ? top[1] : top[0]));
        const float s = block_scale<UE>(amax);
        const BlockDivisor d = block_divisor<UE>(s);
        // lane i of the row's 16 stores row i's scale
        if ((t & 15) < 4 && (held >> mine & 1))
            store_block_scale<FMT == kSfPacked>(static_cast<uint32_t *>(p.sf), p.R, (int64_t)m0 + rg + 32 * mine, tn, K / 128, s);
        auto out = [&](auto general) __attribute__((always_inline)) {
            static_for<4>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                const BlockDivisor di{of_quad<i>(d.y), UE ? 0.f : of_quad<i>(d.s)};
                __builtin_amdgcn_raw_buffer_store_b64(codes(i, general, [&](int) { return di; }), r,
                                                      held & (1u << i) ? at : kPast, 32 * i * K, kNt);
                __builtin_amdgcn_sched_barrier(0);     // row by row: interleaved rows need more registers
            });
        };
        if (strange) out(std::true_type{});
        else out(std::false_type{});
    }
    if (!p.qt) return;                                 // uniform
    // ---- the columns
    __syncthreads();                                   // wmax, and odd is 0
    if (strange && (t & 63) == 0) odd = 1;
    if (t < 128) {
        float m = wmax[0][t];
#pragma unroll
        for (int r = 1; r < 32; ++r) m = fmaxf(m, wmax[r][t]);
        const float s = block_scale<UE>(m);
        const BlockDivisor d = block_divisor<UE>(s);
        div_y[t] = d.y;
        div_s[t] = d.s;
        p.sft[(int64_t)tm * K + n0 + t] = s;
    }
    __syncthreads();
    const __amdgpu_buffer_rsrc_t r = window(p.qt, 1);
    const Raw8<float> y = load8(&div_y[c8]), s = load8(&div_s[c8]);
    auto out = [&](auto general) __attribute__((always_inline)) {
        static_for<4>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            __builtin_amdgcn_raw_buffer_store_b64(codes(i, general, [&](int e) { return BlockDivisor{get8(y, e), get8(s, e)}; }), r,
                                                  at, 32 * i * K, kNt);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    if (odd) out(std::true_type{});
    else out(std::false_type{});
}

template <typename TX, bool kW, bool kDot>
static hipError_t launch_tile_f(const TileArgs &a, int format, hipStream_t stream) {
    const int64_t grid = (int64_t)a.tiles_m * (a.K / 128) + (kDot ? a.T : 0);
    if (!grid_fits(grid, 512)) return hipErrorInvalidValue;
    const dim3 g((unsigned)grid), b(512);
    if (format == kSfFp32) hipLaunchKernelGGL((moe_dispatch_tile_kernel<TX, kSfFp32, kW, kDot>), g, b, 0, stream, a);
    else if (format == kSfUe8m0) hipLaunchKernelGGL((moe_dispatch_tile_kernel<TX, kSfUe8m0, kW, kDot>), g, b, 0, stream, a);
    else hipLaunchKernelGGL((moe_dispatch_tile_kernel<TX, kSfPacked, kW, kDot>), g, b, 0, stream, a);
    return hipGetLastError();
}

template <typename TX>
static hipError_t launch_tile(const MoeDispatchProblem &p, hipStream_t stream) {
    const TileArgs a{p.x, p.weights, p.src, p.y, p.q, p.sf, p.qt, p.sft, p.ld_x, p.T * p.top_k, p.K, p.R, p.R / 128,
                     Divisor(p.top_k), p.rows, p.ye, p.dw, p.T, p.top_k};
    if (p.dw)
        return p.weights ? launch_tile_f<TX, true, true>(a, p.format, stream) : launch_tile_f<TX, false, true>(a, p.format, stream);
    return p.weights ? launch_tile_f<TX, true, false>(a, p.format, stream) : launch_tile_f<TX, false, false>(a, p.format, stream);
}

// By tile where column-scaled codes are wanted, by token otherwise.
hipError_t launch_moe_dispatch(const MoeDispatchProblem &p, int num_cus, hipStream_t stream) {
    if (p.qt && p.R > 0) return p.x_type == kBf16 ? launch_tile<uint16_t>(p, stream) : launch_tile<float>(p, stream);
    if (p.T == 0 || (!p.dw && !p.q && !p.y)) return hipSuccess;
    const DispatchArgs a{p.x, p.weights, p.rows, p.ye, p.dw, p.y, p.q, p.sf, p.ld_x, p.sf_group, p.T, p.top_k, p.K, p.R, p.cap,
                         p.ld_sf, p.format};
    return p.x_type == kBf16 ? launch_dispatch_w<uint16_t>(a, num_cus, stream) : launch_dispatch_w<float>(a, num_cus, stream);
}

// ---------------------------------------------------------------- dispatch of codes

struct CopyArgs {
    const uint8_t *x;
    const uint32_t *sf_in;
    const int32_t *rows;
    uint8_t *q;
    uint32_t *sf;
    int64_t sf_group;
    int T, top_k, K, R, cap, ld_in, ld_sf, words;   // words of a token's scales
};

// A workgroup of 256 threads per token: its codes (16 per lane) and scales are
// read once and written to each of its rows (333 tokens of 2048 to 6 rows: 3.5 us,
// 4.7 with the rows looked up one after the other).
__global__ void __launch_bounds__(256) moe_dispatch_codes_kernel(CopyArgs p) {
    const int lane = threadIdx.x & 63;
    const int tok = xcd_remap(blockIdx.x, gridDim.x);
    const int32_t *rows = p.rows + (int64_t)tok * p.top_k;
    for (int j0 = 0; j0 < p.top_k; j0 += 64) {
        const int n = min(p.top_k - j0, 64);
        const int row64 = lane < n ? rows[j0 + lane] : -1;   // in the lanes: one load, not one after the other
        for (int b = threadIdx.x; b < p.words; b += 256) {
            const uint32_t s = p.sf_in[(int64_t)b * p.ld_in + tok];
            for (int j = 0; j < n; ++j) {
                const int r = __builtin_amdgcn_readlane(row64, j);
                if ((unsigned)r >= (unsigned)p.R) continue;
                const int g = p.cap == p.R ? 0 : r / p.cap;
                p.sf[g * p.sf_group + (int64_t)b * p.ld_sf + (r - g * p.cap)] = s;
            }
        }
        for (int c = threadIdx.x; c < p.K / 16; c += 256) {
            const v4i v = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p.x + (int64_t)tok * p.K) + c);
            for (int j = 0; j < n; ++j) {
                const int r = __builtin_amdgcn_readlane(row64, j);
                if ((unsigned)r < (unsigned)p.R) __builtin_nontemporal_store(v, reinterpret_cast<v4i *>(p.q + (int64_t)r * p.K) + c);
            }
        }
    }
}

hipError_t launch_moe_dispatch_codes(const MoeCopyProblem &p, hipStream_t stream) {
    if (!grid_fits(p.T, 256)) return hipErrorInvalidValue;
    const CopyArgs a{p.x, p.sf_in, p.rows, p.q, p.sf, p.sf_group, p.T, p.top_k, p.K, p.R, p.cap, p.ld_in, p.ld_sf, p.words};
    hipLaunchKernelGGL(moe_dispatch_codes_kernel, dim3((unsigned)p.T), dim3(256), 0, stream, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- combine

struct CombineArgs {
    const uint16_t *y;
    const float *weights;
    const int32_t *rows;
    const void *res;
    void *out;
    int T, top_k, K, R, chunks;   // 512-column chunks of a row
    Divisor by_chunks;
};

// A wave per token and 512 columns (lane l: columns 8 l .. 8 l + 7 of them);
// nothing is shared between waves.  kBatch choices at a time, whose loads are all
// in flight together: a choice without a row reads row 0 (and counts as nothing),
// since a load under a condition waits for the one before it (64 tokens of 7168,
// 8 choices: 4.3 us, 6.9 so).  Four of them: 4096 tokens 103.6 us in a graph, 4.6
// TB/s of rows; all 8 at once, 103.5, and 4.6 for the 64.  Two for one or two
// choices (4096 tokens of 7168, one choice: 30.6 us, 35.1 with four, two choices:
// 39.0 and 40.2; 333 of 2048: 3.2 and 3.5, 3.3 and 3.7).  Workgroups in launch
// order: 112 us with neighbours on one XCD.  The sum runs in the order of the
// choices, in fp32.
template <typename TO, bool kRes, bool kW, int kBatch>
__global__ void __launch_bounds__(256) moe_combine_kernel(CombineArgs p) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t item = blockIdx.x * 4 + wave;     // below 2^26
    const int tok = (int)p.by_chunks.quotient(item);
    if (tok >= p.T) return;
    const int K = p.K, top_k = p.top_k;
    const int col = (int)(item - (uint32_t)tok * p.chunks) * 512 + 8 * lane;
    const bool in = col < K;
    const int at = min(col, K - 8);
    const int32_t *rows = p.rows + (int64_t)tok * top_k;
    const float *ws = kW ? p.weights + (int64_t)tok * top_k : nullptr;
    Raw8<TO> res{};
    if constexpr (kRes) res = load8<true>(static_cast<const TO *>(p.res) + (int64_t)tok * K + at);
    float acc[8];
    for (int j0 = 0; j0 < top_k; j0 += kBatch) {
        Raw8<uint16_t> v[kBatch];
        bool live[kBatch];
        float w[kBatch];
        int r[kBatch];
        // past the last choice, that one's entry again
        static_for<kBatch>([&](auto jc) __attribute__((always_inline)) {
            constexpr int j = decltype(jc)::value;
            r[j] = rows[min(j0 + j, top_k - 1)];
            w[j] = kW ? ws[min(j0 + j, top_k - 1)] : 1.f;
        });
        static_for<kBatch>([&](auto jc) __attribute__((always_inline)) {
            constexpr int j = decltype(jc)::value;
            live[j] = j0 + j < top_k && (unsigned)r[j] < (unsigned)p.R;     // uniform
            v[j] = load8<true>(p.y + (int64_t)(live[j] ? r[j] : 0) * K + at);
        });
        if (j0 == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = kRes ? get8(res, i) : 0.f;
        }
        static_for<kBatch>([&](auto jc) __attribute__((always_inline)) {
            constexpr int j = decltype(jc)::value;
            if (live[j]) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] = kW ? __builtin_fmaf(w[j], get8(v[j], i), acc[i]) : acc[i] + get8(v[j], i);
            }
        });
    }
    if (in) store8<true>(static_cast<TO *>(p.out) + (int64_t)tok * K + col, acc);
}

template <typename TO, bool kRes, bool kW>
static hipError_t launch_combine_b(const CombineArgs &a, hipStream_t stream) {
    const int64_t groups = ((int64_t)a.T * a.chunks + 3) / 4;
    if (!grid_fits(groups, 256)) return hipErrorInvalidValue;
    const dim3 g((unsigned)groups), b(256);
    if (a.top_k <= 2) hipLaunchKernelGGL((moe_combine_kernel<TO, kRes, kW, 2>), g, b, 0, stream, a);
    else hipLaunchKernelGGL((moe_combine_kernel<TO, kRes, kW, 4>), g, b, 0, stream, a);
    return hipGetLastError();
}

template <typename TO>
static hipError_t launch_combine_t(const CombineArgs &a, hipStream_t stream) {
    if (a.res) return a.weights ? launch_combine_b<TO, true, true>(a, stream) : launch_combine_b<TO, true, false>(a, stream);
    return a.weights ? launch_combine_b<TO, false, true>(a, stream) : launch_combine_b<TO, false, false>(a, stream);
}

// Without rows there is nothing to read, not even row 0: out is the residual, or
// zeros.
template <typename TO>
__global__ void __launch_bounds__(256) moe_residual_kernel(const TO *res, TO *out, int64_t n8) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        float v[8];
        const Raw8<TO> r = res ? load8(res + 8 * i) : Raw8<TO>{};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = res ? get8(r, e) : 0.f;
        store8(out + 8 * i, v);
    }
}

hipError_t launch_moe_combine(const MoeCombineProblem &p, hipStream_t stream) {
    if (p.R == 0) {
        const int64_t n8 = (int64_t)p.T * p.K / 8;
        const dim3 g((unsigned)(n8 < 1 << 18 ? (n8 + 255) / 256 : 1024)), b(256);
        if (p.out_type == kBf16)
            hipLaunchKernelGGL(moe_residual_kernel<uint16_t>, g, b, 0, stream, static_cast<const uint16_t *>(p.residual),
                               static_cast<uint16_t *>(p.out), n8);
        else
            hipLaunchKernelGGL(moe_residual_kernel<float>, g, b, 0, stream, static_cast<const float *>(p.residual),
                               static_cast<float *>(p.out), n8);
        return hipGetLastError();
    }
    const int chunks = runs_of(p.K, 512);
    const CombineArgs a{p.y, p.weights, p.rows, p.residual, p.out, p.T, p.top_k, p.K, p.R, chunks, Divisor(chunks)};
    return p.out_type == kBf16 ? launch_combine_t<uint16_t>(a, stream) : launch_combine_t<float>(a, stream);
}

}  // namespace dg
