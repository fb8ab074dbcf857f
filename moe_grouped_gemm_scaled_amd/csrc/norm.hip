// norm.hip -- RMS norm for gfx950: the residual's addition, the norm and the
// E4M3 quantisation of the normalised row in one pass, and the gradient.
//
// Forward, per row of K values (fp32 throughout, each output rounded once):
//     h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  y = h * r * w
//     per 128-column block: sf = max(amax |y|, 1e-4) / 448, q = e4m3(y / sf)
// Backward, from h as stored (r is recomputed from it, so nothing but h is
// kept between the passes), with g = dy * w:
//     dx = dres + r * (g - h * r^2 * mean(g * h));   dw = sum_rows dy * h * r
//
// Both are HBM-bound: a row is read once, held in registers between its
// reduction and its outputs, and written once.
#include "dg_layer.h"
#include "dg_quant.h"
#include "dg_rows.h"

namespace dg {

struct NoRes {};   // no residual

struct NormFwdArgs {
    const void *x, *res, *w;
    void *res_out;
    uint16_t *y;
    uint8_t *q;
    void *sf;
    int64_t ld_x;
    int rows, K, ld_sf;
    float eps;
    int format;   // of sf (SfFormat)
};

// WPR waves share a row (WPR = 1: four rows per workgroup, one per wave; no
// barrier).  Lane l of wave w holds the 8 columns from
// 8 * (64 * (WPR * c + w) + l), c < NCH, so one load instruction reads 1 KB
// (bf16) of consecutive columns, 16 lanes hold a 128-column block, and the
// four blocks of a wave's 512 columns are the four bytes of one packed scale
// word.  Columns past K (a multiple of 128) are loaded from the row's end and
// zeroed.  residual_out may be the residual itself: a lane's loads all come
// before its stores.
template <typename TX, typename TR, typename TW, int WPR, int NCH>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR)
rmsnorm_quant_kernel(NormFwdArgs p) {
    constexpr bool kRes = !std::is_same<TR, NoRes>::value;
    using TRS = typename std::conditional<kRes, TR, TX>::type;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // consecutive rows on one XCD: their scales share cache lines
    const int blk = xcd_remap(blockIdx.x, gridDim.x);
    const int row = WPR == 1 ? blk * 4 + wave : blk;
    const int w0 = WPR == 1 ? 0 : wave;
    const int K = p.K;
    if (WPR == 1 && row >= p.rows) return;

    const TX *xr = static_cast<const TX *>(p.x) + (int64_t)row * p.ld_x;
    const TRS *rr = static_cast<const TRS *>(p.res) + (int64_t)row * K;
    const TW *wr = static_cast<const TW *>(p.w);
    Raw8<TX> xv[NCH];
    Raw8<TRS> rv[kRes ? NCH : 1];
    Raw8<TW> wv[NCH];
    int col[NCH];
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        col[c] = 8 * (64 * (WPR * c + w0) + lane);
        xv[c] = load8<true>(xr + min(col[c], K - 8));
        if constexpr (kRes) rv[c] = load8<true>(rr + min(col[c], K - 8));
    });
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        wv[c] = load8(wr + min(col[c], K - 8));
    });
    float h[NCH][8];
    float ss = 0.f;
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        const bool in = col[c] < K;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = get8(xv[c], i);
            if constexpr (kRes) v += get8(rv[c], i);
            h[c][i] = in ? v : 0.f;
            ss = __builtin_fmaf(h[c][i], h[c][i], ss);
        }
    });
    ss = sum64(ss);
    if constexpr (WPR > 1) {
        __shared__ float red[WPR];
        if (lane == 0) red[wave] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) ss += red[i];
    }
    const float r = 1.0f / sqrtf(ss / (float)K + p.eps);

    TRS *ro = kRes ? static_cast<TRS *>(p.res_out) + (int64_t)row * K : nullptr;
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        const bool in = col[c] < K;
        float y[8];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = h[c][i] * r * get8(wv[c], i);
            amax = fmaxf(amax, fabsf(y[i]));
        }
        amax = max16(amax);
        if constexpr (kRes) {
            if (in && p.res_out) store8<true>(ro + col[c], h[c]);
        }
        if (p.y && in) store8<true>(p.y + (int64_t)row * K + col[c], y);
        if (p.q) {                                     // uniform
            const float s = p.format == kSfFp32 ? block_scale<false>(amax) : block_scale<true>(amax);
            const v4f lo = v4f{y[0], y[1], y[2], y[3]}, hi = v4f{y[4], y[5], y[6], y[7]};
            uint2 w;
            if (p.format == kSfFp32) {
                const BlockDivisor d = block_divisor<false>(s);
                w = uint2{encode4<false>(lo, d), encode4<false>(hi, d)};
            } else {
                const BlockDivisor d = block_divisor<true>(s);
                w = uint2{encode4<true>(lo, d), encode4<true>(hi, d)};
            }
            if (in) *reinterpret_cast<uint2 *>(p.q + (int64_t)row * K + col[c]) = w;
            if (p.format == kSfPacked) {
                // byte j of the word: the exponent of block j of these 512 columns, 0 past K
                uint32_t e = in ? (__float_as_uint(s) >> 23) << (8 * (lane >> 4)) : 0u;
                e |= (uint32_t)__shfl_xor((int)e, 16);
                e |= (uint32_t)__shfl_xor((int)e, 32);
                if (lane == 0 && in)
                    static_cast<uint32_t *>(p.sf)[(int64_t)(WPR * c + w0) * p.ld_sf + row] = e;
            } else if ((lane & 15) == 0 && in) {
                static_cast<float *>(p.sf)[(int64_t)(col[c] / kKBlock) * p.ld_sf + row] = s;
            }
        }
    });
}

// A grid of 2^32 threads or more is not refused but taken modulo 2^32: more
// rows than a grid holds go in several launches.
template <typename TX, typename TR, typename TW, int WPR, int NCH>
static hipError_t launch_fwd_t(const NormFwdArgs &a, hipStream_t stream) {
    constexpr int kThreads = WPR == 1 ? 256 : 64 * WPR, kRows = WPR == 1 ? 4 : 1;      // of a workgroup
    constexpr int64_t kMost = ((int64_t)1 << 32) / kThreads / 2 * kRows;               // rows of a launch
    using TRS = typename std::conditional<std::is_same<TR, NoRes>::value, TX, TR>::type;
    for (int64_t r = 0; r < a.rows; r += kMost) {
        NormFwdArgs p = a;
        p.rows = (int)(a.rows - r < kMost ? a.rows - r : kMost);
        p.x = static_cast<const TX *>(a.x) + r * a.ld_x;
        if (a.res) p.res = static_cast<const TRS *>(a.res) + r * a.K;
        if (a.res_out) p.res_out = static_cast<TRS *>(a.res_out) + r * a.K;
        if (a.y) p.y = a.y + r * a.K;
        if (a.q) {
            p.q = a.q + r * a.K;
            p.sf = static_cast<float *>(a.sf) + r;
        }
        hipLaunchKernelGGL((rmsnorm_quant_kernel<TX, TR, TW, WPR, NCH>), dim3((unsigned)((p.rows + kRows - 1) / kRows)),
                           dim3(kThreads), 0, stream, p);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// Waves per row: one up to 1024 columns (16384 rows: 14 against 25 us with
// four at 512 columns, 22 against 27 at 1024), four from there (4096 rows of
// 7168: 40.7 us, 5.1 TB/s, against 47 us with one; nontemporal loads and
// stores: 45.4 us without), sixteen for few long rows, where a row's latency is
// the call's.
template <typename TX, typename TR, typename TW>
static hipError_t launch_fwd_k(const NormFwdArgs &a, hipStream_t stream) {
    const int n = (a.K + 511) / 512;                   // 512-column chunks
    if (n <= 1) return launch_fwd_t<TX, TR, TW, 1, 1>(a, stream);
    if (n <= 2) return launch_fwd_t<TX, TR, TW, 1, 2>(a, stream);
    if (n <= 4) return launch_fwd_t<TX, TR, TW, 4, 1>(a, stream);
    if (n <= 16 && a.rows < 512) return launch_fwd_t<TX, TR, TW, 16, 1>(a, stream);
    if (n <= 8) return launch_fwd_t<TX, TR, TW, 4, 2>(a, stream);
    if (n <= 16) return launch_fwd_t<TX, TR, TW, 4, 4>(a, stream);
    if (n <= 32) return launch_fwd_t<TX, TR, TW, 16, 2>(a, stream);
    return hipErrorInvalidValue;
}

template <typename TX, typename TR>
static hipError_t launch_fwd_w(const NormFwdArgs &a, int w_type, hipStream_t stream) {
    return w_type == kBf16 ? launch_fwd_k<TX, TR, uint16_t>(a, stream) : launch_fwd_k<TX, TR, float>(a, stream);
}

template <typename TX>
static hipError_t launch_fwd_r(const NormFwdArgs &a, int res_type, int w_type, hipStream_t stream) {
    if (!a.res) return launch_fwd_w<TX, NoRes>(a, w_type, stream);
    return res_type == kBf16 ? launch_fwd_w<TX, uint16_t>(a, w_type, stream)
                             : launch_fwd_w<TX, float>(a, w_type, stream);
}

hipError_t launch_rmsnorm_quant(const RmsNormProblem &p, hipStream_t stream) {
    const NormFwdArgs a{p.x, p.residual, p.weight, p.residual_out, p.y, p.q, p.sf, p.ld_x, p.rows, p.K, p.ld_sf,
                        p.eps, (int)p.format};
    return p.x_type == kBf16 ? launch_fwd_r<uint16_t>(a, p.res_type, p.w_type, stream)
                             : launch_fwd_r<float>(a, p.res_type, p.w_type, stream);
}

// ---------------------------------------------------------------- backward

struct NormBwdArgs {
    const void *dy, *h, *w, *dres;
    void *dx;
    float *dw;     // the result, or (more than one workgroup) a partial row per workgroup
    int rows, K;
    float eps;
};

// WPR waves share a row; the workgroup walks its own run of consecutive rows,
// NR = 4 / WPR of them at a time (WPR < 4), and keeps its sum of dw in registers (each lane owns
// the same columns of every row).  The next row's h and dy are loaded while
// the current row is reduced.  dw leaves as one fp32 row per workgroup, added
// up in workgroup order by a second kernel: the same bits on every run.
template <typename TH, typename TY, typename TW, int WPR, int NCH>
__global__ void __launch_bounds__(WPR <= 4 ? 256 : 64 * WPR)
rmsnorm_bwd_kernel(NormBwdArgs p) {
    constexpr int NR = WPR < 4 ? 4 / WPR : 1;          // rows at a time
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int w0 = wave % WPR, r0 = wave / WPR;
    const int K = p.K;
    const int64_t lo = (int64_t)p.rows * blockIdx.x / gridDim.x, hi = (int64_t)p.rows * (blockIdx.x + 1) / gridDim.x;

    const TH *H = static_cast<const TH *>(p.h);
    const TY *Y = static_cast<const TY *>(p.dy);
    const TH *R = static_cast<const TH *>(p.dres);
    TH *DX = static_cast<TH *>(p.dx);
    int col[NCH], at[NCH];
    Raw8<TW> wv[NCH];
    float dw[NCH][8];
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        col[c] = 8 * (64 * (WPR * c + w0) + lane);
        at[c] = min(col[c], K - 8);
        wv[c] = load8(static_cast<const TW *>(p.w) + at[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0.f;
    });
    Raw8<TH> hn[NCH];
    Raw8<TY> yn[NCH];
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
        static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            hn[c] = load8<true>(H + row * K + at[c]);
            yn[c] = load8<true>(Y + row * K + at[c]);
        });
    };
    __shared__ float2 red[2][WPR];                     // WPR >= 4: sums of the row, alternating
    const int64_t n_it = (hi - lo + NR - 1) / NR;
    if (n_it > 0) fetch(lo + r0 < hi ? lo + r0 : hi - 1);
    for (int64_t it = 0; it < n_it; ++it) {
        const int64_t row = lo + it * NR + r0;
        const bool live = row < hi;                    // uniform per wave
        Raw8<TH> hc[NCH], rc[NCH];
        Raw8<TY> yc[NCH];
        static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            hc[c] = hn[c];
            yc[c] = yn[c];
        });
        if (p.dres && live) {
            static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
                constexpr int c = decltype(cc)::value;
                rc[c] = load8<true>(R + row * K + at[c]);
            });
        }
        if (it + 1 < n_it) fetch(row + NR < hi ? row + NR : hi - 1);
        float ss = 0.f, sg = 0.f;
        static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            if (col[c] < K) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float hv = get8(hc[c], i);
                    ss = __builtin_fmaf(hv, hv, ss);
                    sg = __builtin_fmaf(get8(yc[c], i) * get8(wv[c], i), hv, sg);
                }
            }
        });
        ss = sum64(ss);
        sg = sum64(sg);
        if constexpr (WPR >= 4) {
            if (lane == 0) red[it & 1][w0] = float2{ss, sg};
            __syncthreads();
            ss = 0.f;
            sg = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                ss += red[it & 1][i].x;
                sg += red[it & 1][i].y;
            }
        }
        const float r = 1.0f / sqrtf(ss / (float)K + p.eps);
        const float k = r * r * (sg / (float)K);
        if (live) {
            static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
                constexpr int c = decltype(cc)::value;
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float hv = get8(hc[c], i), yv = get8(yc[c], i);
                    o[i] = r * __builtin_fmaf(-hv, k, yv * get8(wv[c], i));
                    if (p.dres) o[i] += get8(rc[c], i);
                    dw[c][i] = __builtin_fmaf(yv, hv * r, dw[c][i]);
                }
                if (col[c] < K) store8<true>(DX + row * K + col[c], o);
            });
        }
    }
    // one fp32 row per workgroup; rows handled side by side (WPR < 4) first
    // add up through LDS, in wave order
    float *out = p.dw + (int64_t)blockIdx.x * K;
    if constexpr (NR > 1) {
        __shared__ float part[NR][WPR * NCH * 512];
        static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            store8(&part[r0][col[c]], dw[c]);
        });
        __syncthreads();
        for (int j = threadIdx.x; j < K; j += 256) {
            float s = part[0][j];
#pragma unroll
            for (int q = 1; q < NR; ++q) s += part[q][j];
            out[j] = s;
        }
    } else {
        static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            if (col[c] < K) store8(out + col[c], dw[c]);
        });
    }
}

// dw[k] = sum over n partial rows, in a fixed order: 64 columns per
// workgroup, 16 waves each adding every 16th row, then the waves in order.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float *__restrict__ part, float *__restrict__ dw, int n, int K) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k = blockIdx.x * 64 + lane;              // K is a multiple of 128
    float a = 0.f;
#pragma unroll 8
    for (int i = wave; i < n; i += 16) a += part[(int64_t)i * K + k];
    s[wave][lane] = a;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) a += s[i][lane];
        dw[k] = a;
    }
}

// Workgroups of the backward pass.  One for a few short rows: its dw needs no
// second kernel, whose launch costs the host 2.6 us (8 rows of 1536: 8.4 us
// against 3.2 + 2.2 and a gap).  A row each up to as many rows as CUs (87 rows
// of 16000, fp32: 12.7 against 16.4 us with two), two rows or more above, so
// that the partial rows of dw stay small next to the rows (500 rows of 7168:
// 11.3 + 4.7 against 13.6 + 5.5 us with one; 333 of 2048: 5.6 against 7.5 us
// with four).  Two workgroups per CU at most, one above 8192 columns, where two
// do not fit (1059 rows of 10240, fp32: 38.9 against 44.3 us).
static int bwd_groups(int rows, int K, int num_cus) {
    if ((int64_t)rows * K < 16384) return 1;
    const int64_t most = K > 8192 ? num_cus : 2 * (int64_t)num_cus;
    const int64_t g = rows <= num_cus ? rows : ((int64_t)rows + 1) / 2;
    return (int)(g < most ? (g > 0 ? g : 1) : most);
}

size_t rmsnorm_bwd_workspace(int rows, int K, int num_cus) {
    const int g = bwd_groups(rows, K, num_cus);
    return g > 1 ? (size_t)g * K * sizeof(float) : 0;
}

template <typename TH, typename TY, typename TW, int WPR, int NCH>
static hipError_t launch_bwd_t(const RmsNormBwdProblem &p, int groups, hipStream_t stream) {
    const NormBwdArgs a{p.dy, p.h, p.weight, p.dres, p.dx, groups > 1 ? static_cast<float *>(p.ws) : p.dw, p.rows,
                        p.K, p.eps};
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<TH, TY, TW, WPR, NCH>), dim3((unsigned)groups),
                       dim3(WPR <= 4 ? 256 : 64 * WPR), 0, stream, a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || groups <= 1) return err;
    hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((unsigned)(p.K / 64)), dim3(1024), 0, stream,
                       static_cast<const float *>(p.ws), p.dw, groups, p.K);
    return hipGetLastError();
}

template <typename TH, typename TY, typename TW>
static hipError_t launch_bwd_k(const RmsNormBwdProblem &p, int num_cus, hipStream_t stream) {
    const int g = bwd_groups(p.rows, p.K, num_cus);
    const int n = (p.K + 511) / 512;
    if (n <= 1) return launch_bwd_t<TH, TY, TW, 1, 1>(p, g, stream);
    if (n <= 2) return launch_bwd_t<TH, TY, TW, 1, 2>(p, g, stream);
    if (n <= 4) return launch_bwd_t<TH, TY, TW, 4, 1>(p, g, stream);
    if (n <= 8) return launch_bwd_t<TH, TY, TW, 4, 2>(p, g, stream);
    if (n <= 16) return launch_bwd_t<TH, TY, TW, 4, 4>(p, g, stream);
    if (n <= 32) return launch_bwd_t<TH, TY, TW, 8, 4>(p, g, stream);
    return hipErrorInvalidValue;
}

template <typename TH, typename TY>
static hipError_t launch_bwd_w(const RmsNormBwdProblem &p, int num_cus, hipStream_t stream) {
    return p.w_type == kBf16 ? launch_bwd_k<TH, TY, uint16_t>(p, num_cus, stream)
                             : launch_bwd_k<TH, TY, float>(p, num_cus, stream);
}

hipError_t launch_rmsnorm_bwd(const RmsNormBwdProblem &p, int num_cus, hipStream_t stream) {
    if (p.rows == 0) {                                 // no rows: dw is zero
        hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((unsigned)(p.K / 64)), dim3(1024), 0, stream,
                           static_cast<const float *>(nullptr), p.dw, 0, p.K);
        return hipGetLastError();
    }
    if (p.h_type == kBf16)
        return p.dy_type == kBf16 ? launch_bwd_w<uint16_t, uint16_t>(p, num_cus, stream)
                                  : launch_bwd_w<uint16_t, float>(p, num_cus, stream);
    return p.dy_type == kBf16 ? launch_bwd_w<float, uint16_t>(p, num_cus, stream)
                              : launch_bwd_w<float, float>(p, num_cus, stream);
}

}  // namespace dg
