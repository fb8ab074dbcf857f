// layernorm.hip -- layer norm for gfx950: the residual's addition, the norm and
// the E4M3 quantisation of the normalised row in one pass, and the gradient.
//
// Forward, per row of K values (fp32 throughout, each output rounded once):
//     h = x + residual;  m = mean(h);  r = 1 / sqrt(mean((h - m)^2) + eps)
//     y = (h - m) * r * w + b
//     per 128-column block: sf = max(amax |y|, 1e-4) / 448, q = e4m3(y / sf)
// Backward, from h as stored (m and r are recomputed from it), with
// n = (h - m) r and g = dy * w:
//     dx = dres + r * (g - mean(g) - n * mean(g * n))
//     dw = sum_rows dy * n;   db = sum_rows dy
//
// The variance is the mean of squared differences from the mean, which is known
// first: the row is in registers, so the second sum costs no traffic, and
// nothing cancels where the mean is large beside the spread (mean(h^2) - m^2
// would lose twice as many bits as |m| / spread has).
//
// A row is read once, held in registers between its reductions and its outputs,
// and written once, so that HBM bounds both (4096 rows of 7168, bf16: 43.4 us,
// 4.8 TB/s; 64 rows: 4.9 us; the gradient of 16384: 183 us, 5.1 TB/s, and 4.6 for
// the sums of dw and db), except the gradient of more than 4096 columns with fp32
// h or dy, whose registers do not suffice (LnBwdShape).  A second meeting of a row's waves for the variance
// costs less than joining each wave's own mean and squared differences in one
// (the gradient of 4096 rows 58.5 against 68.6 us).
#include "dg_codes8.h"

namespace dg {

struct NoRes {};   // no residual

struct LnFwdArgs {
    const void *x, *res, *w, *b;
    void *res_out;
    uint16_t *y;
    uint8_t *q;
    void *sf;
    int64_t ld_x;
    int rows, K, ld_sf;
    float eps;
    int format;   // of sf (SfFormat)
};

// Eight ones (the weight that is not there) or zeros (the bias).
template <typename T>
__device__ __forceinline__ Raw8<T> same8(bool one) {
    if constexpr (std::is_same<T, float>::value) {
        const float v = one ? 1.f : 0.f;
        return {v4f{v, v, v, v}, v4f{v, v, v, v}};
    } else {
        const int v = one ? 0x3f803f80 : 0;
        return {v4i{v, v, v, v}};
    }
}

// Sum over the WPR waves of a row; `red` is not used again before a barrier.
template <int WPR>
__device__ __forceinline__ float sum_row(float v, float *red, int lane, int wave) {
    v = sum64(v);
    if constexpr (WPR > 1) {
        if (lane == 0) red[wave] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) v += red[i];
    }
    return v;
}

// WPR waves share a row (WPR = 1: four rows per workgroup, one per wave; no
// barrier).  Lane l of wave w holds the 8 columns from
// 8 * (64 * (WPR * c + w) + l), c < NCH: one load instruction reads 1 KB (bf16)
// of consecutive columns, 16 lanes hold a 128-column block, and the four blocks
// of a wave's 512 columns are the four bytes of one packed scale word.  Columns
// past K (a multiple of 8, of 128 where codes are written) are loaded from the
// row's end and count as nothing.  residual_out may be the residual itself: a
// lane's loads all come before its stores.
template <typename TX, typename TR, typename TW, int WPR, int NCH>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR)
layernorm_quant_kernel(LnFwdArgs p) {
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
    Raw8<TX> xv[NCH];
    Raw8<TRS> rv[kRes ? NCH : 1];
    Raw8<TW> wv[NCH], bv[NCH];
    int col[NCH];
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        col[c] = 8 * (64 * (WPR * c + w0) + lane);
        xv[c] = load8<true>(xr + min(col[c], K - 8));
        if constexpr (kRes) rv[c] = load8<true>(rr + min(col[c], K - 8));
    });
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        const int at = min(col[c], K - 8);
        wv[c] = p.w ? load8(static_cast<const TW *>(p.w) + at) : same8<TW>(true);       // uniform
        bv[c] = p.b ? load8(static_cast<const TW *>(p.b) + at) : same8<TW>(false);
    });
    __shared__ float red[2][WPR];
    float h[NCH][8];
    float sum = 0.f;
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        const bool in = col[c] < K;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = get8(xv[c], i);
            if constexpr (kRes) v += get8(rv[c], i);
            h[c][i] = v;
            sum += in ? v : 0.f;
        }
    });
    TRS *ro = kRes ? static_cast<TRS *>(p.res_out) + (int64_t)row * K : nullptr;
    if constexpr (kRes) {
        if (p.res_out) {                               // uniform; before h is centred
            static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
                constexpr int c = decltype(cc)::value;
                if (col[c] < K) store8<true>(ro + col[c], h[c]);
            });
        }
    }
    const float mean = sum_row<WPR>(sum, red[0], lane, w0) / (float)K;
    float ss = 0.f;
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        const bool in = col[c] < K;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[c][i] = in ? h[c][i] - mean : 0.f;
            ss = __builtin_fmaf(h[c][i], h[c][i], ss);
        }
    });
    const float r = 1.0f / sqrtf(sum_row<WPR>(ss, red[1], lane, w0) / (float)K + p.eps);

    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        const bool in = col[c] < K;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(h[c][i] * r, get8(wv[c], i), get8(bv[c], i));
        if (p.y && in) store8<true>(p.y + (int64_t)row * K + col[c], y);
        if (p.q) {                                     // uniform
            float s;
            const uint2 w = codes8(y, max16(amax8(y)), p.format, s);
            if (in) *reinterpret_cast<uint2 *>(p.q + (int64_t)row * K + col[c]) = w;
            if (p.format == kSfPacked) {
                const uint32_t e = scale_word(s, in, lane);
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
static hipError_t launch_fwd_t(const LnFwdArgs &a, hipStream_t stream) {
    constexpr int kThreads = WPR == 1 ? 256 : 64 * WPR, kRows = WPR == 1 ? 4 : 1;      // of a workgroup
    constexpr int64_t kMost = ((int64_t)1 << 32) / kThreads / 2 * kRows;               // rows of a launch
    using TRS = typename std::conditional<std::is_same<TR, NoRes>::value, TX, TR>::type;
    for (int64_t r = 0; r < a.rows; r += kMost) {
        LnFwdArgs p = a;
        p.rows = (int)(a.rows - r < kMost ? a.rows - r : kMost);
        p.x = static_cast<const TX *>(a.x) + r * a.ld_x;
        if (a.res) p.res = static_cast<const TRS *>(a.res) + r * a.K;
        if (a.res_out) p.res_out = static_cast<TRS *>(a.res_out) + r * a.K;
        if (a.y) p.y = a.y + r * a.K;
        if (a.q) {
            p.q = a.q + r * a.K;
            p.sf = static_cast<float *>(a.sf) + r;
        }
        hipLaunchKernelGGL((layernorm_quant_kernel<TX, TR, TW, WPR, NCH>),
                           dim3((unsigned)((p.rows + kRows - 1) / kRows)), dim3(kThreads), 0, stream, p);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// Waves per row, as in the RMS norm, whose traffic is the same: one up to 1024
// columns, four from there, sixteen for few long rows, where a row's latency is
// the call's.  Calls among others, bf16 with residual, the RMS norm's beside them:
// 64 x 7168 6.7 us (6.2), 4096 x 1024 7.6 (7.2), x 4096 24.1 (24.4), x 7168 41.3
// (40.6), 2048 x 16384 51.8 (51.6).  Lanes are dealt columns in powers of two, so
// just past a step nearly half of them count as nothing: 4096 x 1152 10.8 us, 3.1
// TB/s (9.4), x 2176 15.5, 4.1 TB/s (14.5), x 4224 27.9, 4.4 TB/s (26.1).
template <typename TX, typename TR, typename TW>
static hipError_t launch_fwd_k(const LnFwdArgs &a, hipStream_t stream) {
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
static hipError_t launch_fwd_w(const LnFwdArgs &a, int w_type, hipStream_t stream) {
    return w_type == kBf16 ? launch_fwd_k<TX, TR, uint16_t>(a, stream) : launch_fwd_k<TX, TR, float>(a, stream);
}

template <typename TX>
static hipError_t launch_fwd_r(const LnFwdArgs &a, int res_type, int w_type, hipStream_t stream) {
    if (!a.res) return launch_fwd_w<TX, NoRes>(a, w_type, stream);
    return res_type == kBf16 ? launch_fwd_w<TX, uint16_t>(a, w_type, stream)
                             : launch_fwd_w<TX, float>(a, w_type, stream);
}

hipError_t launch_layernorm_quant(const LayerNormProblem &p, hipStream_t stream) {
    const LnFwdArgs a{p.x, p.residual, p.weight, p.bias, p.residual_out, p.y, p.q, p.sf, p.ld_x, p.rows, p.K, p.ld_sf,
                      p.eps, p.format};
    return p.x_type == kBf16 ? launch_fwd_r<uint16_t>(a, p.res_type, p.w_type, stream)
                             : launch_fwd_r<float>(a, p.res_type, p.w_type, stream);
}

// ---------------------------------------------------------------- backward

struct LnBwdArgs {
    const void *dy, *h, *w, *dres;
    void *dx;
    float *dw, *db;   // the results, or partial rows: workgroup g's at g * stride
    int64_t stride;
    int rows, K;
    float eps;
};

// Waves of a workgroup and workgroups of a CU: as many rows side by side as
// registers allow (h, dy and dres of the row, h and dy of the next, sums of dw
// and db), in one workgroup rather than in two where that costs no time, because
// each workgroup leaves partial rows of dw and db.  Eight waves: 4096 rows of
// 7168: 57.3 us, 60.0 with two workgroups of four; 16384 of 1024: 31.0, 31.6;
// two such workgroups per CU where a thread holds 8 columns: 16384 rows of 2048:
// 63.0, 76.5 with four waves, 82 with one workgroup; sixteen waves: 60.6 there,
// but 9.9 against 8.7 for 333 rows.
// With fp32 h or dy and four chunks per lane the 256 registers do not hold all of
// it: 17 to 68 are spilled to scratch.  4096 rows of 7168 take 89 us with fp32 dy,
// 137 with fp32 h and 185 with both (3.3 to 2.5 TB/s), 56 with neither; up to 4096
// columns nothing is spilled (4096 rows of 4096: 41, 54 and 62 us, 4.1 to 4.4 TB/s).
template <int WPR, int NCH>
struct LnBwdShape {
    static constexpr int kThreads = 512;
    static constexpr int kRows = kThreads / (64 * WPR);   // side by side
    static constexpr int kPerCu = WPR == 4 && NCH == 1 ? 2 : 1;
};

// WPR waves share a row; the workgroup walks its own run of consecutive rows,
// NR of them at a time, and keeps its sums of dw and db in registers (each lane
// owns the same columns of every row).  The next row's h and dy are loaded while
// the current row is reduced.  dw and db leave as one fp32 row each per
// workgroup, added up in workgroup order by a second kernel: the same bits on
// every run.
template <typename TH, typename TY, typename TW, int WPR, int NCH>
__global__ void __launch_bounds__(512)
layernorm_bwd_kernel(LnBwdArgs p) {
    constexpr int NR = LnBwdShape<WPR, NCH>::kRows;
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
    float dw[NCH][8], db[NCH][8];
    static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value;
        col[c] = 8 * (64 * (WPR * c + w0) + lane);
        at[c] = min(col[c], K - 8);
        wv[c] = p.w ? load8(static_cast<const TW *>(p.w) + at[c]) : same8<TW>(true);     // uniform
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0.f;
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
    // WPR > 1: sums over the row's waves.  Each array is written again only
    // behind the other one's barrier, so behind every read of it.
    __shared__ float2 red1[NR][WPR], red2[NR][WPR];
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
        auto over_row = [&](float2 v, float2 *red) __attribute__((always_inline)) {
            v.x = sum64(v.x);
            v.y = sum64(v.y);
            if constexpr (WPR > 1) {
                if (lane == 0) red[w0] = v;
                __syncthreads();
                v = float2{0.f, 0.f};
#pragma unroll
                for (int i = 0; i < WPR; ++i) {
                    v.x += red[i].x;
                    v.y += red[i].y;
                }
            }
            return v;
        };
        float2 a = float2{0.f, 0.f}, b = float2{0.f, 0.f};
        static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            if (col[c] < K) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a.x += get8(hc[c], i);
                    a.y = __builtin_fmaf(get8(yc[c], i), get8(wv[c], i), a.y);
                }
            }
        });
        a = over_row(a, red1[r0]);
        const float mean = a.x / (float)K, mg = a.y / (float)K;
        static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(cc)::value;
            if (col[c] < K) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = get8(hc[c], i) - mean;
                    b.x = __builtin_fmaf(d, d, b.x);
                    b.y = __builtin_fmaf(__builtin_fmaf(get8(yc[c], i), get8(wv[c], i), -mg), d, b.y);
                }
            }
        });
        b = over_row(b, red2[r0]);
        const float r = 1.0f / sqrtf(b.x / (float)K + p.eps);
        const float k = r * r * (b.y / (float)K);      // n * mean(g n) = d * k
        if (live) {
            static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
                constexpr int c = decltype(cc)::value;
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = get8(hc[c], i) - mean, yv = get8(yc[c], i);
                    o[i] = r * __builtin_fmaf(-d, k, __builtin_fmaf(yv, get8(wv[c], i), -mg));
                    if (p.dres) o[i] += get8(rc[c], i);
                    dw[c][i] = __builtin_fmaf(yv, d * r, dw[c][i]);
                    db[c][i] += yv;
                }
                if (col[c] < K) store8<true>(DX + row * K + col[c], o);
            });
        }
    }
    // one fp32 row each per workgroup: of the rows handled side by side, the first
    // one's waves add the others' to theirs, in order (a single row leaves as it is)
    auto leave = [&](float (&v)[NCH][8], float *dst) __attribute__((always_inline)) {
        float *out = dst + (int64_t)blockIdx.x * p.stride;
        if constexpr (NR > 1) {
            __shared__ __attribute__((aligned(16))) float part[NR - 1][WPR * NCH * 512];
            const bool join = hi - lo > 1;             // uniform
            if (join && r0 > 0) {
                static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
                    constexpr int c = decltype(cc)::value;
                    store8(&part[r0 - 1][col[c]], v[c]);
                });
            }
            if (join) __syncthreads();
            if (join && r0 == 0) {
                static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
                    constexpr int c = decltype(cc)::value;
#pragma unroll
                    for (int q = 0; q < NR - 1; ++q) {
                        const Raw8<float> o = load8(&part[q][col[c]]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[c][i] += get8(o, i);
                    }
                });
            }
            if (join) __syncthreads();
        }
        if (r0 == 0) {
            static_for<NCH>([&](auto cc) __attribute__((always_inline)) {
                constexpr int c = decltype(cc)::value;
                if (col[c] < K) store8(out + col[c], v[c]);
            });
        }
    };
    if (p.dw) leave(dw, p.dw);                         // uniform
    if (p.db) leave(db, p.db);
}

// Column j of `dst` = sum over the n partial rows (of `stride` values), in a
// fixed order: 64 columns per workgroup, 16 waves each adding every 16th row,
// then the waves in order.  blockIdx.y: dw's half of a partial row, or db's.
__global__ void __launch_bounds__(1024) layernorm_dw_kernel(const float *__restrict__ part, float *__restrict__ dw,
                                                            float *__restrict__ db, int n, int K, int64_t stride) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k = blockIdx.x * 64 + lane, at = min(k, K - 1);
    float *dst = blockIdx.y ? db : dw;
    if (!dst) return;                                  // uniform
    const float *src = part + (blockIdx.y ? K : 0);
    float a = 0.f;
#pragma unroll 8
    for (int i = wave; i < n; i += 16) a += src[(int64_t)i * stride + at];
    s[wave][lane] = a;
    __syncthreads();
    if (wave == 0 && k < K) {
#pragma unroll
        for (int i = 1; i < 16; ++i) a += s[i][lane];
        dst[k] = a;
    }
}

// Workgroups of the backward pass, each of which takes `at_once` rows side by
// side: one where it takes its rows in two steps (no second kernel, whose launch
// costs more), else as many as the rows fill.  The workspace covers every shape:
// its groups are counted with one row at a time and two per CU.
static int bwd_groups(int rows, int at_once, int most) {
    if (rows <= 2 * at_once) return 1;
    const int64_t g = ((int64_t)rows + at_once - 1) / at_once;
    return (int)(g < most ? g : most);
}

size_t layernorm_bwd_workspace(int rows, int K, int num_cus) {
    const int g = bwd_groups(rows, 1, 2 * num_cus);
    return g > 1 ? (size_t)g * 2 * K * sizeof(float) : 0;
}

static hipError_t launch_dw(const float *part, int n, const LayerNormBwdProblem &p, hipStream_t stream) {
    hipLaunchKernelGGL(layernorm_dw_kernel, dim3((unsigned)((p.K + 63) / 64), 2), dim3(1024), 0, stream, part, p.dw, p.db,
                       n, p.K, 2 * (int64_t)p.K);
    return hipGetLastError();
}

template <typename TH, typename TY, typename TW, int WPR, int NCH>
static hipError_t launch_bwd_t(const LayerNormBwdProblem &p, int num_cus, hipStream_t stream) {
    using Shape = LnBwdShape<WPR, NCH>;
    const int groups = bwd_groups(p.rows, Shape::kRows, Shape::kPerCu * num_cus);
    float *part = static_cast<float *>(p.ws);
    const bool parts = groups > 1;
    const LnBwdArgs a{p.dy, p.h, p.weight, p.dres, p.dx, p.dw && parts ? part : p.dw, p.db && parts ? part + p.K : p.db,
                      2 * (int64_t)p.K, p.rows, p.K, p.eps};
    hipLaunchKernelGGL((layernorm_bwd_kernel<TH, TY, TW, WPR, NCH>), dim3((unsigned)groups), dim3(Shape::kThreads), 0, stream,
                       a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || !parts || (!p.dw && !p.db)) return err;
    return launch_dw(part, groups, p, stream);
}

template <typename TH, typename TY, typename TW>
static hipError_t launch_bwd_k(const LayerNormBwdProblem &p, int num_cus, hipStream_t stream) {
    const int n = (p.K + 511) / 512;
    if (n <= 1) return launch_bwd_t<TH, TY, TW, 1, 1>(p, num_cus, stream);
    if (n <= 2) return launch_bwd_t<TH, TY, TW, 1, 2>(p, num_cus, stream);
    if (n <= 4) return launch_bwd_t<TH, TY, TW, 4, 1>(p, num_cus, stream);
    if (n <= 8) return launch_bwd_t<TH, TY, TW, 4, 2>(p, num_cus, stream);
    if (n <= 16) return launch_bwd_t<TH, TY, TW, 4, 4>(p, num_cus, stream);
    if (n <= 32) return launch_bwd_t<TH, TY, TW, 8, 4>(p, num_cus, stream);
    return hipErrorInvalidValue;
}

template <typename TH, typename TY>
static hipError_t launch_bwd_w(const LayerNormBwdProblem &p, int num_cus, hipStream_t stream) {
    return p.w_type == kBf16 ? launch_bwd_k<TH, TY, uint16_t>(p, num_cus, stream)
                             : launch_bwd_k<TH, TY, float>(p, num_cus, stream);
}

hipError_t launch_layernorm_bwd(const LayerNormBwdProblem &p, int num_cus, hipStream_t stream) {
    if (p.rows == 0) return p.dw || p.db ? launch_dw(nullptr, 0, p, stream) : hipSuccess;   // zeros
    if (p.h_type == kBf16)
        return p.dy_type == kBf16 ? launch_bwd_w<uint16_t, uint16_t>(p, num_cus, stream)
                                  : launch_bwd_w<uint16_t, float>(p, num_cus, stream);
    return p.dy_type == kBf16 ? launch_bwd_w<float, uint16_t>(p, num_cus, stream)
                              : launch_bwd_w<float, float>(p, num_cus, stream);
}

}  // namespace dg
