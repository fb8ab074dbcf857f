// gated_bwd.hip -- gradient of the gated activation h = act(gate) * up for
// gfx950, quantised for the two gradient GEMMs that follow it.
//
// From the saved projections and dh, in fp32:
//     d_gate = dh * up * act'(gate),  d_up = dh * act(gate),  h = act(gate) * up
// Outputs (each optional): d_gate | d_up in bf16; its E4M3 codes with one scale
// per row and 128 columns (the A operand of the input gradient); its codes and
// those of h with one scale per column and 128 rows (the operands of the weight
// gradients, whose K axis are the rows).
//
// HBM-bound: 6 bytes read and up to 5 written per (row, column) of h, and both
// scale directions need one 128 x 128 tile in registers at a time, so a
// workgroup takes exactly one such tile of gate, up and dh and everything is
// read once.
#include "dg_act.h"
#include "dg_layer.h"
#include "dg_quant.h"
#include "dg_rows.h"

namespace dg {

struct GatedBwdArgs {
    const uint16_t *gu, *dh;
    const int32_t *idx;       // expert of each row, < 0: the row counts as zeros (NULL: every row counts)
    uint16_t *dgu;
    uint8_t *q;
    float *sf;
    uint8_t *qt;
    float *sft;
    uint8_t *ht;
    float *sfht;
    int rows, I, ld_sf, tiles_n;
};

// 512 threads per 128x128 tile: thread t holds columns 8 (t % 16) .. +7 of
// rows t / 16 + 32 i (i < 4), so 16 lanes hold a row's 128 columns (its scale
// is a reduction inside the DPP row) and every access is 16 consecutive bytes
// per lane, 256 per row.  COLS: the column-scaled outputs are wanted; their
// maxima go through LDS, one partial per wave.
template <int ACT, bool UE, bool COLS>
__global__ void __launch_bounds__(512)
gated_bwd_kernel(GatedBwdArgs p) {
    const int t = threadIdx.x;
    const int lane = t & 63, wave = t >> 6;
    const int c8 = 8 * (t & 15), rg = t >> 4;
    const int tm = blockIdx.x / p.tiles_n, tn = blockIdx.x - tm * p.tiles_n;
    const int I = p.I, n0 = tn * 128;
    const int64_t m0 = (int64_t)tm * 128;
    Raw8<uint16_t> g8[4], u8[4], d8[4];
    bool live[4];
    static_for<4>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        const int64_t r = m0 + rg + 32 * i;
        const int64_t rc = r < p.rows ? r : p.rows - 1;
        const uint16_t *gp = p.gu + rc * 2 * I + n0 + c8;
        g8[i] = load8<true>(gp);
        u8[i] = load8<true>(gp + I);
        d8[i] = load8<true>(p.dh + rc * I + n0 + c8);
        live[i] = r < p.rows && (!p.idx || p.idx[rc] >= 0);
    });
    float dg[4][8], du[4][8], hh[4][8];
    static_for<4>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float g = get8(g8[i], e), u = get8(u8[i], e), d = get8(d8[i], e);
            float a, da;
            act_and_grad<ACT>(g, a, da);
            dg[i][e] = live[i] ? d * u * da : 0.f;
            du[i][e] = live[i] ? d * a : 0.f;
            if constexpr (COLS) hh[i][e] = live[i] ? a * u : 0.f;
        }
    });
    auto encode = [&](const float (&v)[8], auto &&inv) __attribute__((always_inline)) {
        uint2 w;
        w.x = e4m3_encode4(inv(v[0], 0), inv(v[1], 1), inv(v[2], 2), inv(v[3], 3));
        w.y = e4m3_encode4(inv(v[4], 4), inv(v[5], 5), inv(v[6], 6), inv(v[7], 7));
        return w;
    };
    // ---- row scales and row outputs
    static_for<4>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        const int64_t r = m0 + rg + 32 * i;
        const bool in = r < p.rows;
        if (p.dgu && in) {
            store8<true>(p.dgu + r * 2 * I + n0 + c8, dg[i]);
            store8<true>(p.dgu + r * 2 * I + I + n0 + c8, du[i]);
        }
        if (p.q) {                                             // uniform
            float mg = 0.f, mu = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                mg = fmaxf(mg, fabsf(dg[i][e]));
                mu = fmaxf(mu, fabsf(du[i][e]));
            }
            const float sg = block_scale<UE>(max16(mg)), su = block_scale<UE>(max16(mu));
            const double ig = 1.0 / (double)sg, iu = 1.0 / (double)su;
            const uint2 wg = encode(dg[i], [&](float x, int) { return div_by_scale(x, ig); });
            const uint2 wu = encode(du[i], [&](float x, int) { return div_by_scale(x, iu); });
            if (in) {
                uint8_t *qr = p.q + r * 2 * I + n0 + c8;
                *reinterpret_cast<uint2 *>(qr) = wg;
                *reinterpret_cast<uint2 *>(qr + I) = wu;
                if (c8 == 0) {
                    p.sf[(int64_t)(n0 / 128) * p.ld_sf + r] = sg;
                    p.sf[(int64_t)((I + n0) / 128) * p.ld_sf + r] = su;
                }
            }
        }
    });
    if constexpr (COLS) {
        // ---- column scales: maxima over the thread's four rows, the wave's
        // four row groups, then the eight waves
        __shared__ __attribute__((aligned(16))) float wmax[8][3][128];
        __shared__ __attribute__((aligned(16))) double inv[3][128];
        float m[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m[0][e] = fmaxf(fmaxf(fabsf(dg[0][e]), fabsf(dg[1][e])), fmaxf(fabsf(dg[2][e]), fabsf(dg[3][e])));
            m[1][e] = fmaxf(fmaxf(fabsf(du[0][e]), fabsf(du[1][e])), fmaxf(fabsf(du[2][e]), fabsf(du[3][e])));
            m[2][e] = fmaxf(fmaxf(fabsf(hh[0][e]), fabsf(hh[1][e])), fmaxf(fabsf(hh[2][e]), fabsf(hh[3][e])));
        }
#pragma unroll
        for (int a = 0; a < 3; ++a)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                m[a][e] = fmaxf(m[a][e], __shfl_xor(m[a][e], 16));
                m[a][e] = fmaxf(m[a][e], __shfl_xor(m[a][e], 32));
            }
        if (lane < 16) {
#pragma unroll
            for (int a = 0; a < 3; ++a) store8(&wmax[wave][a][c8], m[a]);
        }
        __syncthreads();
        if (t < 384) {
            const int a = t / 128, c = t % 128;
            float v = wmax[0][a][c];
#pragma unroll
            for (int w = 1; w < 8; ++w) v = fmaxf(v, wmax[w][a][c]);
            const float s = block_scale<UE>(v);
            inv[a][c] = 1.0 / (double)s;
            if (a < 2) {
                if (p.qt) p.sft[(int64_t)tm * 2 * I + a * I + n0 + c] = s;
            } else if (p.ht) {
                p.sfht[(int64_t)tm * I + n0 + c] = s;
            }
        }
        __syncthreads();
        auto column_codes = [&](const float (&v)[4][8], int a, uint8_t *out, int64_t pitch) __attribute__((always_inline)) {
            double y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = inv[a][c8 + e];
            static_for<4>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                const uint2 w = encode(v[i], [&](float x, int e) { return div_by_scale(x, y[e]); });
                *reinterpret_cast<uint2 *>(out + (m0 + rg + 32 * i) * pitch) = w;
            });
        };
        if (p.qt) {
            column_codes(dg, 0, p.qt + n0 + c8, 2 * I);
            column_codes(du, 1, p.qt + I + n0 + c8, 2 * I);
        }
        if (p.ht) column_codes(hh, 2, p.ht + n0 + c8, I);
    }
}

template <int ACT, bool UE>
static hipError_t launch_t(const GatedBwdArgs &a, unsigned grid, hipStream_t stream) {
    if (a.qt || a.ht) hipLaunchKernelGGL((gated_bwd_kernel<ACT, UE, true>), dim3(grid), dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((gated_bwd_kernel<ACT, UE, false>), dim3(grid), dim3(512), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedBwdProblem &p, hipStream_t stream) {
    const int tiles_n = p.I / 128;
    const int64_t grid = ((int64_t)p.rows + 127) / 128 * tiles_n;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    const GatedBwdArgs a{p.gu, p.dh, p.idx, p.dgu, p.q, p.sf, p.qt, p.sft, p.ht, p.sfht, p.rows, p.I, p.ld_sf, tiles_n};
    if (p.act == kActSilu)
        return p.ue8m0 ? launch_t<kActSilu, true>(a, (unsigned)grid, stream)
                       : launch_t<kActSilu, false>(a, (unsigned)grid, stream);
    return p.ue8m0 ? launch_t<kActGelu, true>(a, (unsigned)grid, stream)
                   : launch_t<kActGelu, false>(a, (unsigned)grid, stream);
}

}  // namespace dg
