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
#include "dg_pipeline.h"
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

// Keeps a value in its register from here on, instead of the operands of the
// product that makes it.
__device__ __forceinline__ void materialise(float &x) { asm volatile("" : "+v"(x)); }

// 512 threads per 128x128 tile: thread t holds columns 8 (t % 16) .. +7 of
// rows t / 16 + 32 i (i < 4), so 16 lanes hold a row's 128 columns (its scale
// is a reduction inside the DPP row) and every access is 16 (codes: 8)
// consecutive bytes per lane, whole lines per row.  COLS: the column-scaled
// outputs are wanted; their maxima go through LDS.
//
// A tile holds three arrays (0: d_gate, 1: d_up, 2: h).  All three in one
// workgroup are 96 values per thread; 128 registers leave room for two
// workgroups on a CU, so that one's loads and stores run under the other's
// arithmetic (17408 rows of 2048: 128 us with one workgroup of 168 registers,
// 86 us with two, 82 us with the division in fp32).  Buffer accesses keep the addresses in scalar registers for
// that, and turn rows past the last into zeros and dropped stores.
// The arithmetic (some 50 vector instructions per column and row) takes about
// as long as the memory traffic, and with few tiles it is all there is: SPLIT
// gives each array of a tile a workgroup of its own.
template <int ACT, bool UE, bool COLS, bool SPLIT>
__global__ void __launch_bounds__(512, 4)
gated_bwd_kernel(GatedBwdArgs p) {
    constexpr int kNt = SPLIT ? 0 : 2;                // nontemporal: read once
    constexpr int NA = SPLIT ? 1 : (COLS ? 3 : 2);    // arrays of this workgroup
    const int t = threadIdx.x;
    const int c8 = 8 * (t & 15), rg = t >> 4;
    const int part = SPLIT ? (int)(blockIdx.x % (COLS ? 3 : 2)) : 0;
    const int tile = SPLIT ? (int)(blockIdx.x / (COLS ? 3 : 2)) : (int)blockIdx.x;
    const int tm = tile / p.tiles_n, tn = tile - tm * p.tiles_n;
    const int I = p.I, n0 = tn * 128;
    const int64_t m0 = (int64_t)tm * 128;
    const int rows = (int)(p.rows - m0 < 128 ? p.rows - m0 : 128);   // of this tile
    // a row-major tensor of `pitch` elements of `size` bytes from column col of the tile's first row
    auto window = [&](const void *base, int pitch, int size, int col, int n) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc((void *)((const char *)base + (m0 * pitch + col) * size), (short)0,
                                                 n * pitch * size, 0x00020000);
    };
    // element offsets of the thread's i-th row in tensors of pitch 2I and I;
    // opaque, so that each is one addition where it is used, not a register
    // held throughout
    const int o2 = rg * 2 * I + c8, o1 = rg * I + c8;
    auto at2 = [&](int i) __attribute__((always_inline)) { return opaque_offset(o2) + 32 * i * 2 * I; };
    auto at1 = [&](int i) __attribute__((always_inline)) { return opaque_offset(o1) + 32 * i * I; };
    float v[NA][4][8];
    {
        const __amdgpu_buffer_rsrc_t rG = window(p.gu, 2 * I, 2, n0, rows), rU = window(p.gu, 2 * I, 2, I + n0, rows),
                                     rD = window(p.dh, I, 2, n0, rows);
        // NULL idx: an empty window, which reads as 0, a row that counts; rows
        // past the last read as zeros and so count as nothing
        const __amdgpu_buffer_rsrc_t rI =
            __builtin_amdgcn_make_buffer_rsrc((void *)(p.idx + (p.idx ? m0 : 0)), (short)0, p.idx ? rows * 4 : 0, 0x00020000);
        Raw8<uint16_t> g8[4], u8[4], d8[4];
        int id[4];
        static_for<4>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            g8[i].a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rG, 2 * at2(i), 0, kNt));
            u8[i].a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rU, 2 * at2(i), 0, kNt));
            d8[i].a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rD, 2 * at1(i), 0, kNt));
            id[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(rI, 4 * (rg + 32 * i), 0, 0);
        });
        static_for<4>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            const v4i zero = v4i{0, 0, 0, 0};
            const Raw8<uint16_t> gr{id[i] < 0 ? zero : g8[i].a}, ur{id[i] < 0 ? zero : u8[i].a},
                dr{id[i] < 0 ? zero : d8[i].a};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = get8(gr, e), u = get8(ur, e), d = get8(dr, e);
                float a, da;
                act_and_grad<ACT>(g, a, da);
                if constexpr (SPLIT) {
                    v[0][i][e] = part == 0 ? d * u * da : part == 1 ? d * a : a * u;   // uniform
                } else {
                    v[0][i][e] = d * u * da;
                    v[1][i][e] = d * a;
                    if constexpr (COLS) v[2][i][e] = a * u;
                    // otherwise a, u and d stay live beside the products
#pragma unroll
                    for (int k = 0; k < NA; ++k) materialise(v[k][i][e]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);        // row by row: interleaved rows need more registers
        });
    }
    typedef unsigned v2u __attribute__((ext_vector_type(2)));
    auto encode = [&](const float (&x)[8], auto &&div) __attribute__((always_inline)) {
        return v2u{e4m3_encode4(div(x[0], 0), div(x[1], 1), div(x[2], 2), div(x[3], 3)),
                   e4m3_encode4(div(x[4], 4), div(x[5], 5), div(x[6], 6), div(x[7], 7))};
    };
    __shared__ __attribute__((aligned(16))) float wmax[COLS ? NA : 1][COLS ? 32 : 1][128];
    __shared__ __attribute__((aligned(16))) float div_y[COLS ? NA : 1][128], div_s[COLS ? NA : 1][128];
    if constexpr (COLS) {
        // ---- column maxima of the thread's four rows
        static_for<NA>([&](auto kc) __attribute__((always_inline)) {
            constexpr int k = decltype(kc)::value;
            float m[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                m[e] = fmaxf(fmaxf(fabsf(v[k][0][e]), fabsf(v[k][1][e])), fmaxf(fabsf(v[k][2][e]), fabsf(v[k][3][e])));
            store8(&wmax[k][rg][c8], m);
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    // ---- row scales and row outputs of d_gate and d_up
    static_for<NA>([&](auto kc) __attribute__((always_inline)) {
        constexpr int k = decltype(kc)::value;
        const int id = SPLIT ? part : k;
        if (id == 2) return;                          // uniform
        const int col = id * I + n0;
        if (p.dgu) {
            const __amdgpu_buffer_rsrc_t r = window(p.dgu, 2 * I, 2, col, rows);
            static_for<4>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                const v4i w = v4i{(int)pack_bf16x2_rne(v[k][i][0], v[k][i][1]), (int)pack_bf16x2_rne(v[k][i][2], v[k][i][3]),
                                  (int)pack_bf16x2_rne(v[k][i][4], v[k][i][5]), (int)pack_bf16x2_rne(v[k][i][6], v[k][i][7])};
                __builtin_amdgcn_raw_buffer_store_b128(w, r, 2 * at2(i), 0, 2);
            });
        }
        if (p.q) {                                    // uniform
            const __amdgpu_buffer_rsrc_t r = window(p.q, 2 * I, 1, col, rows);
            float *sf = p.sf + (int64_t)(col / 128) * p.ld_sf + m0;
            static_for<4>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[k][i][e]));
                const float s = block_scale<UE>(max16(m));
                const BlockDivisor d = block_divisor<UE>(s);
                const v2u w = encode(v[k][i], [&](float x, int) __attribute__((always_inline)) { return divide<UE>(x, d); });
                __builtin_amdgcn_raw_buffer_store_b64(w, r, at2(i), 0, 0);
                const int row = rg + 32 * i;
                if (c8 == 0 && row < rows) sf[row] = s;
                __builtin_amdgcn_sched_barrier(0);
            });
        }
    });
    if constexpr (COLS) {
        __syncthreads();
        for (int x = t; x < NA * 128; x += 512) {
            const int k = x / 128, c = x % 128;
            float m = wmax[k][0][c];
#pragma unroll
            for (int w = 1; w < 32; ++w) m = fmaxf(m, wmax[k][w][c]);
            const float s = block_scale<UE>(m);
            const BlockDivisor d = block_divisor<UE>(s);
            div_y[k][c] = d.y;
            div_s[k][c] = d.s;
            const int id = SPLIT ? part : k;
            if (id < 2) {
                if (p.qt) p.sft[(int64_t)tm * 2 * I + id * I + n0 + c] = s;
            } else if (p.ht) {
                p.sfht[(int64_t)tm * I + n0 + c] = s;
            }
        }
        __syncthreads();
        static_for<NA>([&](auto kc) __attribute__((always_inline)) {
            constexpr int k = decltype(kc)::value;
            const int id = SPLIT ? part : k;
            uint8_t *out = id == 2 ? p.ht : p.qt;
            if (!out) return;                         // uniform
            // these have 128 rows per tile, whatever the number of rows
            const __amdgpu_buffer_rsrc_t r =
                id == 2 ? window(out, I, 1, n0, 128) : window(out, 2 * I, 1, id * I + n0, 128);
            const Raw8<float> y = load8(&div_y[k][c8]), s = load8(&div_s[k][c8]);
            static_for<4>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                const v2u w = encode(v[k][i], [&](float x, int e) __attribute__((always_inline)) {
                    return divide<UE>(x, BlockDivisor{get8(y, e), get8(s, e)});
                });
                __builtin_amdgcn_raw_buffer_store_b64(w, r, id == 2 ? at1(i) : at2(i), 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            });
        });
    }
}

template <int ACT, bool UE>
static hipError_t launch_t(const GatedBwdArgs &a, int64_t tiles, int num_cus, hipStream_t stream) {
    const bool cols = a.qt || a.ht;
    const int parts = cols ? 3 : 2;
    // one workgroup per array while those all find room at once (two per CU);
    // measured at 200 rows of 2048 (32 tiles): 14.4 -> 10.4 us
    const bool split = tiles * parts <= 2 * (int64_t)num_cus;
    const dim3 grid((unsigned)(split ? tiles * parts : tiles));
    if (cols) {
        if (split) hipLaunchKernelGGL((gated_bwd_kernel<ACT, UE, true, true>), grid, dim3(512), 0, stream, a);
        else hipLaunchKernelGGL((gated_bwd_kernel<ACT, UE, true, false>), grid, dim3(512), 0, stream, a);
    } else {
        if (split) hipLaunchKernelGGL((gated_bwd_kernel<ACT, UE, false, true>), grid, dim3(512), 0, stream, a);
        else hipLaunchKernelGGL((gated_bwd_kernel<ACT, UE, false, false>), grid, dim3(512), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedBwdProblem &p, int num_cus, hipStream_t stream) {
    const int tiles_n = p.I / 128;
    const int64_t grid = ((int64_t)p.rows + 127) / 128 * tiles_n;
    if (!grid_fits(grid, 512)) return hipErrorInvalidValue;
    const GatedBwdArgs a{p.gu, p.dh, p.idx, p.dgu, p.q, p.sf, p.qt, p.sft, p.ht, p.sfht, p.rows, p.I, p.ld_sf, tiles_n};
    if (p.act == kActSilu)
        return p.ue8m0 ? launch_t<kActSilu, true>(a, grid, num_cus, stream)
                       : launch_t<kActSilu, false>(a, grid, num_cus, stream);
    return p.ue8m0 ? launch_t<kActGelu, true>(a, grid, num_cus, stream)
                   : launch_t<kActGelu, false>(a, grid, num_cus, stream);
}

}  // namespace dg
