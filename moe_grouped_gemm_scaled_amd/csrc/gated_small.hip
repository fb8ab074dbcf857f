// gated_small.hip -- the gated GEMM for few rows (decode) on gfx950: the run
// time is the stream of both weight matrices from HBM.
//
// Arithmetic as in gated.hip.  Organisation: a workgroup takes 8 columns of h,
// that is one 16-row B fragment of the MFMA (8 gate rows, the 8 up rows of the
// same columns), all rows of A, and all of K, which is split over its waves.
// Each wave streams its K blocks (16 B rows and all A rows of the block)
// through a ring of NST LDS stages of its own, filled by DMA, so no barrier
// stands in the K loop, and I / 8 workgroups (or half as many) spread B over the
// CUs.  The rings of a workgroup hold 65 to 80 KB up to 64 rows, so about 150 KB
// per CU where the grid gives every CU two workgroups, and half of that where it
// gives one (I = 2048); above 64 rows 127 to 154 KB.  A is read by every
// workgroup, from L2.  Loading
// fragments straight into registers needs no LDS, but 16 lanes then touch 16
// rows: 33 KB/us per CU against 80 to 100 with 8 lanes on each 128-byte line
// (measured on L2-resident data), 20.8 against 10.9 us at 64 rows, I = 2048,
// K = 7168.  The waves' fp32 sums meet in LDS and are added in wave order.
//
// K may further be split over S workgroups, which lets a workgroup take more
// columns and so read A less often; and a quantised output needs a row's
// maximum over 128 columns, which no workgroup has.  In both cases the sums
// go to the caller's workspace in fp32, and a second kernel adds the S partial
// sums in order and finishes h: one wave per 4 (row, 128-column) blocks.  (A
// single kernel whose last workgroup finishes a block, behind device-coherent
// stores and a counter, took about 1 us longer per call and needed the
// workspace zeroed.)
#include <stdio.h>

#include "dg_act.h"
#include "dg_gated.h"
#include "dg_internal.h"
#include "dg_layer.h"
#include "dg_quant.h"
#include "dg_rows.h"

namespace dg {

struct GatedSmallArgs {
    const uint8_t *a;
    const float *sfa;
    const uint8_t *b;
    const float *sfb;
    uint16_t *gu, *h;
    uint8_t *q;
    void *sf;
    float *ws;        // partial sums [S][M][2][I], or NULL: this kernel finishes h
    int M, I, K, ld_sfa, ld_sf, S;
};

// MT 16-row tiles of A, NF fragments of B (8 columns of h each), NW waves, NST
// stages per wave.
template <int MT, int NF, int NW, int NST, int ACT, bool PK>
__global__ void __launch_bounds__(64 * NW)
gated_small_kernel(GatedSmallArgs p) {
    constexpr int NS = (16 * MT + 63) / 64;           // loads of A scales per K block
    constexpr int OFF_B = MT * 2048;                  // a stage: A rows, B rows, A scales, B scales
    constexpr int OFF_SA = OFF_B + NF * 2048;
    constexpr int OFF_SB = OFF_SA + NS * 256;
    constexpr int STAGE = OFF_SB + 256;
    constexpr int PER_BLOCK = 2 * MT + 2 * NF + NS + 1;    // loads per K block
    static_assert(NST >= 2 && NST <= 4 && NST * NW * STAGE <= 160 * 1024 - 64, "stages fit the LDS");
    static_assert((NST - 1) * PER_BLOCK < 64, "vmcnt immediate");
    static_assert(MT * NF * 1024 <= STAGE, "the waves' sums fit the first stage of each");
    // one object per stage, so that the compiler can tell reads of one from
    // DMA into another
    __shared__ __attribute__((aligned(16))) uint8_t stage0[NW * STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t stage1[NW * STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t stage2[NST > 2 ? NW * STAGE : 16];
    __shared__ __attribute__((aligned(16))) uint8_t stage3[NST > 3 ? NW * STAGE : 16];
    auto stage_of = [&](auto sc) __attribute__((always_inline)) -> uint8_t * {
        constexpr int s = decltype(sc)::value;
        if constexpr (s == 0) return stage0;
        else if constexpr (s == 1) return stage1;
        else if constexpr (s == 2) return stage2;
        else return stage3;
    };
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int K = p.K, I = p.I, M = p.M;
    const int nkb = K / kKBlock, nnb = (I + 127) / 128;
    const int nkw = PK ? (nkb + 3) / 4 : nkb;
    // column tile and K share; the wave's blocks are its part of that share
    const int split = blockIdx.x % p.S;
    const int n0 = 8 * NF * (int)(blockIdx.x / p.S);
    const int part_id = split * NW + wave, parts = p.S * NW;
    const int kb0 = (int)((int64_t)nkb * part_id / parts);
    const int nblk = (int)((int64_t)nkb * (part_id + 1) / parts) - kb0;

    const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc((void *)p.a, (short)0, M * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc((void *)p.b, (short)0, 2 * I * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t rSA =
        __builtin_amdgcn_make_buffer_rsrc((void *)p.sfa, (short)0, nkw * p.ld_sfa * 4, 0x00020000);
    const __amdgpu_buffer_rsrc_t rSB =
        __builtin_amdgcn_make_buffer_rsrc((void *)p.sfb, (short)0, 2 * nnb * nkw * 4, 0x00020000);
    // DMA: a load brings 8 rows of 128 bytes; lane l lands at row +l/8, 16-byte
    // chunk l%8 and fetches chunk (l%8) ^ (l/8), so that fragment reads of 16
    // rows spread over the banks.  Rows of A past M read as zeros without
    // memory traffic; columns past I repeat the last one.
    const int dchunk = ((lane & 7) ^ (lane >> 3)) * 16;
    const int va = (lane >> 3) * K + dchunk;
    int vb[NF];                                       // gate rows; the up rows lie I * K further
    static_for<NF>([&](auto fc) __attribute__((always_inline)) {
        constexpr int f = decltype(fc)::value;
        vb[f] = min(n0 + 8 * f + (lane >> 3), I - 1) * K + dchunk;
    });
    const int v_sb = lane < 2 ? (lane * nnb + n0 / 128) * nkw * 4 : kOutOfRange;
    auto fetch = [&](uint8_t *base, int kb) __attribute__((always_inline)) {
        uint8_t *stg = base + wave * STAGE;
        static_for<2 * MT>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            dma_lds16(rA, stg + i * 1024, va + 8 * i * K, kb * kKBlock);
        });
        static_for<NF>([&](auto fc) __attribute__((always_inline)) {
            constexpr int f = decltype(fc)::value;
            dma_lds16(rB, stg + OFF_B + f * 2048, vb[f], kb * kKBlock);
            dma_lds16(rB, stg + OFF_B + f * 2048 + 1024, vb[f] + I * K, kb * kKBlock);
        });
        const int ks = PK ? kb >> 2 : kb;
        static_for<NS>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            const int row = 64 * i + lane;
            dma_lds4(rSA, stg + OFF_SA + i * 256, row < p.ld_sfa ? row * 4 : kOutOfRange, ks * p.ld_sfa * 4);
        });
        dma_lds4(rSB, stg + OFF_SB, v_sb, ks * 4);
    };

    v4f acc[MT][NF];
    static_for<MT>([&](auto ic) __attribute__((always_inline)) {
        static_for<NF>([&](auto fc) __attribute__((always_inline)) {
            acc[decltype(ic)::value][decltype(fc)::value] = v4f{0.f, 0.f, 0.f, 0.f};
        });
    });
    // fragment offsets: row l%16, chunks l/16 and l/16 + 4; opaque, so that
    // every read is one address computation from its stage object
    const int off0 = opaque_offset(wave * STAGE + l16 * kKBlock + ((g4 ^ (l16 & 7)) << 4));
    const int off1 = opaque_offset(wave * STAGE + l16 * kKBlock + (((g4 + 4) ^ (l16 & 7)) << 4));
    const int off_sa = opaque_offset(wave * STAGE + OFF_SA + 4 * l16);
    // scale of the lane's B rows: an fp32 scale multiplies the result, whose
    // columns 4(l/16) .. +3 are gate for l < 32; an exponent goes with the operand
    const int off_sb = opaque_offset(wave * STAGE + OFF_SB + 4 * (PK ? l16 >> 3 : g4 >> 1));
    auto compute = [&](const uint8_t *stg, int kb) __attribute__((always_inline)) {
        auto frag = [&](int row16) __attribute__((always_inline)) {
            const v4i lo = *reinterpret_cast<const v4i *>(stg + off0 + row16 * 2048);
            const v4i hi = *reinterpret_cast<const v4i *>(stg + off1 + row16 * 2048);
            return v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        };
        v8i bf[NF];
        static_for<NF>([&](auto fc) __attribute__((always_inline)) {
            bf[decltype(fc)::value] = frag(MT + decltype(fc)::value);
        });
        const uint32_t sb = *reinterpret_cast<const uint32_t *>(stg + off_sb);
        const int sh = 8 * (kb & 3);
        static_for<MT>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            const v8i af = frag(i);
            const uint32_t sa = *reinterpret_cast<const uint32_t *>(stg + off_sa + 64 * i);
            static_for<NF>([&](auto fc) __attribute__((always_inline)) {
                constexpr int f = decltype(fc)::value;
                if constexpr (PK) {
                    acc[i][f] = mfma_16x16x128_e4m3_scaled(bf[f], af, acc[i][f], (int)((sb >> sh) & 0xffu),
                                                           (int)((sa >> sh) & 0xffu));
                } else {
                    const v4f pp = mfma_16x16x128_e4m3(bf[f], af, v4f{0.f, 0.f, 0.f, 0.f});
                    acc[i][f] = promote(acc[i][f], pp, __uint_as_float(sa) * __uint_as_float(sb));
                }
            });
        });
    };

    // ---- K loop of the wave: block j lives in stage (j + NST - 1) mod NST.
    // Step j refills the stage read in step j-1 (once its reads are done) with
    // block j + NST - 1, waits for block j and multiplies it.  It starts NST-1
    // steps early; indices past the end fetch the last block again, which is
    // then not multiplied.
    constexpr int kWait = wait_vmcnt((NST - 1) * PER_BLOCK);
    if (nblk > 0) {                                   // uniform per wave
#pragma clang loop unroll(disable)   // one copy of every load keeps the wait counts exact
        for (int b = -(NST - 1); b < nblk; b += NST) {
            nested_steps<0, NST>(b, nblk, [&](auto sc) __attribute__((always_inline)) {
                constexpr int u = decltype(sc)::value;
                const int j = b + u;
                lds_reads_done();
                fetch(stage_of(sc), kb0 + min(j + NST - 1, nblk - 1));
                __builtin_amdgcn_s_waitcnt(kWait);
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");   // no read moves above the wait
                if (j >= 0) compute(stage_of(std::integral_constant<int, (u + 1) % NST>{}), kb0 + j);
            });
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_vmcnt(0));        // no DMA is left that could land in the sums
    __syncthreads();
    v4f(*part)[MT * NF][64] = reinterpret_cast<v4f(*)[MT * NF][64]>(stage0);
    static_for<MT>([&](auto ic) __attribute__((always_inline)) {
        static_for<NF>([&](auto fc) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value, f = decltype(fc)::value;
            part[wave][i * NF + f][lane] = acc[i][f];
        });
    });
    __syncthreads();

    // Wave w finishes the (row tile, fragment) pairs w, w + NW, ..: it adds the
    // waves' sums; lane l then holds row 16i + l%16, gate columns 4(l/16) .. +3
    // for l < 32 and the up values of the same columns in lane l + 32.
    const bool vec = (I % 8) == 0;
    for (int t = wave; t < MT * NF; t += NW) {        // uniform
        v4f s = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += part[w][t][lane];
        const int row = 16 * (t / NF) + l16;
        const int c = n0 + 8 * (t % NF) + 4 * (g4 & 1);       // of h
        const int half = g4 >> 1;                             // 0: gate, 1: up
        if (p.ws) {                                           // uniform; I is a multiple of 8
            if (row < M && c < I)
                *reinterpret_cast<v4f *>(p.ws + (((int64_t)split * M + row) * 2 + half) * I + c) = s;
            continue;
        }
        v4f u;
        u.x = __shfl_xor(s.x, 32);
        u.y = __shfl_xor(s.y, 32);
        u.z = __shfl_xor(s.z, 32);
        u.w = __shfl_xor(s.w, 32);
        auto store4 = [&](uint16_t *o, const v4f &v) __attribute__((always_inline)) {
            if (vec) {
                *reinterpret_cast<uint2 *>(o) = uint2{pack_bf16x2_rne(v.x, v.y), pack_bf16x2_rne(v.z, v.w)};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < I) o[e] = f32_to_bf16_rne(v[e]);
            }
        };
        if (row < M && c < I) {
            if (p.gu) store4(p.gu + ((int64_t)row * 2 + half) * I + c, s);
            if (half == 0)
                store4(p.h + (int64_t)row * I + c, v4f{act_value<ACT>(s.x) * u.x, act_value<ACT>(s.y) * u.y,
                                                       act_value<ACT>(s.z) * u.z, act_value<ACT>(s.w) * u.w});
        }
    }
}

// h from the partial sums: 16 lanes per (row, 128-column block), 8 columns
// each; the S sums are added in order.
template <int ACT, bool PK>
__global__ void __launch_bounds__(64) gated_finish_kernel(GatedSmallArgs p) {
    const int lane = threadIdx.x;
    const int I = p.I, nnb = (I + 127) / 128;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (lane >> 4);
    const int nb = (int)(unit % nnb);
    const int row = (int)(unit / nnb);
    const int c = 128 * nb + 8 * (lane & 15);
    const bool in = row < p.M && c < I;
    float g[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.f;
    const float *w = p.ws + (in ? (int64_t)row * 2 * I + c : 0);
    for (int s = 0; s < p.S; ++s, w += (int64_t)p.M * 2 * I) {
        const Raw8<float> a = load8(w), b = load8(w + I);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[e] += get8(a, e);
            u[e] += get8(b, e);
        }
    }
    if (p.gu && in) {
        store8(p.gu + (int64_t)row * 2 * I + c, g);
        store8(p.gu + ((int64_t)row * 2 + 1) * I + c, u);
    }
    float h[8], m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        h[e] = act_value<ACT>(g[e]) * u[e];
        m = fmaxf(m, fabsf(h[e]));
    }
    if (p.h && in) store8(p.h + (int64_t)row * I + c, h);
    if (!p.q) return;                                 // uniform; I is a multiple of 128
    const float s = block_scale<PK>(max16(m));
    const BlockDivisor d = block_divisor<PK>(s);
    if (in)
        *reinterpret_cast<uint2 *>(p.q + (int64_t)row * I + c) =
            uint2{encode4<PK>(v4f{h[0], h[1], h[2], h[3]}, d), encode4<PK>(v4f{h[4], h[5], h[6], h[7]}, d)};
    if (in && (lane & 15) == 0) store_block_scale<PK>(static_cast<uint32_t *>(p.sf), p.ld_sf, row, nb, nnb, s);
}

// Fragments per workgroup and K splits.  A workgroup reads all of A (of its K
// share) for its 8 * nf columns, so above 16 rows two fragments are taken once
// 16-column tiles alone give every CU one (measured, K = 7168, I = 4096: 17.1
// -> 13.0 us at 64 rows, 25.2 -> 19.4 us at 128, 12.2 -> 11.0 us at 32, 10.8 ->
// 11.2 us at 16).  With fewer columns they are taken when the second kernel
// runs anyway (a quantised output), K split so that every CU still has work
// (I = 2048: 11.0 -> 9.3 us at 64 rows, 17.4 -> 13.2 us at 128); without it
// the split does not pay for that kernel's 3 us.
struct SmallPlan {
    int nf, splits;
};
static SmallPlan small_plan(int M, int I, int K, bool quant, int num_cus) {
    const int tiles = (I + 15) / 16;
    if (M <= 16) return {1, 1};
    if (tiles >= num_cus) return {2, 1};
    if (!quant || M <= 32) return {1, 1};
    int s = num_cus / tiles;
    s = s > 4 ? 4 : s;
    const int most = K / kKBlock;
    return {2, s > most ? most : s};
}

// A quantised output with a short K goes to the tiles instead: as fast there,
// in one launch and without scratch (K = 1024: 1 row of 768 columns 7.8 us
// against 3.5 + 2.0 and a gap, 64 rows of 2048 9.4 against 4.8 + 3.2, 128 rows
// 9.6 against 7.2 + 2.8; K = 2048: 13.9 against 5 + 3).
constexpr int kQuantMinK = 1024;

// Scratch of a quantised output: the partial sums.  (Other outputs need none.)
size_t gated_small_workspace(int M, int I, int K, int num_cus) {
    if (M < 1 || M > kGatedSmallMaxM || I % 128 != 0 || K <= kQuantMinK) return 0;
    return (size_t)small_plan(M, I, K, true, num_cus).splits * M * 2 * I * sizeof(float);
}

bool gated_small_takes(const GatedProblem &p, int num_cus) {
    if (p.mode != Mode::Dense || p.rows_a > kGatedSmallMaxM || (int64_t)p.rows_a * p.K >= (int64_t)1 << 31) return false;
    if (!p.q) return true;
    return p.K > kQuantMinK && p.ws && p.ws_bytes >= gated_small_workspace(p.rows_a, p.I, p.K, num_cus);
}

template <int MT, int NF, int NW, int NST>
static hipError_t launch_t(const GatedProblem &p, int S, hipStream_t stream, std::string &config) {
    GatedSmallArgs k{p.a, p.sfa, p.b, p.sfb, p.gu, p.h, p.q, p.sf, nullptr, p.rows_a, p.I, p.K, p.ld_sfa, p.ld_sf, S};
    if (p.q) k.ws = static_cast<float *>(p.ws);
    const unsigned grid = (unsigned)((p.I + 8 * NF - 1) / (8 * NF) * S);
    const unsigned grid2 = (unsigned)(((int64_t)p.rows_a * ((p.I + 127) / 128) + 3) / 4);
    char buf[120];
    snprintf(buf, sizeof buf, "family=gated_small rows=%d cols=%d waves=%d stages=%d splits=%d grid=%u%s", 16 * MT,
             8 * NF, NW, NST, S, grid, p.packed ? " scales=ue8m0_packed" : "");
    config = buf;
    auto go = [&](auto ac, auto pc) -> hipError_t {
        constexpr int ACT = decltype(ac)::value;
        constexpr bool PK = decltype(pc)::value;
        hipLaunchKernelGGL((gated_small_kernel<MT, NF, NW, NST, ACT, PK>), dim3(grid), dim3(64 * NW), 0, stream, k);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess || !k.ws) return err;
        hipLaunchKernelGGL((gated_finish_kernel<ACT, PK>), dim3(grid2), dim3(64), 0, stream, k);
        return hipGetLastError();
    };
    using Silu = std::integral_constant<int, kActSilu>;
    using Gelu = std::integral_constant<int, kActGelu>;
    if (p.packed) return p.act == kActSilu ? go(Silu{}, std::true_type{}) : go(Gelu{}, std::true_type{});
    return p.act == kActSilu ? go(Silu{}, std::false_type{}) : go(Gelu{}, std::false_type{});
}

hipError_t launch_gated_small(const GatedProblem &p, int num_cus, hipStream_t stream, std::string &config) {
    const SmallPlan pl = small_plan(p.rows_a, p.I, p.K, p.q != nullptr, num_cus);
    // waves and stages: two workgroups' rings fit the LDS of a CU up to 64 rows, one above
    if (p.rows_a <= 16) return launch_t<1, 1, 4, 4>(p, pl.splits, stream, config);
    if (pl.nf == 1) {
        if (p.rows_a <= 32) return launch_t<2, 1, 4, 3>(p, pl.splits, stream, config);
        if (p.rows_a <= 64) return launch_t<4, 1, 3, 2>(p, pl.splits, stream, config);
        return launch_t<8, 1, 4, 2>(p, pl.splits, stream, config);
    }
    if (p.rows_a <= 32) return launch_t<2, 2, 4, 2>(p, pl.splits, stream, config);
    if (p.rows_a <= 64) return launch_t<4, 2, 3, 2>(p, pl.splits, stream, config);
    return launch_t<8, 2, 3, 2>(p, pl.splits, stream, config);
}

}  // namespace dg
