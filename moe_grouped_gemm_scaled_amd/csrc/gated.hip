// gated.hip -- the first half of a gated feed-forward block on gfx950 in one
// kernel: both FP8 block-scaled projections, the activation and the product,
// with a bf16 or an E4M3 output.
//
//     gate = A . Wg^T,  up = A . Wu^T   (b holds Wg, then Wu: [2][I][K])
//     h = act(gate) * up
//
// Arithmetic of the projections as in the plain GEMM: one
// v_mfma_f32_16x16x128_f8f6f4 partial per 16x16 subtile and 128-wide K block,
// promoted into fp32 with sfa * sfb (packed power-of-two scales: applied by
// the scaled MFMA itself).  Nothing is rounded before the outputs.
//
// Organisation: the LDS-DMA pipeline of the plain GEMM (constant-count waits,
// XOR-swizzled stages, see pipelined.hip), with a column tile that holds the
// same columns of both projections: of the B rows that a wave multiplies, half
// are gate rows and half the up rows of the same columns, so a lane ends up
// with both factors of its h values in its own registers and the product needs
// no exchange.  128 columns are also one quantisation block of the next GEMM's
// K axis: a row's scale is a maximum over the tile's row, four values per row
// through LDS.  Narrower tiles, which fill the CUs where 128 columns would
// leave most of them idle, hold no whole block: they leave h in fp32 in the
// caller's workspace, and a second kernel encodes it (4 us, 901 rows, I = 512).
// Outputs are staged in LDS as whole rows, so that every store instruction
// writes whole lines.
#include <stdio.h>

#include "dg_act.h"
#include "dg_gated.h"
#include "dg_internal.h"
#include "dg_layer.h"
#include "dg_quant.h"
#include "dg_rows.h"

namespace dg {

struct GatedArgs {
    const uint8_t *a;
    const float *sfa;
    const uint8_t *b;
    const float *sfb;
    const int32_t *idx;        // m_indices (contiguous) or masked_m (masked)
    uint16_t *gu, *h;
    uint8_t *q;
    void *sf;
    int rows_a, I, K, ld_sfa, ld_sf, G, act;
    int tiles_m, tiles_n, gm;
    int cus;                   // contiguous, 256-row tiles: the CUs that a round fills
    int sa_cols;               // columns of sfa from the first row on (ld_sfa, less the rows before it)
    float *hq;                 // tiles of fewer than 128 columns: h of a quantised output in fp32, [rows][I]
};

// Contiguous layout in 256-row units: those of the full rounds over the CUs, or
// all of them, where the rest would not find room at once in 128-row blocks.
__device__ __forceinline__ int head_units(int units, int tiles_n, int cus) {
    const int64_t tiles = (int64_t)units * tiles_n;
    const int full = (int)(tiles / cus * cus / tiles_n);
    return 2 * (int64_t)(units - full) * tiles_n <= cus ? full : units;
}

// 16-byte chunk c of row r in a staged output tile of CPR chunks per row: the
// chunk index is XORed with the row, so that the 16 rows that a wave writes
// together fall on different banks.
template <int CPR>
__device__ __forceinline__ int staged(int r, int c) {
    return (r * CPR + (c ^ (r & (CPR - 1)))) * 16;
}

// Bytes of a stage: A rows, B rows, and 1 KB each for the scales of A, of B and
// the scale loads of the waves that fetch none.
constexpr int stage_bytes(int bm, int bh) { return (bm + 2 * bh) * kKBlock + 3 * 1024; }

// One tile: rows m0 .. m0 + BM - 1 (of group grp), columns BH * tn .. +BH-1.
// The stages are separate LDS objects, so that the compiler can tell reads of
// one from DMA into another.
template <int BM, int BH, int NST, Mode MODE, bool PK>
__device__ __forceinline__ void gated_tile(const GatedArgs &p, const int m0, const int tn, const int grp, uint8_t *stage0,
                                           uint8_t *stage1, uint8_t *stage2, float *row_max, uint8_t *of_expert) {
    constexpr int BN = 2 * BH;                    // B rows of a tile
    constexpr int NW = 8, WGN = BN >= 128 ? 4 : BN / 32, WGM = NW / WGN;   // waves
    constexpr int TM = BM / WGM, TN = BN / WGN;   // wave tile
    constexpr int TH = TN / 2;                    // columns of h per wave
    constexpr int SM = TM / 16, SN = TN / 16;     // MFMA subtiles per wave
    constexpr int SH = SN / 2;                    // of them gate (the others up)
    constexpr int BLK_A = BM * kKBlock, BLK_B = BN * kKBlock;
    constexpr int OFF_B = BLK_A;
    constexpr int OFF_SA = OFF_B + BLK_B;         // sfa[kb][m0 + 4l .. +3] at 16 l
    constexpr int OFF_SB = OFF_SA + 1024;         // gate, up: 16 bytes of sfb from K block kb
    constexpr int OFF_JUNK = OFF_SB + 1024;       // scale loads of the waves that fetch none (zeros)
    constexpr int STAGE = OFF_JUNK + 1024;
    static_assert(STAGE == stage_bytes(BM, BH), "stage");
    constexpr int DA = BM / (8 * NW), DB = BN / (8 * NW);   // 1-KB LDS-DMA chunks per wave per K block
    constexpr int PER_BLOCK = DA + DB + 1;
    static_assert(NST >= 2 && NST <= 3 && NST * STAGE + BM * (WGN * 4 + 1) <= 160 * 1024, "LDS");
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BM / 4 <= 64 && NW >= 2, "DMA chunks");
    static_assert((NST - 2) * PER_BLOCK < 64, "vmcnt immediate");
    static_assert(TH % 16 == 0 && BM * BH * 2 <= STAGE, "a staged output tile fits one stage");

    auto stage_of = [&](auto sc) __attribute__((always_inline)) -> uint8_t * {
        constexpr int s = decltype(sc)::value;
        if constexpr (s == 0) return stage0;
        else if constexpr (s == 1) return stage1;
        else return stage2;
    };

    const int K = p.K, I = p.I;
    const int nkb = K / kKBlock;
    const int nnb = (I + 127) / 128;
    const int nkw = PK ? (nkb + 3) / 4 : nkb;
    const int n0 = tn * BH;

    const uint8_t *A = p.a;
    const float *SFA = p.sfa;
    const uint8_t *B = p.b;
    const float *SFB = p.sfb;
    int64_t row_base = 0;                          // output row of row 0
    const int ld = p.ld_sfa;
    int rows = p.rows_a - m0;                      // rows of the tile that hold data
    int expert = 0;
    int64_t sf_base = 0;                           // of the group's output scales
    if (MODE == Mode::Masked) {
        const int mm = min(max(p.idx[grp], 0), p.rows_a);
        if (m0 >= mm) return;                      // uniform exit, before any barrier
        rows = mm - m0;
        A += (int64_t)grp * p.rows_a * K;
        SFA += (int64_t)grp * nkw * ld;
        B += (int64_t)grp * 2 * I * K;
        SFB += (int64_t)grp * 2 * nnb * nkw;
        row_base = (int64_t)grp * p.rows_a;
        sf_base = (int64_t)grp * (PK ? (nnb + 3) / 4 : nnb) * p.ld_sf;
    }
    if (MODE == Mode::Contig) {
        expert = p.idx[m0];
        if (expert < 0 || expert >= p.G) return;   // padding (or an invalid id): uniform exit
        B += (int64_t)expert * 2 * I * K;
        SFB += (int64_t)expert * 2 * nnb * nkw;
        if (BM == 256 && !(m0 + 128 < p.rows_a && p.idx[m0 + 128] == expert)) rows = 128;
    }
    rows = min(rows, BM);
    A += (int64_t)m0 * K;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WGN, wn = wave % WGN;
    const int l16 = lane & 15;
    const int g4 = lane >> 4;
    const bool wave_live = wm * TM < rows;         // the wave has rows to multiply
    int row_id = -1;                               // contiguous: the expert of tile row tid
    if (MODE == Mode::Contig && tid < rows) row_id = p.idx[m0 + tid];

    // ---- DMA plan: chunk c = wave + NW*i holds tile rows 8c .. 8c+7; lane l
    // lands at row +l/8, 16-byte chunk l%8 and fetches chunk (l%8) ^ (l/8).
    // A ends at its last row with data: rows past it read as zeros, with no
    // memory traffic.  B row r of the tile belongs to wave column r / TN; its
    // first TH rows are gate rows, the others the up rows of the same columns
    // (columns past I repeat the last one, and are never stored).
    const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc((void *)A, (short)0, rows * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc((void *)B, (short)0, 2 * I * K, 0x00020000);
    const int dchunk = ((lane & 7) ^ (lane >> 3)) * 16;
    int va[DA], vb[DB];
    static_for<DA>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        va[i] = (8 * (wave + NW * i) + (lane >> 3)) * K + dchunk;
    });
    static_for<DB>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        const int r = 8 * (wave + NW * i) + (lane >> 3);
        const int o = r % TN;
        const int col = min(n0 + (r / TN) * TH + o % TH, I - 1);
        vb[i] = ((o / TH) * I + col) * K + dchunk;
    });
    const int lds_a = wave * 1024, lds_b = OFF_B + wave * 1024;
    // scales: lane l of wave 0 fetches sfa[kb][m0 + 4l .. +3], lanes 0 and 1 of
    // wave 1 the 16 bytes from K block kb of the gate's and of the up
    // projection's scale row; every other load points out of range, so that
    // every wave issues the same number
    const bool wsa = wave == 0;
    const __amdgpu_buffer_rsrc_t rS = __builtin_amdgcn_make_buffer_rsrc(
        wsa ? (void *)SFA : (void *)SFB, (short)0,
        wsa ? ((nkw - 1) * ld + p.sa_cols) * 4 : 2 * nnb * nkw * 4, 0x00020000);
    const int sa_row = m0 + 4 * lane;
    const int v_s = wsa ? (4 * lane < BM && sa_row < p.sa_cols ? sa_row * 4 : kOutOfRange)
                        : (wave == 1 && lane < 2 ? (lane * nnb + n0 / 128) * nkw * 4 : kOutOfRange);
    const int lds_s = wsa ? OFF_SA : (wave == 1 ? OFF_SB : OFF_JUNK);
    auto dma = [&](uint8_t *stg, int kb) __attribute__((always_inline)) {
        const int ks = PK ? kb >> 2 : kb;
        dma_step<DA, DB, NW * 1024, NW * 1024>(stg, rA, rB, rS, va, vb, v_s, lds_a, lds_b, lds_s, kb * kKBlock,
                                               kb * kKBlock, wsa ? ks * ld * 4 : ks * 4);
    };

    v4f acc[SM][SN];
    static_for<SM>([&](auto ic) __attribute__((always_inline)) {
        static_for<SN>([&](auto jc) __attribute__((always_inline)) {
            acc[decltype(ic)::value][decltype(jc)::value] = v4f{0.f, 0.f, 0.f, 0.f};
        });
    });
    int off_a0[2], off_b0[2], off_sa;
    {
        const int rowa = wm * TM + l16, rowb = wn * TN + l16;
        off_a0[0] = opaque_offset(rowa * kKBlock + ((g4 ^ (l16 & 7)) << 4));
        off_a0[1] = opaque_offset(rowa * kKBlock + (((g4 + 4) ^ (l16 & 7)) << 4));
        off_b0[0] = opaque_offset(OFF_B + rowb * kKBlock + ((g4 ^ (l16 & 7)) << 4));
        off_b0[1] = opaque_offset(OFF_B + rowb * kKBlock + (((g4 + 4) ^ (l16 & 7)) << 4));
        off_sa = opaque_offset(OFF_SA + rowa * 4);
    }
    auto frag = [&](const uint8_t *lo_p, const uint8_t *hi_p) __attribute__((always_inline)) {
        const v4i lo = *reinterpret_cast<const v4i *>(lo_p);
        const v4i hi = *reinterpret_cast<const v4i *>(hi_p);
        return v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    };

    // Multiply the K block held in `stg`.  The B fragment is the MFMA's first
    // operand: lane l holds row 16i + l%16 and columns 4(l/16) .. +3 of
    // subtile (i, j); subtiles j < SH are gate, j + SH the up projection of the
    // same columns.
    auto compute = [&](const uint8_t *stg, int kb) __attribute__((always_inline)) {
        v8i bf[SN];
        static_for<SN>([&](auto jc) __attribute__((always_inline)) {
            constexpr int j = decltype(jc)::value;
            bf[j] = frag(stg + off_b0[0] + j * 16 * kKBlock, stg + off_b0[1] + j * 16 * kKBlock);
        });
        if constexpr (PK) {
            int eb[2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                eb[x] = (int)((reinterpret_cast<const uint32_t *>(stg + OFF_SB + 16 * x)[0] >> (8 * (kb & 3))) & 0xffu);
            static_for<SM>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                const v8i af = frag(stg + off_a0[0] + i * 16 * kKBlock, stg + off_a0[1] + i * 16 * kKBlock);
                const uint32_t wa = *reinterpret_cast<const uint32_t *>(stg + off_sa + i * 64);
                const int ea = (int)((wa >> (8 * (kb & 3))) & 0xffu);
                static_for<SN>([&](auto jc) __attribute__((always_inline)) {
                    constexpr int j = decltype(jc)::value;
                    acc[i][j] = mfma_16x16x128_e4m3_scaled(bf[j], af, acc[i][j], eb[j / SH], ea);
                });
            });
        } else {
            const float sbg = *reinterpret_cast<const float *>(stg + OFF_SB);
            const float sbu = *reinterpret_cast<const float *>(stg + OFF_SB + 16);
            auto read_a = [&](auto ic, v8i &af, float &sa) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                af = frag(stg + off_a0[0] + i * 16 * kKBlock, stg + off_a0[1] + i * 16 * kKBlock);
                sa = *reinterpret_cast<const float *>(stg + off_sa + i * 64);
            };
            // the A fragment of subtile i+1 is read, and subtile i-1 promoted,
            // while the MFMAs of subtile i run
            v8i af_cur, af_nxt;
            float sa_cur, sa_nxt, sa_prv;
            v4f pp_prv[SN];
            read_a(std::integral_constant<int, 0>{}, af_cur, sa_cur);
            static_for<SM>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                if constexpr (i + 1 < SM) read_a(std::integral_constant<int, i + 1>{}, af_nxt, sa_nxt);
                v4f pp[SN];
                static_for<SN>([&](auto jc) __attribute__((always_inline)) {
                    constexpr int j = decltype(jc)::value;
                    pp[j] = mfma_16x16x128_e4m3(bf[j], af_cur, v4f{0.f, 0.f, 0.f, 0.f});
                });
                if constexpr (i > 0) {
                    static_for<SN>([&](auto jc) __attribute__((always_inline)) {
                        constexpr int j = decltype(jc)::value;
                        acc[i - 1][j] = promote(acc[i - 1][j], pp_prv[j], sa_prv * (j < SH ? sbg : sbu));
                    });
                }
                static_for<SN>([&](auto jc) __attribute__((always_inline)) {
                    pp_prv[decltype(jc)::value] = pp[decltype(jc)::value];
                });
                sa_prv = sa_cur;
                if constexpr (i + 1 < SM) {
                    af_cur = af_nxt;
                    sa_cur = sa_nxt;
                }
            });
            static_for<SN>([&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                acc[SM - 1][j] = promote(acc[SM - 1][j], pp_prv[j], sa_prv * (j < SH ? sbg : sbu));
            });
        }
    };

    // ---- K loop: step j waits for its block, meets the other waves, refills
    // the stage read in step j-1 and multiplies; it starts NST-1 steps early so
    // that one copy of every DMA keeps the wait counts exact
    constexpr int kWaitPipe = wait_vmcnt((NST - 2) * PER_BLOCK);
#pragma clang loop unroll(disable)
    for (int b = -(NST - 1); b < nkb; b += NST) {
        nested_steps<0, NST>(b, nkb, [&](auto sc) __attribute__((always_inline)) {
            constexpr int u = decltype(sc)::value;
            const int j = b + u;
            __builtin_amdgcn_s_waitcnt(kWaitPipe);
            lds_barrier();
            dma(stage_of(sc), min(j + NST - 1, nkb - 1));
            if (j >= 0 && wave_live) compute(stage_of(std::integral_constant<int, (u + 1) % NST>{}), j);
        });
    }
    __builtin_amdgcn_s_waitcnt(wait_vmcnt(0));
    lds_barrier();

    // ---- epilogue.  Row r of the tile is stored when it holds data (its
    // output row is row_base + m0 + r).
    // Contiguous: a row of the expert, looked up once per row (looked up with
    // every 16 bytes stored it took 17 us of a 136 us round).
    if constexpr (MODE == Mode::Contig) {
        if (tid < BM) of_expert[tid] = row_id == expert;
        lds_barrier();
    }
    auto row_ok = [&](int r) __attribute__((always_inline)) {
        return r < rows && (MODE != Mode::Contig || of_expert[r]);
    };
    const int64_t row0 = row_base + m0;
    // staged bf16 tile to columns n0 .. n0+BH-1 of out [..][pitch]
    constexpr int CPR = BH / 8;                    // 16-byte chunks per row
    auto store_bf16 = [&](const uint8_t *stg, uint16_t *out, int64_t pitch) __attribute__((always_inline)) {
        const bool vec = (I % 8) == 0;
        for (int item = tid; item < BM * CPR; item += 64 * NW) {
            const int r = item / CPR, c = item % CPR;
            const int col = n0 + 8 * c;
            if (!row_ok(r) || col >= I) continue;
            const v4i v = *reinterpret_cast<const v4i *>(stg + staged<CPR>(r, c));
            uint16_t *o = out + (row0 + r) * pitch + col;
            if (vec) {
                __builtin_nontemporal_store(v, reinterpret_cast<v4i *>(o));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col + e < I) o[e] = (uint16_t)((uint32_t)v[e >> 1] >> (16 * (e & 1)));
            }
        }
    };
    // subtile (i, j)'s four values of this lane as bf16 into a staged tile
    auto stage_bf16 = [&](uint8_t *stg, int i, int j, const v4f &v) __attribute__((always_inline)) {
        const int r = wm * TM + 16 * i + l16;
        const int c = (wn * TH + 16 * j) / 8 + (g4 >> 1);
        *reinterpret_cast<uint2 *>(stg + staged<CPR>(r, c) + 8 * (g4 & 1)) =
            uint2{pack_bf16x2_rne(v.x, v.y), pack_bf16x2_rne(v.z, v.w)};
    };
    if (p.gu) {                                    // uniform
        static_for<SM>([&](auto ic) __attribute__((always_inline)) {
            static_for<SH>([&](auto jc) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
                stage_bf16(stage0, i, j, acc[i][j]);
                stage_bf16(stage1, i, j, acc[i][j + SH]);
            });
        });
        lds_barrier();
        store_bf16(stage0, p.gu, 2 * (int64_t)I);
        store_bf16(stage1, p.gu + I, 2 * (int64_t)I);
        lds_barrier();
    }
    // h = act(gate) * up, into the gate's registers
    if (p.act == kActSilu) {
        static_for<SM>([&](auto ic) __attribute__((always_inline)) {
            static_for<SH>([&](auto jc) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
                const v4f g = acc[i][j], u = acc[i][j + SH];
                acc[i][j] = v4f{act_value<kActSilu>(g.x) * u.x, act_value<kActSilu>(g.y) * u.y,
                                act_value<kActSilu>(g.z) * u.z, act_value<kActSilu>(g.w) * u.w};
            });
        });
    } else {
        static_for<SM>([&](auto ic) __attribute__((always_inline)) {
            static_for<SH>([&](auto jc) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
                const v4f g = acc[i][j], u = acc[i][j + SH];
                acc[i][j] = v4f{act_value<kActGelu>(g.x) * u.x, act_value<kActGelu>(g.y) * u.y,
                                act_value<kActGelu>(g.z) * u.z, act_value<kActGelu>(g.w) * u.w};
            });
        });
    }
    if (p.h) {                                     // uniform
        static_for<SM>([&](auto ic) __attribute__((always_inline)) {
            static_for<SH>([&](auto jc) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
                stage_bf16(stage0, i, j, acc[i][j]);
            });
        });
        lds_barrier();
        store_bf16(stage0, p.h, I);
    }
    if constexpr (BH < 128) {                      // no whole quantisation block: gated_encode_kernel takes over
        if (p.hq) {                                // uniform; I is a multiple of 128
            static_for<SM>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                const int r = wm * TM + 16 * i + l16;
                static_for<SH>([&](auto jc) __attribute__((always_inline)) {
                    constexpr int j = decltype(jc)::value;
                    if (r < rows)
                        *reinterpret_cast<v4f *>(p.hq + (row0 + r) * I + n0 + wn * TH + 16 * j + 4 * g4) = acc[i][j];
                });
            });
        }
    } else if (p.q) {                              // uniform; I is a multiple of 128
        // the row's maximum over this wave's TH columns, then over the waves
        static_for<SM>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            float m = 0.f;
            static_for<SH>([&](auto jc) __attribute__((always_inline)) {
                const v4f v = acc[i][decltype(jc)::value];
                m = fmaxf(m, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
            });
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            if (g4 == 0) row_max[wn * BM + wm * TM + 16 * i + l16] = m;
        });
        lds_barrier();
        static_for<SM>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            const int r = wm * TM + 16 * i + l16;
            float m = row_max[r];
#pragma unroll
            for (int x = 1; x < WGN; ++x) m = fmaxf(m, row_max[x * BM + r]);
            const float s = block_scale<PK>(m);
            const BlockDivisor d = block_divisor<PK>(s);
            static_for<SH>([&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                *reinterpret_cast<uint32_t *>(stage1 + staged<8>(r, wn * SH + j) + 4 * g4) =
                    encode4<PK>(acc[i][j], d);
            });
            if (wn == 0 && g4 == 0 && row_ok(r))
                store_block_scale<PK>(static_cast<uint32_t *>(p.sf) + sf_base, p.ld_sf, m0 + r, n0 / 128, nnb, s);
        });
        lds_barrier();
        for (int item = tid; item < BM * 8; item += 64 * NW) {
            const int r = item >> 3, c = item & 7;
            if (row_ok(r))
                *reinterpret_cast<v4i *>(p.q + (row0 + r) * I + n0 + 16 * c) =
                    *reinterpret_cast<const v4i *>(stage1 + staged<8>(r, c));
        }
    }
}

// One tile per workgroup, in all layouts.
template <int BM, int BH, int NST, Mode MODE, bool PK>
__global__ void __launch_bounds__(512, BH == 32 ? 4 : 2)   // waves per SIMD: two workgroups of the smallest tile share a CU
gated_kernel(GatedArgs p) {
    constexpr int STAGE = stage_bytes(BM, BH);
    __shared__ __attribute__((aligned(16))) uint8_t stage0[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t stage1[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t stage2[NST > 2 ? STAGE : 16];
    __shared__ float row_max[BH == 128 ? 4 * BM : 1];
    __shared__ uint8_t of_expert[MODE == Mode::Contig ? BM : 1];
    const int tiles_per_group = p.tiles_m * p.tiles_n;
    int t_lin = xcd_remap(blockIdx.x, gridDim.x);
    int grp = 0;
    if (MODE == Mode::Masked) {
        grp = t_lin / tiles_per_group;
        t_lin -= grp * tiles_per_group;
    }
    int tm, tn;
    raster(t_lin, p.tiles_m, p.tiles_n, p.gm, tm, tn);
    gated_tile<BM, BH, NST, MODE, PK>(p, tm * BM, tn, grp, stage0, stage1, stage2, row_max, of_expert);
}

// Contiguous layout, many rows: tiles of 256-row units for the full rounds over
// the CUs, then the remaining rows in 128-row blocks, when those fit the CUs at
// once: a last, partly filled round of 256-row tiles costs as much as a full
// one.  How many units there are is known on the device only, so every
// workgroup works out its tile from m_indices.  In one launch the blocks fill
// the CUs as the units' tiles end, of which those with one block of rows are
// early.
// The first `first` workgroups take a tile each, which is all of them where
// every expert has one segment.  Where the experts' blocks alternate there are
// up to twice as many units; the workgroups behind go over the tiles past the
// first ones, block by block.  (A workgroup for each such tile would end at
// once in the usual case, but takes 2 us to find that out: 1024 blocks, 16
// experts, I = 256, K = 512: 126 against 119 us, 118 without any.)
template <bool PK>
__global__ void __launch_bounds__(512, 2) gated_units_kernel(GatedArgs p, int first) {
    constexpr int STAGE = stage_bytes(256, 128);
    __shared__ __attribute__((aligned(16))) uint8_t stage0[STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t stage1[STAGE];
    __shared__ float row_max[4 * 256];
    __shared__ uint8_t of_expert[256];
    const int nblocks = p.rows_a / 128;
    const ContigBlocks blocks = contig_load(p.idx, nblocks, 0);
    int units = 0;
    contig_scan(p.idx, nblocks, blocks, -1, units);
    units = __builtin_amdgcn_readfirstlane(units);
    const int head = head_units(units, p.tiles_n, p.cus);
    const int head_tiles = head * p.tiles_n, tail_m = 2 * (units - head);
    const int tiles = head_tiles + tail_m * p.tiles_n;
    // tile t of the rest: the first block of its unit, and whether the tile is the unit's second block
    auto rest_tile = [&](int t, int &tn, int &second) __attribute__((always_inline)) {
        int tm;
        raster(xcd_remap(t - head_tiles, tail_m * p.tiles_n), tail_m, p.tiles_n, p.gm, tm, tn);
        second = tm & 1;
        return __builtin_amdgcn_readfirstlane(contig_scan(p.idx, nblocks, blocks, head + tm / 2, units));
    };
    auto head_tile = [&](int t, int &tn) __attribute__((always_inline)) {
        int tm;
        raster(xcd_remap(t, head_tiles), head, p.tiles_n, p.gm, tm, tn);
        return __builtin_amdgcn_readfirstlane(contig_scan(p.idx, nblocks, blocks, tm, units));
    };
    // a unit's second block, where it has one
    auto has_second = [&](int b) __attribute__((always_inline)) {
        return b + 1 < nblocks && p.idx[((int64_t)b + 1) * 128] == p.idx[(int64_t)b * 128];
    };
    int tn, second = 0;
    if ((int)blockIdx.x < first) {
        const int t = blockIdx.x;
        if (t < head_tiles) {
            const int b = head_tile(t, tn);
            gated_tile<256, 128, 2, Mode::Contig, PK>(p, b * 128, tn, 0, stage0, stage1, nullptr, row_max, of_expert);
        } else if (t < tiles) {
            const int b = rest_tile(t, tn, second);
            if (second && !has_second(b)) return;  // uniform exit
            gated_tile<128, 128, 2, Mode::Contig, PK>(p, (b + second) * 128, tn, 0, stage0, stage1, nullptr, row_max, of_expert);
        }
        return;
    }
    for (int t = (int)blockIdx.x; t < tiles; t += (int)gridDim.x - first) {     // uniform
        const bool whole = t < head_tiles;
        const int b = whole ? head_tile(t, tn) : rest_tile(t, tn, second);
        for (int k = whole ? 0 : second; k <= (whole ? 1 : second); ++k) {
            if (k && !has_second(b)) break;
            gated_tile<128, 128, 2, Mode::Contig, PK>(p, (b + k) * 128, tn, 0, stage0, stage1, nullptr, row_max, of_expert);
            __syncthreads();                       // the next tile's loads overwrite the stages
        }
    }
}

// E4M3 blocks of h from fp32: 16 lanes per (row, 128-column block).
template <bool PK>
__global__ void __launch_bounds__(256) gated_encode_kernel(GatedArgs p) {
    const int lane16 = threadIdx.x & 15;
    const int I = p.I, nnb = I / 128;
    const int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int nb = (int)(unit % nnb);
    const int64_t row = unit / nnb;
    if (row >= p.rows_a) return;                   // whole groups of 16 lanes
    const int64_t o = row * I + 128 * nb + 8 * lane16;
    const Raw8<float> v = load8(p.hq + o);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(get8(v, e)));
    const float s = block_scale<PK>(max16(m));
    const BlockDivisor d = block_divisor<PK>(s);
    *reinterpret_cast<uint2 *>(p.q + o) =
        uint2{encode4<PK>(v4f{get8(v, 0), get8(v, 1), get8(v, 2), get8(v, 3)}, d),
              encode4<PK>(v4f{get8(v, 4), get8(v, 5), get8(v, 6), get8(v, 7)}, d)};
    if (lane16 == 0) store_block_scale<PK>(static_cast<uint32_t *>(p.sf), p.ld_sf, row, nb, nnb, s);
}

static GatedArgs args_of(const GatedProblem &p, int bm, int bh, int num_cus) {
    return {p.a, p.sfa, p.b, p.sfb, p.idx, p.gu, p.h, p.q, p.sf, p.rows_a, p.I, p.K, p.ld_sfa, p.ld_sf, p.G, p.act,
            (p.rows_a + bm - 1) / bm, (p.I + bh - 1) / bh, 4, num_cus, p.ld_sfa - p.row0,
            bh < 128 && p.q ? static_cast<float *>(p.ws) : nullptr};
}

static void describe(std::string &config, Mode mode, const char *tile, int stages, int64_t grid, bool packed) {
    char buf[160];
    snprintf(buf, sizeof buf, "%sfamily=gated mode=%d %s stages=%d grid=%lld%s", config.empty() ? "" : " + ", (int)mode,
             tile, stages, (long long)grid, packed ? " scales=ue8m0_packed" : "");
    config += buf;
}

template <int BM, int BH, int NST, Mode MODE, bool PK>
static hipError_t launch_t(const GatedProblem &p, int num_cus, hipStream_t stream, std::string &config) {
    const GatedArgs k = args_of(p, BM, BH, num_cus);
    const int64_t grid = (int64_t)k.tiles_m * k.tiles_n * (MODE == Mode::Masked ? p.G : 1);
    if (!grid_fits(grid, 512)) return hipErrorInvalidValue;
    char tile[32];
    snprintf(tile, sizeof tile, "tile=%dx%dx128", BM, 2 * BH);
    describe(config, MODE, tile, NST, grid, PK);
    hipLaunchKernelGGL((gated_kernel<BM, BH, NST, MODE, PK>), dim3((unsigned)grid), dim3(512), 0, stream, k);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || !k.hq) return err;
    const int64_t blocks = (int64_t)p.rows_a * (p.I / 128);
    hipLaunchKernelGGL(gated_encode_kernel<PK>, dim3((unsigned)((blocks + 15) / 16)), dim3(256), 0, stream, k);
    return hipGetLastError();
}

template <bool PK>
static hipError_t launch_units(const GatedProblem &p, int num_cus, hipStream_t stream, std::string &config) {
    const GatedArgs k = args_of(p, 256, 128, num_cus);
    // With one segment per expert, every expert's last unit may hold one block,
    // and no unit holds less; the rest takes at most one workgroup per CU, half
    // of them in place of units.  Other orders have up to a unit per block.
    const int64_t nblocks = p.rows_a / 128, most = nblocks / 2 + p.G + 1;
    const int64_t first = (most < nblocks ? most : nblocks) * k.tiles_n + num_cus / 2;
    const int64_t more = nblocks * k.tiles_n + num_cus / 2 - first;
    const int64_t grid = first + (more < num_cus ? more : num_cus);
    if (!grid_fits(grid, 512)) return hipErrorInvalidValue;
    describe(config, Mode::Contig, "tile=256x256x128 rest: tile=128x256x128", 2, grid, PK);
    hipLaunchKernelGGL((gated_units_kernel<PK>), dim3((unsigned)grid), dim3(512), 0, stream, k, (int)first);
    return hipGetLastError();
}

// Tiles, rows x columns of h, and what a round of them over the CUs costs per K
// block, in hundredths of a round of 256x128 (measured, I = 2048, K = 7168:
// 97 to 103 us at 256x128 with packed scales, 57 to 60 at 128x128, 39 to 41 at
// 128x64, 38 (packed) to 46 (fp32 scales) at 64x128, 26.3 at 64x64 and 18.0 at
// 64x32).  Small tiles multiply less per byte they load, but fill the CUs: 256
// rows take 18.0 us in 64x32 tiles, 33 in 64x128 ones.  Three stages: two cost
// 30 to 40 % more with the narrow tiles, four gain nothing.
struct Tile {
    int rows, cols, cost;
};
constexpr Tile kTiles[] = {{256, 128, 100}, {128, 128, 60}, {128, 64, 38}, {64, 128, 41}, {64, 64, 25}, {64, 32, 17}};
// Prologue and epilogue of a round, and the second kernel of a narrow tile with
// a quantised output, in the same unit (18 ns).
constexpr int kRoundCost = 150, kEncodeCost = 300;

// narrow: tiles of fewer than 128 columns can serve.  encode: they need the
// second kernel.  spare: rows that 256-row tiles waste besides.  cap: rows that
// are launched, of which `rows` are expected to hold data.
static Tile choose_tile(int rows, int cap, int spare, int groups, int I, int K, bool narrow, bool encode, int num_cus) {
    Tile best = kTiles[0];
    int64_t least = INT64_MAX;
    for (const Tile &t : kTiles) {
        if (t.cols < 128 && !narrow) continue;
        const int64_t tiles = groups * ((rows + (t.rows == 256 ? (int64_t)spare : 0) + t.rows - 1) / t.rows) * ((I + t.cols - 1) / t.cols);
        // many groups of few columns: a larger tile
        if (!grid_fits(groups * (((int64_t)cap + t.rows - 1) / t.rows) * ((I + t.cols - 1) / t.cols), 512)) continue;
        const int64_t c = (tiles + num_cus - 1) / num_cus * ((int64_t)t.cost * (K / kKBlock) + kRoundCost) +
                          (t.cols < 128 && encode ? kEncodeCost : 0);
        if (c < least) {
            least = c;
            best = t;
        }
    }
    return best;
}

template <Mode MODE, bool PK>
static hipError_t launch_tile(Tile t, const GatedProblem &p, int num_cus, hipStream_t stream, std::string &config) {
    if constexpr (MODE != Mode::Contig) {           // contiguous: launch_units
        if (t.rows == 256) return launch_t<256, 128, 2, MODE, PK>(p, num_cus, stream, config);
    }
    if (t.rows == 128)
        return t.cols == 128 ? launch_t<128, 128, 3, MODE, PK>(p, num_cus, stream, config)
                             : launch_t<128, 64, 3, MODE, PK>(p, num_cus, stream, config);
    return t.cols == 128  ? launch_t<64, 128, 3, MODE, PK>(p, num_cus, stream, config)
           : t.cols == 64 ? launch_t<64, 64, 3, MODE, PK>(p, num_cus, stream, config)
                          : launch_t<64, 32, 3, MODE, PK>(p, num_cus, stream, config);
}

// Dense: rows of the full rounds of 256x128 tiles.
static int head_rows(int rows, int I, int num_cus) {
    const int64_t tiles_n = (I + 127) / 128;
    return (int)(rows / 256 * tiles_n / num_cus * num_cus / tiles_n * 256);
}

template <bool PK>
static hipError_t launch_pk(const GatedProblem &p, int num_cus, hipStream_t stream, std::string &config) {
    const int64_t tiles_n = (p.I + 127) / 128;
    switch (p.mode) {
    case Mode::Dense: {
        // full rounds of 256-row tiles, then the rows that are left in tiles of
        // their own choice (4500 rows: 16 row tiles of 256, then 64-row tiles)
        const int head = head_rows(p.rows_a, p.I, num_cus), rest = p.rows_a - head;
        if (head > 0) {
            GatedProblem q = p;
            q.rows_a = head;
            const hipError_t err = launch_t<256, 128, 2, Mode::Dense, PK>(q, num_cus, stream, config);
            if (err != hipSuccess || rest == 0) return err;
        }
        GatedProblem q = p;
        q.rows_a = rest;
        q.row0 = head;
        q.a += (int64_t)head * p.K;
        q.sfa += head;
        if (q.gu) q.gu += (int64_t)head * 2 * p.I;
        if (q.h) q.h += (int64_t)head * p.I;
        if (q.q) {
            q.q += (int64_t)head * p.I;
            q.sf = static_cast<uint32_t *>(p.sf) + head;
        }
        const bool scratch = p.ws && p.ws_bytes >= (size_t)rest * p.I * sizeof(float);
        const Tile t = choose_tile(rest, rest, 0, 1, p.I, p.K, !p.q || scratch, p.q != nullptr, num_cus);
        return launch_tile<Mode::Dense, PK>(t, q, num_cus, stream, config);
    }
    case Mode::Contig: {
        // every expert's last unit may hold one block only: one more 256-row tile each
        const Tile t = choose_tile(p.rows_a, p.rows_a, 128 * p.G, 1, p.I, p.K, !p.q, false, num_cus);
        if (t.rows == 64 || t.cols < 128) return launch_tile<Mode::Contig, PK>(t, p, num_cus, stream, config);
        if (p.rows_a < 256 || (t.rows == 128 && p.rows_a / 128 * tiles_n <= num_cus))
            return launch_tile<Mode::Contig, PK>(kTiles[1], p, num_cus, stream, config);
        return launch_units<PK>(p, num_cus, stream, config);
    }
    case Mode::Masked: {
        // the groups' counts are on the device: the caller's hint, or the capacity
        const int expect = p.expected_m > 0 && p.expected_m < p.rows_a ? p.expected_m : p.rows_a;
        const Tile t = choose_tile(expect, p.rows_a, 0, p.G, p.I, p.K, !p.q, false, num_cus);
        return launch_tile<Mode::Masked, PK>(t, p, num_cus, stream, config);
    }
    case Mode::KGrouped: break;
    }
    return hipErrorInvalidValue;
}

size_t gated_workspace(int M, int I, int K, int num_cus) {
    if (M <= kGatedSmallMaxM) return gated_small_workspace(M, I, K, num_cus);
    if (I % 128 != 0) return 0;                    // no quantised output
    const int rest = M - head_rows(M, I, num_cus);
    return rest > 0 && choose_tile(rest, rest, 0, 1, I, K, true, true, num_cus).cols < 128 ? (size_t)rest * I * sizeof(float) : 0;
}

hipError_t launch_gated(const GatedProblem &p, int num_cus, hipStream_t stream, std::string &config) {
    if (gated_small_takes(p, num_cus)) return launch_gated_small(p, num_cus, stream, config);
    return p.packed ? launch_pk<true>(p, num_cus, stream, config) : launch_pk<false>(p, num_cus, stream, config);
}

}  // namespace dg
