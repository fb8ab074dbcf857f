/*
 * dg.h -- C ABI of the MI355X (gfx950) FP8 block-scaled GEMM library: the
 * NT GEMM and its M-grouped MoE forms, the E4M3 quantisers, the NN/TN/TT
 * layouts, the K-grouped weight-gradient GEMM, power-of-two (UE8M0) scale
 * variants, the FP8 MQA logits, and the operators around the GEMMs of a
 * gated feed-forward layer (norms, gating, the tokens' way to the experts'
 * rows and back, and their gradients).
 *
 * Operation (the "DeepGEMM" README summary on GeekNews, ja.news.hada.io topic
 * 19459, section "GEMM interface and layout constraints"): D = C + A . B^T in
 * the NT layout, A and B in FP8 E4M3, FP32 scaling factors with the LHS
 * scales stored transposed, the caller doing the casting and transposition.
 * Scales are applied during accumulation: for every 128-wide K block the FP8
 * matrix-core partial is promoted into an FP32 accumulator after multiplying
 * by sfa * sfb (two-level accumulation, "DeepSeek open-sources DeepGEMM",
 * picoinsstore.com, paragraph on the Hopper design).  Granularity: one scale
 * per row and 128-wide K block of A (1x128), one per 128x128 block of B.
 *
 *   D[m,n] = C[m,n] + sum_kb sfa[kb][m] * sfb[n/128][kb] * sum_{k in kb} A[m,k] B[n,k]
 *
 * Conventions for every entry point (a declaration below states any
 * exception, e.g. the fp32 outputs of the K-grouped GEMM and the MQA logits):
 *  - Types: E4M3 values are uint8_t bit patterns (OCP E4M3FN: bias 7, no
 *    infinities, max 448); bf16 values are uint16_t bit patterns; scales fp32.
 *  - All tensors are dense, row-major (last index fastest), in device memory
 *    owned by the caller; base pointers must be 16-byte aligned.  The library
 *    keeps no pointer after the call returns.
 *  - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default
 *    stream).  Argument errors are detected on the host and returned before
 *    anything is launched; nothing is written then.  A failed launch returns
 *    DG_ERR_HIP, and so do sizes that would take a grid of 2^32 threads (some
 *    10^6 to 10^7 workgroups).  Device faults surface at the caller's next synchronisation.
 *  - D is bf16, rounded to nearest even from the fp32 accumulator.  C is bf16
 *    of the same shape as D, or NULL for C = 0; C may alias D exactly.
 *  - K must be a positive multiple of 128.  M and N may be any positive size
 *    (partial row and column tiles are handled), except where an operand is
 *    stored MN-major (multiples of 16).
 *  - The library allocates no device memory and never synchronises.  Dense
 *    calls with a small M run fastest with K split over several workgroups,
 *    which needs scratch memory: the *_ws entry points take it from the
 *    caller (size from dg_get_workspace_size), the others run without
 *    split-K.
 *  - Thread-safe.  Process-wide settings: the CU cap only.  Per thread: the
 *    kernel-family setting and the last-config string.
 */
#ifndef DG_H
#define DG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dg_status {
    DG_OK = 0,
    DG_ERR_NULL = -1,        /* a required pointer is NULL */
    DG_ERR_SHAPE = -2,       /* a size is out of range (K % 128, M, N, G <= 0, M_total % 128) */
    DG_ERR_ALIGN = -3,       /* a pointer or leading dimension is misaligned */
    DG_ERR_ARG = -4,         /* any other invalid argument */
    DG_ERR_UNSUPPORTED = -5, /* valid but not supported here (e.g. not a gfx950 device) */
    DG_ERR_HIP = -6,         /* a HIP runtime call failed */
    DG_ERR_SCRATCH = -7      /* more scratch needed than dg_fp8_gemm_nt_noalloc holds */
} dg_status;

/*
 * Dense FP8 NT GEMM, D = C + A . B^T.
 *   a   [M][K]                E4M3
 *   sfa [K/128][ld_sfa]       fp32, sfa[kb*ld_sfa + m] scales A[m, 128kb : 128kb+128];
 *                             ld_sfa >= M and ld_sfa % 4 == 0 (the transposed,
 *                             16-byte aligned LHS scale layout); entries with
 *                             m >= M are never used for results.
 *   b   [N][K]                E4M3 (row n is column n of B^T)
 *   sfb [ceil(N/128)][K/128]  fp32, sfb[nb*(K/128) + kb] scales the 128x128 block
 *   c   [M][N] bf16 or NULL;  d [M][N] bf16 (written entirely).
 * Errors: DG_ERR_NULL (a, sfa, b, sfb, d), DG_ERR_SHAPE (M, N < 1; K < 128 or
 * K % 128), DG_ERR_ALIGN (ld_sfa < M or ld_sfa % 4; pointer not 16-B aligned).
 */
int dg_fp8_gemm_nt(const uint8_t *a, const float *sfa, int ld_sfa,
                   const uint8_t *b, const float *sfb,
                   const uint16_t *c, uint16_t *d,
                   int M, int N, int K, void *stream);

/*
 * The dense GEMM with caller-provided split-K scratch.  Same arguments,
 * results and errors as dg_fp8_gemm_nt (and dg_fp8_gemm_nt_ue8m0), plus:
 *   workspace        device memory, 16-byte aligned, or NULL (then K is
 *                    never split: the dg_fp8_gemm_nt path);
 *   workspace_bytes  its size; at least dg_get_workspace_size(M, N, K) for
 *                    the configuration the call chooses (DG_ERR_ARG
 *                    otherwise, before anything is launched).
 * Layout: the workspace starts with a fixed 16 KiB region of int32 arrival
 * counters (one per output tile of a split call), which must be ZERO when a
 * call starts; every call that completes leaves them zero again, so memory
 * zeroed once (hipMemset, torch.zeros) serves any number of calls of any
 * shapes in stream order, eager or captured in a graph.  The rest holds the
 * fp32 partial tiles of the K splits.  The caller owns
 * the workspace; it must stay allocated until the call's work completes, and
 * two calls that may run at the same time (other streams, concurrently
 * replayed graphs) need two workspaces.  The partials of the splits are
 * added in split order, so the result does not depend on the order in which
 * the splits finish.
 */
int dg_fp8_gemm_nt_ws(const uint8_t *a, const float *sfa, int ld_sfa,
                      const uint8_t *b, const float *sfb,
                      const uint16_t *c, uint16_t *d,
                      int M, int N, int K,
                      void *workspace, size_t workspace_bytes, void *stream);
int dg_fp8_gemm_nt_ue8m0_ws(const uint8_t *a, const float *sfa, int ld_sfa,
                            const uint8_t *b, const float *sfb,
                            const uint16_t *c, uint16_t *d,
                            int M, int N, int K,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * Allocation-free dense GEMM, for callers that cannot allocate device memory
 * (code under graph capture, serving loops that forbid allocation): the
 * results of dg_fp8_gemm_nt_ws with a large enough workspace, the split-K
 * scratch being the library's own device array of 32 MiB per GPU (loaded
 * with the library's code and held until the process ends; its counters are
 * cleared on the first call per device).  Allocates and frees nothing.
 * Every call on a GPU shares that GPU's array: calls that may overlap in time
 * on one GPU (other streams, concurrently replayed graphs) race, and must use
 * dg_fp8_gemm_nt_ws with separate workspaces instead.  Same arguments and
 * errors as dg_fp8_gemm_nt, plus DG_ERR_SCRATCH when the configuration the
 * call chooses needs more scratch than the array holds (more than 32 MiB
 * with its 16 KiB of counters); nothing is launched then.
 */
int dg_fp8_gemm_nt_noalloc(const uint8_t *a, const float *sfa, int ld_sfa,
                           const uint8_t *b, const float *sfb,
                           const uint16_t *c, uint16_t *d,
                           int M, int N, int K, void *stream);

/*
 * Workspace bytes for dg_fp8_gemm_nt_ws and dg_fp8_gemm_nt_ue8m0_ws on an
 * M x N x K problem on the current device, with the calling thread's kernel
 * family setting and the CU cap in force (0: the problem is not split).
 * Negative dg_status on error: DG_ERR_SHAPE (M, N < 1; K), DG_ERR_HIP or
 * DG_ERR_UNSUPPORTED (no usable device).  The pages' library keeps such
 * buffers itself; here the caller owns all memory, so that every call is
 * asynchronous and can be captured into a graph.
 */
int64_t dg_get_workspace_size(int M, int N, int K);

/*
 * The other memory layouts of the dense GEMM ("DeepGEMM" README summary,
 * sections "GEMM interface and layout constraints" and "Dense and Grouped
 * GEMM": fp8_gemm_{nt, nn, tn, tt}, D = C + A @ B with each operand either
 * as stored or transposed).  The product, the scales and their layouts are
 * those of dg_fp8_gemm_nt:
 *   D[m,n] = C[m,n] + sum_kb sfa[kb][m] * sfb[n/128][kb] * sum_{k in kb} A(m,k) B(n,k)
 * only where A(m,k) and B(n,k) are stored differs:
 *   nn: a [M][K] (A(m,k) = a[m*K + k]),  b [K][N] (B(n,k) = b[k*N + n])
 *   tn: a [K][M] (A(m,k) = a[k*M + m]),  b [K][N]
 *   tt: a [K][M],                        b [N][K] (as in nt)
 * An operand stored [K][M] or [K][N] (MN-major) needs M (resp. N) a multiple
 * of 16, so that its rows are 16-byte aligned, and K*M (K*N) below 2^31.
 * Same arguments otherwise, same tolerance, same errors as dg_fp8_gemm_nt,
 * plus DG_ERR_ALIGN (M or N of an MN-major operand not a multiple of 16) and
 * DG_ERR_SHAPE (K*M or K*N reaching 2^31).  These always run on the
 * pipelined kernel family, whatever dg_set_kernel_family selects.
 */
int dg_fp8_gemm_nn(const uint8_t *a, const float *sfa, int ld_sfa,
                   const uint8_t *b, const float *sfb,
                   const uint16_t *c, uint16_t *d,
                   int M, int N, int K, void *stream);
int dg_fp8_gemm_tn(const uint8_t *a, const float *sfa, int ld_sfa,
                   const uint8_t *b, const float *sfb,
                   const uint16_t *c, uint16_t *d,
                   int M, int N, int K, void *stream);
int dg_fp8_gemm_tt(const uint8_t *a, const float *sfa, int ld_sfa,
                   const uint8_t *b, const float *sfb,
                   const uint16_t *c, uint16_t *d,
                   int M, int N, int K, void *stream);

/*
 * M-grouped contiguous layout ("DeepGEMM" README summary, section "Dense and
 * Grouped GEMM"): the tokens of all experts are concatenated along M, N and K
 * are shared, and every expert segment starts at a multiple of the M block
 * (dg_get_mk_alignment_for_contiguous_layout(), 128 rows).
 *   a   [M_total][K] E4M3;  sfa [K/128][M_total] fp32
 *   b   [G][N][K] E4M3;     sfb [G][ceil(N/128)][K/128] fp32
 *   c   [M_total][N] bf16 or NULL;  d [M_total][N] bf16
 *   m_indices [M_total] int32 in device memory: the expert of each row, or -1
 *             on padding rows.  Rows with -1 are neither computed nor written;
 *             a 128-row block whose first id lies outside [0, G) is treated
 *             as padding too (so a bad id never reads outside b and sfb).
 * Precondition (not checked on the device): each aligned 128-row block holds
 * rows of at most one expert, valid rows first.  The blocks may come in any
 * order (an expert may own several segments).
 * Errors: DG_ERR_NULL, DG_ERR_SHAPE (M_total % 128, N, K, G < 1), DG_ERR_ALIGN.
 */
int dg_m_grouped_fp8_gemm_nt_contiguous(const uint8_t *a, const float *sfa,
                                        const uint8_t *b, const float *sfb,
                                        const uint16_t *c, uint16_t *d,
                                        const int32_t *m_indices,
                                        int M_total, int N, int K, int G,
                                        void *stream);

/*
 * M-grouped masked layout (same section): every group owns M_cap rows and
 * only its first masked_m[g] rows are valid; the counts live on the device,
 * so the host never reads them and the call is safe to capture in a graph.
 *   a   [G][M_cap][K] E4M3;  sfa [G][K/128][round_up(M_cap,4)] fp32
 *   b   [G][N][K] E4M3;      sfb [G][ceil(N/128)][K/128] fp32
 *   c   [G][M_cap][N] bf16 or NULL;  d [G][M_cap][N] bf16
 *   masked_m [G] int32 in device memory, clamped to [0, M_cap] on the device.
 *   expected_m: host hint of the typical count (<= 0: unknown); it only
 *               steers the tile choice and never changes results.
 * Rows r >= masked_m[g] of d are left untouched.
 * Errors: DG_ERR_NULL, DG_ERR_SHAPE (G, M_cap, N < 1; K), DG_ERR_ALIGN.
 */
int dg_m_grouped_fp8_gemm_nt_masked(const uint8_t *a, const float *sfa,
                                    const uint8_t *b, const float *sfb,
                                    const uint16_t *c, uint16_t *d,
                                    const int32_t *masked_m,
                                    int G, int M_cap, int N, int K,
                                    int expected_m, void *stream);

/*
 * E4M3 quantiser, one scale per row and 128-wide K block (the LHS layout):
 *   x [groups][rows][K] fp32  ->  q [groups][rows][K] E4M3,
 *   sf [groups][K/128][ld_sf] fp32 with sf = max(amax, 1e-4) / 448 (one IEEE
 *   fp32 division) and q = round-to-nearest-even(x / sf) (IEEE division,
 *   saturating at +-448).  Entries of sf with row >= rows are not written.
 * The pages leave the cast to the user ("GEMM interface and layout
 * constraints"); this kernel writes the required scale layout directly.
 * Errors: DG_ERR_NULL, DG_ERR_SHAPE (groups, rows < 1; K), DG_ERR_ALIGN
 * (ld_sf < rows or ld_sf % 4).
 */
int dg_quantize_e4m3_1x128(const float *x, int groups, int rows, int K,
                           uint8_t *q, float *sf, int ld_sf, void *stream);

/*
 * E4M3 quantiser, one scale per 128x128 block (the RHS layout):
 *   x [groups][rows][K] -> q, sf [groups][ceil(rows/128)][K/128].
 * The last row block of each group may be partial; blocks never straddle
 * groups.  Same scale formula and rounding as the 1x128 quantiser.
 */
int dg_quantize_e4m3_128x128(const float *x, int groups, int rows, int K,
                             uint8_t *q, float *sf, void *stream);

/*
 * Power-of-two (UE8M0) scale variants.  The DeepGEMM README summary
 * ("GEMM interface and layout constraints") describes packed UE8M0 scaling
 * factors for its SM100 kernels: every scale a power of two.
 *
 * Quantisers: as above, but the block scale is max(amax, 1e-4)/448 (one
 * IEEE fp32 division) rounded up to the next power of two, so |x/sf| <= 448
 * still holds and the division is exact.  Same layouts and errors.
 */
int dg_quantize_e4m3_1x128_ue8m0(const float *x, int groups, int rows, int K,
                                 uint8_t *q, float *sf, int ld_sf, void *stream);
int dg_quantize_e4m3_128x128_ue8m0(const float *x, int groups, int rows, int K,
                                   uint8_t *q, float *sf, void *stream);

/*
 * GEMMs on power-of-two scales: same arguments, layouts, results (to the
 * same tolerance) and errors as the three GEMMs above, but every entry of
 * sfa and sfb that scales a computed element must be a positive normal
 * power of two, as the *_ue8m0 quantisers write them.  gfx950's FP8 matrix
 * instruction then applies the scales itself, as exponents, and
 * accumulates across K blocks without a separate promotion step.  The
 * mantissa bits of a scale are not read: a scale that is not a power of
 * two gives a wrong result (nothing checks this on the device).
 */
int dg_fp8_gemm_nt_ue8m0(const uint8_t *a, const float *sfa, int ld_sfa,
                         const uint8_t *b, const float *sfb,
                         const uint16_t *c, uint16_t *d,
                         int M, int N, int K, void *stream);
int dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0(const uint8_t *a, const float *sfa,
                                              const uint8_t *b, const float *sfb,
                                              const uint16_t *c, uint16_t *d,
                                              const int32_t *m_indices,
                                              int M_total, int N, int K, int G,
                                              void *stream);
int dg_m_grouped_fp8_gemm_nt_masked_ue8m0(const uint8_t *a, const float *sfa,
                                          const uint8_t *b, const float *sfb,
                                          const uint16_t *c, uint16_t *d,
                                          const int32_t *masked_m,
                                          int G, int M_cap, int N, int K,
                                          int expected_m, void *stream);
/* The same for the other layouts and the K-grouped form (declared below),
 * with the same power-of-two requirement on every scale.  In the K-grouped
 * form each lane hands the matrix instruction the exponent of its own B
 * column, so the per-column scales cost no promotion either. */
int dg_fp8_gemm_nn_ue8m0(const uint8_t *a, const float *sfa, int ld_sfa,
                         const uint8_t *b, const float *sfb,
                         const uint16_t *c, uint16_t *d,
                         int M, int N, int K, void *stream);
int dg_fp8_gemm_tn_ue8m0(const uint8_t *a, const float *sfa, int ld_sfa,
                         const uint8_t *b, const float *sfb,
                         const uint16_t *c, uint16_t *d,
                         int M, int N, int K, void *stream);
int dg_fp8_gemm_tt_ue8m0(const uint8_t *a, const float *sfa, int ld_sfa,
                         const uint8_t *b, const float *sfb,
                         const uint16_t *c, uint16_t *d,
                         int M, int N, int K, void *stream);
int dg_k_grouped_fp8_gemm_tn_contiguous_ue8m0(const uint8_t *a, const float *sfa,
                                              const uint8_t *b, const float *sfb,
                                              const int32_t *ks, const float *c, float *d,
                                              int M, int N, int K, int G, void *stream);

/*
 * Packed UE8M0 scales.  The DeepGEMM README summary ("GEMM interface and
 * layout constraints") states that the SM100 kernels take their scaling
 * factors as UE8M0 exponents packed four to a 32-bit integer.  The pages do
 * not fix the packing order; here the four share one row (A) or 128-column
 * block (B) and four consecutive K blocks: with nkw = ceil(K/512), byte j
 * (bits 8j .. 8j+7) of word q holds the biased exponent of K block 4q + j
 * (the fp32 exponent field of the power-of-two scale 2^(e-127)); bytes past
 * the last K block are ignored.
 *
 *   sfa   uint32 [nkw][ld_sfa]           (dense; ld_sfa >= M, multiple of 4)
 *         uint32 [nkw][M_total]          (contiguous)
 *         uint32 [G][nkw][ceil4(M_cap)]  (masked)
 *   sfb   uint32 [ceil(N/128)][nkw]      (dense)
 *         uint32 [G][ceil(N/128)][nkw]   (grouped)
 *
 * Every other argument, the result (bit-identical to the matching *_ue8m0
 * entry point on the scales the words encode) and the errors are as for
 * dg_fp8_gemm_nt_ws, dg_m_grouped_fp8_gemm_nt_contiguous and
 * dg_m_grouped_fp8_gemm_nt_masked, plus DG_ERR_SHAPE when K times M (M_total,
 * M_cap) or K times N reaches 2^31.  The byte 0 (2^-127) is not a valid
 * scale, as a scale that is not a normal power of two is not for the
 * *_ue8m0 forms.
 */
int dg_fp8_gemm_nt_ue8m0_packed(const uint8_t *a, const uint32_t *sfa, int ld_sfa,
                                const uint8_t *b, const uint32_t *sfb,
                                const uint16_t *c, uint16_t *d,
                                int M, int N, int K,
                                void *workspace, size_t workspace_bytes, void *stream);
int dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0_packed(const uint8_t *a, const uint32_t *sfa,
                                                     const uint8_t *b, const uint32_t *sfb,
                                                     const uint16_t *c, uint16_t *d,
                                                     const int32_t *m_indices,
                                                     int M_total, int N, int K, int G,
                                                     void *stream);
int dg_m_grouped_fp8_gemm_nt_masked_ue8m0_packed(const uint8_t *a, const uint32_t *sfa,
                                                 const uint8_t *b, const uint32_t *sfb,
                                                 const uint16_t *c, uint16_t *d,
                                                 const int32_t *masked_m,
                                                 int G, int M_cap, int N, int K,
                                                 int expected_m, void *stream);

/*
 * Packs power-of-two fp32 scales into the words above (the pages' library
 * offers a scale layout transform, transform_sf_into_required_layout, among
 * its utilities: "Utilities and environment variables").  sf is viewed as
 * fp32 [outer][kblocks][inner], out as uint32 [outer][ceil(kblocks/4)][inner];
 * byte j of out[o][q][i] = bits 23..30 of sf[o][4q+j][i], 0 where 4q+j >=
 * kblocks.  For sfa: outer = groups (1 when dense), kblocks = K/128, inner =
 * the scale leading dimension; for sfb: outer = G * ceil(N/128), kblocks =
 * K/128, inner = 1.  sf and out device memory, 4-byte aligned, not
 * overlapping; enqueued on `stream`.
 * Errors: DG_ERR_NULL (sf, out), DG_ERR_SHAPE (outer, kblocks, inner < 1;
 * more than 2^31 workgroups), DG_ERR_ALIGN, DG_ERR_HIP.
 */
int dg_pack_sf_ue8m0(const float *sf, int outer, int kblocks, int inner,
                     uint32_t *out, void *stream);

/*
 * FP8 MQA logits, non-paged (the DeepSeek v3.2 indexer's scoring kernel;
 * GeekNews summary of the DeepGEMM README, section on the MQA kernels for the
 * v3.2 Indexer).  For every query token i and key token j in
 * [k_start[i], k_end[i]) (both clamped to [0, S_kv]; empty when end <= start):
 *   logits[i][j] = sum_h weights[i][h] * ReLU(kv_scale[j] * (q[i,h,:] . kv[j,:]))
 *   q         [S][H][D]  E4M3
 *   kv        [S_kv][D]  E4M3
 *   kv_scale  [S_kv]     fp32, positive and finite (the kernel applies it
 *                        after the ReLU and the head sum, which equals the
 *                        formula only for positive scales; not checked)
 *   weights   [S][H]     fp32
 *   k_start, k_end [S]   int32
 *   logits    [S][S_kv]  fp32 (row i at logits + i*S_kv).  Positions of row
 *                        i outside its range are set to -inf when
 *                        clean_logits != 0 and left untouched otherwise.
 * Accuracy: the FP8 matrix instruction sums each group of 8 consecutive
 * head-dim products in a window 13 bits below the group's leading bit
 * (truncating) and the group sums in fp32; the weighted head sum is fp32.  A
 * logit is within 2^-10 * kv_scale[j] * sum_h |weights[i][h]| *
 * sum_d |q[i,h,d] kv[j,d]| of the exact value.
 * Supported: D == 128, H in {16, 32, 48, 64}, S_kv * D < 2^31.
 * Errors: DG_ERR_NULL (any pointer), DG_ERR_SHAPE (S, S_kv < 1; D, H
 * unsupported; S_kv too large), DG_ERR_ALIGN (q, kv, weights not 16-B
 * aligned; kv_scale, k_start, k_end, logits not 4-B aligned).  Rows are
 * written with 16-byte stores when S_kv % 4 == 0 and logits is 16-B aligned,
 * with 4-byte stores otherwise.
 */
int dg_fp8_mqa_logits(const uint8_t *q, const uint8_t *kv, const float *kv_scale,
                      const float *weights, const int32_t *k_start, const int32_t *k_end,
                      int clean_logits, float *logits,
                      int S, int H, int D, int S_kv, void *stream);

/*
 * K-grouped FP8 GEMM, TN contiguous layout (the MoE weight-gradient form;
 * "DeepGEMM" README summary, section "Dense and Grouped GEMM": groups along
 * K, M and N fixed, k_grouped_fp8_gemm_tn_contiguous).  The K rows of G
 * groups are concatenated; group g owns rows [k0_g, k0_g + ks[g]) with
 * k0_g = ks[0] + .. + ks[g-1], and for every group (an empty one included)
 *   D[g][m][n] = C[g][m][n] + sum_{kb in g} sfa[kb][m] * sfb[kb][n] * sum_{k in kb} A[k][m] B[k][n]
 *   a   [K][M]        E4M3 (stored K-major in rows: A^T of the usual layout)
 *   sfa [K/128][M]    fp32, one scale per 128 K rows and column m
 *   b   [K][N]        E4M3
 *   sfb [K/128][N]    fp32, one scale per 128 K rows and column n (both
 *                     operands are activations or gradients, quantised
 *                     1x128 along K)
 *   ks  [G]           int32 group sizes in K rows, in DEVICE memory: each a
 *                     multiple of 128, sum <= K.  Not checked on the host; a
 *                     negative size counts as 0 and ranges are clamped to
 *                     K, so a bad size gives wrong groups but no access
 *                     outside the operands.
 *   c   [G][M][N]     fp32 or NULL (= 0); may alias d exactly
 *   d   [G][M][N]     fp32, written entirely.
 * Accumulation as in dg_fp8_gemm_nt (fp32, one promotion per 128-row K
 * block), so D meets the GEMMs' bar without their final bf16 rounding:
 * |D - D_ref| <= 2^-20 |D_ref| + 1e-4 max|D_ref|, where many products of like
 * size make a result.  The FP8 instruction keeps 13 bits below the largest of
 * eight consecutive products, which is up to 2^-12 of the sum of the products'
 * magnitudes: with one or two K blocks and operands of a few large values
 * (gradients) that alone may pass 1e-4 max|D_ref|.  Needs M and N multiples of
 * 16, K*M and K*N below 2^31.
 * Errors: DG_ERR_NULL (a, sfa, b, sfb, ks, d), DG_ERR_SHAPE (M, N, G < 1;
 * K < 128 or K % 128; K*M or K*N too large), DG_ERR_ALIGN (M or N not a
 * multiple of 16; a, sfa, b, sfb, c, d not 16-B aligned; ks not 4-B aligned).
 */
int dg_k_grouped_fp8_gemm_tn_contiguous(const uint8_t *a, const float *sfa,
                                        const uint8_t *b, const float *sfb,
                                        const int32_t *ks, const float *c, float *d,
                                        int M, int N, int K, int G, void *stream);

/* ------------------------------------------------------------------------
 * The feed-forward layer around the GEMMs: the norm that makes the first
 * GEMM's operand, the gated projections that make the second's, and the
 * gradients of both.  Conventions as above, except that
 *  - a call with no rows (rows, M or M_total = 0) is valid: it writes nothing
 *    (dg_rmsnorm_backward: dw = 0) and returns DG_OK; pointers may be NULL then;
 *  - outputs marked optional may be NULL and are then not computed;
 *  - tensors whose element type varies are void pointers with a dg_type.
 * Statistics, activations and maxima are computed in fp32; every output is
 * rounded once, from fp32.  NaN and infinities follow the formulas in fp32;
 * in the quantised outputs they are treated as by the quantisers above.
 * ------------------------------------------------------------------------ */
typedef enum dg_type { DG_BF16 = 0, DG_F32 = 1 } dg_type;
typedef enum dg_act {
    DG_ACT_SILU = 0,      /* g / (1 + exp(-g)) */
    DG_ACT_GELU_TANH = 1  /* 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */
} dg_act;

/*
 * Residual addition, RMS norm and 1x128 E4M3 quantisation in one pass:
 *   h = x + residual;  y = h / sqrt(mean_k(h^2) + eps) * weight
 *   q, sf = the 1x128 quantiser's output on y (before any rounding of y)
 *   x [rows][ld_x >= K]        DG_BF16 or DG_F32; the row pitch lets the norm
 *                              read a column range of a wider matrix
 *   residual [rows][K]         or NULL (= 0); its type is also residual_out's
 *   weight [K]                 DG_BF16 or DG_F32
 *   residual_out [rows][K]     optional: h, rounded to its type; may be the
 *                              residual itself (in place).  The norm uses h
 *                              before that rounding.
 *   y [rows][K] bf16           optional
 *   q [rows][K] E4M3, sf       optional (q and sf together; y or q is needed)
 * The scales are those of dg_quantize_e4m3_1x128 (sf [K/128][ld_sf] fp32), of
 * its _ue8m0 form, or (_ue8m0_packed) the packed words of the latter,
 * sf [ceil(K/512)][ld_sf] with the unused high bytes zero; entries of rows
 * past the last are not written.
 * Sums of squares overflow fp32 for |h| above about 1e19: mean(h^2) is then
 * infinite and y zero.
 * Errors: DG_ERR_NULL; DG_ERR_SHAPE (rows < 0; K < 128, K % 128, K > 16384);
 * DG_ERR_ARG (a type; eps negative or NaN; residual_out without residual);
 * DG_ERR_ALIGN (a pointer not 16-byte aligned; ld_x < K or its rows not
 * 16-byte aligned; ld_sf < rows or ld_sf % 4).
 */
int dg_rmsnorm_quantize_e4m3_1x128(const void *x, int x_type, int64_t ld_x,
                                   const void *residual, int residual_type,
                                   const void *weight, int weight_type, float eps,
                                   void *residual_out, uint16_t *y,
                                   uint8_t *q, float *sf, int ld_sf,
                                   int rows, int K, void *stream);
int dg_rmsnorm_quantize_e4m3_1x128_ue8m0(const void *x, int x_type, int64_t ld_x,
                                         const void *residual, int residual_type,
                                         const void *weight, int weight_type, float eps,
                                         void *residual_out, uint16_t *y,
                                         uint8_t *q, float *sf, int ld_sf,
                                         int rows, int K, void *stream);
int dg_rmsnorm_quantize_e4m3_1x128_ue8m0_packed(const void *x, int x_type, int64_t ld_x,
                                                const void *residual, int residual_type,
                                                const void *weight, int weight_type, float eps,
                                                void *residual_out, uint16_t *y,
                                                uint8_t *q, uint32_t *sf, int ld_sf,
                                                int rows, int K, void *stream);

/*
 * Gradient of the norm, from its input h as stored (residual_out, or x where
 * there is no residual); the quantisation is taken as the identity.
 *   r = 1 / sqrt(mean_k(h^2) + eps),  g = dy * weight
 *   dx = dres + r * (g - h * r^2 * mean_k(g * h))   [rows][K], h's type
 *   dw = sum over rows of dy * h * r                [K] fp32
 *   dy [rows][K]; h, dres (or NULL = 0), dx [rows][K] of one type; dx may be
 *   dres or h (in place).  dx is the gradient of x and of the residual alike.
 * dw is added up in a fixed order: the same bits on every run.
 *   workspace: dg_get_rmsnorm_backward_workspace_size(rows, K) bytes of device
 *   memory, 16-byte aligned (NULL when that is 0), of any content.
 * Errors as above, and DG_ERR_ARG for a workspace that is too small.
 */
int dg_rmsnorm_backward(const void *dy, int dy_type, const void *h, int h_type,
                        const void *weight, int weight_type, float eps,
                        const void *dres, void *dx, float *dw, int rows, int K,
                        void *workspace, size_t workspace_bytes, void *stream);
int64_t dg_get_rmsnorm_backward_workspace_size(int rows, int K);

/*
 * Gated projections: both GEMMs, the activation and the product in one kernel.
 *   gate = A . Wg^T,  up = A . Wu^T  (block-scaled as in dg_fp8_gemm_nt)
 *   h = act(gate) * up
 *   a [M][K], sfa [K/128][ld_sfa]  as for dg_fp8_gemm_nt
 *   b [2][I][K] E4M3               Wg, then Wu
 *   sfb [2][ceil(I/128)][K/128]    (what dg_quantize_e4m3_128x128 writes for
 *                                  two groups of I rows)
 *   gu [M][2][I] bf16              optional: gate and up, for the backward pass
 *   h [M][I] bf16                  optional
 *   q [M][I] E4M3, sf [I/128][ld_sf] fp32   optional: h through the 1x128
 *                                  quantiser (before any rounding), the A
 *                                  operand of the next GEMM; needs I % 128 == 0
 * h or q is needed; act is a dg_act.
 * The _ue8m0_packed form takes packed power-of-two scales (sfa
 * [ceil(K/512)][ld_sfa], sfb [2][ceil(I/128)][ceil(K/512)]) and writes such
 * scales (sf [ceil(I/512)][ld_sf]), as dg_fp8_gemm_nt_ue8m0_packed takes them.
 *   workspace: dg_get_gated_workspace_size(M, I, K) bytes of device memory,
 *   16-byte aligned, of any content, for a q output of problems too small to
 *   fill the CUs with 128-column tiles (0 bytes elsewhere); calls that may run
 *   at the same time need one each.  With NULL,
 *   or too few bytes, a kernel that needs none (and is slower there) computes
 *   the same outputs.
 * Errors: DG_ERR_NULL; DG_ERR_SHAPE (M < 0; I < 1; K < 128 or K % 128; q with
 * I % 128; 2*I*K, 256*K or the bytes of sfa reaching 2^31); DG_ERR_ARG (act);
 * DG_ERR_ALIGN.
 */
int dg_fp8_gated_gemm_nt(const uint8_t *a, const float *sfa, int ld_sfa,
                         const uint8_t *b, const float *sfb, int act,
                         uint16_t *gu, uint16_t *h, uint8_t *q, float *sf, int ld_sf,
                         int M, int I, int K,
                         void *workspace, size_t workspace_bytes, void *stream);
int dg_fp8_gated_gemm_nt_ue8m0_packed(const uint8_t *a, const uint32_t *sfa, int ld_sfa,
                                      const uint8_t *b, const uint32_t *sfb, int act,
                                      uint16_t *gu, uint16_t *h, uint8_t *q, uint32_t *sf, int ld_sf,
                                      int M, int I, int K,
                                      void *workspace, size_t workspace_bytes, void *stream);
int64_t dg_get_gated_workspace_size(int M, int I, int K);

/*
 * Its M-grouped forms, with the row layouts of the plain M-grouped GEMMs: b
 * [G][2][I][K], sfb [G][2][ceil(I/128)][K/128].
 * Contiguous: a, gu, h, q of M_total rows (a multiple of 128), sfa
 * [K/128][M_total], sf [I/128][M_total], m_indices [M_total] (16-byte aligned);
 * the experts' 128-row blocks may come in any order.
 * Masked: a [G][M_cap][K], sfa [G][K/128][round_up(M_cap,4)], outputs
 * [G][M_cap][..], sf [G][I/128][round_up(M_cap,4)], masked_m [G] on the device.
 * Rows that hold no data are not written, in any output, sf included.
 */
int dg_m_grouped_fp8_gated_gemm_nt_contiguous(const uint8_t *a, const float *sfa,
                                              const uint8_t *b, const float *sfb, int act,
                                              uint16_t *gu, uint16_t *h, uint8_t *q, float *sf,
                                              const int32_t *m_indices,
                                              int M_total, int I, int K, int G, void *stream);
int dg_m_grouped_fp8_gated_gemm_nt_contiguous_ue8m0_packed(const uint8_t *a, const uint32_t *sfa,
                                                           const uint8_t *b, const uint32_t *sfb, int act,
                                                           uint16_t *gu, uint16_t *h, uint8_t *q, uint32_t *sf,
                                                           const int32_t *m_indices,
                                                           int M_total, int I, int K, int G, void *stream);
int dg_m_grouped_fp8_gated_gemm_nt_masked(const uint8_t *a, const float *sfa,
                                          const uint8_t *b, const float *sfb, int act,
                                          uint16_t *gu, uint16_t *h, uint8_t *q, float *sf,
                                          const int32_t *masked_m,
                                          int G, int M_cap, int I, int K, int expected_m, void *stream);
int dg_m_grouped_fp8_gated_gemm_nt_masked_ue8m0_packed(const uint8_t *a, const uint32_t *sfa,
                                                       const uint8_t *b, const uint32_t *sfb, int act,
                                                       uint16_t *gu, uint16_t *h, uint8_t *q, uint32_t *sf,
                                                       const int32_t *masked_m,
                                                       int G, int M_cap, int I, int K, int expected_m,
                                                       void *stream);

/*
 * Gradient of h = act(gate) * up, quantised for the gradient GEMMs that follow:
 *   d_gate = dh * up * act'(gate),  d_up = dh * act(gate)
 *   gu [rows][2][I] bf16 (as saved by the gated GEMM), dh [rows][I] bf16
 *   m_indices [rows] int32 or NULL: rows with a negative index count as zeros
 *       in every output (whatever gu and dh hold there), so the padding of the
 *       contiguous layout adds nothing to a weight gradient
 * Outputs, each optional, at least one:
 *   dgu [rows][2][I] bf16                        d_gate, d_up
 *   q [rows][2I] E4M3, sf [2I/128][ld_sf]        1x128 scales along 2I: the A
 *       operand of the input gradient, d_x = [d_gate d_up] . [Wg; Wu]
 *   qt [rows up to a multiple of 128][2I] E4M3, sft [ceil(rows/128)][2I]   one
 *       scale per column and 128 rows: the A operand, stored [K][M], of
 *       dg_fp8_gemm_tn and dg_k_grouped_fp8_gemm_tn_contiguous for the weight
 *       gradient of [Wg; Wu]; rows past the last are written as zeros
 *   ht [.. as qt ..][I] E4M3, sfht [ceil(rows/128)][I]   the same of h =
 *       act(gate) * up, for the weight gradient of the projection that follows
 * The _ue8m0 form rounds every scale up to a power of two.
 * Errors: DG_ERR_NULL; DG_ERR_SHAPE (rows < 0; I < 128, I % 128, or 512*I
 * reaching 2^31); DG_ERR_ARG (act); DG_ERR_ALIGN (m_indices: 4 bytes, the
 * others 16; ld_sf < rows or ld_sf % 4).
 */
int dg_gated_backward_quantize_e4m3(const uint16_t *gu, const uint16_t *dh, int act, const int32_t *m_indices,
                                    uint16_t *dgu, uint8_t *q, float *sf, int ld_sf,
                                    uint8_t *qt, float *sft, uint8_t *ht, float *sfht,
                                    int rows, int I, void *stream);
int dg_gated_backward_quantize_e4m3_ue8m0(const uint16_t *gu, const uint16_t *dh, int act, const int32_t *m_indices,
                                          uint16_t *dgu, uint8_t *q, float *sf, int ld_sf,
                                          uint8_t *qt, float *sft, uint8_t *ht, float *sfht,
                                          int rows, int I, void *stream);

/*
 * Layer norm: the RMS norm's calls with the mean taken out and a bias,
 *   h = x + residual;  m = mean_k(h);  v = mean_k((h - m)^2)
 *   y = (h - m) / sqrt(v + eps) * weight + bias
 *   q, sf = the 1x128 quantiser's output on y (before any rounding of y)
 * Arguments as for dg_rmsnorm_quantize_e4m3_1x128, and
 *   weight, bias [K]   each optional (NULL: ones, zeros), of one type
 *   K                  a multiple of 128 where q is asked for, of 8 otherwise;
 *                      8 to 16384
 * The mean is subtracted before the squares are summed, so a mean that is large
 * beside the spread costs no more bits than h itself holds.  Sums of squares
 * overflow fp32 for differences above about 1e19: v is then infinite and y the
 * bias.  A row with an infinity or NaN in it is NaN throughout (codes 0x7f); so
 * is a row whose sum passes fp32, and with eps = 0 a row of equal values.
 * Errors as there.
 */
int dg_layernorm_quantize_e4m3_1x128(const void *x, int x_type, int64_t ld_x,
                                     const void *residual, int residual_type,
                                     const void *weight, const void *bias, int weight_type, float eps,
                                     void *residual_out, uint16_t *y,
                                     uint8_t *q, float *sf, int ld_sf,
                                     int rows, int K, void *stream);
int dg_layernorm_quantize_e4m3_1x128_ue8m0(const void *x, int x_type, int64_t ld_x,
                                           const void *residual, int residual_type,
                                           const void *weight, const void *bias, int weight_type, float eps,
                                           void *residual_out, uint16_t *y,
                                           uint8_t *q, float *sf, int ld_sf,
                                           int rows, int K, void *stream);
int dg_layernorm_quantize_e4m3_1x128_ue8m0_packed(const void *x, int x_type, int64_t ld_x,
                                                  const void *residual, int residual_type,
                                                  const void *weight, const void *bias, int weight_type, float eps,
                                                  void *residual_out, uint16_t *y,
                                                  uint8_t *q, uint32_t *sf, int ld_sf,
                                                  int rows, int K, void *stream);

/*
 * Gradient of the layer norm, from its input h as stored (residual_out, or x
 * where there is no residual); the quantisation is taken as the identity.
 *   r = 1 / sqrt(v + eps),  n = (h - m) * r,  g = dy * weight
 *   dx = dres + r * (g - mean_k(g) - n * mean_k(g * n))   [rows][K], h's type
 *                     (r^2 is formed: v + eps above 2.9e-39)
 *   dw = sum over rows of dy * n,  db = sum over rows of dy   [K] fp32, each optional
 * weight, dres optional; the rest as for dg_rmsnorm_backward, K a multiple of 8.
 *   workspace: dg_get_layernorm_backward_workspace_size(rows, K) bytes of
 *   device memory, 16-byte aligned (NULL when that is 0, or neither dw nor db
 *   is asked for), of any content; calls that may run at the same time (other
 *   streams, graphs replayed concurrently) need one each.
 */
int dg_layernorm_backward(const void *dy, int dy_type, const void *h, int h_type,
                          const void *weight, int weight_type, float eps,
                          const void *dres, void *dx, float *dw, float *db, int rows, int K,
                          void *workspace, size_t workspace_bytes, void *stream);
int64_t dg_get_layernorm_backward_workspace_size(int rows, int K);

/* ------------------------------------------------------------------------
 * Tokens to the experts' rows and back.  T tokens choose top_k of G experts
 * each; pair t * top_k + j is token t's choice j.  A pair whose id lies outside
 * [0, G) (an expert that lives elsewhere, a token that was dropped) has no row:
 * its entry of `rows` is -1, it is neither dispatched nor combined, and its
 * weight's gradient is 0.  Index arrays are int32, 4-byte aligned; weights are
 * fp32, 4-byte aligned.  Every result is computed in a fixed order: the same
 * bits on every run.
 * ------------------------------------------------------------------------ */

/*
 * The sort: a row for every pair, in pair order within an expert.
 *   ids  [T][top_k]   in device memory; an expert may occur twice in a token
 *   rows [T][top_k]   the pair's row, -1 where it has none
 * Contiguous: expert e's segment starts at the sum of the sizes before it, each
 * rounded up to 128 rows.
 *   m_indices [M_total]   optional, 16-byte aligned: the expert of each row, -1
 *                         on rows that hold no pair
 *   src       [M_total]   optional: the pair of each row, -1 likewise
 *   counts    [G]         optional: rows that hold a pair
 *   ks        [G]         optional: rows of the segment (a multiple of 128): the
 *                         group sizes of the K-grouped GEMM
 *   M_total   a multiple of 128.  dg_get_moe_rows(T, top_k, G) rows hold the
 *             pairs however they fall; with fewer, pairs whose row would lie at
 *             or past M_total have none.
 * Masked: expert e's rows are e * M_cap onwards; pairs past M_cap have no row.
 *   masked_m [G]          rows that hold a pair
 *   src      [G][M_cap]   optional
 *   workspace: dg_get_moe_sort_workspace_size(T, top_k, G) bytes of device
 *   memory, 16-byte aligned, of any content; with NULL or too few bytes the
 *   same results take longer where that is not 0.  Calls that may run at the
 *   same time need one each.
 * A call with T = 0 writes the plan of no pairs.
 * Errors: DG_ERR_NULL (ids, rows with T > 0; masked_m); DG_ERR_SHAPE (T < 0,
 * top_k < 1, T * top_k > 2^26, G < 1 or > 1024, M_total < 0 or % 128, M_cap < 1;
 * the rows reaching 2^31); DG_ERR_ALIGN.
 */
int dg_moe_sort_contiguous(const int32_t *ids, int T, int top_k, int G,
                           int32_t *rows, int32_t *src, int32_t *m_indices, int32_t *counts, int32_t *ks,
                           int M_total, void *workspace, size_t workspace_bytes, void *stream);
int dg_moe_sort_masked(const int32_t *ids, int T, int top_k, int G,
                       int32_t *rows, int32_t *src, int32_t *masked_m,
                       int M_cap, void *workspace, size_t workspace_bytes, void *stream);
int64_t dg_get_moe_rows(int T, int top_k, int G);
int64_t dg_get_moe_sort_workspace_size(int T, int top_k, int G);

/*
 * Dispatch: v = weights[t, j] * x[t] (weights NULL: x[t]) for every pair, in the
 * row rows[t, j].
 *   x [T][ld_x >= K]       DG_BF16 or DG_F32, rows 16-byte aligned
 *   weights [T][top_k]     fp32 or NULL
 *   rows [T][top_k]        from the sort: each row at most once (not checked;
 *                          a row outside the layout counts as -1)
 * Outputs, each optional, at least one; rows that hold no pair are not written,
 * in y, q and sf:
 *   y [..][K] bf16
 *   q [..][K] E4M3, sf     v through the 1x128 quantiser (the _ue8m0 forms: its
 *                          _ue8m0 form, packed words), in the A operand's layout
 *                          of the M-grouped GEMMs:
 *       contiguous: q [M_total][K], sf [K/128][M_total] (packed: [ceil(K/512)])
 *       masked: q [G][M_cap][K], sf [G][K/128][round_up(M_cap,4)]
 *   contiguous only, written entirely, zeros on rows that hold no pair:
 *   qt [M_total][K] E4M3, sft [M_total/128][K] fp32   one scale per column and
 *       128 rows (power-of-two scales in the _ue8m0 forms): an operand of
 *       dg_k_grouped_fp8_gemm_tn_contiguous (for the weight gradient); needs src
 *       (the sort's, of the same rows)
 * Errors: DG_ERR_NULL; DG_ERR_SHAPE (T < 0; top_k, G, M_cap < 1; M_total < 0 or
 * % 128; K < 128, K % 128, K > 16384; top_k > 2^30; T * top_k or the rows
 * reaching 2^31); DG_ERR_ARG (x_type); DG_ERR_ALIGN.
 */
int dg_moe_dispatch_quantize_e4m3_contiguous(const void *x, int x_type, int64_t ld_x, const float *weights,
                                             const int32_t *rows, const int32_t *src,
                                             uint16_t *y, uint8_t *q, float *sf, uint8_t *qt, float *sft,
                                             int T, int top_k, int K, int M_total, void *stream);
int dg_moe_dispatch_quantize_e4m3_contiguous_ue8m0(const void *x, int x_type, int64_t ld_x, const float *weights,
                                                   const int32_t *rows, const int32_t *src,
                                                   uint16_t *y, uint8_t *q, float *sf, uint8_t *qt, float *sft,
                                                   int T, int top_k, int K, int M_total, void *stream);
int dg_moe_dispatch_quantize_e4m3_contiguous_ue8m0_packed(const void *x, int x_type, int64_t ld_x,
                                                          const float *weights,
                                                          const int32_t *rows, const int32_t *src,
                                                          uint16_t *y, uint8_t *q, uint32_t *sf,
                                                          uint8_t *qt, float *sft,
                                                          int T, int top_k, int K, int M_total, void *stream);
int dg_moe_dispatch_quantize_e4m3_masked(const void *x, int x_type, int64_t ld_x, const float *weights,
                                         const int32_t *rows, uint16_t *y, uint8_t *q, float *sf,
                                         int T, int top_k, int K, int G, int M_cap, void *stream);
int dg_moe_dispatch_quantize_e4m3_masked_ue8m0(const void *x, int x_type, int64_t ld_x, const float *weights,
                                               const int32_t *rows, uint16_t *y, uint8_t *q, float *sf,
                                               int T, int top_k, int K, int G, int M_cap, void *stream);
int dg_moe_dispatch_quantize_e4m3_masked_ue8m0_packed(const void *x, int x_type, int64_t ld_x, const float *weights,
                                                      const int32_t *rows, uint16_t *y, uint8_t *q, uint32_t *sf,
                                                      int T, int top_k, int K, int G, int M_cap, void *stream);

/*
 * Dispatch of codes that are quantised already (a norm's, or another rank's):
 * codes and scales are copied as they are.
 *   q_in [T][K] E4M3;  sf_in [K/128][ld_in] fp32, or packed words [ceil(K/512)][ld_in]
 *   (ld_in >= T, a multiple of 4); q, sf as above, sf in sf_in's format.
 * Errors as above (K of any multiple of 128).
 */
int dg_moe_dispatch_e4m3_contiguous(const uint8_t *q_in, const float *sf_in, int ld_in, const int32_t *rows,
                                    uint8_t *q, float *sf, int T, int top_k, int K, int M_total, void *stream);
int dg_moe_dispatch_e4m3_contiguous_ue8m0_packed(const uint8_t *q_in, const uint32_t *sf_in, int ld_in,
                                                 const int32_t *rows, uint8_t *q, uint32_t *sf,
                                                 int T, int top_k, int K, int M_total, void *stream);
int dg_moe_dispatch_e4m3_masked(const uint8_t *q_in, const float *sf_in, int ld_in, const int32_t *rows,
                                uint8_t *q, float *sf, int T, int top_k, int K, int G, int M_cap, void *stream);
int dg_moe_dispatch_e4m3_masked_ue8m0_packed(const uint8_t *q_in, const uint32_t *sf_in, int ld_in,
                                             const int32_t *rows, uint8_t *q, uint32_t *sf,
                                             int T, int top_k, int K, int G, int M_cap, void *stream);

/*
 * Combine: the experts' rows back to their tokens,
 *   out[t] = residual[t] + sum_j weights[t, j] * y[rows[t, j]]
 * summed in fp32 in the order of the choices and rounded once.
 *   y [R][K] bf16          the experts' outputs (R = M_total, or G * M_cap)
 *   weights [T][top_k]     fp32 or NULL (ones: the gradient of dispatch without
 *                          weights)
 *   residual, out [T][K]   out_type DG_BF16 or DG_F32; residual NULL = 0, and
 *                          may be out (in place)
 * Errors: DG_ERR_NULL; DG_ERR_SHAPE (T, R < 0; top_k < 1 or > 2^30; K < 8 or
 * K % 8; T * top_k reaching 2^31); DG_ERR_ARG (out_type); DG_ERR_ALIGN.
 */
int dg_moe_combine(const uint16_t *y, const float *weights, const int32_t *rows, const void *residual,
                   void *out, int out_type, int T, int top_k, int K, int R, void *stream);

/*
 * Gradient of combine (contiguous layout):
 *   dw[t, j] = sum_k dout[t, k] * y[rows[t, j], k]         [T][top_k] fp32, optional
 *   dy[rows[t, j]] = weights[t, j] * dout[t]               a dispatch of dout: its
 *                                                          outputs dy, q, sf, qt, sft
 * dout [T][ld_dout >= K] DG_BF16 or DG_F32; y [M_total][K] bf16 (needed for dw);
 * the gradient of residual is dout.  Arguments, forms and errors as for
 * dg_moe_dispatch_quantize_e4m3_contiguous; at least one output.
 */
int dg_moe_combine_backward_quantize_e4m3_contiguous(const void *dout, int dout_type, int64_t ld_dout,
                                                     const uint16_t *y, const float *weights,
                                                     const int32_t *rows, const int32_t *src,
                                                     float *dw, uint16_t *dy, uint8_t *q, float *sf,
                                                     uint8_t *qt, float *sft,
                                                     int T, int top_k, int K, int M_total, void *stream);
int dg_moe_combine_backward_quantize_e4m3_contiguous_ue8m0(const void *dout, int dout_type, int64_t ld_dout,
                                                           const uint16_t *y, const float *weights,
                                                           const int32_t *rows, const int32_t *src,
                                                           float *dw, uint16_t *dy, uint8_t *q, float *sf,
                                                           uint8_t *qt, float *sft,
                                                           int T, int top_k, int K, int M_total, void *stream);
int dg_moe_combine_backward_quantize_e4m3_contiguous_ue8m0_packed(const void *dout, int dout_type, int64_t ld_dout,
                                                                  const uint16_t *y, const float *weights,
                                                                  const int32_t *rows, const int32_t *src,
                                                                  float *dw, uint16_t *dy, uint8_t *q, uint32_t *sf,
                                                                  uint8_t *qt, float *sft,
                                                                  int T, int top_k, int K, int M_total,
                                                                  void *stream);

/* Row alignment of expert segments in the contiguous layout (128): the
 * set_/get_mk_alignment_for_contiguous_layout utilities of the "DeepGEMM"
 * README summary, section "Utilities and environment variables".  The
 * setter accepts only 128 and returns DG_ERR_ARG otherwise. */
int dg_get_mk_alignment_for_contiguous_layout(void);
int dg_set_mk_alignment_for_contiguous_layout(int alignment);

/* Leading dimension for a transposed scale array over mn rows: round_up(mn, 4)
 * (16-byte aligned columns).  The analogue of get_tma_aligned_size in the
 * same section (the LHS scales must be stored transposed and aligned,
 * section "GEMM interface and layout constraints"). */
int dg_get_sf_aligned_size(int mn);

/* Cap on the number of compute units the tile scheduler plans for: the
 * analogue of set_num_sms / get_num_sms in the same section.  n >= 1 sets
 * the cap, n == 0 restores the device's CU count; negative -> DG_ERR_ARG.
 * get returns the cap in force (the device's CU count when none is set, or
 * a negative dg_status when no device can be queried).  Process-wide. */
int dg_set_num_cus(int n);
int dg_get_num_cus(void);

/* Kernel family used by the GEMM entry points called from this thread, for
 * tuning and testing: "auto" (the default: chosen per problem), "pipe",
 * "persist", "skinny", "stream" or "tiled".  Not on the pages (whose JIT picks one
 * kernel per shape, "Utilities and environment variables"); here every
 * family stays reachable so each can be tested.  A family that cannot take a
 * problem falls back to the automatic choice; results agree to the
 * documented tolerance whichever family runs, but are not bit-identical
 * across families.  Every thread starts from the environment variable
 * DG_KERNEL_FAMILY.  set returns DG_ERR_NULL or DG_ERR_ARG for a NULL or
 * unknown name; get returns the calling thread's setting. */
int dg_set_kernel_family(const char *name);
const char *dg_get_kernel_family(void);

/* Static string for a status code.  The pages' Python interface raises
 * exceptions; a C ABI returns codes instead, and this names them. */
const char *dg_status_string(int status);

/* Description of the kernel configuration chosen by this thread's last GEMM
 * call (family, tile, grid, split).  Also printed to stderr for every call
 * when the environment variable DG_PRINT_CONFIGS is set to a non-zero value:
 * the DG_PRINT_CONFIGS variable of the same section, which prints the config
 * chosen for each shape. */
const char *dg_last_config(void);

#ifdef __cplusplus
}
#endif
#endif /* DG_H */
