// dg_layer.h -- host-side declarations of the feed-forward layer's kernels:
// the norms, the gated GEMM, the tokens' way to the experts' rows and back, and
// their gradients.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <stddef.h>

#include <string>

#include "dg_internal.h"

namespace dg {

// Element types and scale formats as the C ABI numbers them.
constexpr int kBf16 = 0, kF32 = 1;
constexpr int kSfFp32 = 0, kSfUe8m0 = 1, kSfPacked = 2;

// The calling thread's device, checked to be gfx950, and its CU count under
// the CU cap; a dg_status.
int current_device_cus(int &cus);
// Records what dg_last_config returns.
void set_last_config(const std::string &config);

struct RmsNormProblem {
    const void *x, *residual, *weight;
    void *residual_out;
    uint16_t *y;
    uint8_t *q;
    void *sf;
    int64_t ld_x;
    int rows, K, ld_sf;
    float eps;
    int x_type, res_type, w_type, format;
};
// Needs rows >= 1, K a multiple of 128 up to kNormMaxK.
constexpr int kNormMaxK = 16384;
hipError_t launch_rmsnorm_quant(const RmsNormProblem &p, hipStream_t stream);

struct RmsNormBwdProblem {
    const void *dy, *h, *weight, *dres;
    void *dx;
    float *dw;
    void *ws;
    int rows, K;
    float eps;
    int h_type, dy_type, w_type;
};
size_t rmsnorm_bwd_workspace(int rows, int K, int num_cus);
hipError_t launch_rmsnorm_bwd(const RmsNormBwdProblem &p, int num_cus, hipStream_t stream);

struct LayerNormProblem {
    const void *x, *residual, *weight, *bias;
    void *residual_out;
    uint16_t *y;
    uint8_t *q;
    void *sf;
    int64_t ld_x;
    int rows, K, ld_sf;
    float eps;
    int x_type, res_type, w_type, format;
};
// Needs rows >= 1, K a multiple of 8 (with q: of 128) up to kNormMaxK.
hipError_t launch_layernorm_quant(const LayerNormProblem &p, hipStream_t stream);

struct LayerNormBwdProblem {
    const void *dy, *h, *weight, *dres;
    void *dx;
    float *dw, *db;
    void *ws;
    int rows, K;
    float eps;
    int h_type, dy_type, w_type;
};
size_t layernorm_bwd_workspace(int rows, int K, int num_cus);
hipError_t launch_layernorm_bwd(const LayerNormBwdProblem &p, int num_cus, hipStream_t stream);

// Rows of the n pairs ids[0 .. n) sorted by expert: R rows in segments of whole
// 128-row blocks (cap = 0) or of cap rows.  counts: pairs that have a row,
// ks: padded sizes.
constexpr int kMoeMaxExperts = 1024;
constexpr int64_t kMoeMaxPairs = (int64_t)1 << 26;   // of a sort
struct MoeSortProblem {
    const int32_t *ids;
    int32_t *rows, *src, *expert, *counts, *ks;
    void *ws;
    size_t ws_bytes;
    int n, G, cap, R;
};
// Needs 1 <= G <= kMoeMaxExperts, n <= kMoeMaxPairs, R below 2^31.
size_t moe_sort_workspace(int64_t n, int G);
hipError_t launch_moe_sort(const MoeSortProblem &p, hipStream_t stream);

// Tokens to the experts' rows; with ye and dw also dw[t, j] = x[t] . ye[rows[t, j]].
// Groups of cap rows (contiguous: R), sf_group scale words each.
struct MoeDispatchProblem {
    const void *x;
    const float *weights;
    const int32_t *rows, *src;
    const uint16_t *ye;
    float *dw;
    uint16_t *y;
    uint8_t *q;
    void *sf;
    uint8_t *qt;
    float *sft;
    int64_t ld_x, sf_group;
    int T, top_k, K, R, cap, ld_sf, x_type, format;
};
// Needs K a multiple of 128 up to kNormMaxK; with qt one group, R a multiple of 128.
hipError_t launch_moe_dispatch(const MoeDispatchProblem &p, int num_cus, hipStream_t stream);

struct MoeCopyProblem {
    const uint8_t *x;
    const uint32_t *sf_in;
    const int32_t *rows;
    uint8_t *q;
    uint32_t *sf;
    int64_t sf_group;
    int T, top_k, K, R, cap, ld_in, ld_sf, words;
};
// Needs T >= 1, K a multiple of 128.
hipError_t launch_moe_dispatch_codes(const MoeCopyProblem &p, hipStream_t stream);

struct MoeCombineProblem {
    const uint16_t *y;
    const float *weights;
    const int32_t *rows;
    const void *residual;
    void *out;
    int T, top_k, K, R, out_type;
};
// Needs T >= 1, K a multiple of 8.
hipError_t launch_moe_combine(const MoeCombineProblem &p, hipStream_t stream);

// Gated GEMM: h = act(A Wg^T) * (A Wu^T).  Per group, A has `rows_a` rows
// (dense: M, contiguous: M_total, masked: M_cap); `idx` is m_indices
// (contiguous) or masked_m (masked).  packed: sfa, sfb and sf hold words of
// four power-of-two exponents.
struct GatedProblem {
    const uint8_t *a;
    const float *sfa;
    const uint8_t *b;
    const float *sfb;
    const int32_t *idx;
    uint16_t *gu, *h;
    uint8_t *q;
    void *sf;
    int rows_a, I, K, ld_sfa, ld_sf, G, act;
    Mode mode;
    int expected_m;
    bool packed;
    void *ws;          // caller's scratch (dense), or NULL
    size_t ws_bytes;
    int row0 = 0;      // rows of the caller's problem before `a` (set by the launcher that cuts it)
};
// Needs rows_a >= 1 and 2 * I * K and the bytes of sfa below 2^31 per group.
hipError_t launch_gated(const GatedProblem &p, int num_cus, hipStream_t stream, std::string &config);

// Its kernel for few rows (dense): takes the problem or not (a quantised
// output needs scratch of gated_small_workspace bytes).
constexpr int kGatedSmallMaxM = 128;
bool gated_small_takes(const GatedProblem &p, int num_cus);
size_t gated_small_workspace(int M, int I, int K, int num_cus);
hipError_t launch_gated_small(const GatedProblem &p, int num_cus, hipStream_t stream, std::string &config);

// Scratch bytes a dense problem with a quantised output can use.
size_t gated_workspace(int M, int I, int K, int num_cus);

struct GatedBwdProblem {
    const uint16_t *gu, *dh;
    const int32_t *idx;
    uint16_t *dgu;
    uint8_t *q;
    float *sf;
    uint8_t *qt;
    float *sft;
    uint8_t *ht;
    float *sfht;
    int rows, I, ld_sf, act;
    bool ue8m0;
};
// Needs rows >= 1, I a multiple of 128.
hipError_t launch_gated_bwd(const GatedBwdProblem &p, int num_cus, hipStream_t stream);

}  // namespace dg
