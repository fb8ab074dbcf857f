// moe_api.cpp -- C ABI of the layer norm and of the tokens' way to the experts'
// rows and back (the third part of include/dg.h): argument validation on the
// host, before any HIP call, and kernel dispatch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dg.h"
#include "dg_layer.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool type_ok(int t) { return t == DG_BF16 || t == DG_F32; }
int64_t type_size(int t) { return t == DG_BF16 ? 2 : 4; }
constexpr int64_t kIndexLimit = (int64_t)1 << 31;    // pairs and rows are int32

int status(hipError_t e) { return e == hipSuccess ? DG_OK : DG_ERR_HIP; }

// K of the norms: a multiple of 128 for codes, of 8 (16-byte rows of bf16) otherwise.
bool layernorm_k(int K, bool codes) { return K >= 8 && K % (codes ? 128 : 8) == 0 && K <= dg::kNormMaxK; }

int layernorm_impl(const void *x, int x_type, int64_t ld_x, const void *residual, int residual_type, const void *weight,
                   const void *bias, int weight_type, float eps, void *residual_out, uint16_t *y, uint8_t *q, void *sf,
                   int ld_sf, int rows, int K, void *stream, int format) {
    if (rows < 0 || !layernorm_k(K, q != nullptr)) return DG_ERR_SHAPE;
    if (!type_ok(x_type) || !type_ok(residual_type) || !type_ok(weight_type) || !(eps >= 0.0f)) return DG_ERR_ARG;
    if (rows > 0 && (!x || (!q && !y) || (q && !sf))) return DG_ERR_NULL;
    if (residual_out && !residual) return DG_ERR_ARG;
    if (ld_x < K || ld_x % (16 / type_size(x_type)) != 0) return DG_ERR_ALIGN;
    if (q && (ld_sf < rows || ld_sf % 4 != 0)) return DG_ERR_ALIGN;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(bias) || !aligned16(residual_out) ||
        !aligned16(y) || !aligned16(q) || !aligned16(sf))
        return DG_ERR_ALIGN;
    if (rows == 0) return DG_OK;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const dg::LayerNormProblem p{x, residual, weight, bias, residual_out, y, q, sf, ld_x, rows, K, ld_sf, eps, x_type,
                                 residual_type, weight_type, format};
    return status(dg::launch_layernorm_quant(p, static_cast<hipStream_t>(stream)));
}

// Pairs of T tokens, or -1 where they reach 2^31 or a token's choices pass 2^30:
// kernels walk these in steps of up to 64 and hold the next step's start in an int.
constexpr int kMaxTopK = 1 << 30;
int64_t moe_pairs(int T, int top_k) {
    const int64_t n = (int64_t)T * top_k;
    return T < 0 || top_k < 1 || top_k > kMaxTopK || n >= kIndexLimit ? -1 : n;
}

bool moe_sort_sizes(int64_t n, int G) { return n >= 0 && n <= dg::kMoeMaxPairs && G >= 1 && G <= dg::kMoeMaxExperts; }

int64_t moe_rows(int64_t n, int G) { return (n + 127 * (n < G ? n : G)) / 128 * 128; }

int moe_sort(const int32_t *ids, int T, int top_k, int G, int32_t *rows, int32_t *src, int32_t *expert, int32_t *counts,
             int32_t *ks, int cap, int64_t R, void *workspace, size_t bytes, void *stream) {
    const int64_t n = moe_pairs(T, top_k);
    if (!moe_sort_sizes(n, G) || R < 0 || R >= kIndexLimit) return DG_ERR_SHAPE;
    if (n > 0 && (!ids || !rows)) return DG_ERR_NULL;
    if (!aligned4(ids) || !aligned4(rows) || !aligned4(src) || !aligned16(expert) || !aligned4(counts) || !aligned4(ks) ||
        !aligned16(workspace))
        return DG_ERR_ALIGN;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const dg::MoeSortProblem p{ids, rows, src, expert, counts, ks, workspace, workspace ? bytes : 0, (int)n, G, cap, (int)R};
    return status(dg::launch_moe_sort(p, static_cast<hipStream_t>(stream)));
}

struct MoeOut {
    float *dw;
    uint16_t *y;
    uint8_t *q;
    void *sf;
    uint8_t *qt;
    float *sft;
};

// cap: rows of a group (contiguous: R, one group).
int moe_dispatch(const void *x, int x_type, int64_t ld_x, const uint16_t *ye, const float *weights, const int32_t *rows,
                 const int32_t *src, const MoeOut &o, int T, int top_k, int K, int64_t cap, int64_t G, void *stream,
                 int format) {
    if (moe_pairs(T, top_k) < 0 || K < 128 || K % 128 != 0 || K > dg::kNormMaxK || cap < 0 || G < 1 ||
        cap > INT32_MAX - 3 || G * cap >= kIndexLimit)
        return DG_ERR_SHAPE;
    if (!type_ok(x_type)) return DG_ERR_ARG;
    const int64_t R = G * cap;
    // the tensors of no rows may be NULL
    if (R > 0 && ((o.q && !o.sf) || (o.qt && (!o.sft || !src)) || (!o.dw && !o.y && !o.q && !o.qt))) return DG_ERR_NULL;
    if (T > 0 && (!x || !rows || (o.dw && R > 0 && !ye))) return DG_ERR_NULL;
    if (ld_x < K || ld_x % (16 / type_size(x_type)) != 0) return DG_ERR_ALIGN;
    if (!aligned16(x) || !aligned16(ye) || !aligned4(weights) || !aligned4(rows) || !aligned4(src) || !aligned4(o.dw) ||
        !aligned16(o.y) || !aligned16(o.q) || !aligned16(o.sf) || !aligned16(o.qt) || !aligned16(o.sft))
        return DG_ERR_ALIGN;
    if ((T == 0 && !o.qt) || (R == 0 && !o.dw)) return DG_OK;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const int ld = (int)((cap + 3) / 4 * 4);
    const int64_t words = format == dg::kSfPacked ? (K / 128 + 3) / 4 : K / 128;
    const dg::MoeDispatchProblem p{x, weights, rows, src, ye, o.dw, o.y, o.q, o.sf, o.qt, o.sft, ld_x, words * ld, T, top_k,
                                   K, (int)R, (int)cap, ld, x_type, format};
    return status(dg::launch_moe_dispatch(p, cus, static_cast<hipStream_t>(stream)));
}

int moe_contiguous(const void *x, int x_type, int64_t ld_x, const uint16_t *ye, const float *weights, const int32_t *rows,
                   const int32_t *src, const MoeOut &o, int T, int top_k, int K, int M_total, void *stream, int format) {
    if (M_total < 0 || M_total % 128 != 0) return DG_ERR_SHAPE;
    return moe_dispatch(x, x_type, ld_x, ye, weights, rows, src, o, T, top_k, K, M_total, 1, stream, format);
}

int moe_masked(const void *x, int x_type, int64_t ld_x, const float *weights, const int32_t *rows, const MoeOut &o, int T,
               int top_k, int K, int G, int M_cap, void *stream, int format) {
    if (G < 1 || M_cap < 1) return DG_ERR_SHAPE;
    return moe_dispatch(x, x_type, ld_x, nullptr, weights, rows, nullptr, o, T, top_k, K, M_cap, G, stream, format);
}

int moe_codes(const uint8_t *q_in, const void *sf_in, int ld_in, const int32_t *rows, uint8_t *q, void *sf, int T, int top_k,
              int K, int64_t cap, int64_t G, void *stream, bool packed) {
    if (moe_pairs(T, top_k) < 0 || K < 128 || K % 128 != 0 || cap < 0 || G < 1 || cap > INT32_MAX - 3 ||
        G * cap >= kIndexLimit)
        return DG_ERR_SHAPE;
    if (T > 0 && (!q_in || !sf_in || !rows || (G * cap > 0 && (!q || !sf)))) return DG_ERR_NULL;
    if (ld_in < T || ld_in % 4 != 0) return DG_ERR_ALIGN;
    if (!aligned16(q_in) || !aligned16(sf_in) || !aligned4(rows) || !aligned16(q) || !aligned16(sf)) return DG_ERR_ALIGN;
    if (T == 0 || G * cap == 0) return DG_OK;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const int ld = (int)((cap + 3) / 4 * 4), words = packed ? (K / 128 + 3) / 4 : K / 128;
    const dg::MoeCopyProblem p{q_in, static_cast<const uint32_t *>(sf_in), rows, q, static_cast<uint32_t *>(sf),
                               (int64_t)words * ld, T, top_k, K, (int)(G * cap), (int)cap, ld_in, ld, words};
    return status(dg::launch_moe_dispatch_codes(p, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int dg_layernorm_quantize_e4m3_1x128(const void *x, int x_type, int64_t ld_x, const void *residual, int residual_type,
                                     const void *weight, const void *bias, int weight_type, float eps,
                                     void *residual_out, uint16_t *y, uint8_t *q, float *sf, int ld_sf, int rows, int K,
                                     void *stream) {
    return layernorm_impl(x, x_type, ld_x, residual, residual_type, weight, bias, weight_type, eps, residual_out, y, q, sf,
                          ld_sf, rows, K, stream, dg::kSfFp32);
}

int dg_layernorm_quantize_e4m3_1x128_ue8m0(const void *x, int x_type, int64_t ld_x, const void *residual, int residual_type,
                                     const void *weight, const void *bias, int weight_type, float eps,
                                     void *residual_out, uint16_t *y, uint8_t *q, float *sf, int ld_sf, int rows, int K,
                                     void *stream) {
    return layernorm_impl(x, x_type, ld_x, residual, residual_type, weight, bias, weight_type, eps, residual_out, y, q, sf,
                          ld_sf, rows, K, stream, dg::kSfUe8m0);
}

int dg_layernorm_quantize_e4m3_1x128_ue8m0_packed(const void *x, int x_type, int64_t ld_x, const void *residual, int residual_type,
                                     const void *weight, const void *bias, int weight_type, float eps,
                                     void *residual_out, uint16_t *y, uint8_t *q, uint32_t *sf, int ld_sf, int rows, int K,
                                     void *stream) {
    return layernorm_impl(x, x_type, ld_x, residual, residual_type, weight, bias, weight_type, eps, residual_out, y, q, sf,
                          ld_sf, rows, K, stream, dg::kSfPacked);
}

int64_t dg_get_layernorm_backward_workspace_size(int rows, int K) {
    if (rows < 0 || !layernorm_k(K, false)) return DG_ERR_SHAPE;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    return (int64_t)dg::layernorm_bwd_workspace(rows, K, cus);
}

int dg_layernorm_backward(const void *dy, int dy_type, const void *h, int h_type, const void *weight, int weight_type,
                          float eps, const void *dres, void *dx, float *dw, float *db, int rows, int K, void *workspace,
                          size_t workspace_bytes, void *stream) {
    if (rows < 0 || !layernorm_k(K, false)) return DG_ERR_SHAPE;
    if (!type_ok(dy_type) || !type_ok(h_type) || !type_ok(weight_type) || !(eps >= 0.0f)) return DG_ERR_ARG;
    if (rows > 0 && (!dy || !h || !dx)) return DG_ERR_NULL;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(dres) || !aligned16(dx) || !aligned16(dw) ||
        !aligned16(db) || !aligned16(workspace))
        return DG_ERR_ALIGN;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const size_t need = dw || db ? dg::layernorm_bwd_workspace(rows, K, cus) : 0;
    if (need > 0 && !workspace) return DG_ERR_NULL;
    if (workspace_bytes < need) return DG_ERR_ARG;
    const dg::LayerNormBwdProblem p{dy, h, weight, dres, dx, dw, db, workspace, rows, K, eps, h_type, dy_type, weight_type};
    return status(dg::launch_layernorm_bwd(p, cus, static_cast<hipStream_t>(stream)));
}

int64_t dg_get_moe_rows(int T, int top_k, int G) {
    const int64_t n = moe_pairs(T, top_k);
    if (!moe_sort_sizes(n, G)) return DG_ERR_SHAPE;
    return moe_rows(n, G);
}

int64_t dg_get_moe_sort_workspace_size(int T, int top_k, int G) {
    const int64_t n = moe_pairs(T, top_k);
    if (!moe_sort_sizes(n, G)) return DG_ERR_SHAPE;
    return (int64_t)dg::moe_sort_workspace(n, G);
}

int dg_moe_sort_contiguous(const int32_t *ids, int T, int top_k, int G, int32_t *rows, int32_t *src, int32_t *m_indices,
                           int32_t *counts, int32_t *ks, int M_total, void *workspace, size_t workspace_bytes,
                           void *stream) {
    if (M_total % 128 != 0) return DG_ERR_SHAPE;
    return moe_sort(ids, T, top_k, G, rows, src, m_indices, counts, ks, 0, M_total, workspace, workspace_bytes, stream);
}

int dg_moe_sort_masked(const int32_t *ids, int T, int top_k, int G, int32_t *rows, int32_t *src, int32_t *masked_m,
                       int M_cap, void *workspace, size_t workspace_bytes, void *stream) {
    if (M_cap < 1) return DG_ERR_SHAPE;
    if (!masked_m) return DG_ERR_NULL;
    return moe_sort(ids, T, top_k, G, rows, src, nullptr, masked_m, nullptr, M_cap, (int64_t)G * M_cap, workspace,
                    workspace_bytes, stream);
}

int dg_moe_dispatch_quantize_e4m3_contiguous(const void *x, int x_type, int64_t ld_x, const float *weights,
                                             const int32_t *rows, const int32_t *src, uint16_t *y, uint8_t *q, float *sf,
                                             uint8_t *qt, float *sft, int T, int top_k, int K, int M_total, void *stream) {
    return moe_contiguous(x, x_type, ld_x, nullptr, weights, rows, src, {nullptr, y, q, sf, qt, sft}, T, top_k, K, M_total,
                          stream, dg::kSfFp32);
}

int dg_moe_dispatch_quantize_e4m3_masked(const void *x, int x_type, int64_t ld_x, const float *weights,
                                         const int32_t *rows, uint16_t *y, uint8_t *q, float *sf, int T, int top_k, int K,
                                         int G, int M_cap, void *stream) {
    return moe_masked(x, x_type, ld_x, weights, rows, {nullptr, y, q, sf, nullptr, nullptr}, T, top_k, K, G, M_cap, stream,
                      dg::kSfFp32);
}

int dg_moe_combine_backward_quantize_e4m3_contiguous(const void *dout, int dout_type, int64_t ld_dout, const uint16_t *y,
                                                     const float *weights, const int32_t *rows, const int32_t *src,
                                                     float *dw, uint16_t *dy, uint8_t *q, float *sf, uint8_t *qt,
                                                     float *sft, int T, int top_k, int K, int M_total, void *stream) {
    return moe_contiguous(dout, dout_type, ld_dout, y, weights, rows, src, {dw, dy, q, sf, qt, sft}, T, top_k, K, M_total,
                          stream, dg::kSfFp32);
}

int dg_moe_dispatch_quantize_e4m3_contiguous_ue8m0(const void *x, int x_type, int64_t ld_x, const float *weights,
                                             const int32_t *rows, const int32_t *src, uint16_t *y, uint8_t *q, float *sf,
                                             uint8_t *qt, float *sft, int T, int top_k, int K, int M_total, void *stream) {
    return moe_contiguous(x, x_type, ld_x, nullptr, weights, rows, src, {nullptr, y, q, sf, qt, sft}, T, top_k, K, M_total,
                          stream, dg::kSfUe8m0);
}

int dg_moe_dispatch_quantize_e4m3_masked_ue8m0(const void *x, int x_type, int64_t ld_x, const float *weights,
                                         const int32_t *rows, uint16_t *y, uint8_t *q, float *sf, int T, int top_k, int K,
                                         int G, int M_cap, void *stream) {
    return moe_masked(x, x_type, ld_x, weights, rows, {nullptr, y, q, sf, nullptr, nullptr}, T, top_k, K, G, M_cap, stream,
                      dg::kSfUe8m0);
}

int dg_moe_combine_backward_quantize_e4m3_contiguous_ue8m0(const void *dout, int dout_type, int64_t ld_dout, const uint16_t *y,
                                                     const float *weights, const int32_t *rows, const int32_t *src,
                                                     float *dw, uint16_t *dy, uint8_t *q, float *sf, uint8_t *qt,
                                                     float *sft, int T, int top_k, int K, int M_total, void *stream) {
    return moe_contiguous(dout, dout_type, ld_dout, y, weights, rows, src, {dw, dy, q, sf, qt, sft}, T, top_k, K, M_total,
                          stream, dg::kSfUe8m0);
}

int dg_moe_dispatch_quantize_e4m3_contiguous_ue8m0_packed(const void *x, int x_type, int64_t ld_x, const float *weights,
                                             const int32_t *rows, const int32_t *src, uint16_t *y, uint8_t *q, uint32_t *sf,
                                             uint8_t *qt, float *sft, int T, int top_k, int K, int M_total, void *stream) {
    return moe_contiguous(x, x_type, ld_x, nullptr, weights, rows, src, {nullptr, y, q, sf, qt, sft}, T, top_k, K, M_total,
                          stream, dg::kSfPacked);
}

int dg_moe_dispatch_quantize_e4m3_masked_ue8m0_packed(const void *x, int x_type, int64_t ld_x, const float *weights,
                                         const int32_t *rows, uint16_t *y, uint8_t *q, uint32_t *sf, int T, int top_k, int K,
                                         int G, int M_cap, void *stream) {
    return moe_masked(x, x_type, ld_x, weights, rows, {nullptr, y, q, sf, nullptr, nullptr}, T, top_k, K, G, M_cap, stream,
                      dg::kSfPacked);
}

int dg_moe_combine_backward_quantize_e4m3_contiguous_ue8m0_packed(const void *dout, int dout_type, int64_t ld_dout, const uint16_t *y,
                                                     const float *weights, const int32_t *rows, const int32_t *src,
                                                     float *dw, uint16_t *dy, uint8_t *q, uint32_t *sf, uint8_t *qt,
                                                     float *sft, int T, int top_k, int K, int M_total, void *stream) {
    return moe_contiguous(dout, dout_type, ld_dout, y, weights, rows, src, {dw, dy, q, sf, qt, sft}, T, top_k, K, M_total,
                          stream, dg::kSfPacked);
}

int dg_moe_dispatch_e4m3_contiguous(const uint8_t *q_in, const float *sf_in, int ld_in, const int32_t *rows, uint8_t *q,
                                    float *sf, int T, int top_k, int K, int M_total, void *stream) {
    if (M_total < 0 || M_total % 128 != 0) return DG_ERR_SHAPE;
    return moe_codes(q_in, sf_in, ld_in, rows, q, sf, T, top_k, K, M_total, 1, stream, false);
}

int dg_moe_dispatch_e4m3_masked(const uint8_t *q_in, const float *sf_in, int ld_in, const int32_t *rows, uint8_t *q,
                                float *sf, int T, int top_k, int K, int G, int M_cap, void *stream) {
    if (G < 1 || M_cap < 1) return DG_ERR_SHAPE;
    return moe_codes(q_in, sf_in, ld_in, rows, q, sf, T, top_k, K, M_cap, G, stream, false);
}

int dg_moe_dispatch_e4m3_contiguous_ue8m0_packed(const uint8_t *q_in, const uint32_t *sf_in, int ld_in, const int32_t *rows, uint8_t *q,
                                    uint32_t *sf, int T, int top_k, int K, int M_total, void *stream) {
    if (M_total < 0 || M_total % 128 != 0) return DG_ERR_SHAPE;
    return moe_codes(q_in, sf_in, ld_in, rows, q, sf, T, top_k, K, M_total, 1, stream, true);
}

int dg_moe_dispatch_e4m3_masked_ue8m0_packed(const uint8_t *q_in, const uint32_t *sf_in, int ld_in, const int32_t *rows, uint8_t *q,
                                uint32_t *sf, int T, int top_k, int K, int G, int M_cap, void *stream) {
    if (G < 1 || M_cap < 1) return DG_ERR_SHAPE;
    return moe_codes(q_in, sf_in, ld_in, rows, q, sf, T, top_k, K, M_cap, G, stream, true);
}

int dg_moe_combine(const uint16_t *y, const float *weights, const int32_t *rows, const void *residual, void *out,
                   int out_type, int T, int top_k, int K, int R, void *stream) {
    if (moe_pairs(T, top_k) < 0 || R < 0 || K < 8 || K % 8 != 0) return DG_ERR_SHAPE;
    if (!type_ok(out_type)) return DG_ERR_ARG;
    if (T > 0 && ((R > 0 && !y) || !rows || !out)) return DG_ERR_NULL;
    if (!aligned16(y) || !aligned4(weights) || !aligned4(rows) || !aligned16(residual) || !aligned16(out)) return DG_ERR_ALIGN;
    if (T == 0) return DG_OK;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const dg::MoeCombineProblem p{y, weights, rows, residual, out, T, top_k, K, R, out_type};
    return status(dg::launch_moe_combine(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
