// layer_api.cpp -- C ABI of the feed-forward layer's operators (the second
// part of include/dg.h): argument validation on the host, before any HIP call,
// and kernel dispatch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "../../include/dg.h"
#include "dg_layer.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool type_ok(int t) { return t == DG_BF16 || t == DG_F32; }
bool act_ok(int a) { return a == DG_ACT_SILU || a == DG_ACT_GELU_TANH; }
int64_t type_size(int t) { return t == DG_BF16 ? 2 : 4; }
constexpr int64_t kOffsetLimit = (int64_t)1 << 31;   // 32-bit buffer offsets

int status(hipError_t e) { return e == hipSuccess ? DG_OK : DG_ERR_HIP; }

int rmsnorm_impl(const void *x, int x_type, int64_t ld_x, const void *residual, int residual_type, const void *weight,
                 int weight_type, float eps, void *residual_out, uint16_t *y, uint8_t *q, void *sf, int ld_sf, int rows,
                 int K, void *stream, int format) {
    if (rows < 0 || K < 128 || K % 128 != 0 || K > dg::kNormMaxK) return DG_ERR_SHAPE;
    if (!type_ok(x_type) || !type_ok(residual_type) || !type_ok(weight_type) || !(eps >= 0.0f)) return DG_ERR_ARG;
    if (rows > 0 && (!x || !weight || (!q && !y) || (q && !sf))) return DG_ERR_NULL;
    if (residual_out && !residual) return DG_ERR_ARG;
    if (ld_x < K || ld_x % (16 / type_size(x_type)) != 0) return DG_ERR_ALIGN;
    if (q && (ld_sf < rows || ld_sf % 4 != 0)) return DG_ERR_ALIGN;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) || !aligned16(y) ||
        !aligned16(q) || !aligned16(sf))
        return DG_ERR_ALIGN;
    if (rows == 0) return DG_OK;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const dg::RmsNormProblem p{x, residual, weight, residual_out, y, q, sf, ld_x, rows, K, ld_sf, eps, x_type,
                               residual_type, weight_type, format};
    return status(dg::launch_rmsnorm_quant(p, static_cast<hipStream_t>(stream)));
}

struct GatedOut {
    uint16_t *gu, *h;
    uint8_t *q;
    void *sf;
    int ld_sf;
};

// What the three layouts of the gated GEMM have in common.
int gated_check(const void *a, const void *sfa, const void *b, const void *sfb, int act, const GatedOut &o, int rows,
                int ld_sfa, int I, int K) {
    if (rows < 0 || I < 1 || K < 128 || K % 128 != 0) return DG_ERR_SHAPE;
    if (2 * (int64_t)I * K >= kOffsetLimit || 256 * (int64_t)K >= kOffsetLimit ||
        (int64_t)(K / 128) * ld_sfa * 4 >= kOffsetLimit)
        return DG_ERR_SHAPE;
    if (o.q && I % 128 != 0) return DG_ERR_SHAPE;
    if (!act_ok(act)) return DG_ERR_ARG;
    if (rows > 0 && (!a || !sfa || !b || !sfb || (!o.h && !o.q) || (o.q && !o.sf))) return DG_ERR_NULL;
    if (ld_sfa < rows || ld_sfa % 4 != 0) return DG_ERR_ALIGN;
    if (o.q && (o.ld_sf < rows || o.ld_sf % 4 != 0)) return DG_ERR_ALIGN;
    if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(o.gu) || !aligned16(o.h) ||
        !aligned16(o.q) || !aligned16(o.sf))
        return DG_ERR_ALIGN;
    return DG_OK;
}

int gated_run(const dg::GatedProblem &p, void *stream) {
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    try {
        std::string config;
        const hipError_t err = dg::launch_gated(p, cus, static_cast<hipStream_t>(stream), config);
        dg::set_last_config(config);
        return status(err);
    } catch (...) {   // no memory for the description: no exception leaves a C entry
        return DG_ERR_HIP;
    }
}

int gated_dense(const uint8_t *a, const void *sfa, int ld_sfa, const uint8_t *b, const void *sfb, int act,
                const GatedOut &o, int M, int I, int K, void *workspace, size_t bytes, void *stream, bool packed) {
    const int st = gated_check(a, sfa, b, sfb, act, o, M, ld_sfa, I, K);
    if (st != DG_OK) return st;
    if (!aligned16(workspace)) return DG_ERR_ALIGN;
    if (M == 0) return DG_OK;
    return gated_run({a, static_cast<const float *>(sfa), b, static_cast<const float *>(sfb), nullptr, o.gu, o.h, o.q,
                      o.sf, M, I, K, ld_sfa, o.ld_sf, 1, act, dg::Mode::Dense, 0, packed, workspace,
                      workspace ? bytes : 0},
                     stream);
}

int gated_contiguous(const uint8_t *a, const void *sfa, const uint8_t *b, const void *sfb, int act, const GatedOut &o,
                     const int32_t *m_indices, int M_total, int I, int K, int G, void *stream, bool packed) {
    if (M_total % 128 != 0 || G < 1) return DG_ERR_SHAPE;
    const int st = gated_check(a, sfa, b, sfb, act, o, M_total, M_total, I, K);
    if (st != DG_OK) return st;
    if (M_total > 0 && !m_indices) return DG_ERR_NULL;
    if (!aligned16(m_indices)) return DG_ERR_ALIGN;
    if (M_total == 0) return DG_OK;
    return gated_run({a, static_cast<const float *>(sfa), b, static_cast<const float *>(sfb), m_indices, o.gu, o.h, o.q,
                      o.sf, M_total, I, K, M_total, o.ld_sf, G, act, dg::Mode::Contig, 0, packed, nullptr, 0},
                     stream);
}

int gated_masked(const uint8_t *a, const void *sfa, const uint8_t *b, const void *sfb, int act, GatedOut o,
                 const int32_t *masked_m, int G, int M_cap, int I, int K, int expected_m, void *stream, bool packed) {
    if (G < 1 || M_cap < 1 || M_cap > INT32_MAX - 3) return DG_ERR_SHAPE;
    o.ld_sf = (M_cap + 3) / 4 * 4;                     // of sfa too
    const int st = gated_check(a, sfa, b, sfb, act, o, M_cap, o.ld_sf, I, K);
    if (st != DG_OK) return st;
    if (!masked_m) return DG_ERR_NULL;
    if (!aligned4(masked_m)) return DG_ERR_ALIGN;
    return gated_run({a, static_cast<const float *>(sfa), b, static_cast<const float *>(sfb), masked_m, o.gu, o.h, o.q,
                      o.sf, M_cap, I, K, o.ld_sf, o.ld_sf, G, act, dg::Mode::Masked, expected_m, packed,
                      nullptr, 0},
                     stream);
}

int gated_bwd_impl(const uint16_t *gu, const uint16_t *dh, int act, const int32_t *m_indices, uint16_t *dgu, uint8_t *q,
                   float *sf, int ld_sf, uint8_t *qt, float *sft, uint8_t *ht, float *sfht, int rows, int I,
                   void *stream, bool ue8m0) {
    if (rows < 0 || I < 128 || I % 128 != 0 || 512 * (int64_t)I >= kOffsetLimit) return DG_ERR_SHAPE;
    if (!act_ok(act)) return DG_ERR_ARG;
    if (rows > 0 && (!gu || !dh || (!dgu && !q && !qt && !ht) || (q && !sf) || (qt && !sft) || (ht && !sfht)))
        return DG_ERR_NULL;
    if (q && (ld_sf < rows || ld_sf % 4 != 0)) return DG_ERR_ALIGN;
    if (!aligned16(gu) || !aligned16(dh) || !aligned4(m_indices) || !aligned16(dgu) || !aligned16(q) || !aligned16(sf) ||
        !aligned16(qt) || !aligned16(sft) || !aligned16(ht) || !aligned16(sfht))
        return DG_ERR_ALIGN;
    if (rows == 0) return DG_OK;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const dg::GatedBwdProblem p{gu, dh, m_indices, dgu, q, sf, qt, sft, ht, sfht, rows, I, ld_sf, act, ue8m0};
    return status(dg::launch_gated_bwd(p, cus, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int dg_rmsnorm_quantize_e4m3_1x128(const void *x, int x_type, int64_t ld_x, const void *residual, int residual_type,
                                   const void *weight, int weight_type, float eps, void *residual_out, uint16_t *y,
                                   uint8_t *q, float *sf, int ld_sf, int rows, int K, void *stream) {
    return rmsnorm_impl(x, x_type, ld_x, residual, residual_type, weight, weight_type, eps, residual_out, y, q, sf,
                        ld_sf, rows, K, stream, dg::kSfFp32);
}

int dg_rmsnorm_quantize_e4m3_1x128_ue8m0(const void *x, int x_type, int64_t ld_x, const void *residual,
                                         int residual_type, const void *weight, int weight_type, float eps,
                                         void *residual_out, uint16_t *y, uint8_t *q, float *sf, int ld_sf, int rows,
                                         int K, void *stream) {
    return rmsnorm_impl(x, x_type, ld_x, residual, residual_type, weight, weight_type, eps, residual_out, y, q, sf,
                        ld_sf, rows, K, stream, dg::kSfUe8m0);
}

int dg_rmsnorm_quantize_e4m3_1x128_ue8m0_packed(const void *x, int x_type, int64_t ld_x, const void *residual,
                                                int residual_type, const void *weight, int weight_type, float eps,
                                                void *residual_out, uint16_t *y, uint8_t *q, uint32_t *sf, int ld_sf,
                                                int rows, int K, void *stream) {
    return rmsnorm_impl(x, x_type, ld_x, residual, residual_type, weight, weight_type, eps, residual_out, y, q, sf,
                        ld_sf, rows, K, stream, dg::kSfPacked);
}

int64_t dg_get_rmsnorm_backward_workspace_size(int rows, int K) {
    if (rows < 0 || K < 128 || K % 128 != 0 || K > dg::kNormMaxK) return DG_ERR_SHAPE;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    return (int64_t)dg::rmsnorm_bwd_workspace(rows, K, cus);
}

int dg_rmsnorm_backward(const void *dy, int dy_type, const void *h, int h_type, const void *weight, int weight_type,
                        float eps, const void *dres, void *dx, float *dw, int rows, int K, void *workspace,
                        size_t workspace_bytes, void *stream) {
    if (rows < 0 || K < 128 || K % 128 != 0 || K > dg::kNormMaxK) return DG_ERR_SHAPE;
    if (!type_ok(dy_type) || !type_ok(h_type) || !type_ok(weight_type) || !(eps >= 0.0f)) return DG_ERR_ARG;
    if (!dw || (rows > 0 && (!dy || !h || !weight || !dx))) return DG_ERR_NULL;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(dres) || !aligned16(dx) || !aligned16(dw) ||
        !aligned16(workspace))
        return DG_ERR_ALIGN;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    const size_t need = dg::rmsnorm_bwd_workspace(rows, K, cus);
    if (need > 0 && !workspace) return DG_ERR_NULL;
    if (workspace_bytes < need) return DG_ERR_ARG;
    const dg::RmsNormBwdProblem p{dy, h, weight, dres, dx, dw, workspace, rows, K, eps, h_type, dy_type, weight_type};
    return status(dg::launch_rmsnorm_bwd(p, cus, static_cast<hipStream_t>(stream)));
}

int64_t dg_get_gated_workspace_size(int M, int I, int K) {
    if (M < 0 || I < 1 || K < 128 || K % 128 != 0 || 2 * (int64_t)I * K >= kOffsetLimit ||
        256 * (int64_t)K >= kOffsetLimit)
        return DG_ERR_SHAPE;
    int cus = 0;
    const int st = dg::current_device_cus(cus);
    if (st != DG_OK) return st;
    return (int64_t)dg::gated_workspace(M, I, K, cus);
}

int dg_fp8_gated_gemm_nt(const uint8_t *a, const float *sfa, int ld_sfa, const uint8_t *b, const float *sfb, int act,
                         uint16_t *gu, uint16_t *h, uint8_t *q, float *sf, int ld_sf, int M, int I, int K,
                         void *workspace, size_t workspace_bytes, void *stream) {
    return gated_dense(a, sfa, ld_sfa, b, sfb, act, {gu, h, q, sf, ld_sf}, M, I, K, workspace, workspace_bytes, stream,
                       false);
}

int dg_fp8_gated_gemm_nt_ue8m0_packed(const uint8_t *a, const uint32_t *sfa, int ld_sfa, const uint8_t *b,
                                      const uint32_t *sfb, int act, uint16_t *gu, uint16_t *h, uint8_t *q, uint32_t *sf,
                                      int ld_sf, int M, int I, int K, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    return gated_dense(a, sfa, ld_sfa, b, sfb, act, {gu, h, q, sf, ld_sf}, M, I, K, workspace, workspace_bytes, stream,
                       true);
}

int dg_m_grouped_fp8_gated_gemm_nt_contiguous(const uint8_t *a, const float *sfa, const uint8_t *b, const float *sfb,
                                              int act, uint16_t *gu, uint16_t *h, uint8_t *q, float *sf,
                                              const int32_t *m_indices, int M_total, int I, int K, int G, void *stream) {
    return gated_contiguous(a, sfa, b, sfb, act, {gu, h, q, sf, M_total}, m_indices, M_total, I, K, G, stream, false);
}

int dg_m_grouped_fp8_gated_gemm_nt_contiguous_ue8m0_packed(const uint8_t *a, const uint32_t *sfa, const uint8_t *b,
                                                           const uint32_t *sfb, int act, uint16_t *gu, uint16_t *h,
                                                           uint8_t *q, uint32_t *sf, const int32_t *m_indices,
                                                           int M_total, int I, int K, int G, void *stream) {
    return gated_contiguous(a, sfa, b, sfb, act, {gu, h, q, sf, M_total}, m_indices, M_total, I, K, G, stream, true);
}

int dg_m_grouped_fp8_gated_gemm_nt_masked(const uint8_t *a, const float *sfa, const uint8_t *b, const float *sfb,
                                          int act, uint16_t *gu, uint16_t *h, uint8_t *q, float *sf,
                                          const int32_t *masked_m, int G, int M_cap, int I, int K, int expected_m,
                                          void *stream) {
    return gated_masked(a, sfa, b, sfb, act, {gu, h, q, sf, 0}, masked_m, G, M_cap, I, K, expected_m,
                        stream, false);
}

int dg_m_grouped_fp8_gated_gemm_nt_masked_ue8m0_packed(const uint8_t *a, const uint32_t *sfa, const uint8_t *b,
                                                       const uint32_t *sfb, int act, uint16_t *gu, uint16_t *h,
                                                       uint8_t *q, uint32_t *sf, const int32_t *masked_m, int G,
                                                       int M_cap, int I, int K, int expected_m, void *stream) {
    return gated_masked(a, sfa, b, sfb, act, {gu, h, q, sf, 0}, masked_m, G, M_cap, I, K, expected_m,
                        stream, true);
}

int dg_gated_backward_quantize_e4m3(const uint16_t *gu, const uint16_t *dh, int act, const int32_t *m_indices,
                                    uint16_t *dgu, uint8_t *q, float *sf, int ld_sf, uint8_t *qt, float *sft,
                                    uint8_t *ht, float *sfht, int rows, int I, void *stream) {
    return gated_bwd_impl(gu, dh, act, m_indices, dgu, q, sf, ld_sf, qt, sft, ht, sfht, rows, I, stream, false);
}

int dg_gated_backward_quantize_e4m3_ue8m0(const uint16_t *gu, const uint16_t *dh, int act, const int32_t *m_indices,
                                          uint16_t *dgu, uint8_t *q, float *sf, int ld_sf, uint8_t *qt, float *sft,
                                          uint8_t *ht, float *sfht, int rows, int I, void *stream) {
    return gated_bwd_impl(gu, dh, act, m_indices, dgu, q, sf, ld_sf, qt, sft, ht, sfht, rows, I, stream, true);
}

}  // extern "C"
