// Host-only sanitizer driver for the argument validation of the feed-forward
// layer's entry points (layer_api.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer.  The device query and the launchers are stand-ins
// that check what reaches them: every size that validation lets through is one
// that the kernels' offsets can take.  Every integer argument runs over its
// extremes; an exception in a launcher must not leave the C entry.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/dg.h"
#include "../../moe_grouped_gemm_scaled_amd/csrc/dg_layer.h"

static int failures = 0, launches = 0;
static bool throwing = false;
#define CHECK(cond)                                                         \
    do {                                                                    \
        if (!(cond)) {                                                      \
            fprintf(stderr, "line %d: %s does not hold\n", __LINE__, #cond); \
            ++failures;                                                     \
        }                                                                   \
    } while (0)

namespace dg {

int current_device_cus(int &cus) {
    cus = 256;
    return DG_OK;
}
void set_last_config(const std::string &) {}
hipError_t launch_rmsnorm_quant(const RmsNormProblem &p, hipStream_t) {
    ++launches;
    CHECK(p.rows >= 1 && p.K >= 128 && p.K % 128 == 0 && p.K <= kNormMaxK && p.ld_x >= p.K);
    return hipSuccess;
}
size_t rmsnorm_bwd_workspace(int rows, int K, int cus) { return rows > 4 ? (size_t)2 * cus * K * 4 : 0; }
hipError_t launch_rmsnorm_bwd(const RmsNormBwdProblem &p, int, hipStream_t) {
    ++launches;
    CHECK(p.rows >= 0 && p.K >= 128 && p.K % 128 == 0 && p.K <= kNormMaxK);
    return hipSuccess;
}
size_t gated_workspace(int, int, int, int) { return 16; }
hipError_t launch_gated(const GatedProblem &p, int, hipStream_t, std::string &config) {
    ++launches;
    if (throwing) throw std::bad_alloc();
    config = "stub";
    CHECK(p.rows_a >= 1 && p.I >= 1 && p.G >= 1 && p.ld_sfa >= p.rows_a && p.ld_sfa % 4 == 0);
    CHECK(2 * (int64_t)p.I * p.K < (int64_t)1 << 31 && 256 * (int64_t)p.K < (int64_t)1 << 31);
    CHECK((int64_t)(p.K / 128) * p.ld_sfa * 4 < (int64_t)1 << 31);
    CHECK(!p.q || p.I % 128 == 0);
    return hipSuccess;
}
hipError_t launch_gated_bwd(const GatedBwdProblem &p, int, hipStream_t) {
    ++launches;
    CHECK(p.rows >= 1 && p.I >= 128 && p.I % 128 == 0 && 512 * (int64_t)p.I < (int64_t)1 << 31);
    return hipSuccess;
}

}  // namespace dg

int main() {
    uint8_t *const P = reinterpret_cast<uint8_t *>(0x10000);   // never dereferenced
    float *const F = reinterpret_cast<float *>(P);
    uint16_t *const H = reinterpret_cast<uint16_t *>(P);
    const uint32_t *W = reinterpret_cast<const uint32_t *>(P);
    const int32_t *X = reinterpret_cast<const int32_t *>(P);
    const int sizes[] = {INT_MIN, -1, 0, 1, 100, 128, 256, 16384, 1 << 20, 1 << 22, 1 << 23, 1 << 30, INT_MAX - 127, INT_MAX - 3, INT_MAX};
    const int64_t pitches[] = {INT64_MIN, -1, 0, 128, 1 << 20, INT64_MAX - 7, INT64_MAX};
    for (int rows : sizes)
        for (int K : sizes) {
            for (int64_t ld : pitches)
                for (int ld_sf : {INT_MIN, 0, 128, INT_MAX - 3, INT_MAX})
                    for (int type : {-1, 0, 1, 2}) {
                        dg_rmsnorm_quantize_e4m3_1x128(P, type, ld, P, type, P, 0, 1e-6f, P, H, P, F, ld_sf, rows, K, nullptr);
                        dg_rmsnorm_quantize_e4m3_1x128_ue8m0(P, 0, ld, P, type, P, 0, 1e-6f, P, H, P, F, ld_sf, rows, K, nullptr);
                        dg_rmsnorm_quantize_e4m3_1x128_ue8m0_packed(P, 0, ld, P, 0, P, type, 1e-6f, P, H, P, const_cast<uint32_t *>(W),
                                                                    ld_sf, rows, K, nullptr);
                    }
            dg_rmsnorm_backward(P, 0, P, 1, P, 0, 1e-6f, P, P, F, rows, K, P, (size_t)-1, nullptr);
            dg_get_rmsnorm_backward_workspace_size(rows, K);
            for (int I : sizes) {
                dg_get_gated_workspace_size(rows, I, K);
                for (int ld : {INT_MIN, 0, 128, 1 << 29, INT_MAX - 3, INT_MAX}) {
                    dg_fp8_gated_gemm_nt(P, F, ld, P, F, 0, H, H, P, F, ld, rows, I, K, P, 1 << 20, nullptr);
                    dg_fp8_gated_gemm_nt_ue8m0_packed(P, W, ld, P, W, 1, H, H, nullptr, nullptr, ld, rows, I, K, nullptr, 0, nullptr);
                }
                for (int G : {INT_MIN, 0, 1, INT_MAX}) {
                    dg_m_grouped_fp8_gated_gemm_nt_contiguous(P, F, P, F, 0, H, H, P, F, X, rows, I, K, G, nullptr);
                    dg_m_grouped_fp8_gated_gemm_nt_contiguous_ue8m0_packed(P, W, P, W, 0, H, H, nullptr, nullptr, X, rows, I, K, G, nullptr);
                    dg_m_grouped_fp8_gated_gemm_nt_masked(P, F, P, F, 0, H, H, P, F, X, G, rows, I, K, INT_MAX, nullptr);
                    dg_m_grouped_fp8_gated_gemm_nt_masked_ue8m0_packed(P, W, P, W, 0, H, H, nullptr, nullptr, X, G, rows, I, K, INT_MIN, nullptr);
                }
            }
            dg_gated_backward_quantize_e4m3(H, H, 0, X, H, P, F, K, P, F, P, F, rows, K, nullptr);
            dg_gated_backward_quantize_e4m3_ue8m0(H, H, 1, nullptr, H, nullptr, nullptr, 0, P, F, P, F, rows, K, nullptr);
        }
    CHECK(launches > 100);
    throwing = true;
    CHECK(dg_fp8_gated_gemm_nt(P, F, 128, P, F, 0, H, H, P, F, 128, 128, 128, 128, P, 16, nullptr) == DG_ERR_HIP);
    throwing = false;
    CHECK(dg_fp8_gated_gemm_nt(P, F, 128, P, F, 0, H, H, P, F, 128, 128, 128, 128, P, 16, nullptr) == DG_OK);
    if (!failures) printf("layer driver ok, %d launches\n", launches);
    return failures != 0;
}
