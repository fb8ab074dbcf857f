// Host-only sanitizer driver for the argument validation of the layer norm's and
// the experts' row operators' entry points (moe_api.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer.  The device query and the
// launchers are stand-ins that check what reaches them; every integer argument
// runs over its extremes.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/dg.h"
#include "../../moe_grouped_gemm_scaled_amd/csrc/dg_layer.h"

static int failures = 0, launches = 0;
#define CHECK(cond)                                                         \
    do {                                                                    \
        if (!(cond)) {                                                      \
            fprintf(stderr, "line %d: %s does not hold\n", __LINE__, #cond); \
            ++failures;                                                     \
        }                                                                   \
    } while (0)

namespace dg {

constexpr int64_t kLimit = (int64_t)1 << 31;

int current_device_cus(int &cus) {
    cus = 256;
    return DG_OK;
}
hipError_t launch_layernorm_quant(const LayerNormProblem &p, hipStream_t) {
    ++launches;
    CHECK(p.rows >= 1 && p.K >= 8 && p.K % (p.q ? 128 : 8) == 0 && p.K <= kNormMaxK && p.ld_x >= p.K && (p.q || p.y));
    return hipSuccess;
}
size_t layernorm_bwd_workspace(int rows, int K, int cus) { return rows > 1 ? (size_t)4 * cus * K * 4 : 0; }
hipError_t launch_layernorm_bwd(const LayerNormBwdProblem &p, int, hipStream_t) {
    ++launches;
    CHECK(p.rows >= 0 && p.K >= 8 && p.K % 8 == 0 && p.K <= kNormMaxK);
    return hipSuccess;
}
size_t moe_sort_workspace(int64_t n, int G) {
    CHECK(n >= 0 && n <= kMoeMaxPairs && G >= 1 && G <= kMoeMaxExperts);
    return (size_t)n;
}
hipError_t launch_moe_sort(const MoeSortProblem &p, hipStream_t) {
    ++launches;
    CHECK(p.n >= 0 && p.n <= kMoeMaxPairs && p.G >= 1 && p.G <= kMoeMaxExperts && p.R >= 0 && p.cap >= 0);
    CHECK(p.cap ? (int64_t)p.G * p.cap == p.R : p.R % 128 == 0);
    return hipSuccess;
}
hipError_t launch_moe_dispatch(const MoeDispatchProblem &p, int, hipStream_t) {
    ++launches;
    CHECK(p.T >= 0 && p.top_k >= 1 && (int64_t)p.T * p.top_k < kLimit && p.K >= 128 && p.K % 128 == 0 && p.K <= kNormMaxK);
    CHECK(p.R >= 0 && p.cap >= 0 && p.cap <= p.R && p.ld_x >= p.K && p.ld_sf >= p.cap && p.sf_group >= 0);
    CHECK(!p.qt || p.R == 0 || (p.cap == p.R && p.R % 128 == 0 && p.src && p.sft));
    return hipSuccess;
}
hipError_t launch_moe_dispatch_codes(const MoeCopyProblem &p, hipStream_t) {
    ++launches;
    CHECK(p.T >= 1 && p.top_k >= 1 && (int64_t)p.T * p.top_k < kLimit && p.K >= 128 && p.K % 128 == 0);
    CHECK(p.R >= 1 && p.cap >= 1 && p.R % p.cap == 0 && p.ld_in >= p.T && p.ld_sf >= p.cap && p.words >= 1);
    return hipSuccess;
}
hipError_t launch_moe_combine(const MoeCombineProblem &p, hipStream_t) {
    ++launches;
    CHECK(p.T >= 1 && p.top_k >= 1 && (int64_t)p.T * p.top_k < kLimit && p.K >= 8 && p.K % 8 == 0 && p.R >= 0);
    return hipSuccess;
}

}  // namespace dg

int main() {
    alignas(16) static uint8_t mem[64];
    const int ends[] = {INT_MIN, INT_MIN + 1, -128, -1, 0, 1, 2, 8, 100, 128, 256, 1000, 1024, 1025, 16384, 16512, 65536,
                        1 << 26, (1 << 26) + 1, 1 << 30, INT_MAX - 127, INT_MAX - 3, INT_MAX - 1, INT_MAX};
    const int64_t pitches[] = {INT64_MIN, -8, 0, 8, 128, 256, 16384, 1 << 20, INT64_MAX, INT64_MAX - 7};
    const int kinds[] = {INT_MIN, -1, 0, 1, 2, INT_MAX};
    void *p = mem;
    uint16_t *h = reinterpret_cast<uint16_t *>(mem);
    float *f = reinterpret_cast<float *>(mem);
    uint32_t *u = reinterpret_cast<uint32_t *>(mem);
    int32_t *i32 = reinterpret_cast<int32_t *>(mem);
    for (int a : ends) {
        for (int b : ends) {
            dg_get_layernorm_backward_workspace_size(a, b);
            dg_layernorm_backward(p, 0, p, 0, p, 0, 1e-5f, p, p, f, f, a, b, p, SIZE_MAX, nullptr);
            for (int64_t ld : pitches)
                for (int q = 0; q < 2; ++q)
                    dg_layernorm_quantize_e4m3_1x128(p, 1, ld, p, 0, p, p, 0, 1e-5f, p, h, q ? mem : nullptr, f, a, a, b,
                                                     nullptr);
            for (int c : ends) {
                const int64_t rows = dg_get_moe_rows(a, b, c);
                CHECK(rows < 0 || (rows % 128 == 0 && rows < (int64_t)1 << 31));
                dg_get_moe_sort_workspace_size(a, b, c);
                for (int d : ends) {
                    dg_moe_sort_contiguous(i32, a, b, c, i32, i32, i32, i32, i32, d, p, SIZE_MAX, nullptr);
                    dg_moe_sort_masked(i32, a, b, c, i32, i32, i32, d, p, 0, nullptr);
                    dg_moe_combine(h, f, i32, p, p, 0, a, b, c, d, nullptr);
                    for (int64_t ld : {(int64_t)256, (int64_t)INT64_MAX - 7})
                        dg_moe_combine_backward_quantize_e4m3_contiguous_ue8m0_packed(p, 0, ld, h, f, i32, i32, f, h, mem, u,
                                                                                     mem, f, a, b, c, d, nullptr);
                    for (int e : {1, 3, 1024, INT_MAX}) {
                        dg_moe_dispatch_quantize_e4m3_masked(p, 1, 16384, f, i32, h, mem, f, a, b, c, e, d, nullptr);
                        dg_moe_dispatch_e4m3_masked(mem, f, a, i32, mem, f, a, b, c, e, d, nullptr);
                    }
                    dg_moe_dispatch_e4m3_contiguous_ue8m0_packed(mem, u, a, i32, mem, u, a, b, c, d, nullptr);
                }
            }
        }
    }
    for (int k : kinds) {
        CHECK((dg_moe_combine(h, f, i32, p, p, k, 1, 1, 8, 8, nullptr) == DG_OK) == (k == 0 || k == 1));
        CHECK((dg_moe_dispatch_quantize_e4m3_contiguous(p, k, 128, f, i32, i32, h, mem, f, nullptr, nullptr, 1, 1, 128, 128,
                                                        nullptr) == DG_OK) == (k == 0 || k == 1));
        CHECK((dg_layernorm_backward(p, k, p, 0, p, 0, 0.f, p, p, f, f, 1, 8, p, 0, nullptr) == DG_OK) == (k == 0 || k == 1));
    }
    CHECK(launches > 1000);
    if (!failures) printf("ok: %d launches\n", launches);
    return failures != 0;
}
