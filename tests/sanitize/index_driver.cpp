// Host-only driver of dg_index.h's arithmetic at the ends of its sizes, built
// with AddressSanitizer and UndefinedBehaviorSanitizer.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <vector>

#include "../../moe_grouped_gemm_scaled_amd/csrc/dg_index.h"

static int failures = 0;
#define CHECK(cond)                                                         \
    do {                                                                    \
        if (!(cond)) {                                                      \
            fprintf(stderr, "line %d: %s does not hold\n", __LINE__, #cond); \
            if (++failures > 20) return 1;                                  \
        }                                                                   \
    } while (0)

static int test_for_share() {
    // every index once, in order within a part
    for (int n : {0, 1, 63, 64, 65, 1000, 4096, 4097}) {
        for (int parts : {1, 2, 3, 64}) {
            std::vector<int> seen(n + 1);
            for (int part = 0; part < parts; ++part)
                for (int t = 0; t < 128; ++t)
                    dg::for_share(n, part, parts, t, 128, [&](int i) { ++seen[i < 0 || i > n ? n : i]; });
            for (int i = 0; i < n; ++i) CHECK(seen[i] == 1);
            CHECK(seen[n] == 0);
        }
    }
    // the last part of the most rows: the step after the last index passes 2^31
    for (int n : {INT32_MAX, INT32_MAX - 1, INT32_MAX - 1022, INT32_MAX - 1023, INT32_MAX - 1024}) {
        for (int parts : {1, 3, 64}) {
            for (int t : {0, 1, 511, 1022, 1023}) {
                int64_t count = 0, last = -1, bad = 0;
                const int64_t lo = (int64_t)n * (parts - 1) / parts, want = (n - lo - t + 1023) / 1024;
                dg::for_share(n, parts - 1, parts, t, 1024, [&](int i) {
                    bad += i < lo || i >= n || (last >= 0 && i != last + 1024);
                    last = i;
                    ++count;
                });
                CHECK(bad == 0);
                CHECK(count == want);
            }
        }
    }
    return 0;
}

static int test_share_of() {
    for (int n : {0, 1, 7, 8, 255, 256, 257, 1000, (1 << 23) - 1, 1 << 23, 1 << 24, (1 << 26) - 1, 1 << 26, 1 << 30, INT32_MAX}) {
        for (int parts : {1, 2, 5, 255, 256, 304, 1024}) {
            int at = 0;
            for (int part = 0; part < parts; ++part) {
                const dg::Share s = dg::share_of(n, part, parts);
                CHECK(s.lo == at);
                CHECK(s.hi - s.lo - n / parts == 0 || s.hi - s.lo - n / parts == 1);
                at = s.hi;
            }
            CHECK(at == n);
        }
    }
    return 0;
}

static int test_runs_of() {
    for (int n : {0, 8, 504, 512, 520, 1024, 16384, 1 << 30, INT32_MAX - 519, INT32_MAX - 511, INT32_MAX - 510, INT32_MAX - 7}) {
        const int64_t runs = dg::runs_of(n, 512);
        CHECK(runs * 512 >= n && (runs - 1) * 512 < n);
        // the columns of the last run's last lane still fit an int
        CHECK((runs - 1) * 512 + 8 * 63 <= INT32_MAX);
    }
    return 0;
}

int main(int argc, char **argv) {
    const char *what = argc > 1 ? argv[1] : "";
    if (!strcmp(what, "for_share")) test_for_share();
    else if (!strcmp(what, "share_of")) test_share_of();
    else if (!strcmp(what, "runs_of")) test_runs_of();
    else return 2;
    if (!failures) printf("ok: %s\n", what);
    return failures != 0;
}
