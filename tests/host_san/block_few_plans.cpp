// Plans of the feed-forward block of few rows, over every number of rows that takes them: slices of the reductions, none
// without work, whose sums fit the region behind the plan's others, and regions that do not overlap.  Built with the sanitizers by
// tests/test_block_few_plans.py; exits nonzero on an unexpected value.
#include <stdint.h>
#include <stdio.h>

#include "block/block_plan.h"

static int failures = 0, plans = 0;

static void check(bool good, const char* what, int64_t t, int64_t d, int64_t f, int k) {
    if (good) return;
    if (failures++ < 20) fprintf(stderr, "FAIL %s: %ld x %ld x %ld, form %d\n", what, (long)t, (long)d, (long)f, k);
}

int main() {
    const int64_t ds[] = {1, 8, 15, 64, 65, 255, 1000, 1024, 1040, 2048, 4096, 8192, 20279, 28672, 65535, dion::kWidthMax};
    const int64_t fs[] = {1, 8, 63, 64, 75, 513, 1013, 1024, 1040, 4096, 5632, 28672, 65537, dion::kHiddenMax};
    for (int64_t t = 0; t <= 65; ++t)
        for (int64_t d : ds)
            for (int64_t f : fs)
                for (int k = 0; k < 16; ++k) {
                    dion::FfnPlan p;
                    const int bf16 = k & 1, x8 = k >> 1 & 1, g = k >> 2 & 1, saved = k >> 3;
                    if ((!g && saved) || !dion::make_ffn_plan(t, d, f, bf16, x8, g, saved, &p) || !p.few) continue;
                    ++plans;
                    const int64_t n = t < 1 ? 1 : t;
                    const size_t sums = p.total - p.acc;
                    // reductions over k: a slice of `unit` at least; sums of `cols` columns
                    auto slices = [&](const char* what, int s, int64_t k_, int64_t unit, int64_t cols, bool joined) {
                        check(s >= 1 && (s == 1 || s * unit <= k_), what, t, d, f, k);
                        check((s == 1 && !joined) || (size_t)(s * n * cols * 4) <= sums, what, t, d, f, k);
                    };
                    if (!saved) slices("a, b", p.fgu, d, 512, 2 * p.fk, false);
                    if (!g) slices("Y", p.fy, f, 512, p.dk, false);
                    if (g) {   // (these are always joined; a group of 16 k may be ragged)
                        slices("du", p.fdu, (d + 15) / 16, 16, p.fk, true);
                        slices("dX", p.fdx, (f + 15) / 16 * 2, 16, p.dk, true);
                    }
                    // u | dab | gate | up | sums, in this order
                    size_t at = 0;
                    auto region = [&](const char* what, size_t off, int64_t bytes) {
                        check(off >= at && off % 256 == 0, what, t, d, f, k);
                        at = off + (size_t)bytes;
                    };
                    region("u", p.u, n * p.fk * 4);   // fp32, or two bf16 parts
                    if (g) {
                        region("da, db", p.dab, 2 * n * p.fk * 4);
                        if (!saved) {
                            region("gate", p.gate, n * f * 4);
                            region("up", p.up, n * f * 4);
                        }
                    }
                    region("sums", p.acc, 0);
                    check(p.total >= at, "total", t, d, f, k);
                }
    if (failures) return 1;
    printf("all %d plans as expected\n", plans);
    return plans > 10000 ? 0 : 2;
}
