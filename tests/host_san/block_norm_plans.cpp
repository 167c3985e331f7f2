// Plans of the norm over every width, with the rows that a wave holds up to 2048 elements of (bf16 to 8 bits) and without:
// a team holds its row, and is one that the kernels are built for.  Built with the sanitizers by tests/test_block_norm_plans.py.
#include <stdint.h>
#include <stdio.h>

#include "block/block_plan.h"

int main() {
    int failures = 0;
    for (int wave = 0; wave < 2; ++wave)
        for (int64_t d = 1; d <= dion::kWidthMax; ++d) {
            const dion::NormPlan p = dion::make_norm_plan(1000, d, wave);
            const bool holds = (int64_t)p.team * p.vecs * 8 >= d && (p.vecs == 1 || (int64_t)p.team * p.vecs * 4 < d);
            const bool built = p.team == 64 ? p.vecs <= 2 || (wave && p.vecs == 4) : p.team == 256 ? p.vecs <= 8 : p.team == 1024 && p.vecs >= 4;
            const bool rule = (p.team == 64) == (d <= (wave ? 2048 : 1024)) && p.per_block == (p.team == 64 ? 4 : 1);
            if ((!holds || !built || !rule || p.vecs > 8) && failures++ < 10) fprintf(stderr, "FAIL %ld, wave %d: %d x %d\n", (long)d, wave, p.team, p.vecs);
        }
    if (failures) return 1;
    printf("all plans as expected\n");
    return 0;
}
