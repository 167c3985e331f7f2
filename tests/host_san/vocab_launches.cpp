// The grids of the vocabulary operators' launches over every size that the planners accept: HIP takes fewer than 2^32 threads
// per dimension of a grid, and at most 65535 workgroups in its second.  Built with the sanitizers by
// tests/test_vocab_launches.py; exits nonzero on the first grid outside.
#include <stdint.h>
#include <stdio.h>

#include "dion_vocab.h"
#include "vocab_plan.h"

static int failures = 0;
static int64_t largest = 0;

static void grid(const char* what, int64_t blocks, int64_t threads, int64_t second, const dion::XentPlan& x) {
    if (blocks * threads > largest) largest = blocks * threads;
    if (blocks >= 1 && blocks * threads < ((int64_t)1 << 32) && second <= 65535) return;
    fprintf(stderr, "%s of %ld x %ld x %ld: %ld workgroups of %ld threads, %ld in the second dimension\n", what, (long)x.n, (long)x.v,
            (long)x.d, (long)blocks, (long)threads, (long)second);
    ++failures;
}

int main() {
    using dion::ceil_div64;
    const int64_t lim = DION_VOCAB_MAX_TOKENS;
    const int64_t ts[] = {1, 2, 16, 17, 33, 128, 129, 257, 4096, 16384, 16385, 65536, 131073, lim / 2, lim};
    const int64_t vs[] = {1, 255, 1000, 1100, 32000, 131072, 1000003, dion::kVocabMax};
    const int64_t ds[] = {1, 8, 64, 255, 1024, 4096, 16384, 32768, 65535, dion::kWidthMax};
    for (int64_t t : ts)
        for (int64_t v : vs)
            for (int64_t d : ds) {
                for (int k = 0; k < 8; ++k) {
                    dion::XentPlan x;
                    if (!dion::make_xent_plan(t, v, d, k & 1, (k >> 1) & 1, k >> 2, &x)) continue;
                    grid("gathering", ceil_div64(t, 8), 512, 1, x);
                    grid("planes", ceil_div64(x.piece, 4), 256, 1, x);
                    grid("loss", ceil_div64(t, 4), 256, 1, x);
                    if (x.split_z > 1) grid("sliced logits", t, 256, t, x);
                    if (!(k >> 2)) continue;
                    grid("dH", dion::join_blocks(t, x.dp, x.split_h), 256, 1, x);
                    grid("dW", dion::join_blocks(x.piece, x.dp, x.split_w), 256, 1, x);
                }
                // lookup and table gradient: at least one token or chunk a workgroup, at most 256 elements of a row in the first
                // dimension's share
                dion::XentPlan x{};
                x.n = t; x.v = v; x.d = d;
                dion::EmbedGradPlan e;
                dion::make_embed_grad_plan(t, v, d, &e);
                grid("lookup", t, 256, ceil_div64(ceil_div64(d, 4), 256), x);
                grid("table sums", e.nchunk, 256, ceil_div64(ceil_div64(d, 4), 32), x);
                grid("sorting", e.sort_blocks ? e.sort_blocks + 4 * 2048 : ceil_div64(t, 64) + 2048, 1024, 1, x);
            }
    if (failures) return 1;
    printf("every grid fits, the largest has %ld threads\n", (long)largest);
    return 0;
}
