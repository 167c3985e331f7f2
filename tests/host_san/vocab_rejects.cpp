// Drives the host validation of the vocabulary operators (csrc/vocab/vocab_api.cpp) through refused, empty and accepted
// calls with fake device addresses (never dereferenced), and the workspace planners over a range of sizes.  The device
// entry points are stand-ins that count their calls and return a fixed hipError_t-like value.  Built with the sanitizers
// by tests/test_vocab_host_sanitizers.py; exits nonzero on the first unexpected status.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "dion_vocab.h"
#include "vocab_plan.h"

static int calls = 0;
constexpr int kError = 7;
namespace dion {
int run_embedding(const EmbedArgs&, void*) { ++calls; return kError; }
int run_embedding_grad(const EmbedArgs&, const EmbedGradPlan&, char*, void*) { ++calls; return kError; }
int run_xent(const XentArgs&, const XentPlan&, char*, void*) { ++calls; return kError; }
int run_xent_grad(const XentArgs&, const XentPlan&, char*, void*) { ++calls; return kError; }
}  // namespace dion

static int failures = 0;
static void expect(const char* what, long got, long want) {
    if (got != want) {
        fprintf(stderr, "FAIL %s: got %ld, want %ld\n", what, got, want);
        ++failures;
    }
}

static char* P(int gib, uintptr_t off = 0) { return (char*)(((uintptr_t)1 << 40) + ((uintptr_t)gib << 30) + off); }

int main() {
    const size_t ws = (size_t)4 << 30;
    const int64_t lim = DION_VOCAB_MAX_TOKENS;
    auto look = [&](void* ids, void* W, void* out, int64_t t, int64_t v, int64_t d, float s) {
        return dion_embedding(ids, W, out, t, v, d, s, DION_I64, DION_BF16, DION_F32, nullptr);
    };
    expect("lookup", look(P(0), P(1), P(2), 10, 100, 24, 1.f), DION_ERR_HIP - kError);
    expect("lookup nan", look(P(0), P(1), P(2), 10, 100, 24, NAN), DION_ERR_HYPER);
    expect("lookup empty", look(nullptr, nullptr, nullptr, 0, 100, 24, 1.f), DION_OK);
    expect("lookup null", look(P(0), nullptr, P(2), 10, 100, 24, 1.f), DION_ERR_NULL);
    expect("lookup tokens", look(P(0), P(1), P(2), lim + 1, 100, 24, 1.f), DION_ERR_SHAPE);
    expect("lookup align", look(P(0, 4), P(1), P(2), 10, 100, 24, 1.f), DION_ERR_ALIGN);
    expect("lookup overlap", look(P(0), P(1), P(1, 16), 10, 100, 24, 1.f), DION_ERR_OVERLAP);
    expect("lookup largest", look(P(0), P(1), P(1000000), lim, ((int64_t)1 << 24) - 1, 1 << 16, 1.f), DION_ERR_HIP - kError);
    auto table = [&](void* dY, void* dW, int64_t t, int64_t v, int acc, void* w, size_t n) {
        return dion_embedding_grad(P(0), dY, dW, t, v, 24, 1.f, -1, DION_I32, DION_F32, DION_BF16, acc, w, n, nullptr);
    };
    expect("table", table(P(1), P(2), 10, 100, 0, P(3), ws), DION_ERR_HIP - kError);
    expect("table empty", table(nullptr, nullptr, 0, 100, 1, nullptr, 0), DION_OK);
    expect("table of nothing", table(nullptr, P(2), 0, 100, 0, nullptr, 0), DION_ERR_HIP - kError);
    expect("table option", table(P(1), P(2), 10, 100, 2, P(3), ws), DION_ERR_OPTION);
    expect("table small workspace", table(P(1), P(2), 10, 100, 0, P(3), 100), DION_ERR_WORKSPACE);
    expect("table overlap", table(P(2), P(2), 10, 100, 0, P(3), ws), DION_ERR_OVERLAP);
    auto loss = [&](void* H, float* l, int64_t t, int64_t v, int64_t d, void* w, size_t n) {
        return dion_linear_xent(H, P(1), P(2), l, (float*)P(4), t, v, d, -100, DION_I64, DION_F32, w, n, nullptr);
    };
    expect("loss", loss(P(0), (float*)P(3), 10, 100, 24, P(5), ws), DION_ERR_HIP - kError);
    expect("loss empty", loss(nullptr, nullptr, 0, 100, 24, nullptr, 0), DION_OK);
    expect("loss workspace", loss(P(0), (float*)P(3), 10, 100, 24, P(5), 10), DION_ERR_WORKSPACE);
    expect("loss overlap", loss(P(0), (float*)P(0), 10, 100, 24, P(5), ws), DION_ERR_OVERLAP);
    expect("loss width", loss(P(0), (float*)P(3), 10, 100, 0, P(5), ws), DION_ERR_SHAPE);
    auto grad = [&](int64_t gn, void* dH, void* dW, int64_t t, int acc, size_t n) {
        return dion_linear_xent_grad(P(0), P(1), P(2), (float*)P(3), (float*)P(4), gn, dH, dW, t, 100, 24, -100, DION_I64,
                                     DION_BF16, DION_F32, acc, P(7), n, nullptr);
    };
    expect("grad", grad(1, P(5), P(6), 10, 0, ws), DION_ERR_HIP - kError);
    expect("grad dH", grad(10, P(5), nullptr, 10, 1, ws), DION_ERR_HIP - kError);
    expect("grad dW", grad(10, nullptr, P(6), 10, 1, ws), DION_ERR_HIP - kError);
    expect("grad none", grad(1, nullptr, nullptr, 10, 0, ws), DION_ERR_NULL);
    expect("grad count", grad(3, P(5), P(6), 10, 0, ws), DION_ERR_SHAPE);
    expect("grad empty", grad(0, P(5), nullptr, 0, 0, 0), DION_OK);
    expect("grad of nothing", grad(0, P(5), P(6), 0, 0, ws), DION_ERR_HIP - kError);
    expect("grad workspace", grad(1, P(5), P(6), 10, 0, 0), DION_ERR_WORKSPACE);

    // the planners: every size they are asked for keeps their invariants
    const int64_t ts[] = {0, 1, 2, 31, 32, 33, 64, 192, 193, 255, 256, 257, 4096, 16384, 16385, 65536, 131072, 131073, lim};
    const int64_t vs[] = {1, 2, 255, 256, 257, 5000, 32000, 131072, 1000003, ((int64_t)1 << 24) - 1};
    const int64_t ds[] = {1, 3, 8, 63, 64, 65, 255, 1024, 4096, 65536};
    for (int64_t t : ts)
        for (int64_t v : vs)
            for (int64_t d : ds) {
                dion::EmbedGradPlan e;
                expect("table plan", dion::make_embed_grad_plan(t, v, d, &e), 1);
                expect("chunks cover", e.nchunk * e.chunk >= t && (t == 0 || (e.nchunk - 1) * e.chunk < t) && e.nchunk <= 1024, 1);
                expect("digits cover", (v >> (dion::kDigitBits * e.digits)) == 0, 1);
                expect("sort blocks", e.sort_blocks <= 256, 1);
                for (int k = 0; k < 8; ++k) {
                    dion::XentPlan x;
                    if (!dion::make_xent_plan(t, v, d, k & 1, (k >> 1) & 1, k >> 2, &x)) continue;
                    const int64_t bm = dion::tile_m(x.tile_z);
                    const bool ok = x.piece % 256 == 0 && x.piece * x.pieces >= v && x.piece * (x.pieces - 1) < v &&
                                    x.kp % 64 == 0 && x.kp >= d && x.np % 256 == 0 && x.np >= t && x.nvt * bm >= v &&
                                    (!(k >> 2) || (x.split_h >= 1 && x.split_w >= 1 && x.split_h <= 256 && x.split_w <= 256)) &&
                                    (!x.few || (t <= dion::kFewTokens && !(k & 1))) &&
                                    // slices of the logits: of one piece, none empty, tokens within a grid's second dimension
                                    (x.split_z == 1 || (x.split_z > 1 && x.pieces == 1 && t < 65536 &&
                                                        dion::ceil_div64(x.kp / 64, x.split_z) * (x.split_z - 1) < x.kp / 64));
                    if (!ok) fprintf(stderr, "plan of %ld x %ld x %ld, kind %d\n", (long)t, (long)v, (long)d, k);
                    expect("cross entropy plan", ok, 1);
                }
            }
    if (failures) return 1;
    printf("all cases as expected, %d device calls\n", calls);
    return 0;
}
