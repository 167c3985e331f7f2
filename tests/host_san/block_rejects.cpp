// Drives the host validation of the residual blocks' operators (csrc/block/block_api.cpp) through refused, empty and
// accepted calls with fake device addresses (never dereferenced), and the planners over every size that is accepted: their
// grids fit HIP's limits (fewer than 2^32 threads per dimension), their slices cover the reductions, their workspaces hold
// what they say.  The device entry points are stand-ins that count their calls and return a fixed hipError_t-like value.
// Built with the sanitizers by tests/test_block_host_sanitizers.py; exits nonzero on the first unexpected value.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "block/block_plan.h"
#include "dion_block.h"

static int calls = 0;
constexpr int kError = 7;
namespace dion {
int run_dropout(const DropoutArgs&, void*) { ++calls; return kError; }
int run_rms_norm(const NormArgs&, void*) { ++calls; return kError; }
int run_rms_norm_grad(const NormGradArgs&, const NormPlan&, void*) { ++calls; return kError; }
int run_ffn(const FfnArgs&, const FfnPlan&, char*, void*) { ++calls; return kError; }
int run_ffn_grad(const FfnArgs&, const FfnPlan&, char*, void*) { ++calls; return kError; }
int run_zeros(void*, int64_t, void*) { ++calls; return 0; }
}  // namespace dion

static int failures = 0;
static void expect(const char* what, long got, long want) {
    if (got != want) {
        fprintf(stderr, "FAIL %s: got %ld, want %ld\n", what, got, want);
        ++failures;
    }
}
static char* P(int gib, uintptr_t off = 0) { return (char*)(((uintptr_t)1 << 40) + ((uintptr_t)gib << 30) + off); }

static void product(const char* what, const dion::Product& r, int64_t m, int64_t n, int64_t k, int64_t m2, int64_t n2, size_t acc) {
    const int64_t all = dion::tiles(m, n, r.tile) + (m2 ? dion::tiles(m2, n2, r.tile) : 0);
    const dion::Cut& c = r.cut;
    const int64_t parts = r.tile == dion::TILE_256 ? 8 * 4 * 512 : r.tile == dion::TILE_128 ? 4 * 4 * 256 : 2 * 2 * 256;   // a tile's sums, by fours
    const bool covered = c.full + c.rem == all && c.k >= k && c.k < k + 64 && c.k % 64 == 0 && c.k_per % 64 == 0 &&
                         (c.rem == 0 ? c.slices == 0
                                     : c.slices > 1 && (int64_t)c.k_per * c.slices >= c.k && (int64_t)c.k_per * (c.slices - 1) < c.k);
    const bool held = r.acc >= (size_t)c.rem * c.slices * parts * 16 && r.acc <= acc;
    const int64_t most = c.full > (int64_t)c.rem * c.slices ? c.full : (int64_t)c.rem * c.slices;
    if (!covered || !held || most < 1 || most >= (int64_t)1 << 31 || (int64_t)c.rem * 4 * 512 >= (int64_t)1 << 32) {
        fprintf(stderr, "FAIL %s %ld x %ld x %ld: tile %d full %d rem %d slices %d k_per %d\n", what, (long)m, (long)n, (long)k, r.tile, c.full,
                c.rem, c.slices, c.k_per);
        ++failures;
    }
}

int main() {
    const size_t ws = (size_t)1 << 30;
    auto drop = [&](void* x, void* out, int64_t n, double p) {
        return dion_dropout(x, nullptr, out, n, p, (int64_t*)P(9), -1, DION_F32, DION_BF16, nullptr);
    };
    expect("dropout", drop(P(0), P(1), 10, 0.5), DION_ERR_HIP - kError);
    expect("dropout nan", drop(P(0), P(1), 10, NAN), DION_ERR_HYPER);
    expect("dropout empty", drop(nullptr, nullptr, 0, 0.5), DION_OK);
    expect("dropout itself", drop(P(0), P(0), 10, 0.5), DION_ERR_OVERLAP);
    auto norm = [&](void* x, void* r, void* h, void* y, int64_t t, int64_t d) {
        return dion_rms_norm(x, r, P(2), h, y, nullptr, nullptr, t, d, 1e-6, 0.0, nullptr, 0, DION_BF16, DION_F32, DION_F32, DION_BF16, nullptr);
    };
    expect("norm", norm(P(0), P(1), P(3), P(4), 10, 100), DION_ERR_HIP - kError);
    expect("norm in place", norm(P(0), P(1), P(1), P(4), 10, 100), DION_ERR_HIP - kError);
    expect("norm onto x", norm(P(0), P(1), P(0), P(4), 10, 100), DION_ERR_OVERLAP);
    expect("norm null", norm(P(0), P(1), P(3), nullptr, 10, 100), DION_ERR_NULL);
    expect("norm largest", norm(P(0), nullptr, nullptr, P(512), DION_BLOCK_MAX_ROWS, 1 << 16), DION_ERR_HIP - kError);
    auto grad = [&](void* dsum, void* dh, int64_t t, int64_t d, size_t n) {
        return dion_rms_norm_grad(P(0), P(10), P(20), (float*)P(21), dsum, dh, nullptr, P(22), t, d, 0.0, nullptr, 0, DION_F32, DION_F32,
                                  DION_F32, DION_F32, 0, P(23), n, nullptr);
    };
    expect("norm gradient", grad(P(30), P(40), 1000, 100, ws), DION_ERR_HIP - kError);
    expect("norm gradient in place", grad(P(30), P(30), 1000, 100, ws), DION_ERR_HIP - kError);
    expect("norm gradient workspace", grad(P(30), P(40), 1000, 100, 1000), DION_ERR_WORKSPACE);
    expect("norm gradient of nothing", grad(P(30), P(40), 0, 100, 0), DION_ERR_HIP - kError);   // dw is zero
    auto ffn = [&](void* Y, int64_t t, int64_t d, int64_t f, size_t n) {
        return dion_gated_ffn(P(0), nullptr, P(1), P(2), P(3), nullptr, nullptr, Y, t, d, f, DION_GELU, DION_BF16, DION_BF16, P(20), n, nullptr);
    };
    expect("ffn", ffn(P(4), 100, 24, 40, ws), DION_ERR_HIP - kError);
    expect("ffn workspace", ffn(P(4), 100, 24, 40, 10), DION_ERR_WORKSPACE);
    expect("ffn onto X", ffn(P(0), 100, 24, 40, ws), DION_ERR_OVERLAP);
    const int before = calls;
    expect("ffn gradient of nothing", dion_gated_ffn_grad(nullptr, nullptr, P(1), P(2), P(3), nullptr, nullptr, nullptr, nullptr, P(4), P(5), P(6),
                                                          0, 24, 40, DION_SILU, DION_F32, DION_F32, DION_F32, 0, nullptr, 0, nullptr), DION_OK);
    expect("its zeros", calls - before, 3);

    const int64_t lim = DION_BLOCK_MAX_ROWS;
    const int64_t ts[] = {1, 2, 8, 9, 16, 17, 33, 48, 49, 128, 257, 1000, 4096, 8192, 65536, 131073, lim};
    const int64_t ds[] = {1, 8, 64, 255, 1000, 2048, 8192, 28672, 65535, dion::kWidthMax};
    const int64_t fs[] = {1, 63, 64, 1013, 5632, 28672, dion::kHiddenMax};
    for (int64_t t : ts)
        for (int64_t d : ds) {
            const dion::NormPlan np = dion::make_norm_plan(t, d);
            if (np.team * np.vecs * 8 < d || np.blocks < 1 || np.blocks * 1024 >= (int64_t)1 << 32 || np.blocks > 1024 || t * 1024 >= (int64_t)1 << 32 ||
                (np.blocks > 1 && np.total < (size_t)(np.blocks * d * 4))) {
                fprintf(stderr, "FAIL norm plan %ld x %ld\n", (long)t, (long)d);
                ++failures;
            }
            for (int64_t f : fs)
                for (int k = 0; k < 16; ++k) {
                    dion::FfnPlan p;
                    const int bf16 = k & 1, x8 = k >> 1 & 1, g = k >> 2 & 1, saved = k >> 3;
                    if (!g && saved) continue;
                    if (!dion::make_ffn_plan(t, d, f, bf16, x8, g, saved, &p)) continue;
                    if (p.few) continue;
                    const int64_t rows = 2 * p.fk + 2 * d + 2 * t;   // of the packing, four to a workgroup
                    if ((rows / 4 + 5) * 256 >= (int64_t)1 << 32) { fprintf(stderr, "FAIL packing\n"); ++failures; }
                    const size_t acc = p.total - p.acc;
                    if (p.mid) {
                        // slices: of the reductions, none without a step; their sums; offsets in the rows' planes in 32 bits
                        auto slices = [&](const char* what, int n, int64_t steps, int64_t sums, int64_t planes) {
                            if (n < 1 || n > (steps + 3) / 4 || (n > 1 && (size_t)(n * sums * t * 4) > acc) || planes * t * 2 >= (int64_t)1 << 31) {
                                fprintf(stderr, "FAIL slices of %s: %ld x %ld x %ld\n", what, (long)t, (long)d, (long)f);
                                ++failures;
                            }
                        };
                        if (!saved) slices("a, b", p.mgu, p.dk / 32, 2 * p.fk, 3 * p.dk);
                        if (!g) slices("Y", p.my, p.fk / 32, p.dk, 3 * p.fk);
                        if (g) {
                            slices("du", p.mdu, p.dk / 32, p.fk, 3 * p.dk);
                            slices("dX", p.mdx, p.fk / 16, p.dk, 6 * p.fk);
                            product("dWg, dWu", p.dgu, d, 2 * p.fk, t, 0, 0, acc);
                            product("dWd", p.dd, f, d, t, 0, 0, acc);
                            product("dW", p.dw, d, 2 * p.fk, t, f, d, acc);
                        }
                        continue;
                    }
                    product("a, b", p.gu, 2 * p.fk, t, d, 0, 0, acc);
                    if (!g) {
                        product("Y", p.y, d, t, f, 0, 0, acc);
                    } else {
                        product("du", p.du, p.fk, t, d, 0, 0, acc);
                        product("dX", p.dx, d, t, p.wpack ? 2 * p.fk : f, 0, 0, acc);
                        product("dWg, dWu", p.dgu, d, 2 * p.fk, t, 0, 0, acc);
                        product("dWd", p.dd, f, d, t, 0, 0, acc);
                        product("dW", p.dw, d, 2 * p.fk, t, f, d, acc);
                        if (p.dgu.tile == dion::TILE_32 || p.dd.tile == dion::TILE_32 || p.dw.tile == dion::TILE_32) {
                            fprintf(stderr, "FAIL narrow tiles for a weight's gradient\n");
                            ++failures;
                        }
                    }
                }
        }
    if (failures) return 1;
    printf("all cases as expected\n");
    return 0;
}
