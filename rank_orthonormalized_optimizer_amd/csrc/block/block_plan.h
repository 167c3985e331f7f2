// Host-side sizes and launch entry points of the residual blocks' operators (arguments validated in
// block_api.cpp).  Every run_* returns a hipError_t value.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "vocab/vocab_plan.h"

namespace dion {

constexpr int64_t kHiddenMax = (int64_t)1 << 17;

// The mask of dropout: an element is kept where its word is at least `threshold`, and multiplied by `scale`.
struct Mask {
    const int64_t* seed;
    int64_t site;
    uint32_t threshold;
    double scale;
    int on;
};

struct DropoutArgs {
    const void* x;
    const void* residual;
    void* out;
    int64_t n;
    Mask mask;
    int x_bf16, out_bf16;
};
int run_dropout(const DropoutArgs& a, void* stream);

struct NormArgs {
    const void* x;
    const void* residual;
    const void* w;
    void* h;
    void* y;
    float* scale;
    float* rstd;
    int64_t rows;
    int d;
    double eps;
    Mask mask;
    int x_bf16, s_bf16, w_bf16, y_bf16;   // (scale is given: y in 8 bits)
};
int run_rms_norm(const NormArgs& a, void* stream);

struct NormGradArgs {
    const void* dy;
    const void* h;
    const void* w;
    const float* rstd;
    const void* dsum;
    void* dh;
    void* dx;
    void* dw;
    float* part;        // [blocks][d] sums of dw, where there are several blocks
    int64_t rows;
    int d;
    Mask mask;
    int y_bf16, s_bf16, w_bf16, dw_bf16, accumulate;
};

// A row is a team's: the threads that hold it in registers, `vecs` vectors of eight elements each.  A wave needs no barrier for
// its sums, and a narrow team leaves a CU more rows at a time.  2^26 elements, norm, to 8 bits and gradient (us): bf16 rows of
// 1024 by a wave 92, 86, 81, by four 100, 182, 95; of 2048 by a wave 94, 94, 75, by four 92, 101, 73; of 8192 by four 96, 95, 75,
// by sixteen 108, 161, 78; of 16384 by four 96, 98, 94, by sixteen 94, 134, 92, in fp32 210, 201, 153 and 199, 198, 198.
// bf16 rows of 1025 to 2048 that go to 8 bits are a wave's too: 16384 rows of 2048 with dropout, calls in a row over buffers that no
// cache holds, by a wave 61, by four 72, of 1536 64 and 69, 32768 rows of 2048 without dropout 93 and 105; in fp32 by a wave 86, by
// four 81, its gradient 111 and 104.
struct NormPlan {
    int team, vecs;
    int64_t per_block;   // rows of a workgroup at a time
    int64_t blocks;      // gradient: workgroups, which stride over the rows and leave one partial dw each
    size_t total;        // bytes of the partial sums
};

// wave: of bf16 rows that go to 8 bits, which a wave holds twice as much of
inline NormPlan make_norm_plan(int64_t rows, int64_t width, bool wave = false) {
    NormPlan p{};
    const int64_t v = ceil_div64(width, 8);   // vectors of a row
    p.team = v <= (wave ? 256 : 128) ? 64 : v <= 2048 ? 256 : 1024;
    p.vecs = 1;
    while ((int64_t)p.team * p.vecs < v) p.vecs *= 2;
    p.per_block = p.team == 64 ? 4 : 1;
    const int64_t most = p.team == 1024 ? kCUs : kCUs * 4, all = ceil_div64(rows, p.per_block);
    p.blocks = all < most ? all : most;
    p.total = p.blocks > 1 ? align256((size_t)(p.blocks * width * 4)) : 0;
    return p;
}
int run_rms_norm_grad(const NormGradArgs& a, const NormPlan& p, void* stream);

// Layout of a feed-forward call.  bf16 operands are one part each, in place where rows are a multiple of 64 elements, else
// in packed planes with rows of a multiple of 64 and zeros behind the matrix.  fp32 operands always go through planes: two
// fp16 ones (scaled rows) for a, b and du, three bf16 ones for the other products.  Wg's and Wu's planes are one matrix of 2 fk
// rows, da and db one of 2 fk columns.
// How a product's tiles go over the chip: `full` of them whole, the `rem` others cut into slices of the reduction.
struct Cut {
    int full, rem, slices;
    int k, k_per;   // the reduction's length, and a slice's, multiples of 64
};
struct Product {
    int tile;       // TILE_*
    Cut cut;
    size_t acc;     // bytes of the slices' sums
};
struct FfnPlan {
    int64_t t, d, f, dk, fk;
    bool few;                          // few rows: the weights are read in place (run_ffn_few; fp32 gradients: run_ffn_few_grad)
    bool mid;                          // a moderate number of fp32 rows: the weights are read in place (run_mid_*), rows in planes
    int fgu, fy, fdu, fdx;             // slices of few rows' reductions: of a and b, Y, du, dX
    int mgu, my, mdu, mdx;             // of a moderate number's
    int parts;                         // of the operands that are not fp16 planes: 1 or 3
    int uparts;                        // of u, da and db: 1, 2 or 3
    bool xpack, wpack, dpack, ypack;   // X, Wg and Wu, Wd, dY go through planes in the workspace
    Product gu, y, du, dx, dgu, dd, dw;   // (dw: dgu and dd at once)
    size_t x, w, wd, dy;               // their planes
    size_t x16, w16, wd16, dy16;       // fp16 planes
    size_t xinv, winv, dinv, yinv;     // inverse scales of their rows
    size_t u, dab, gate, up, acc;
    size_t total;
};
// fp32: inverse scales are read for whole tiles
inline int64_t scale_rows(int64_t rows) { return ceil_div64(rows, 256) * 256 + 256; }

// Times in microseconds of a tile's slab of 64 k and of its start and epilogue, and the workgroups that a CU holds; `busy` is
// how many of the chip's CUs have one.  Measured over seven shapes from 64 x 2048 x 5632 to 2000 x 2048 x 5632, each tile
// and 1, 2, 4 and 8 slices: a slab of 256 x 256 takes 1.1 where few CUs work and 1.6 where all do, one of 128 x 128 0.67 alone on
// its CU and 1.2 beside another, one of 64 x 64 0.34.
struct TileCost {
    int tile;
    double few, all, ends;
    int64_t per_cu;
    double slab(int64_t workgroups) const {
        if (per_cu > 1) return workgroups > kCUs ? all : few;
        return few + (all - few) * (workgroups < kCUs ? (double)workgroups / kCUs : 1.0);
    }
};
constexpr TileCost kTileCosts[] = {{TILE_256, 1.08, 1.6, 9.0, 1}, {TILE_128, 0.67, 1.2, 6.0, 2}, {TILE_64, 0.3, 0.34, 5.0, 1}};

// The tile and the cut of least estimated time for one product of m x n, or two (whose tiles are counted together).
// narrow: few rows go in tiles of 128 x 32.
inline Product pick_product(int64_t m, int64_t n, int64_t k, int64_t terms, bool narrow, int64_t m2 = 0, int64_t n2 = 0) {
    Product best{};
    double least = 1e300;
    const int64_t slabs = ceil_div64(k, 64);
    for (const TileCost& c : kTileCosts) {
        const TileCost t = narrow && n <= 32 ? TileCost{TILE_32, 0.3, 0.34, 4.0, 1} : c;
        const int64_t slots = kCUs * t.per_cu, all = tiles(m, n, t.tile) + (m2 ? tiles(m2, n2, t.tile) : 0);
        const int64_t rounds = all / slots, rest = all % slots;
        const double bytes = 4.0 * (double)(tile_m(t.tile) * tile_n(t.tile));
        for (int64_t s = 1; s <= 16 && (s == 1 || (s <= slabs && rest * s <= slots)); ++s) {
            const int64_t per = ceil_div64(slabs, s);
            if (s > 1 && ceil_div64(slabs, per) != s) continue;   // a slice without any k
            double time = (double)rounds * ((double)(slabs * terms) * t.slab(slots) + t.ends);
            if (rest) time += (double)(per * terms) * t.slab(rest * s) + t.ends;
            if (rest && s > 1) time += 4.5 + (double)(rest * s) * bytes * 0.4e-6;   // a launch, sums written and read
            if (time >= least) continue;
            least = time;
            best.tile = t.tile;
            best.cut = Cut{(int)(s > 1 ? all - rest : all), (int)(s > 1 ? rest : 0), (int)(s > 1 ? s : 0), (int)(slabs * 64), (int)(per * 64)};
            best.acc = s > 1 ? (size_t)(rest * s) * (size_t)bytes : 0;
        }
    }
    return best;
}

// Forward calls of so few rows read weights and rows in place (run_ffn_few), more go through tiles.  That way and by tiles: bf16
// 2048 x 5632 1 row 24 us and 28, 4 rows 26 and 28, 16 rows 32 and 29, 8192 x 8192 4 rows 72 and 99, 16 rows 90 and 100; fp32
// 2048 x 5632 1 row 45 and 110, 32 rows 79 and 111, 48 rows 120 and 123, 64 rows 139 and 124, 8192 x 8192 48 rows 351 and 652.
constexpr int64_t kFewRows = 8, kFewRowsF32 = 64;
// Slices of the reduction over k for an output of `cols` columns, 16 to a workgroup: where they are fewer than a quarter of the
// CUs and k is long, a workgroup for every CU (forward, fp32 4 x 65 x 20279: 60 -> 18 us, 22 x 4001 x 75: 40 -> 18).  More columns
// are left uncut, though a quarter of the CUs has little to stream with: width 1024, whose 64 blocks are cut, and 1040, whose 65 are
// not, hidden 28672: one bf16 row 40 us and 67, 16 fp32 rows 96 and 194; hidden 5632: 16 and 19, 32 and 45.
inline int64_t few_gate_slices(int64_t cols, int64_t k) {
    const int64_t blocks = ceil_div64(cols, 16), most = k / 512;
    if (blocks * 4 > kCUs || most < 2) return 1;
    return kCUs / blocks < most ? kCUs / blocks : most;
}
constexpr int64_t kFewGradRowsF32 = 64;
// Slices of the reduction over k (of `matrices` in a row) for an output of `cols` columns, 64 to a workgroup: two workgroups
// for every CU, if each of its eight waves has two groups of 16 k.
inline int64_t few_slices(int64_t cols, int64_t k, int64_t matrices) {
    const int64_t blocks = ceil_div64(cols, 64), most = ceil_div64(k, 16) * matrices / 16;
    int64_t s = 2 * kCUs / blocks;
    if (s > most) s = most;
    return s < 1 ? 1 : s;
}

// fp32 calls that read the weights in place beside planes of the rows (run_mid_*).  That way, and few rows' way or by tiles,
// width x hidden (us): forward, 2048 x 5632 16 rows 64 and 60, 24 rows 64 and 87, 64 rows 71 and 146, 128 rows 102 and 148, 512 rows
// 232 and 242; 1024 x 4096 64 rows 45 and 37, 96 rows 53 and 64, 512 rows 102 and 108; 768 x 2048 96 rows 52 and 41; 8192 x 8192 96
// rows 278 and 683, 640 rows 1657 and 1432.  Gradients, 2048 x 5632 32 rows 121 and 114, 40 rows 124 and 134, 128 rows 188 and 273,
// 512 rows 424 and 496; 1024 x 4096 48 rows 66 and 63, 64 rows 69 and 83; 768 x 2048 128 rows 77 and 75, 256 rows 90 and 101; 1024 x 1024
// 256 rows 82 and 78.
constexpr int64_t kMidRowsF32 = 512;
inline bool mid_rows(int64_t rows, int64_t elements, int for_grad) {   // elements: of a weight matrix
    if (rows > kMidRowsF32) return false;
    if (for_grad) return rows > 64 ? elements >= (3 << 19) : rows > 32 && elements >= (1 << 22);
    return rows > 64 ? elements >= (1 << 22) : rows > 16 && elements >= (1 << 23);
}
// Slices of the reduction's `steps` of 32, four of which are under way, for an output of `cols` columns, `per` to a workgroup:
// a workgroup for every CU.
inline int mid_slices(int64_t rows, int64_t cols, int64_t per, int64_t steps) {
    const int64_t blocks = ceil_div64(cols, per) * ceil_div64(rows, 128), units = ceil_div64(steps, 4);
    int64_t s = kCUs / blocks;
    if (s > units) s = units;
    if (s < 1) s = 1;
    return (int)ceil_div64(units, ceil_div64(units, s));   // (all slices as long as the longest)
}

// bf16 calls of so few rows take two bf16 parts of u, da and db, whose rounding adds as much to the outputs' errors as the
// outputs' own does.  That way and with one part (us): forward, 2048 x 5632 16 rows 28.0 and 26.7, 64 rows 29.7 and 26.7, 8192 x 8192 16
// rows 99.4 and 99.1, 64 rows 107 and 97; gradients, 2048 x 5632 16 rows 63.6 and 55.5, 64 rows 75.2 and 64.0.
constexpr int64_t kTwoPartRows = 64, kTwoPartGradRows = 16;   // (narrow tiles for gradients)

// for_grad: the gradient; saved: gate and up are given to it
inline bool make_ffn_plan(int64_t rows, int64_t width, int64_t hidden, int bf16, int x8, int for_grad, int saved, FfnPlan* p) {
    FfnPlan q{};
    q.t = rows; q.d = width; q.f = hidden;
    q.dk = ceil_div64(width, 64) * 64;
    q.fk = ceil_div64(hidden, 64) * 64;
    q.parts = bf16 ? 1 : 3;
    q.uparts = bf16 ? rows <= (for_grad ? kTwoPartGradRows : kTwoPartRows) ? 2 : 1 : 3;
    q.xpack = !bf16 || x8 || width != q.dk;
    q.wpack = !bf16 || width != q.dk;
    q.dpack = !bf16 || hidden != q.fk;
    q.ypack = !bf16 || width != q.dk;
    const int64_t n = rows < 1 ? 1 : rows, terms = bf16 ? q.uparts : 6, scaled = bf16 ? 1 : 3;
    size_t off = 0, acc = 0;
    auto take = [&](int64_t bytes) { const size_t at = off; off += align256((size_t)bytes); return at; };
    auto plan = [&](Product& r, int64_t m, int64_t n, int64_t k, int64_t t, bool narrow, int64_t m2 = 0, int64_t n2 = 0) {
        r = pick_product(m, n, k, t, narrow, m2, n2);
        if (r.acc > acc) acc = r.acc;
    };
    q.mid = !bf16 && mid_rows(rows, width * hidden, for_grad);
    q.few = !q.mid && rows <= (for_grad ? bf16 ? 0 : kFewGradRowsF32 : bf16 ? kFewRows : kFewRowsF32);
    if (q.few) {
        int64_t sums = 0;
        auto most = [&](int64_t e) { if (e > sums) sums = e; };
        if (!for_grad || !saved) {
            q.fgu = (int)few_gate_slices(hidden, width);
            if (q.fgu > 1) most(q.fgu * 2 * q.fk);
        }
        q.u = take(n * q.fk * 4);   // (fp32, or two bf16 parts)
        if (for_grad) {
            q.dab = take(2 * n * q.fk * 4);
            q.fdu = (int)few_slices(hidden, width, 1);
            q.fdx = (int)few_slices(width, hidden, 2);
            most(q.fdu * q.fk);
            most(q.fdx * q.dk);
            if (!saved) {
                q.gate = take(n * hidden * 4);
                q.up = take(n * hidden * 4);
            }
        } else {
            q.fy = (int)few_gate_slices(width, hidden);
            if (q.fy > 1) most(q.fy * q.dk);
        }
        q.acc = take(sums * n * 4);
        q.total = off;
        *p = q;
        return true;
    }
    const bool forms = !for_grad || !saved;   // a and b are formed
    if (q.mid) {
        int64_t sums = 0;
        auto slice = [&](int64_t cols, int64_t per, int64_t steps, int64_t ld, int64_t outputs) {
            const int s = mid_slices(n, cols, per, steps);
            if (s > 1 && s * ld * outputs > sums) sums = s * ld * outputs;
            return s;
        };
        q.x = take(3 * n * q.dk * 2);
        q.u = take(3 * n * q.fk * 2);
        if (forms) q.mgu = slice(hidden, 128, q.dk / 32, q.fk, 2);
        if (!for_grad) {
            q.my = slice(width, 256, q.fk / 32, q.dk, 1);
        } else {
            if (!saved) {
                q.gate = take(n * hidden * 4);
                q.up = take(n * hidden * 4);
            }
            q.dy = take(3 * n * q.dk * 2);
            q.dab = take(3 * n * 2 * q.fk * 2);
            q.mdu = slice(hidden, 256, q.dk / 32, q.fk, 1);
            q.mdx = slice(width, 256, 2 * q.fk / 32, q.dk, 1);
            plan(q.dgu, width, 2 * q.fk, n, terms, false);
            plan(q.dd, hidden, width, n, terms, false);
            plan(q.dw, width, 2 * q.fk, n, terms, false, hidden, width);
        }
        if (acc < (size_t)(sums * n * 4)) acc = (size_t)(sums * n * 4);
        q.acc = take((int64_t)acc);
        q.total = off;
        *p = q;
        return true;
    }
    if (bf16 ? q.xpack : for_grad) q.x = take(q.parts * n * q.dk * 2);
    if (bf16 ? q.wpack : for_grad) q.w = take(q.parts * 2 * q.fk * q.dk * 2);
    if (bf16 ? q.dpack : !for_grad) q.wd = take(q.parts * width * q.fk * 2);
    if (!bf16 && forms) {
        q.x16 = take(2 * n * q.dk * 2);
        q.w16 = take(2 * 2 * q.fk * q.dk * 2);
        q.xinv = take(scale_rows(n) * 4);
        q.winv = take(2 * scale_rows(q.fk) * 4);
    }
    q.u = take(q.uparts * n * q.fk * 2);
    plan(q.gu, 2 * q.fk, n, width, scaled, true);
    if (!for_grad) {
        plan(q.y, width, n, hidden, terms, true);
    } else {
        if (!saved) {
            q.gate = take(n * hidden * (bf16 ? 2 : 4));
            q.up = take(n * hidden * (bf16 ? 2 : 4));
        }
        if (q.ypack) q.dy = take(q.parts * n * q.dk * 2);
        if (!bf16) {
            q.wd16 = take(2 * width * q.fk * 2);
            q.dy16 = take(2 * n * q.dk * 2);
            q.dinv = take(scale_rows(q.dk) * 4);
            q.yinv = take(scale_rows(n) * 4);
        }
        q.dab = take(q.uparts * n * 2 * q.fk * 2);
        plan(q.du, q.fk, n, width, scaled, true);
        plan(q.dx, width, n, q.wpack ? 2 * q.fk : hidden, q.wpack ? terms : 2 * terms, true);   // (in place: twice the terms, of hidden)
        plan(q.dgu, width, 2 * q.fk, n, terms, false);
        plan(q.dd, hidden, width, n, terms, false);
        plan(q.dw, width, 2 * q.fk, n, terms, false, hidden, width);
    }
    q.acc = take((int64_t)acc);
    q.total = off;
    *p = q;
    return off < ((size_t)1 << 46);
}

struct FfnArgs {
    const void* X;
    const float* x_scale;   // X in 8 bits, or null
    const void* Wg;
    const void* Wu;
    const void* Wd;
    void* Y;                // forward
    void* gate;             // forward: written, or null.  Gradient: read, or null: formed again
    void* up;
    const void* dY;         // gradient
    void* dX;
    void* dWg;
    void* dWu;
    void* dWd;
    int act, bf16, dw_bf16, accumulate;
    int even;               // the form of gate and up, for bf16 operands
};
int run_ffn(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream);
int run_ffn_few(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream);
int run_ffn_few_gate(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream);   // gate and up alone, fp32
int run_ffn_few_grad(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream);
// a and b (gate and up, planes of u), Y, du (planes of da, db and u), dX from the rows' planes
int run_mid_gate(const FfnArgs& a, const FfnPlan& p, bool u, char* ws, void* stream);
int run_mid_out(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream);
int run_mid_du(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream);
int run_mid_dx(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream);
int run_ffn_grad(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream);
// nothing but zeros, in n 16-bit words
int run_zeros(void* out, int64_t n, void* stream);

}  // namespace dion
