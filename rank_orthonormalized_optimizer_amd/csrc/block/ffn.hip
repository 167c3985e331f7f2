// Gated feed-forward block and its gradients.
//
//   a = X Wg^T;  b = X Wu^T;  u = act(a) b;  Y = u Wd^T
//   du = dY Wd;  da = du b act'(a);  db = du act(a);  dX = da Wg + db Wu;  dWg = da^T X;  dWu = db^T X;  dWd = dY^T u
//
// a and b are one product whose tiles take 16 rows of Wg and of Wu in turn, so that a lane holds both for the same elements
// and the epilogue forms u; du's epilogue reads a and b and forms da, db (side by side, one operand of 2 hidden columns)
// and u.  Then dX is one product over both, and so are dWg and dWu.  Every product runs along the contiguous dimension of
// its output in the matrix core's rows, as in cross_entropy.hip.
//
// bf16 operands multiply as they are, in place where rows are a multiple of 64 elements; fp32 operands as three bf16 parts
// in planes in the workspace.  Where the tiles are too few for the chip, the reductions are sliced: the partial sums are
// stored, and a pass over them takes the epilogue's place.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "block_plan.h"
#include "dion_block.h"
#include "rows.hpp"

namespace dion {

namespace {

// ---------------------------------------------------------------------------
// Activations
// ---------------------------------------------------------------------------
// 1 / (1 + exp(-z)), zero below -87.  EXACT: to a few ulp (the rounding of -z log2(e) is carried into the result); else that
// rounding's |z| 2^-24 stays, which is far below bf16's.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z) {
    const float h = z * -1.44269504f;
    float e = __builtin_amdgcn_exp2f(h);
    if constexpr (!EXACT) return __builtin_amdgcn_rcpf(1.f + e);
    const float l = fmaf(z, -1.44269504f, -h) - z * 1.92596299e-8f;   // log2(e) - 1.44269504f
    e = fmaf(e, l * 0.693147181f, e);
    return z < -87.f ? 0.f : 1.f / (1.f + e);
}

// act(a) and its derivative
template <bool EXACT>
__device__ __forceinline__ float activate(int act, float a, float& slope) {
    if (act == DION_SILU) {
        const float r = sigmoid<EXACT>(a);
        slope = r * fmaf(a, 1.f - r, 1.f);
        return a * r;
    }
    // a / (1 + exp(-2 s)) = a (1 + tanh s) / 2 with s = sqrt(2 / pi) (a + 0.044715 a^3), which is past every border at 30
    const float x = fminf(fmaxf(a, -30.f), 30.f), q = x * x;
    const float r = sigmoid<EXACT>(1.59576912f * x * fmaf(0.044715f, q, 1.f));
    slope = fmaf(x * r * (1.f - r), 1.59576912f * fmaf(0.134145f, q, 1.f), r);
    return a * r;
}

// ---------------------------------------------------------------------------
// Planes
// ---------------------------------------------------------------------------
// Rows [rows][d] of a matrix to bf16 planes [PARTS][plane] with `all` rows of kp elements, a wave per row, zeros behind the
// matrix; kind: 0 fp32, 1 bf16, 2 e4m3 with a scale per row.
template <int PARTS>
__global__ __launch_bounds__(256) void planes_kernel(const void* in, const float* scale, int kind, int64_t rows, int64_t all, int d,
                                                     int kp, uint16_t* out, int64_t plane) {
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= all) return;
    const float s = scale && r < rows ? scale[r] : 1.f;
    if (r >= rows) d = 0;
#pragma unroll 4
    for (int c = (threadIdx.x & 63) * 8; c < kp; c += 512) {
        float v[8];
        if (kind == 0) {
            load8<false>(in, r * d, c, d, v);
        } else if (kind == 1) {
            load8<true>(in, r * d, c, d, v);
        } else {
            const uint8_t* p = (const uint8_t*)in + r * d + c;
            uint32_t w[2] = {0, 0};
            if (c + 8 <= d) {
                const u32x2_bytes q = *(const u32x2_bytes*)p;
                w[0] = q[0];
                w[1] = q[1];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < d) w[e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true);
                v[4 * h] = lo[0] * s;
                v[4 * h + 1] = lo[1] * s;
                v[4 * h + 2] = hi[0] * s;
                v[4 * h + 3] = hi[1] * s;
            }
        }
        store8<PARTS>(out, plane, r * kp + c, v);
    }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// The tiles of this workgroup: tm x tn of them times the slices of the reduction; the next tile's loads start before
// epilogue(m0, n0, slice, acc) of this one.
template <class C, class E>
__device__ __forceinline__ void walk_tiles(mm::Product<C>& mul, const mm::Operand& a, const mm::Operand& b, mm::Segments seg, int tm,
                                           int tn, int split, int k, int k_per, E epilogue) {
    Walk walk(tm, tn, split);
    if (walk.done()) return;
    int mt, nt, slice;
    auto start = [&]() {
        walk.tile(mt, nt, slice);
        const int k0 = slice * k_per, k1 = k0 + k_per < k ? k0 + k_per : k;
        mul.start(a, b, mt * C::BM, nt * C::BN, k0, k1, seg);
    };
    start();
    for (;;) {
        const int m0 = mul.m0, n0 = mul.n0, sl = slice;
        typename C::Acc acc = {};
        mul.finish(a, b, acc);
        walk.next();
        const bool more = !walk.done();
        if (more) start();
        epilogue(m0, n0, sl, acc);
        if (!more) return;
    }
}

// Four packed bf16 from four values.
__device__ __forceinline__ void pack4(const float (&v)[4], uint32_t (&w)[2]) {
    w[0] = down16(v[0]) | (down16(v[1]) << 16);
    w[1] = down16(v[2]) | (down16(v[3]) << 16);
}

struct GatedArgs {
    mm::Operand w, x, g;   // Wg and Wu (x), X; du: Wd and dY (g unused)
    mm::Segments seg;
    int64_t rows;
    int f, fk, act;
    int k, k_per, split;
    void* gate;            // [rows][f], or null
    void* up;
    uint16_t* u;           // planes [PARTS][rows][fk], or null (du)
    uint16_t* dab;         // du: planes [PARTS][rows][2 fk], or null
    float* acc;            // slices: [split][rows][2][fk], du: [split][rows][fk]; or null
};

// Columns c .. c + N - 1 (N 4 or 8) of a row of planes.
template <int PARTS, int N>
__device__ __forceinline__ void put_planes(uint16_t* out, int64_t plane, int64_t at, const float (&v)[N]) {
    uint32_t part[N][3];
#pragma unroll
    for (int e = 0; e < N; ++e) split3(v[e], part[e]);
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
        if constexpr (N == 8) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = part[2 * e][q] | (part[2 * e + 1][q] << 16);
            *(u32x4*)(out + q * plane + at) = w;
        } else {
            *(u32x2*)(out + q * plane + at) = u32x2{part[0][q] | (part[1][q] << 16), part[2][q] | (part[3][q] << 16)};
        }
    }
}

// The eight values of two blocks of four as their lane quarter holds them after the trade: trade() for fp32 values.
__device__ __forceinline__ void trade8(const float (&lo)[4], const float (&hi)[4], float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(lo[e]), __float_as_uint(hi[e]), false, false);
        const auto z = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
        v[e] = __uint_as_float(z[0]);
        v[4 + e] = __uint_as_float(z[1]);
    }
}

// u of eight columns from a and b; gate and up are kept where asked for.
template <int PARTS>
__device__ __forceinline__ void gated8(const GatedArgs& g, int64_t n, int c, float (&a)[8], float (&b)[8]) {
    if (g.gate) {
        put8<PARTS == 1>(g.gate, n * g.f, c, g.f, a);
        put8<PARTS == 1>(g.up, n * g.f, c, g.f, b);
    }
    if (!g.u) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float slope;
        a[e] = c + e < g.f ? activate<PARTS != 1>(g.act, a[e], slope) * b[e] : 0.f;
    }
    put_planes<PARTS>(g.u, g.rows * g.fk, n * g.fk + c, a);
}

// da, db and u of eight columns from du.
template <int PARTS>
__device__ __forceinline__ void dgated8(const GatedArgs& g, int64_t n, int c, const float (&du)[8], const Raw8<PARTS == 1>& a,
                                        const Raw8<PARTS == 1>& b) {
    float da[8], db[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // (a and b are zero behind column f, and du may be anything there)
        float slope;
        const float be = b.get(e), v = activate<PARTS != 1>(g.act, a.get(e), slope), d = c + e < g.f ? du[e] : 0.f;
        da[e] = d * be * slope;
        db[e] = d * v;
        u[e] = v * be;
    }
    if (g.dab) {
        put_planes<PARTS>(g.dab, g.rows * 2 * g.fk, n * 2 * g.fk + c, da);
        put_planes<PARTS>(g.dab, g.rows * 2 * g.fk, n * 2 * g.fk + g.fk + c, db);
    }
    if (g.u) put_planes<PARTS>(g.u, g.rows * g.fk, n * g.fk + c, u);
}

template <class C, int PARTS>
__global__ __launch_bounds__(C::THREADS) void gated_kernel(GatedArgs g) {
    __shared__ __attribute__((aligned(1024))) uint16_t lds[C::kLds];
    mm::Product<C> mul(lds);
    const int rows = (int)g.rows, quarter = mul.lane / 16;
    walk_tiles(mul, g.w, g.x, g.seg, (2 * g.fk + C::BM - 1) / C::BM, (rows + C::BN - 1) / C::BN, g.split, g.k, g.k_per,
               [&](int m0, int n0, int slice, typename C::Acc& acc) {
        const int c0 = (m0 + mul.xa) / 2;   // blocks 2 i and 2 i + 1: a and b of columns c0 + 16 i ..
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const int n = n0 + mul.xb + 16 * j + mul.lane % 16;
            if (g.acc) {
#pragma unroll
                for (int i = 0; i < C::MI; ++i) {
                    const int c = c0 + 16 * (i / 2) + 4 * quarter;
                    if (n < rows && c < g.fk) *(f32x4*)(g.acc + ((slice * g.rows + n) * 2 + i % 2) * g.fk + c) = acc[i][j];
                }
                continue;
            }
            if constexpr (C::MI % 4 == 0) {
#pragma unroll
                for (int i = 0; i < C::MI; i += 4) {
                    float v[4][4], a[8], b[8];
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[h][e] = acc[i + h][j][e];
                    trade8(v[0], v[2], a);
                    trade8(v[1], v[3], b);
                    const int c = c0 + 8 * i + 16 * (quarter / 2) + 8 * (quarter % 2);
                    if (n < rows && c < g.fk) gated8<PARTS>(g, n, c, a, b);
                }
            } else {   // one block of 16 columns: two quarters have eight of them
                float v[2][4], zero[4] = {0.f, 0.f, 0.f, 0.f}, a[8], b[8];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[h][e] = acc[h][j][e];
                trade8(v[0], zero, a);
                trade8(v[1], zero, b);
                const int c = c0 + 8 * (quarter % 2);
                if (quarter < 2 && n < rows && c < g.fk) gated8<PARTS>(g, n, c, a, b);
            }
        }
    });
}

template <class C, int PARTS>
__global__ __launch_bounds__(C::THREADS) void dgated_kernel(GatedArgs g) {
    __shared__ __attribute__((aligned(1024))) uint16_t lds[C::kLds];
    mm::Product<C> mul(lds);
    const int rows = (int)g.rows, quarter = mul.lane / 16;
    walk_tiles(mul, g.w, g.x, g.seg, (g.fk + C::BM - 1) / C::BM, (rows + C::BN - 1) / C::BN, g.split, g.k, g.k_per,
               [&](int m0, int n0, int slice, typename C::Acc& acc) {
        const int c0 = m0 + mul.xa;
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const int n = n0 + mul.xb + 16 * j + mul.lane % 16;
            if (g.acc) {
#pragma unroll
                for (int i = 0; i < C::MI; ++i) {
                    const int c = c0 + 16 * i + 4 * quarter;
                    if (n < rows && c < g.fk) *(f32x4*)(g.acc + (slice * g.rows + n) * g.fk + c) = acc[i][j];
                }
                continue;
            }
            Raw8<PARTS == 1> a[C::MI / 2], b[C::MI / 2];
#pragma unroll
            for (int i = 0; i < C::MI; i += 2) {
                const int c = c0 + 16 * i + 16 * (quarter / 2) + 8 * (quarter % 2);
                if (n < rows && c < g.fk) {
                    a[i / 2].load(g.gate, (int64_t)n * g.f, c, g.f);
                    b[i / 2].load(g.up, (int64_t)n * g.f, c, g.f);
                }
            }
#pragma unroll
            for (int i = 0; i < C::MI; i += 2) {
                float v[2][4], du[8];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[h][e] = acc[i + h][j][e];
                trade8(v[0], v[1], du);
                const int c = c0 + 16 * i + 16 * (quarter / 2) + 8 * (quarter % 2);
                if (n < rows && c < g.fk) dgated8<PARTS>(g, n, c, du, a[i / 2], b[i / 2]);
            }
        }
    });
}

// Eight columns of the slices' sums.
__device__ __forceinline__ void sum8(const float* acc, int64_t stride, int split, float (&v)[8]) {
    f32x4 lo{0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll 4
    for (int s = 0; s < split; ++s) {
        lo += *(const f32x4*)(acc + s * stride);
        hi += *(const f32x4*)(acc + s * stride + 4);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = lo[e]; v[4 + e] = hi[e]; }
}

// The epilogues over sliced sums, eight columns a thread.
template <int PARTS, bool GRAD>
__global__ __launch_bounds__(256) void gated_join_kernel(GatedArgs g) {
    const int64_t per = g.fk / 8, all = g.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t n = i / per;
        const int c = (int)(i - n * per) * 8;
        if constexpr (GRAD) {
            Raw8<PARTS == 1> a, b;
            a.load(g.gate, n * g.f, c, g.f);
            b.load(g.up, n * g.f, c, g.f);
            float du[8];
            sum8(g.acc + n * g.fk + c, g.rows * g.fk, g.split, du);
            dgated8<PARTS>(g, n, c, du, a, b);
        } else {
            float a[8], b[8];
            sum8(g.acc + n * 2 * g.fk + c, g.rows * 2 * g.fk, g.split, a);
            sum8(g.acc + n * 2 * g.fk + g.fk + c, g.rows * 2 * g.fk, g.split, b);
            gated8<PARTS>(g, n, c, a, b);
        }
    }
}

struct OutArgs {
    mm::Operand a, b;
    mm::Segments seg;
    int k, k_per, split;
    int cols;               // of the output
    int64_t rows;           // of the product: the output's, or those of two outputs, the second's from row `second`
    int64_t second, valid;  // and how many rows each has (second: rows where there is one output)
    void* out;
    void* out2;
    int out_bf16, accumulate;
    float* acc;             // [split][rows][cols rounded up to 8], or null
    int ldacc;
};

// where row n goes, or null
__device__ __forceinline__ void* out_row(const OutArgs& a, int64_t n, int64_t& row) {
    const bool two = n >= a.second;
    row = two ? n - a.second : n;
    return row < a.valid && n < a.rows ? (two ? a.out2 : a.out) : nullptr;
}

__device__ __forceinline__ void put_out8(const OutArgs& a, void* out, int64_t row, int c, float (&v)[8]) {
    const int64_t at = row * a.cols;
    if (a.out_bf16) {
        if (a.accumulate) {
            Raw8<true> r;
            r.load(out, at, c, a.cols);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r.get(e);
        }
        put8<true>(out, at, c, a.cols, v);
    } else {
        if (a.accumulate) {
            Raw8<false> r;
            r.load(out, at, c, a.cols);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r.get(e);
        }
        put8<false>(out, at, c, a.cols, v);
    }
}

template <class C>
__global__ __launch_bounds__(C::THREADS) void ffn_out_kernel(OutArgs a) {
    __shared__ __attribute__((aligned(1024))) uint16_t lds[C::kLds];
    mm::Product<C> mul(lds);
    const int rows = (int)a.rows, quarter = mul.lane / 16;
    walk_tiles(mul, a.a, a.b, a.seg, (a.cols + C::BM - 1) / C::BM, (rows + C::BN - 1) / C::BN, a.split, a.k, a.k_per,
               [&](int m0, int n0, int slice, typename C::Acc& acc) {
        const int c0 = m0 + mul.xa;
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const int n = n0 + mul.xb + 16 * j + mul.lane % 16;
            if (a.acc) {
#pragma unroll
                for (int i = 0; i < C::MI; ++i) {
                    const int c = c0 + 16 * i + 4 * quarter;
                    if (n < rows && c < a.ldacc) *(f32x4*)(a.acc + (slice * a.rows + n) * a.ldacc + c) = acc[i][j];
                }
                continue;
            }
            int64_t row;
            void* out = out_row(a, n, row);
#pragma unroll
            for (int i = 0; i < C::MI; i += 2) {
                float v[2][4], o[8];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[h][e] = acc[i + h][j][e];
                trade8(v[0], v[1], o);
                const int c = c0 + 16 * i + 16 * (quarter / 2) + 8 * (quarter % 2);
                if (out && c < a.cols) put_out8(a, out, row, c, o);
            }
        }
    });
}

__global__ __launch_bounds__(256) void out_join_kernel(OutArgs a) {
    const int64_t per = a.ldacc / 8, all = a.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t n = i / per;
        const int c = (int)(i - n * per) * 8;
        int64_t row;
        void* out = out_row(a, n, row);
        if (!out || c >= a.cols) continue;
        float v[8];
        sum8(a.acc + n * a.ldacc + c, a.rows * a.ldacc, a.split, v);
        put_out8(a, out, row, c, v);
    }
}

__global__ __launch_bounds__(256) void zeros_kernel(uint16_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <bool TA, bool TB, bool PAIR> using C256 = mm::Config<256, 256, 2, 4, 2, TA, TB, false, PAIR>;
template <bool TA, bool TB, bool PAIR> using C128 = mm::Config<128, 128, 2, 2, 4, TA, TB, false, PAIR>;
template <bool TA, bool TB, bool PAIR> using C64 = mm::Config<64, 64, 2, 2, 8, TA, TB, false, PAIR>;
template <bool TA, bool TB, bool PAIR> using C32 = mm::Config<128, 32, 4, 1, 4, TA, TB, false, PAIR>;

template <bool TA, bool TB, bool PAIR, class F>
void of_tile(int tile, F f) {
    if (tile == TILE_256) f(C256<TA, TB, PAIR>());
    else if (tile == TILE_128) f(C128<TA, TB, PAIR>());
    else if (tile == TILE_64) f(C64<TA, TB, PAIR>());
    else if constexpr (!TB) f(C32<TA, TB, PAIR>());
    else f(C128<TA, TB, PAIR>());
}

template <bool GRAD>
void launch_gated(GatedArgs g, const Product& r, int parts, float* acc, hipStream_t s) {
    g.k = (int)r.k; g.k_per = (int)r.k_per; g.split = (int)r.split;
    g.acc = r.split > 1 ? acc : nullptr;
    of_tile<GRAD, false, !GRAD>(r.tile, [&](auto c) {
        using C = decltype(c);
        const dim3 grid = walkers<C>(ceil_div64(GRAD ? g.fk : 2 * g.fk, C::BM) * ceil_div64(g.rows, C::BN) * r.split);
        if constexpr (GRAD) {
            if (parts == 1) hipLaunchKernelGGL((dgated_kernel<C, 1>), grid, dim3(C::THREADS), 0, s, g);
            else hipLaunchKernelGGL((dgated_kernel<C, 3>), grid, dim3(C::THREADS), 0, s, g);
        } else {
            if (parts == 1) hipLaunchKernelGGL((gated_kernel<C, 1>), grid, dim3(C::THREADS), 0, s, g);
            else hipLaunchKernelGGL((gated_kernel<C, 3>), grid, dim3(C::THREADS), 0, s, g);
        }
    });
    if (!g.acc) return;
    const dim3 grid((unsigned)stride_blocks(ceil_div64(g.rows * (g.fk / 8), 256)));
    if (parts == 1) hipLaunchKernelGGL((gated_join_kernel<1, GRAD>), grid, dim3(256), 0, s, g);
    else hipLaunchKernelGGL((gated_join_kernel<3, GRAD>), grid, dim3(256), 0, s, g);
}

template <bool TA, bool TB>
void launch_out(OutArgs a, const Product& r, float* acc, hipStream_t s) {
    a.k = (int)r.k; a.k_per = (int)r.k_per; a.split = (int)r.split;
    a.acc = r.split > 1 ? acc : nullptr;
    a.ldacc = (a.cols + 7) / 8 * 8;
    of_tile<TA, TB, false>(r.tile, [&](auto c) {
        using C = decltype(c);
        const dim3 grid = walkers<C>(ceil_div64(a.cols, C::BM) * ceil_div64(a.rows, C::BN) * r.split);
        hipLaunchKernelGGL((ffn_out_kernel<C>), grid, dim3(C::THREADS), 0, s, a);
    });
    if (a.acc)
        hipLaunchKernelGGL(out_join_kernel, dim3((unsigned)stride_blocks(ceil_div64(a.rows * (a.ldacc / 8), 256))), dim3(256), 0, s, a);
}

// A matrix as planes in the workspace, or in place.
mm::Operand operand(const void* in, const float* scale, int kind, bool pack, int parts, int64_t rows, int64_t all, int64_t d,
                    uint16_t* out, int64_t plane, hipStream_t s) {
    const int64_t kp = ceil_div64(d, 64) * 64;
    if (!pack) return mm::Operand{(const uint16_t*)in, 0, d, (int)rows};
    const dim3 grid((unsigned)ceil_div64(all, 4));
    if (parts == 1)
        hipLaunchKernelGGL((planes_kernel<1>), grid, dim3(256), 0, s, in, scale, kind, rows, all, (int)d, (int)kp, out, plane);
    else
        hipLaunchKernelGGL((planes_kernel<3>), grid, dim3(256), 0, s, in, scale, kind, rows, all, (int)d, (int)kp, out, plane);
    return mm::Operand{out, plane, kp, (int)rows};
}

struct Inputs {
    mm::Operand x, w, wd;   // w: Wg's rows and, `pair` elements on, Wu's
    mm::Segments seg;
};

Inputs inputs(const FfnArgs& a, const FfnPlan& p, char* ws, bool need_x, hipStream_t s) {
    Inputs in{};
    const int kind = a.bf16 ? 1 : 0;
    in.seg = segments(p.parts, p.parts);
    if (need_x)
        in.x = operand(a.X, a.x_scale, a.x_scale ? 2 : kind, p.xpack, p.parts, p.t, p.t, p.d, (uint16_t*)(ws + p.x), p.t * p.dk, s);
    uint16_t* w = (uint16_t*)(ws + p.w);
    const int64_t plane = 2 * p.fk * p.dk;
    in.w = operand(a.Wg, nullptr, kind, p.wpack, p.parts, p.f, p.fk, p.d, w, plane, s);
    if (p.wpack) {
        operand(a.Wu, nullptr, kind, true, p.parts, p.f, p.fk, p.d, w + p.fk * p.dk, plane, s);
        in.w.pair = p.fk * p.dk;
    } else {
        in.w.pair = ((intptr_t)a.Wu - (intptr_t)a.Wg) / 2;
    }
    in.wd = operand(a.Wd, nullptr, kind, p.dpack, p.parts, p.d, p.d, p.f, (uint16_t*)(ws + p.wd), p.d * p.fk, s);
    return in;
}

GatedArgs gated_args(const FfnArgs& a, const FfnPlan& p, const Inputs& in, char* ws) {
    GatedArgs g{};
    g.w = in.w; g.x = in.x; g.seg = in.seg;
    g.rows = p.t; g.f = (int)p.f; g.fk = (int)p.fk; g.act = a.act;
    g.gate = a.gate; g.up = a.up;
    g.u = (uint16_t*)(ws + p.u);
    return g;
}

}  // namespace

int run_zeros(void* out, int64_t n, void* stream) {
    hipLaunchKernelGGL(zeros_kernel, dim3((unsigned)stride_blocks(ceil_div64(n, 256 * 8))), dim3(256), 0, (hipStream_t)stream,
                       (uint16_t*)out, n);
    return (int)hipGetLastError();
}

int run_ffn(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    const Inputs in = inputs(a, p, ws, true, s);
    float* acc = (float*)(ws + p.acc);
    launch_gated<false>(gated_args(a, p, in, ws), p.gu, p.parts, acc, s);
    OutArgs o{};
    o.a = in.wd;
    o.b = mm::Operand{(uint16_t*)(ws + p.u), p.t * p.fk, p.fk, (int)p.t};
    o.seg = in.seg; o.cols = (int)p.d; o.rows = o.second = o.valid = p.t; o.out = a.Y; o.out_bf16 = a.bf16;
    launch_out<false, false>(o, p.y, acc, s);
    return (int)hipGetLastError();
}

int run_ffn_grad(const FfnArgs& args, const FfnPlan& p, char* ws, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    FfnArgs a = args;
    const Inputs in = inputs(a, p, ws, !a.gate || a.dWg, s);
    float* acc = (float*)(ws + p.acc);
    if (!a.gate) {
        a.gate = ws + p.gate;
        a.up = ws + p.up;
        GatedArgs g = gated_args(a, p, in, ws);
        g.u = nullptr;
        launch_gated<false>(g, p.gu, p.parts, acc, s);
    }
    const mm::Operand dy = operand(a.dY, nullptr, a.bf16 ? 1 : 0, p.ypack, p.parts, p.t, p.t, p.d, (uint16_t*)(ws + p.dy), p.t * p.dk, s);
    GatedArgs g = gated_args(a, p, in, ws);
    g.w = in.wd; g.x = dy;
    g.dab = a.dX || a.dWg ? (uint16_t*)(ws + p.dab) : nullptr;
    if (!a.dWd) g.u = nullptr;
    launch_gated<true>(g, p.du, p.parts, acc, s);
    const mm::Operand dab{(uint16_t*)(ws + p.dab), p.t * 2 * p.fk, 2 * p.fk, (int)p.t};
    OutArgs o{};
    if (a.dX) {   // over da and Wg, db and Wu: two planes of one part each in place, one matrix of 2 fk rows where packed
        o.a = in.w; o.b = dab; o.seg = in.seg;
        if (p.wpack) {
            o.a.rows = (int)(2 * p.fk);
        } else {
            o.a.plane = in.w.pair;
            o.b.plane = p.fk;
            o.seg = mm::Segments{2, 0 | (1 | 1 << 2) << 4};
        }
        o.cols = (int)p.d; o.rows = o.second = o.valid = p.t; o.out = a.dX; o.out_bf16 = a.bf16;
        launch_out<true, false>(o, p.dx, acc, s);
    }
    if (a.dWg) {
        o = OutArgs{};
        o.a = in.x; o.b = dab; o.seg = in.seg;
        o.cols = (int)p.d; o.rows = 2 * p.fk; o.second = p.fk; o.valid = p.f; o.out = a.dWg; o.out2 = a.dWu;
        o.out_bf16 = a.dw_bf16; o.accumulate = a.accumulate;
        launch_out<true, true>(o, p.dgu, acc, s);
    }
    if (a.dWd) {
        o = OutArgs{};
        o.a = mm::Operand{(uint16_t*)(ws + p.u), p.t * p.fk, p.fk, (int)p.t};
        o.b = dy; o.seg = in.seg;
        o.cols = (int)p.f; o.rows = o.second = o.valid = p.d; o.out = a.dWd;
        o.out_bf16 = a.dw_bf16; o.accumulate = a.accumulate;
        launch_out<true, true>(o, p.dd, acc, s);
    }
    return (int)hipGetLastError();
}

}  // namespace dion
