// The gated feed-forward block of few rows: a stream of the three weight matrices, read once and in place, whatever their width.
//
//   u = act(X Wg^T) (X Wu^T);  Y = u Wd^T
//
// Two launches.  A workgroup has 16 output columns (16 rows of a matrix, or of Wg and of Wu); its waves share the reduction,
// each with loads of its own straight to registers, many of them under way at once, and their sums meet in LDS.  bf16 goes
// through v_mfma_f32_16x16x32_bf16, fp32 through v_mfma_f32_16x16x4_f32, whose rate (157 TFLOP/s) is enough for the 2 x 16 NT
// operations that an element of a matrix is worth here.
//
// Bound by the latency of two short kernels: one bf16 row, 2048 x 5632: 12.2 and 8.7 us (69 MB of weights, 14 us at the rate of
// a large copy), where tiles of 128 x 32 with sliced reductions take 26 in four launches.  8192 x 8192 (403 MB): 72 us, 5.6 TB/s.
// With 8 instead of 12 steps under way the second kernel takes 11.0 us; waves that take every eighth step instead of a
// piece of the rows, and twice the workgroups on a CU, measured the same.
//
// Lane layout of both: A[l % 16][k of the lane's quarter l / 16], B likewise, D element v of lane l is D[4 (l / 16) + v][l % 16].
// The order of k is free as long as A and B agree: a quarter takes 16 bytes of a row.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "block_plan.h"
#include "gate.hpp"
#include "rows.hpp"

namespace dion {

namespace {

struct FewArgs {
    const void* w[2];     // [cols][k]
    const void* x;        // [rows][ldx]
    const float* scale;   // x in 8 bits, or null
    int rows, cols, k, ldx;
    int slices;           // of k; several: their sums go to
    float* acc;           // [slices][M][rows][ldout], for few_join_kernel
    int act, even;
    void* out;            // u (M == 2) or null, fp32 [rows][ldout] or bf16 parts [2][rows][ldout]; or Y [rows][cols]
    int ldout;
    void* gate;           // [rows][cols], or null
    void* up;
};

template <bool BF16> struct Few;
template <> struct Few<true> {
    static constexpr int kStep = 32, kPer = 8;   // k of a step, and of a lane
    // elements c .. c + 7 of a row, zeros from k on
    static __device__ __forceinline__ u32x4 load(const void* p, int64_t row, int c, int k) {
        Raw8<true> r;
        r.load(p, row, c, k);
        return r.w[0];
    }
    static __device__ __forceinline__ u32x4 load8bit(const void* p, int64_t row, int c, int k, float s) {
        float v[8];
        load_e4m3<8>(p, row, c, k, s, v);
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = down16(v[2 * e]) | (down16(v[2 * e + 1]) << 16);
        return w;
    }
    static __device__ __forceinline__ f32x4 mma(const u32x4& a, const u32x4& b, const f32x4& c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mm::bf16x8, a), __builtin_bit_cast(mm::bf16x8, b), c, 0, 0, 0);
    }
};
template <> struct Few<false> {
    static constexpr int kStep = 16, kPer = 4;
    static __device__ __forceinline__ u32x4 load(const void* p, int64_t row, int c, int k) {
        const float* q = (const float*)p + row + c;
        if (c + 4 <= k) return __builtin_bit_cast(u32x4, (f32x4)*(const f32x4_any*)q);
        u32x4 w{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < k) w[e] = __float_as_uint(q[e]);
        return w;
    }
    static __device__ __forceinline__ u32x4 load8bit(const void* p, int64_t row, int c, int k, float s) {
        float v[4];
        load_e4m3<4>(p, row, c, k, s, v);
        return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
    static __device__ __forceinline__ f32x4 mma(const u32x4& a, const u32x4& b, f32x4 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
        return c;
    }
};

template <bool BF16>
__device__ __forceinline__ void keep4(void* p, int64_t row, int c, int d, int even, const float (&v)[4]) {
    if constexpr (BF16) {
        uint32_t w[2];
        if (even) {
            w[0] = keep32<true>(v[0], v[1]);
            w[1] = keep32<true>(v[2], v[3]);
        } else {
            w[0] = keep32<false>(v[0], v[1]);
            w[1] = keep32<false>(v[2], v[3]);
        }
        if (c + 4 <= d) {
            *(u32x2_any*)((uint16_t*)p + row + c) = u32x2{w[0], w[1]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < d) ((uint16_t*)p)[row + c + e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
        }
    } else {
        put4<false>(p, row, c, d, v);
    }
}

// Four columns of u (p, q: a and b) or of Y (p).
template <bool BF16, int M>
__device__ __forceinline__ void few_out(const FewArgs& a, int64_t row, int c, const float (&p)[4], const float (&q)[4]) {
    if constexpr (M == 2) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float slope;
            v[e] = activate<!BF16>(a.act, p[e], slope) * q[e];
        }
        if (a.gate) {
            keep4<BF16>(a.gate, row * a.cols, c, a.cols, a.even, p);
            keep4<BF16>(a.up, row * a.cols, c, a.cols, a.even, q);
        }
        if (a.out) {
            put4<BF16>(a.out, row * a.ldout, c, a.cols, v);
            if constexpr (BF16) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] -= up16(down16(v[e]));
                put4<BF16>(a.out, (a.rows + row) * a.ldout, c, a.cols, v);
            }
        }
    } else {
        put4<BF16>(a.out, row * a.cols, c, a.cols, p);
    }
}

// f(n) of a number that is known when it runs, 1 .. N, or nothing for 0
template <int N, class F>
__device__ __forceinline__ void rest(int n, F f) {
    if constexpr (N > 0) {
        if (n == N) f(std::integral_constant<int, N>());
        else rest<N - 1>(n, f);
    }
}

// M: matrices (2: Wg and Wu); NT: blocks of 16 rows of x; X8: which has 8 bits; WAVES share the reduction.
// bf16 with one matrix: x is u in two parts, the second ones of row r in the place of row r + 8, so that u's rounding, which
// would add as much to Y's error as Y's own, costs nothing.
template <bool BF16, int M, int NT, bool X8, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void few_kernel(FewArgs a) {
    using T = Few<BF16>;
    constexpr bool SPLIT = BF16 && M == 1;
    static_assert(!SPLIT || NT == 1, "rows r and r + 8");
    constexpr int U = M + NT <= 2 ? 12 : M + NT <= 3 ? 8 : 4;   // steps under way, as many as the registers hold
    __shared__ __attribute__((aligned(16))) f32x4 sums[WAVES][M * NT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slice = blockIdx.x % a.slices, c0 = blockIdx.x / a.slices * 16, steps = a.k / T::kStep;
    const int share = a.slices * WAVES, me = slice * WAVES + wave;
    const int first = (int)((int64_t)steps * me / share), last = (int)((int64_t)steps * (me + 1) / share);
    const int col = c0 + lane % 16 < a.cols ? c0 + lane % 16 : a.cols - 1;   // (columns and rows behind the last: any, not stored)
    const int64_t wrow = (int64_t)col * a.k;
    int64_t xrow[NT];
    float s[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int own = SPLIT ? lane % 8 : 16 * j + lane % 16, r = own < a.rows ? own : a.rows - 1;
        xrow[j] = (int64_t)(SPLIT && lane % 16 >= 8 ? a.rows + r : r) * a.ldx;
        s[j] = X8 ? a.scale[r] : 1.f;
    }
    f32x4 sum[M][NT] = {};
    const auto batch = [&](int at, auto count) {
        constexpr int N = decltype(count)::value;
        u32x4 w[N][M], x[N][NT];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (at + i) * T::kStep + lane / 16 * T::kPer;
#pragma unroll
            for (int m = 0; m < M; ++m) w[i][m] = T::load(a.w[m], wrow, c, 0x7fffffff);
#pragma unroll
            for (int j = 0; j < NT; ++j) x[i][j] = X8 ? T::load8bit(a.x, xrow[j], c, 0x7fffffff, s[j]) : T::load(a.x, xrow[j], c, 0x7fffffff);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {   // all of them under way before the first is used
#pragma unroll
            for (int m = 0; m < M; ++m) asm volatile("" : "+v"(w[i][m]));
#pragma unroll
            for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(x[i][j]));
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[m][j] = T::mma(w[i][m], x[i][j], sum[m][j]);
    };
    int at = first;
    for (; at + U <= last; at += U) batch(at, std::integral_constant<int, U>());
    rest<U - 1>(last - at, [&](auto count) { batch(at, count); });
    if (me == share - 1 && a.k % T::kStep != 0) {   // the step at the rows' end
        const int c = steps * T::kStep + lane / 16 * T::kPer;
        u32x4 w[M], x[NT];
#pragma unroll
        for (int m = 0; m < M; ++m) w[m] = T::load(a.w[m], wrow, c, a.k);
#pragma unroll
        for (int j = 0; j < NT; ++j) x[j] = X8 ? T::load8bit(a.x, xrow[j], c, a.k, s[j]) : T::load(a.x, xrow[j], c, a.k);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j) sum[m][j] = T::mma(w[m], x[j], sum[m][j]);
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[wave][m * NT + j][lane] = sum[m][j];
    __syncthreads();
    if (wave >= NT) return;
    f32x4 t[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        t[m] = sums[0][m * NT + wave][lane];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) t[m] += sums[i][m * NT + wave][lane];
    }
    const int64_t row = 16 * wave + lane % 16;
    const int c = c0 + 4 * (lane / 16);
    if (row >= a.rows) return;
    if constexpr (SPLIT) {
#pragma unroll
        for (int i = 0; i < WAVES; ++i) t[0] += sums[i][0][lane + 8];
    }
    if (a.slices > 1) {   // (rows of a multiple of 64)
#pragma unroll
        for (int m = 0; m < M; ++m) *(f32x4*)(a.acc + (((int64_t)slice * M + m) * a.rows + row) * a.ldout + c) = t[m];
        return;
    }
    float p[4], q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) { p[e] = t[0][e]; q[e] = t[M - 1][e]; }
    few_out<BF16, M>(a, row, c, p, q);
}

// The slices' sums, four columns a thread.
template <bool BF16, int M>
__global__ __launch_bounds__(256) void few_join_kernel(FewArgs a) {
    const int per = a.ldout / 4, i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.rows * per) return;
    const int64_t row = i / per;
    const int c = (i - (int)row * per) * 4;
    if (c >= a.cols) return;
    f32x4 t[M] = {};
#pragma unroll 4
    for (int s = 0; s < a.slices; ++s)
#pragma unroll
        for (int m = 0; m < M; ++m) t[m] += *(const f32x4*)(a.acc + (((int64_t)s * M + m) * a.rows + row) * a.ldout + c);
    float p[4], q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) { p[e] = t[0][e]; q[e] = t[M - 1][e]; }
    few_out<BF16, M>(a, row, c, p, q);
}

template <bool BF16, int M, int NT>
void launch_few(const FewArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(ceil_div64(a.cols, 16) * a.slices));
    if constexpr (M == 2) {
        if (a.scale) hipLaunchKernelGGL((few_kernel<BF16, 2, NT, true, 8>), grid, dim3(512), 0, s, a);
        else hipLaunchKernelGGL((few_kernel<BF16, 2, NT, false, 8>), grid, dim3(512), 0, s, a);
    } else {   // (twice the waves for each where half the chip's CUs are without a workgroup)
        if (grid.x < kCUs) hipLaunchKernelGGL((few_kernel<BF16, 1, NT, false, 16>), grid, dim3(1024), 0, s, a);
        else hipLaunchKernelGGL((few_kernel<BF16, 1, NT, false, 8>), grid, dim3(512), 0, s, a);
    }
}

template <bool BF16, int M>
void launch_few(const FewArgs& a, hipStream_t s) {
    if (BF16 || a.rows <= 16) launch_few<BF16, M, 1>(a, s);
    else if constexpr (!BF16) {
        if (a.rows <= 32) launch_few<false, M, 2>(a, s);
        else launch_few<false, M, 4>(a, s);
    }
    if (a.slices > 1)
        hipLaunchKernelGGL((few_join_kernel<BF16, M>), dim3((unsigned)ceil_div64((int64_t)a.rows * (a.ldout / 4), 256)), dim3(256), 0, s, a);
}

}  // namespace

namespace {

FewArgs gate_args(const FfnArgs& a, const FfnPlan& p, char* ws) {
    FewArgs g{};
    g.slices = p.fgu; g.acc = (float*)(ws + p.acc); g.ldout = (int)p.fk;
    g.w[0] = a.Wg; g.w[1] = a.Wu; g.x = a.X; g.scale = a.x_scale;
    g.rows = (int)p.t; g.cols = (int)p.f; g.k = (int)p.d; g.ldx = (int)p.d; g.act = a.act; g.even = a.even;
    g.gate = a.gate; g.up = a.up;
    return g;
}

}  // namespace

int run_ffn_few_gate(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream) {
    launch_few<false, 2>(gate_args(a, p, ws), (hipStream_t)stream);
    return (int)hipGetLastError();
}

int run_ffn_few(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    FewArgs g = gate_args(a, p, ws);
    g.out = ws + p.u;
    FewArgs d{};
    d.w[0] = a.Wd; d.x = ws + p.u;
    d.rows = (int)p.t; d.cols = (int)p.d; d.k = (int)p.f; d.ldx = (int)p.fk;
    d.slices = p.fy; d.acc = g.acc; d.ldout = (int)p.dk;
    d.out = a.Y;
    if (a.bf16) {
        launch_few<true, 2>(g, s);
        launch_few<true, 1>(d, s);
    } else {
        launch_few<false, 2>(g, s);
        launch_few<false, 1>(d, s);
    }
    return (int)hipGetLastError();
}

}  // namespace dion
