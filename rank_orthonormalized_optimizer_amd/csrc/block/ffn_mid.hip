// Products of the gated feed-forward block of a moderate number of fp32 rows, with the weight matrices read in place.
//
//   a = X Wg^T, b = X Wu^T, u = act(a) b;  Y = u Wd^T          (reductions along the matrices' rows' elements)
//   du = dY Wd, da = du b act'(a), db = du act(a);  dX = da Wg + db Wu          (reductions over the matrices' rows)
//
// Planes of the weights, which many rows are worth, cost more traffic here than the products: the weights go from memory
// straight to registers, four steps of 32 k under way, where a wave splits its two blocks of 16 columns into three bf16 parts
// (an exact split, six products); the few rows' planes go through LDS, in the order in which the lanes read them, and serve
// the workgroup's eight waves.  Where the columns do not fill the chip the reduction is cut into slices, whose sums a second
// launch joins.
//
// Bound by HBM up to 64 rows, then by both: 8192 x 8192 fp32, a and b 32 rows 140 us (3.8 TB/s; without the products 125),
// 128 rows 199 (2.7 TB/s, 650 TFLOP/s of part products; 161), dX 130 and 188 (93 and 130).  With workgroups of four waves,
// which read the rows' planes twice as often, 238 and 222 for 128 rows; with the next loads all started before the products 222
// and 212, for a wave whose loads are held up starts no product; with two steps under way as with four waves.  (Each the least of
// several runs on one card; on others a and b of 128 rows took 188 to 209 at least and 210 to 225 in the median.)
//
// Lane layout of v_mfma_f32_16x16x32_bf16: A[l % 16][8 values of k of the quarter l / 16], B likewise, D element v of lane l is
// D[4 (l / 16) + v][l % 16].  The order of k is free as long as A and B agree: a quarter has k of 4 q .. 4 q + 3 and 16 behind
// them, so that four lanes load 64 bytes of a row.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "block_plan.h"
#include "gate.hpp"
#include "rows.hpp"

namespace dion {

namespace {

constexpr int kStep = 32;    // k of a step
constexpr int kMayCross = 0x106;   // vector and scalar arithmetic and reads of LDS
constexpr int kWaves = 8;

struct MidArgs {
    const float* w[2];      // Wg and Wu, or Wd twice; [cols][k], or [k][cols] (over the matrices' rows)
    const uint16_t* x;      // planes [3][rows][ldx], zeros behind the last k
    int64_t xplane;
    int rows, cols, k, ldx;
    int steps;              // of all matrices
    int second;             // steps from which the second matrix's rows are meant (over the rows; dX), else `steps`
    int slices, groups;     // of the reduction; of 16 NT rows
    float* acc;             // [slices][1 or 2][rows][ldacc]
    int ldacc;
    int act;
    float* gate;            // a and b, [rows][hidden]: written (or null), or read
    float* up;
    uint16_t* u;            // planes [3][rows][fk], or null
    uint16_t* dab;          // planes [3][rows][2 fk], or null
    int f, fk;
    float* out;             // Y or dX, [rows][cols]
};

enum { GATED = 0, OUT = 1, DGATED = 2 };

__device__ __forceinline__ void put_planes(uint16_t* p, int64_t plane, int64_t at, const float (&v)[4]) {
    uint32_t part[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) split3(v[e], part[e]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
        *(u32x2*)(p + q * plane + at) = u32x2{part[0][q] | (part[1][q] << 16), part[2][q] | (part[3][q] << 16)};
}

__device__ __forceinline__ void get4(const float* p, int64_t row, int c, int d, float (&v)[4]) {
    f32x4 t{0.f, 0.f, 0.f, 0.f};
    if (c + 4 <= d) {
        t = *(const f32x4_any*)(p + row + c);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < d) t[e] = p[row + c + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[e];
}

// Four columns of a and b (p, q), of an output (p) or of du (p); planes are written up to their rows' end.
template <int KIND>
__device__ __forceinline__ void mid_out(const MidArgs& a, int64_t row, int c, float (&p)[4], const float (&q)[4]) {
    if constexpr (KIND == OUT) {
        if (c < a.cols) put4<false>(a.out, row * a.cols, c, a.cols, p);
    } else {
        if (c >= a.fk) return;
        float u[4], da[4], db[4], ka[4], kb[4];
        if constexpr (KIND == GATED) {
            if (a.gate && c < a.f) {
                put4<false>(a.gate, row * a.f, c, a.f, p);
                put4<false>(a.up, row * a.f, c, a.f, q);
            }
        } else {
            get4(a.gate, row * a.f, c, a.f, ka);
            get4(a.up, row * a.f, c, a.f, kb);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float slope;
            const float v = activate<true>(a.act, KIND == GATED ? p[e] : ka[e], slope);
            u[e] = v * (KIND == GATED ? q[e] : kb[e]);
            da[e] = p[e] * kb[e] * slope;
            db[e] = p[e] * v;
            if (c + e >= a.f) u[e] = da[e] = db[e] = 0.f;   // (made of anything there)
        }
        if (a.u) put_planes(a.u, (int64_t)a.rows * a.fk, row * a.fk + c, u);
        if (KIND == DGATED && a.dab) {
            const int64_t plane = (int64_t)a.rows * 2 * a.fk, at = row * 2 * a.fk + c;
            put_planes(a.dab, plane, at, da);
            put_planes(a.dab, plane, at + a.fk, db);
        }
    }
}

// Columns that a workgroup has: those of 2 kWaves blocks, or of half as many where a wave's two blocks are of two matrices.
template <int KIND> constexpr int kCols = KIND == GATED ? 16 * kWaves : 32 * kWaves;

// TRANS (over the matrices' rows): a wave's blocks are the even and the odd ones of 32 columns, so that a lane loads pairs.
template <int KIND, bool TRANS, int NT>
__global__ __launch_bounds__(64 * kWaves, 2) void mid_kernel(MidArgs a) {
    constexpr int FRAGS = 3 * NT, PER = (FRAGS + kWaves - 1) / kWaves, DEEP = 4;   // steps under way
    __shared__ __attribute__((aligned(16))) u32x2 lds[2][FRAGS][64][2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), quarter = lane / 16;
    const int group = blockIdx.x % a.groups, part = blockIdx.x / a.groups, slice = part % a.slices;
    const int c0 = part / a.slices * kCols<KIND> + wave * (KIND == GATED ? 16 : 32);
    const int all = (a.steps + DEEP - 1) / DEEP;   // a slice has a multiple of DEEP steps, in the last one zeros behind the end
    const int first = (int)((int64_t)all * slice / a.slices) * DEEP, end = (int)((int64_t)all * (slice + 1) / a.slices) * DEEP;
    const int last = end < a.steps ? end : a.steps;

    // Weights: offsets from a descriptor that ends with the matrix, behind which zeros are read.
    const auto range = [](int64_t left) { return (int)(left < 0 ? 0 : left < 0x7fffffff ? left : 0x7fffffff); };
    __amdgpu_buffer_rsrc_t rsrc[2];
    uint32_t off;
    if constexpr (!TRANS) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int64_t row = c0 + (KIND == GATED ? 0 : 16 * m);
            rsrc[m] = __builtin_amdgcn_make_buffer_rsrc((void*)(a.w[m] + row * a.k), 0, range((a.cols - row) * a.k * 4), 0x00027000);
        }
        off = (uint32_t)(lane % 16 * a.k + 4 * quarter) * 4u;
    } else {
        off = (uint32_t)(4 * quarter * a.cols + c0 + 2 * (lane % 16)) * 4u;
    }
    u32x4 raw[DEEP][4];
    // piece p of four of a step's weights
    const auto fetch = [&](int s, u32x4 (&to)[4], int p) {
        if constexpr (!TRANS) {
            const uint32_t at = s < last ? off + (uint32_t)s * (kStep * 4u) : mm::kOutside;
            to[p] = __builtin_amdgcn_raw_buffer_load_b128(rsrc[p / 2], at + 64u * (p % 2), 0, 0);
        } else {
            const int which = s >= a.second, row = (s - (which ? a.second : 0)) * kStep;
            const int64_t left = s < last ? ((int64_t)a.k - row) * a.cols * 4 : 0;
            const auto from = __builtin_amdgcn_make_buffer_rsrc((void*)((which ? a.w[1] : a.w[0]) + (int64_t)row * a.cols), 0,
                                                                range(left), 0x00027000);
#pragma unroll
            for (int e = 2 * p; e < 2 * p + 2; ++e) {
                const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(from, off + (uint32_t)((e % 4 + 16 * (e / 4)) * a.cols) * 4u, 0, 0);
                to[e / 4][e % 4] = v[0];
                to[2 + e / 4][e % 4] = v[1];
            }
        }
    };

    // The rows' planes: fragment f is part f / NT of rows 16 (f % NT) on.
    const auto planes = __builtin_amdgcn_make_buffer_rsrc((void*)a.x, 0, range(3 * a.xplane * 2), 0x00027000);
    uint32_t xoff[PER];
    u32x4 next[DEEP][PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int f = wave + kWaves * i, row = (group * NT + f % NT) * 16 + lane % 16;
        xoff[i] = f >= FRAGS ? mm::kOutside : (uint32_t)((f / NT) * a.xplane + (row < a.rows ? row : a.rows - 1) * a.ldx + 8 * quarter) * 2u;
    }
    const auto fetch_x = [&](int s, u32x4 (&to)[PER], int i) {
        to[i] = __builtin_amdgcn_raw_buffer_load_b128(planes, s < last ? xoff[i] + (uint32_t)s * (kStep * 2u) : mm::kOutside, 0, 0);
    };
    const auto all_x = [&](int s, u32x4 (&to)[PER]) {
#pragma unroll
        for (int i = 0; i < PER; ++i) fetch_x(s, to, i);
    };
    const auto stage = [&](int to, const u32x4 (&x)[PER]) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (FRAGS % kWaves == 0 || wave + kWaves * i < FRAGS) {
                auto& f = lds[to][wave + kWaves * i];
                f[32 * (quarter % 2) + lane % 16][quarter / 2] = u32x2{x[i][0], x[i][1]};
                f[32 * (quarter % 2) + 16 + lane % 16][quarter / 2] = u32x2{x[i][2], x[i][3]};
            }
    };

    f32x4 sum[2][NT] = {};
    // Loads end in the order of their start: a step's rows are fetched just before its weights, all as many steps ahead, and
    // those behind the last step are fetched too, as zeros from outside, so that the number under way is always the same.
    all_x(first, next[0]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
#pragma unroll
        for (int p = 0; p < 4; ++p) fetch(first + i, raw[i], p);
        if (i + 1 < DEEP) all_x(first + i + 1, next[i + 1]);
        __builtin_amdgcn_sched_barrier(0);
    }
    stage(0, next[0]);
    all_x(first + DEEP, next[0]);
    __syncthreads();
    for (int s0 = first; s0 < end; s0 += DEEP) {
#pragma unroll
        for (int i = 0; i < DEEP; ++i) {
            const int s = s0 + i;
            u32x4 w[2][3];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(raw[i][2 * m + e / 4][e % 4]);
                if (!TRANS && (s + 1) * kStep > a.k) {   // behind a row's end is the next one
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (s * kStep + 4 * quarter + e % 4 + 16 * (e / 4) >= a.k) v[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    uint32_t p0[3], p1[3];
                    split3(v[e], p0);
                    split3(v[e + 1], p1);
#pragma unroll
                    for (int q = 0; q < 3; ++q) w[m][q][e / 2] = p0[q] | (p1[q] << 16);
                }
            }
            stage((i + 1) & 1, next[(i + 1) % DEEP]);
            // The next loads start between the products: together they would hold up the wave.
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                mm::bf16x8 x[2][3];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        x[h][q] = __builtin_bit_cast(mm::bf16x8, *(const u32x4*)lds[i & 1][q * NT + j + h][lane]);
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    if (p * NT / 8 == j / 2) fetch(s + DEEP, raw[i], p);
#pragma unroll
                for (int p = 0; p < PER; ++p)
                    if (p * NT / 8 == j / 2) fetch_x(s + 1 + DEEP, next[(i + 1) % DEEP], p);
                __builtin_amdgcn_sched_barrier(kMayCross);
                constexpr int WP[6] = {1, 0, 2, 0, 1, 0}, XP[6] = {1, 2, 0, 1, 0, 0};   // small ones first
#pragma unroll
                for (int t = 0; t < 6; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            sum[m][j + h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(mm::bf16x8, w[m][WP[t]]), x[h][XP[t]], sum[m][j + h], 0, 0, 0);
            }
            __syncthreads();
        }
    }

#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t row = (group * NT + j) * 16 + lane % 16;
        if (row >= a.rows) continue;
        float p[2][4], q[4];
        int c[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            c[m] = KIND == GATED ? c0 + 4 * quarter : TRANS ? c0 + 8 * quarter + 4 * m : c0 + 16 * m + 4 * quarter;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[m][e] = TRANS ? sum[e % 2][j][2 * m + e / 2] : sum[m][j][e];
                q[e] = sum[1][j][e];
            }
        }
        if (a.slices > 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int64_t unit = KIND == GATED ? 2 * slice + m : slice;
                if (c[m] < a.ldacc) *(f32x4*)(a.acc + (unit * a.rows + row) * a.ldacc + c[m]) = f32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            }
        } else {
            mid_out<KIND>(a, row, c[0], p[0], q);
            if (KIND != GATED) mid_out<KIND>(a, row, c[1], p[1], q);
        }
    }
}

// The slices' sums, four columns a thread.
template <int KIND>
__global__ __launch_bounds__(256) void mid_join_kernel(MidArgs a) {
    constexpr int M = KIND == GATED ? 2 : 1;
    const int per = a.ldacc / 4, i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.rows * per) return;
    const int64_t row = i / per;
    const int c = (i - (int)row * per) * 4;
    f32x4 t[M] = {};
#pragma unroll 4
    for (int s = 0; s < a.slices; ++s)
#pragma unroll
        for (int m = 0; m < M; ++m) t[m] += *(const f32x4*)(a.acc + (((int64_t)s * M + m) * a.rows + row) * a.ldacc + c);
    float p[4], q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) { p[e] = t[0][e]; q[e] = t[M - 1][e]; }
    mid_out<KIND>(a, row, c, p, q);
}

template <int KIND, bool TRANS>
void launch_mid(MidArgs a, hipStream_t s) {
    // as few groups as can be, of 64, 96 or 128 rows (96 instead of 128: forward, 8192 x 8192, 96 rows 307 us, so 278,
    // 192 rows 539 and 464)
    const int blocks = (int)ceil_div64(a.rows, 16);
    a.groups = (blocks + 7) / 8;
    const int nt = (blocks + a.groups - 1) / a.groups;
    const dim3 grid((unsigned)(ceil_div64(a.cols, kCols<KIND>) * a.slices * a.groups)), block(64 * kWaves);
    if (nt <= 4) hipLaunchKernelGGL((mid_kernel<KIND, TRANS, 4>), grid, block, 0, s, a);
    else if (nt <= 6) hipLaunchKernelGGL((mid_kernel<KIND, TRANS, 6>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((mid_kernel<KIND, TRANS, 8>), grid, block, 0, s, a);
    if (a.slices > 1)
        hipLaunchKernelGGL((mid_join_kernel<KIND>), dim3((unsigned)ceil_div64((int64_t)a.rows * (a.ldacc / 4), 256)), dim3(256), 0, s, a);
}

MidArgs mid_args(const FfnArgs& a, const FfnPlan& p, char* ws) {
    MidArgs g{};
    g.rows = (int)p.t; g.f = (int)p.f; g.fk = (int)p.fk; g.act = a.act;
    g.acc = (float*)(ws + p.acc);
    g.gate = (float*)a.gate; g.up = (float*)a.up;
    return g;
}

}  // namespace

int run_mid_gate(const FfnArgs& a, const FfnPlan& p, bool u, char* ws, void* stream) {
    MidArgs g = mid_args(a, p, ws);
    g.w[0] = (const float*)a.Wg; g.w[1] = (const float*)a.Wu;
    g.x = (const uint16_t*)(ws + p.x); g.xplane = p.t * p.dk; g.ldx = (int)p.dk;
    g.cols = (int)p.f; g.k = (int)p.d;
    g.steps = g.second = (int)(p.dk / kStep);
    g.slices = p.mgu; g.ldacc = (int)p.fk;
    g.u = u ? (uint16_t*)(ws + p.u) : nullptr;
    launch_mid<GATED, false>(g, (hipStream_t)stream);
    return (int)hipGetLastError();
}

int run_mid_out(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream) {
    MidArgs g = mid_args(a, p, ws);
    g.w[0] = g.w[1] = (const float*)a.Wd;
    g.x = (const uint16_t*)(ws + p.u); g.xplane = p.t * p.fk; g.ldx = (int)p.fk;
    g.cols = (int)p.d; g.k = (int)p.f;
    g.steps = g.second = (int)(p.fk / kStep);
    g.slices = p.my; g.ldacc = (int)p.dk;
    g.out = (float*)a.Y;
    launch_mid<OUT, false>(g, (hipStream_t)stream);
    return (int)hipGetLastError();
}

int run_mid_du(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream) {
    MidArgs g = mid_args(a, p, ws);
    g.w[0] = g.w[1] = (const float*)a.Wd;
    g.x = (const uint16_t*)(ws + p.dy); g.xplane = p.t * p.dk; g.ldx = (int)p.dk;
    g.cols = (int)p.f; g.k = (int)p.d;
    g.steps = g.second = (int)(p.dk / kStep);
    g.slices = p.mdu; g.ldacc = (int)p.fk;
    g.u = a.dWd ? (uint16_t*)(ws + p.u) : nullptr;
    g.dab = a.dX || a.dWg ? (uint16_t*)(ws + p.dab) : nullptr;
    launch_mid<DGATED, true>(g, (hipStream_t)stream);
    return (int)hipGetLastError();
}

int run_mid_dx(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream) {
    MidArgs g = mid_args(a, p, ws);
    g.w[0] = (const float*)a.Wg; g.w[1] = (const float*)a.Wu;
    g.x = (const uint16_t*)(ws + p.dab); g.xplane = p.t * 2 * p.fk; g.ldx = (int)(2 * p.fk);
    g.cols = (int)p.d; g.k = (int)p.f;
    g.second = (int)(p.fk / kStep); g.steps = 2 * g.second;
    g.slices = p.mdx; g.ldacc = (int)p.dk;
    g.out = (float*)a.dX;
    launch_mid<OUT, true>(g, (hipStream_t)stream);
    return (int)hipGetLastError();
}

}  // namespace dion
