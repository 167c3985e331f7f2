// Gradients of the gated feed-forward block of few fp32 rows: each weight matrix is read once and each weight's gradient
// written once, in place, whatever their width.
//
//   du = dY Wd;  da = du b act'(a);  db = du act(a);  dX = da Wg + db Wu          (reductions along the matrices' rows)
//   dWg = da^T X;  dWu = db^T X;  dWd = dY^T u                                   (sums over few rows: streams of writes)
//
// Five launches (and one that forms a and b again, where they are not kept): the two products over the matrices' rows are cut
// into slices that fill the chip, whose sums are joined, and the three weights' gradients are one launch.  Everything goes
// through v_mfma_f32_16x16x4_f32, whose 157 TFLOP/s are enough for the 2 rows operations that an element of a matrix is worth
// here.  Bound by HBM.
//
// Lane layout of the instruction: A[l % 16][k = l / 16], B likewise, D element v of lane l is D[4 (l / 16) + v][l % 16].  A lane
// loads V columns in a row of a matrix and gives each to a product of its own, so that product e has the columns V i + e.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "block_plan.h"
#include "gate.hpp"
#include "rows.hpp"

namespace dion {

namespace {

constexpr int V = 4;

// four elements of a row of d from column c, zeros behind it; kind: 0 fp32, 2 e4m3 times s
__device__ __forceinline__ f32x4 load4(const void* p, int64_t row, int c, int d, int kind, float s) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (kind == 0) {
        const float* q = (const float*)p + row + c;
        if (c + 4 <= d) return *(const f32x4_any*)q;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < d) v[e] = q[e];
    } else {
        load_e4m3<4>(p, row, c, d, s, v);
    }
    return f32x4{v[0], v[1], v[2], v[3]};
}

__device__ __forceinline__ f32x4 mma4(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// ---------------------------------------------------------------------------
// out[t][c] = sum over m and k of x_m[t][k] W_m[k][c]
// ---------------------------------------------------------------------------
struct DownArgs {
    const float* w[2];    // [k][cols]
    const float* x[2];    // [rows][ldx]
    int rows, cols, k, ldx;
    int slices, ldacc;
    float* acc;           // [slices][rows][ldacc]
    int act;
    const float* gate;    // du: [rows][cols], kept
    const float* up;
    float* da;            // du: [rows][ldout] each
    float* db;
    float* u;
    int ldout;
    float* out;           // dX [rows][cols]
};

// A workgroup: 64 columns and a slice of the groups of 16 k (of both matrices in a row), shared by its eight waves.
template <int M, int NT>
__global__ __launch_bounds__(512) void down_kernel(DownArgs a) {
    constexpr int WAVES = 8, U = NT == 1 ? 4 : 2;   // groups under way
    __shared__ __attribute__((aligned(16))) f32x4 sums[WAVES][V * NT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), quarter = lane / 16;
    const int slice = blockIdx.x % a.slices, c0 = blockIdx.x / a.slices * 16 * V, c = c0 + V * (lane % 16);
    const bool ragged = c0 + 16 * V > a.cols;
    const int groups = (a.k + 15) / 16, all = M * groups, share = a.slices * WAVES, me = slice * WAVES + wave;
    const int first = (int)((int64_t)all * me / share), last = (int)((int64_t)all * (me + 1) / share);
    int64_t xrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xrow[j] = (int64_t)(16 * j + lane % 16 < a.rows ? 16 * j + lane % 16 : a.rows - 1) * a.ldx;
    f32x4 sum[V][NT] = {};
    const auto multiply = [&](const f32x4 (&w)[4], const f32x4 (&x)[NT]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[v][j] = mma4(w[e][v], x[j][e], sum[v][j]);
    };
    int at = first;
    while (at < last) {
        const int m = M == 2 && at >= groups, g = at - m * groups, whole = a.k / 16;
        const float* wp = m ? a.w[1] : a.w[0];
        const float* xp = m ? a.x[1] : a.x[0];
        if (!ragged && at + U <= last && g + U <= whole) {   // all of one matrix, none behind its last k
            f32x4 w[U][4], x[U][NT];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int k = (g + i) * 16 + 4 * quarter;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[i][e] = *(const f32x4_any*)(wp + (int64_t)(k + e) * a.cols + c);
#pragma unroll
                for (int j = 0; j < NT; ++j) x[i][j] = *(const f32x4_any*)(xp + xrow[j] + k);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {   // all of them under way before the first is used
#pragma unroll
                for (int e = 0; e < 4; ++e) asm volatile("" : "+v"(w[i][e]));
#pragma unroll
                for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(x[i][j]));
            }
#pragma unroll
            for (int i = 0; i < U; ++i) multiply(w[i], x[i]);
            at += U;
        } else {
            const int k = g * 16 + 4 * quarter;
            f32x4 w[4], x[NT];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = load4(wp, (int64_t)(k + e < a.k ? k + e : a.k - 1) * a.cols, c, a.cols, 0, 1.f);
#pragma unroll
            for (int j = 0; j < NT; ++j) x[j] = load4(xp, xrow[j], k, a.k, 0, 1.f);   // (zeros behind the last k)
            multiply(w, x);
            ++at;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[wave][v * NT + j][lane] = sum[v][j];
    __syncthreads();
    if (wave >= NT) return;
    f32x4 t[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        t[v] = sums[0][v * NT + wave][lane];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) t[v] += sums[i][v * NT + wave][lane];
    }
    const int row = 16 * wave + lane % 16;
    if (row >= a.rows) return;
    // element v of product e: column V v + e behind the quarter's first (rows of a multiple of 64)
    f32x4* to = (f32x4*)(a.acc + ((int64_t)slice * a.rows + row) * a.ldacc + c0 + 4 * V * quarter);
#pragma unroll
    for (int v = 0; v < 4; ++v) to[v] = f32x4{t[0][v], t[1][v], t[2][v], t[3][v]};
}

// The slices' sums: dX, or da, db and u.  Four columns a thread.
template <int M>
__global__ __launch_bounds__(256) void down_join_kernel(DownArgs a) {
    const int per = a.ldacc / 4, i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.rows * per) return;
    const int64_t row = i / per;
    const int c = (i - (int)row * per) * 4;
    if (c >= a.cols) return;
    f32x4 t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < a.slices; ++s) t += *(const f32x4*)(a.acc + ((int64_t)s * a.rows + row) * a.ldacc + c);
    float v[4] = {t[0], t[1], t[2], t[3]};
    if constexpr (M == 2) {
        put4<false>(a.out, row * a.cols, c, a.cols, v);
    } else {
        const f32x4 ka = load4(a.gate, row * a.cols, c, a.cols, 0, 1.f), kb = load4(a.up, row * a.cols, c, a.cols, 0, 1.f);
        float da[4], db[4], u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float slope;
            const float s = activate<true>(a.act, ka[e], slope);
            da[e] = v[e] * kb[e] * slope;
            db[e] = v[e] * s;
            u[e] = s * kb[e];
        }
        put4<false>(a.da, row * a.ldout, c, a.cols, da);
        put4<false>(a.db, row * a.ldout, c, a.cols, db);
        put4<false>(a.u, row * a.ldout, c, a.cols, u);
    }
}

// ---------------------------------------------------------------------------
// out[r][c] (+)= sum over t of y[t][r] x[t][c]
// ---------------------------------------------------------------------------
struct RankJob {
    const float* y;       // [rows][ldy]
    const void* x;        // [rows][ldx], fp32, or 8 bits with
    const float* scale;   // a scale per row
    void* out;            // [r][c]
    int ldy, ldx, r, c;
    int across;           // workgroups of 256 columns
    unsigned first;       // its first workgroup
};
struct RankArgs {
    RankJob job[3];
    int n, rows, accumulate;
};
constexpr int kRankRows = 64;   // of out, a workgroup

// Four waves, each 64 columns of kRankRows rows: x stays in registers, y comes 16 rows at a time.
template <bool OB, int STEPS>
__global__ __launch_bounds__(256) void rank_kernel(RankArgs a) {
    int at = 0;
    while (at + 1 < a.n && blockIdx.x >= a.job[at + 1].first) ++at;
    const RankJob& job = a.job[at];
    const int block = (int)(blockIdx.x - job.first), lane = threadIdx.x & 63, wave = threadIdx.x >> 6, quarter = lane / 16;
    const int c0 = (block % job.across * 4 + wave) * 64, r0 = block / job.across * kRankRows;
    if (c0 >= job.c) return;
    f32x4 x[STEPS];   // product e: columns 16 e + l % 16, so that four lanes store 64 bytes of a row
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int t = 4 * s + quarter;
        x[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = c0 + 16 * e + lane % 16;
            if (t >= a.rows || c >= job.c) continue;
            const int64_t i = (int64_t)t * job.ldx + c;
            x[s][e] = job.scale ? __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)job.x)[i], 0) * job.scale[t] : ((const float*)job.x)[i];
        }
    }
    const int end = r0 + kRankRows < job.r ? r0 + kRankRows : job.r;
    float y[2][STEPS];
    const auto fetch = [&](int r, float (&to)[STEPS]) {
        const int row = r + lane % 16 < job.r ? r + lane % 16 : job.r - 1;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int t = 4 * s + quarter;
            to[s] = job.y[(int64_t)(t < a.rows ? t : a.rows - 1) * job.ldy + row];
            if (t >= a.rows) to[s] = 0.f;   // (as x is: a number that is not finite reaches only its own row)
        }
    };
    fetch(r0, y[0]);
#pragma unroll
    for (int i = 0; i < kRankRows / 16; ++i) {
        const int r = r0 + 16 * i;
        if (r >= end) return;
        if (r + 16 < end) fetch(r + 16, y[(i + 1) % 2]);
        f32x4 sum[V] = {};
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int v = 0; v < V; ++v) sum[v] = mma4(x[s][v], y[i % 2][s], sum[v]);
        const int row = r + lane % 16;
        if (row >= end) continue;
        const int64_t to = (int64_t)row * job.c;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int col = c0 + 16 * e + 4 * quarter;
            if (col >= job.c) continue;
            float o[4] = {sum[e][0], sum[e][1], sum[e][2], sum[e][3]};
            if (a.accumulate) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (col + k < job.c) o[k] += OB ? up16(((const uint16_t*)job.out)[to + col + k]) : ((const float*)job.out)[to + col + k];
            }
            put4<OB>(job.out, to, col, job.c, o);
        }
    }
}

template <int M>
void launch_down(const DownArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(ceil_div64(a.cols, 16 * V) * a.slices));
    if (a.rows <= 16) hipLaunchKernelGGL((down_kernel<M, 1>), grid, dim3(512), 0, s, a);
    else if (a.rows <= 32) hipLaunchKernelGGL((down_kernel<M, 2>), grid, dim3(512), 0, s, a);
    else if (a.rows <= 48) hipLaunchKernelGGL((down_kernel<M, 3>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((down_kernel<M, 4>), grid, dim3(512), 0, s, a);
    hipLaunchKernelGGL((down_join_kernel<M>), dim3((unsigned)ceil_div64((int64_t)a.rows * (a.ldacc / 4), 256)), dim3(256), 0, s, a);
}

template <bool OB>
void launch_rank(const RankArgs& a, unsigned blocks, hipStream_t s) {
    if (a.rows <= 4) hipLaunchKernelGGL((rank_kernel<OB, 1>), dim3(blocks), dim3(256), 0, s, a);
    else if (a.rows <= 16) hipLaunchKernelGGL((rank_kernel<OB, 4>), dim3(blocks), dim3(256), 0, s, a);
    else if (a.rows <= 32) hipLaunchKernelGGL((rank_kernel<OB, 8>), dim3(blocks), dim3(256), 0, s, a);
    else if (a.rows <= 48) hipLaunchKernelGGL((rank_kernel<OB, 12>), dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((rank_kernel<OB, 16>), dim3(blocks), dim3(256), 0, s, a);
}

}  // namespace

int run_ffn_few_grad(const FfnArgs& args, const FfnPlan& p, char* ws, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    FfnArgs a = args;
    if (!a.gate) {
        a.gate = ws + p.gate;
        a.up = ws + p.up;
        const int e = run_ffn_few_gate(a, p, ws, stream);
        if (e) return e;
    }
    DownArgs g{};
    g.w[0] = (const float*)a.Wd; g.x[0] = (const float*)a.dY;
    g.rows = (int)p.t; g.cols = (int)p.f; g.k = (int)p.d; g.ldx = (int)p.d; g.act = a.act;
    g.slices = p.fdu; g.ldacc = (int)p.fk; g.acc = (float*)(ws + p.acc);
    g.gate = (const float*)a.gate; g.up = (const float*)a.up;
    g.da = (float*)(ws + p.dab); g.db = g.da + p.t * p.fk; g.u = (float*)(ws + p.u); g.ldout = (int)p.fk;
    launch_down<1>(g, s);
    if (a.dX) {
        DownArgs x{};
        x.w[0] = (const float*)a.Wg; x.w[1] = (const float*)a.Wu; x.x[0] = g.da; x.x[1] = g.db;
        x.rows = (int)p.t; x.cols = (int)p.d; x.k = (int)p.f; x.ldx = (int)p.fk;
        x.slices = p.fdx; x.ldacc = (int)p.dk; x.acc = g.acc;
        x.out = (float*)a.dX;
        launch_down<2>(x, s);
    }
    RankArgs w{};
    w.rows = (int)p.t; w.accumulate = a.accumulate;
    unsigned blocks = 0;
    const auto add = [&](RankJob j) {
        j.across = (int)ceil_div64(j.c, 256);
        j.first = blocks;
        blocks += (unsigned)(j.across * ceil_div64(j.r, kRankRows));
        w.job[w.n++] = j;
    };
    const int f = (int)p.f, d = (int)p.d, fk = (int)p.fk;
    if (a.dWg) {
        add({g.da, a.X, a.x_scale, a.dWg, fk, d, f, d});
        add({g.db, a.X, a.x_scale, a.dWu, fk, d, f, d});
    }
    if (a.dWd) add({(const float*)a.dY, g.u, nullptr, a.dWd, d, fk, d, f});
    if (w.n > 0) {
        if (a.dw_bf16) launch_rank<true>(w, blocks, s);
        else launch_rank<false>(w, blocks, s);
    }
    return (int)hipGetLastError();
}

}  // namespace dion
