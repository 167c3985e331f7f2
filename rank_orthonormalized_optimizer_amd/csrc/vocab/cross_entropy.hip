// Softmax cross entropy of a linear head, and its gradients, the logits formed where they are used.
//
//   z = H W^T (tokens x vocab);  lse = log sum_v exp z;  loss = lse - z[target]
//   D = grad (exp(z - lse) - onehot(target));  dH = D W;  dW = D^T H
//
// The tokens whose target is not ignored are first gathered into H's planes in the workspace
// (order kept, their number left in device memory), so ignored rows cost no products and whatever
// they hold reaches nothing.  The loss: one tile product over W, whose epilogue reduces each tile
// of logits to a maximum and a sum of exponentials per token (online softmax across tiles), then
// one pass over these pairs.  The gradient: per piece of the vocabulary the logits are formed
// again, turned into D (16-bit parts) and multiplied from both sides.
//
// What multiplies: bf16 operands as they are, D in one bf16 part, or two for dW of small products; three parts for an fp32 dW.
// Rounding D to one part would leave the same of every target's element where the factor is the same and the probability
// small, rows of frequent targets then off by up to 2^-8 in one direction.  What it leaves of them goes to dH and dW in fp32:
// rest[t] W[target] as dH is stored, and for dW the sums of rest[t] H[t] over the tokens of each target (sum_weighted_rows),
// which its product adds.  dW of 8192 x 32000 x 2048 against 64 bits, relative: 1.80e-3 without them, 1.65e-3 with them and for
// a correctly rounded dW.
// fp32 operands: logits and dH from two fp16 parts of W's and H's rows, each row scaled by a power of two (three products), dW
// from three bf16 parts of D and H (six: D's columns for rare tokens are too small for fp16).  fp32 and few tokens: W in place,
// split in registers (FewProduct).
//
// Bound by the matrix cores: 2 tokens vocab width flops for the loss, four times that for loss and gradients together, the
// logits formed twice.  8192 tokens (5% ignored) x 32000 x 2048 in bf16: loss 0.80 to 0.82 ms (1.25 to 1.28 PFLOP/s, of the
// 1.42 that the library's product of these sizes reaches), loss and gradients 3.40 to 3.45 ms, 0.08 of them the targets'
// elements of dW (sorting 15 us, sums 24, their rows in the product's epilogue 40); matrix cores busy 59 to 65% of the cycles.
// Without the matrix products the loss kernel takes 0.57 ms and the gradients' products 0.70 and 0.73, without the loads 0.58
// to 0.61: the two overlap but for the barrier of each slab.
//
// Where the tiles are too few for the chip, the logits' reduction over the width is sliced and the partial logits, few then,
// are stored: one pass over them makes the loss or D.
//
// In every product the vocabulary (or width) runs along the matrix core's rows and the tokens (or
// vocabulary) along its columns: a lane then holds four consecutive elements of the contiguous
// dimension of what it writes, and the softmax's reduction runs mostly inside a lane.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "dion_vocab.h"
#include "mm16.hpp"
#include "vocab_plan.h"

namespace dion {

namespace {

using mm::f32x4;
using mm::u32x2;
using mm::u32x4;

__device__ __forceinline__ float up16(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ uint32_t down16(float f) { return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f); }

// a = h + m + l exactly: h = RN(a), m = RN(a - h), l = a - h - m
__device__ __forceinline__ void split3(float a, uint32_t (&part)[3]) {
    part[0] = down16(a);
    const float r = a - up16(part[0]);
    part[1] = down16(r);
    part[2] = down16(r - up16(part[1]));
}

// a = (h + l) / scale to 2^-23 |a| and 2^-38 of the row's largest: fp16 parts of a scale, a power of two that puts the row's
// largest value into [2^13, 2^14); a low part below the normal numbers is off by up to 2^-25
__device__ __forceinline__ void split2(float a, float scale, uint32_t (&part)[2]) {
    const _Float16 h = (_Float16)(a * scale);
    const _Float16 l = (_Float16)(a * scale - (float)h);
    part[0] = (uint32_t)__builtin_bit_cast(uint16_t, h);
    part[1] = (uint32_t)__builtin_bit_cast(uint16_t, l);
}

// That scale for a row whose largest magnitude is `top`, at most 2^100: its inverse, and 2^14 over that as D is scaled, stay
// normal numbers (a row whose largest is below 2^-87 is then good to 2^-125).  And its inverse.  A row of zeros gets the
// largest scale: its inverse must not pass for the largest of a matrix.  (A row that is not finite stays as it is.)
__device__ __forceinline__ float row_scale(float top, float& inverse) {
    int e = 140 - (int)(__float_as_uint(top) >> 23);   // 127 + 13 - biased exponent
    if (!(top < INFINITY)) e = 0;
    e = e > 100 ? 100 : e;   // zero and subnormal numbers among them
    inverse = __uint_as_float((uint32_t)(127 - e) << 23);
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

// The softmax runs in powers of two.  kLog2e is log2(e) rounded to fp32; 2^fma(z, kLog2e, -c) takes e to
// z (1 + 1.3e-8), less than z's own rounding, and a sum's reference point c is kept in the same unit, so that its
// rounding drops out.  kLn2 + kLn2Low is 1 / kLog2e.
constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = (float)(1.0 / (double)kLog2e);
constexpr float kLn2Low = (float)(1.0 / (double)kLog2e - (double)kLn2);
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// exp(z - lse) to about two ulp of the difference: its rounding as a power of two is carried into the result.
__device__ __forceinline__ float exp_exact(float z, float lse) {
    const float x = z - lse, h = x * kLog2e;
    const float l = fmaf(x, kLog2e, -h) + x * 1.92596299e-8f;   // log2(e) - kLog2e
    const float r = __builtin_amdgcn_exp2f(h);
    return x < -87.f ? 0.f : fmaf(r, l * 0.693147181f, r);
}

// ---------------------------------------------------------------------------
// Gathering the rows that count
// ---------------------------------------------------------------------------
struct PackArgs {
    XentArgs x;
    int64_t n, v, d, kp, np;
    uint16_t* h;     // planes [parts][np][kp], null: not needed
    uint16_t* h16;   // fp16 planes [2][np][kp] of fp32 rows and the inverse of their scales
    float* inv;
    int* map;        // gathered row -> token
    int* tgt;        // its target, -1 where that is no row of W
    int* pos;        // token -> gathered row, 0 for the ignored ones, or null
    float2* lg;      // (lse, grad) of the gathered row (gradient)
    float* gscale;   // the power of two in grad (gradient of fp32 operands)
    int* cnt;        // how many rows were gathered
    float* factor;   // the one factor of all of them, 1 where there are none: it may be 1 / 0 then, and dW stays what it is
    int* blocks;     // rows to gather in each kCountBlock tokens, or null: few tokens
};

__device__ __forceinline__ int64_t load_target(const XentArgs& a, int64_t i) {
    return a.t64 ? ((const int64_t*)a.targets)[i] : (int64_t)((const int32_t*)a.targets)[i];
}

// Vectors at any element's address: rows of any length start there, and the memory unit takes such accesses whole.
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;

// eight elements of a row of length d from column c, zeros past its end
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t row, int64_t c, int64_t d, float (&v)[8]) {
    if (c + 8 <= d) {
        if constexpr (BF16) {
            const u32x4 w = *(const u32x4_any*)((const uint16_t*)p + row + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[2 * e] = up16(w[e]); v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u); }
        } else {
            const f32x4_any* q = (const f32x4_any*)((const float*)p + row + c);
            const f32x4 w0 = q[0], w1 = q[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[e] = w0[e]; v[4 + e] = w1[e]; }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = 0.f;
            if (c + e < d) v[e] = BF16 ? up16(((const uint16_t*)p)[row + c + e]) : ((const float*)p)[row + c + e];
        }
    }
}

template <int PARTS>
__device__ __forceinline__ void store8(uint16_t* out, int64_t plane, int64_t i, const float (&v)[8]) {
    uint32_t part[8][3];
#pragma unroll
    for (int e = 0; e < 8; ++e) split3(v[e], part[e]);
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = part[2 * e][q] | (part[2 * e + 1][q] << 16);
        *(u32x4*)(out + q * plane + i) = w;
    }
}

__device__ __forceinline__ void store8_f16(uint16_t* out, int64_t plane, int64_t i, const float (&v)[8], float scale) {
    uint32_t part[8][2];
#pragma unroll
    for (int e = 0; e < 8; ++e) split2(v[e], scale, part[e]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = part[2 * e][q] | (part[2 * e + 1][q] << 16);
        *(u32x4*)(out + q * plane + i) = w;
    }
}

// One row of a matrix to its planes by one wave: fp32 rows become fp16 planes with the row's scale (p16, inv, if p16 is
// given) and bf16 planes (p, if given); bf16 rows are copied to p.  Columns up to kp are zero.
template <bool BF16>
__device__ __forceinline__ void pack_row(const void* in, int64_t row, int64_t d, int64_t kp, uint16_t* p, int64_t plane,
                                         uint16_t* p16, int64_t plane16, float* inv, int64_t to, int lane) {
    float scale = 1.f;
    if (!BF16 && p16) {
        float top = 0.f;
#pragma unroll 4
        for (int64_t c = lane * 8; c < kp; c += 512) {
            float v[8];
            load8<BF16>(in, row * d, c, d, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        float inverse;
        scale = row_scale(top, inverse);
        if (lane == 0) inv[to] = inverse;
    }
#pragma unroll 4
    for (int64_t c = lane * 8; c < kp; c += 512) {
        float v[8];
        load8<BF16>(in, row * d, c, d, v);
        if (!BF16 && p16) store8_f16(p16, plane16, to * kp + c, v, scale);
        if (p) store8<BF16 ? 1 : 3>(p, plane, to * kp + c, v);
    }
}

constexpr int kPackRows = 8;

// How many rows to gather in each kCountBlock tokens.
__global__ __launch_bounds__(512) void count_kernel(PackArgs a) {
    __shared__ int part[8];
    const int64_t t0 = (int64_t)blockIdx.x * kCountBlock;
    int c = 0;
#pragma unroll
    for (int i = 0; i < kCountBlock / 512; ++i) {
        const int64_t t = t0 + i * 512 + threadIdx.x;
        if (t < a.n) c += load_target(a.x, t) != a.x.ignore;
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) c += __shfl_xor(c, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = c;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) c += part[i];
        a.blocks[blockIdx.x] = c;
    }
}

// Eight tokens per workgroup, one per wave.  The workgroup counts the gathered rows before its own itself, a read of
// the targets (or of the counts of whole blocks, and the targets since the last one) from L2.
template <bool BF16, bool GRAD>
__global__ __launch_bounds__(512) void pack_kernel(PackArgs a) {
    __shared__ int before[8], slot[kPackRows];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * kPackRows;
    int c = 0;
    const int64_t from = a.blocks ? t0 / kCountBlock * kCountBlock : 0;
    if (a.blocks)
        for (int64_t i = tid; i < t0 / kCountBlock; i += 512) c += a.blocks[i];
#pragma unroll 8
    for (int64_t i = from + tid; i < t0; i += 512) c += load_target(a.x, i) != a.x.ignore;
#pragma unroll
    for (int o = 32; o; o >>= 1) c += __shfl_xor(c, o);
    if (lane == 0) before[w] = c;
    __syncthreads();
    if (w == 0) {
        const int64_t t = t0 + lane;
        const bool row = lane < kPackRows && t < a.n;
        const int64_t y = row ? load_target(a.x, t) : 0;
        const bool keep = row && y != a.x.ignore;
        const uint64_t kept = __ballot(keep);
        int base = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) base += before[i];
        const int j = base + __popcll(kept & ((1ull << lane) - 1));
        if (lane < kPackRows) slot[lane] = keep ? j : -1;
        if (GRAD && row && a.pos) a.pos[t] = keep ? j : 0;
        if (keep) {
            const bool in = y >= 0 && y < a.v;
            a.map[j] = (int)t;
            a.tgt[j] = in ? (int)y : -1;
            if (GRAD) {
                // one factor for all tokens is applied to the outputs: in D it would be rounded the same way everywhere
                const float g = a.x.grad_n == 1 ? 1.f : a.x.grad[t];
                a.lg[j] = float2{a.x.lse[t], in ? g : __uint_as_float(0x7fc00000u)};
                const int e = (int)(__float_as_uint(g) >> 23 & 255u);
                if (a.gscale) a.gscale[j] = e > 0 && e < 255 ? __uint_as_float((uint32_t)e << 23) : 1.f;   // g / gscale in [1, 2)
            }
        } else if (row && !GRAD) {
            a.x.loss[t] = 0.f;
            a.x.lse_out[t] = 0.f;
        }
        if (lane == 0 && blockIdx.x == gridDim.x - 1) {
            const int all = base + __popcll(kept);
            a.cnt[0] = all;
            if (GRAD && a.x.grad_n == 1) *a.factor = all > 0 ? a.x.grad[0] : 1.f;
        }
    }
    __syncthreads();
    const int64_t t = t0 + w;
    if (t >= a.n) return;
    if (slot[w] >= 0) {
        pack_row<BF16>(a.x.H, t, a.d, a.kp, a.h, a.np * a.kp, a.h16, a.np * a.kp, a.inv, slot[w], lane);
    } else if (GRAD && a.x.dH) {
        for (int64_t col = lane; col < a.d; col += 64) {
            if (BF16) ((uint16_t*)a.x.dH)[t * a.d + col] = 0;
            else ((float*)a.x.dH)[t * a.d + col] = 0.f;
        }
    }
}

// The largest of n inverse scales, to out.
__global__ __launch_bounds__(1024) void top_kernel(const float* inv, int n, float* out) {
    __shared__ float part[16];
    float top = 0.f;
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += 1024) top = fmaxf(top, inv[i]);
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i) top = fmaxf(top, part[i]);
        *out = top;
    }
}

// Planes of `rows` rows of W (from row0), a wave per row: fp16 ones of fp32 rows, a copy of bf16 ones.
template <bool BF16>
__global__ __launch_bounds__(256) void plane_kernel(const void* W, int64_t row0, int64_t rows, int64_t d, int64_t kp,
                                                    uint16_t* p, uint16_t* p16, int64_t plane, float* inv) {
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r < rows)
        pack_row<BF16>((const char*)W + row0 * d * (BF16 ? 2 : 4), r, d, kp, p, plane, p16, plane, inv, r, threadIdx.x & 63);
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// The tiles of this workgroup.  Workgroups go to the eight XCDs in turn; each XCD takes a contiguous
// range of the tiles and its workgroups walk it side by side, in bands of eight tile rows, so that
// its L2 serves the operands' re-reads.
struct Walk {
    int tm, tn, at, end, by;
    __device__ __forceinline__ Walk(int tm_, int tn_, int slices) : tm(tm_), tn(tn_) {
        const int total = tm * tn * slices, q = total / 8, r = total % 8, x = blockIdx.x % 8;
        const int start = x * q + (x < r ? x : r);
        by = ((int)gridDim.x - x + 7) / 8;   // workgroups on this XCD
        at = start + blockIdx.x / 8;
        end = start + q + (x < r ? 1 : 0);
    }
    __device__ __forceinline__ bool done() const { return at >= end; }
    __device__ __forceinline__ void next() { at += by; }
    __device__ __forceinline__ void tile(int& mt, int& nt, int& slice) const {
        constexpr int G = 8;
        slice = at / (tm * tn);
        const int t = at - slice * tm * tn;
        const int band = t / (G * tn), m0 = band * G, g = tm - m0 < G ? tm - m0 : G, in = t - band * G * tn;
        mt = m0 + in % g;
        nt = in / g;
    }
};

struct LogitArgs {
    mm::Operand w, h;      // w.rows: rows of this piece; h.rows is read from cnt
    mm::Segments seg;
    int kp;
    const int* cnt;
    const int* tgt;
    const float* hinv;     // F16: inverse scales of the rows of H's and W's fp16 planes
    const float* winv;
    int v0;                // first vocabulary row of the piece
    // loss
    float2* part;          // [np][nvt] maximum of a tile of logits and sum of exponentials, as powers of two
    float* zt;             // the target's logit
    int nvt;
    // gradient
    const float2* lg;
    uint16_t* dl;          // planes [dparts][np][piece]
    uint16_t* dl16;        // F16: fp16 planes [2][np][piece] of D times W's inverse row scales, for dH
    const float* gscale;
    const float* wtop;     // F16: the largest of the piece's inverse row scales
    float* rest;           // [np] what the first part of D leaves of the target's element, for dH and (one part) dW
    int64_t np, piece;
};

enum { EPI_LOSS, EPI_D1, EPI_D2, EPI_D3 };

// Stores a lane's 4-row pieces of two neighbouring blocks of 16 rows: the lane quarters trade their four rows of one
// against the other's (v_permlane32_swap, v_permlane16_swap), so that a lane stores eight consecutive rows and four lanes
// 64 bytes.  a, b: the four values of each block, packed in two words; to: the address for this lane's quarter.
__device__ __forceinline__ void store_pair(uint16_t* to, const uint32_t (&a)[2], const uint32_t (&b)[2], bool in) {
    u32x4 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto x = __builtin_amdgcn_permlane32_swap(a[h], b[h], false, false);
        const auto z = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
        w[h] = z[0];
        w[2 + h] = z[1];
    }
    if (in) *(u32x4*)to = w;
}

template <class C, int EPI>
__global__ __launch_bounds__(C::THREADS) void logit_kernel(LogitArgs a) {
    __shared__ __attribute__((aligned(1024))) uint16_t lds[C::kLds];
    __shared__ float2 red[EPI == EPI_LOSS ? C::WM * C::BN : 1];
    const int count = a.cnt[0], rows = a.w.rows;
    Walk walk((rows + C::BM - 1) / C::BM, (count + C::BN - 1) / C::BN, 1);
    if (walk.done()) return;
    a.h.rows = count;
    typename mm::ProductOf<C>::type mul(lds);
    int mt, nt, slice;
    walk.tile(mt, nt, slice);
    mul.start(a.w, a.h, mt * C::BM, nt * C::BN, 0, a.kp, a.seg);
    const int rl = mul.xa + 4 * (mul.lane / 16);   // this lane's first row in the tile, + 16 i + v
    const int cl = mul.xb + mul.lane % 16;         // its first column, + 16 j
    for (;;) {
        const int m0 = mul.m0, n0 = mul.n0;
        int y[C::NI];
        float2 lg[C::NI];
        float hinv[C::F16 ? C::NI : 1], gs[C::F16 ? C::NI : 1];
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const int n = n0 + cl + 16 * j, nn = n < count ? n : count - 1;
            y[j] = a.tgt[nn] - a.v0;
            if (C::F16) hinv[j] = a.hinv[nn];
            if (EPI != EPI_LOSS) lg[j] = a.lg[nn];
            if (EPI != EPI_LOSS && C::F16) gs[j] = a.gscale[nn];
        }
        typename C::Acc acc = {};
        mul.finish(a.w, a.h, acc);
        walk.next();
        const bool more = !walk.done();
        if (more) {
            walk.tile(mt, nt, slice);
            mul.start(a.w, a.h, mt * C::BM, nt * C::BN, 0, a.kp, a.seg);
        }
        if constexpr (C::F16) {
#pragma unroll
            for (int i = 0; i < C::MI; ++i) {
                const int m = m0 + rl + 16 * i;   // (winv is allocated for whole tiles)
                const f32x4 s = *(const f32x4*)(a.winv + m);
#pragma unroll
                for (int j = 0; j < C::NI; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] = acc[i][j][v] * hinv[j] * s[v];
            }
        }
        if (m0 + C::BM > rows) {
#pragma unroll
            for (int i = 0; i < C::MI; ++i)
#pragma unroll
                for (int j = 0; j < C::NI; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (m0 + rl + 16 * i + v >= rows) acc[i][j][v] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const int n = n0 + cl + 16 * j;
            // the target's element is this lane's if it is 16 i + v rows behind its first; few tiles of a column have it
            const int at = y[j] - m0 - rl;
            const bool mine = n < count && at >= 0 && (at & 15) < 4 && at < 16 * C::MI && y[j] < rows;
            if constexpr (EPI == EPI_LOSS) {
                if (__any(mine)) {
#pragma unroll
                    for (int i = 0; i < C::MI; ++i)
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (mine && at == 16 * i + v) a.zt[n] = acc[i][j][v];
                }
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < C::MI; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) mx = fmaxf(mx, acc[i][j][v]);
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32)) * kLog2e;
                const float ref = mx == -INFINITY ? 0.f : mx;   // an empty or all-minus-infinity column sums to 0, NaN to NaN
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < C::MI; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) s += exp2_fast(fmaf(acc[i][j][v], kLog2e, -ref));
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                if (mul.lane < 16) red[mul.wave % C::WM * C::BN + cl + 16 * j] = float2{mx, s};
            } else {
                constexpr int PD = EPI == EPI_D3 ? 3 : EPI == EPI_D2 ? 2 : 1;
                const float c = lg[j].x * kLog2e;
#pragma unroll
                for (int i = 0; i < C::MI; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[i][j][v] = PD == 3 ? exp_exact(acc[i][j][v], lg[j].x) : exp2_fast(fmaf(acc[i][j][v], kLog2e, -c));
                if (__any(mine)) {
                    float d = 0.f;
#pragma unroll
                    for (int i = 0; i < C::MI; ++i)
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (mine && at == 16 * i + v) {
                                acc[i][j][v] -= 1.f;
                                d = acc[i][j][v] * lg[j].y;
                            }
                    if (mine) a.rest[n] = d - up16(down16(d));
                }
                // A lane has four consecutive rows of a block of 16, and stores two blocks at a time, where there are two.
                const int quarter = mul.lane / 16;
                const int64_t at8 = n * a.piece + m0 + mul.xa + 16 * (quarter / 2) + 8 * (quarter % 2);
#pragma unroll
                for (int i = 0; i < C::MI; i += 2) {
                    constexpr bool kPairs = C::MI % 2 == 0;
                    uint32_t part[2][4][3];
#pragma unroll
                    for (int h = 0; h < (kPairs ? 2 : 1); ++h)
#pragma unroll
                        for (int v = 0; v < 4; ++v) split3(acc[i + h][j][v] * lg[j].y, part[h][v]);
                    if (a.dl) {
#pragma unroll
                        for (int q = 0; q < PD; ++q) {
                            const uint32_t w0[2] = {part[0][0][q] | (part[0][1][q] << 16), part[0][2][q] | (part[0][3][q] << 16)};
                            if constexpr (kPairs) {
                                const uint32_t w1[2] = {part[1][0][q] | (part[1][1][q] << 16), part[1][2][q] | (part[1][3][q] << 16)};
                                store_pair(a.dl + q * a.np * a.piece + at8 + 16 * i, w0, w1, n < count);
                            } else if (n < count) {
                                *(u32x2*)(a.dl + (q * a.np + n) * a.piece + m0 + rl + 16 * i) = u32x2{w0[0], w0[1]};
                            }
                        }
                    }
                }
                if constexpr (C::F16) {
                    if (a.dl16) {
                        // |D / gscale| < 2 and an inverse scale is at most wtop: the product goes to below 2^15
                        const float unit = lg[j].y / gs[j] * (16384.f / a.wtop[0]);
#pragma unroll
                        for (int i = 0; i < C::MI; i += 2) {
                            uint32_t w[2][2][2];   // [block][part][word]
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                f32x4 s = *(const f32x4*)(a.winv + m0 + rl + 16 * (i + h));
                                if (m0 + C::BM > rows) {   // no scales behind the piece's rows, whose D is 0
#pragma unroll
                                    for (int v = 0; v < 4; ++v)
                                        if (m0 + rl + 16 * (i + h) + v >= rows) s[v] = 0.f;
                                }
                                uint32_t part[4][2];
#pragma unroll
                                for (int v = 0; v < 4; ++v) split2(acc[i + h][j][v], unit * s[v], part[v]);
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    w[h][q][0] = part[0][q] | (part[1][q] << 16);
                                    w[h][q][1] = part[2][q] | (part[3][q] << 16);
                                }
                            }
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                store_pair(a.dl16 + q * a.np * a.piece + at8 + 16 * i, w[0][q], w[1][q], n < count);
                        }
                    }
                }
            }
        }
        if constexpr (EPI == EPI_LOSS) {
            __syncthreads();
            for (int c = threadIdx.x; c < C::BN && n0 + c < count; c += C::THREADS) {
                float2 t = red[c];
#pragma unroll
                for (int i = 1; i < C::WM; ++i) {
                    const float2 u = red[i * C::BN + c];
                    const float m = fmaxf(t.x, u.x), ref = m == -INFINITY ? 0.f : m;
                    t.y = t.y * exp2_fast(t.x - ref) + u.y * exp2_fast(u.x - ref);
                    t.x = m;
                }
                a.part[(int64_t)(n0 + c) * a.nvt + (a.v0 + m0) / C::BM] = t;
            }
        }
        if (!more) return;   // (the barriers of the next tile's product come before red is written again)
    }
}

// loss and lse of the gathered tokens from their tiles' pairs, one wave per token
__global__ __launch_bounds__(256) void loss_kernel(const float2* part, const float* zt, const int* tgt, const int* map,
                                                   const int* cnt, int nvt, float* loss, float* lse) {
    const int j = (int)(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63;
    if (j >= cnt[0]) return;
    float m = -INFINITY, s = 0.f;
    for (int i = lane; i < nvt; i += 64 * 8) {
        float2 u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = i + 64 * e < nvt ? part[(int64_t)j * nvt + i + 64 * e] : float2{-INFINITY, 0.f};
        float top = m;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, u[e].x);
        const float ref = top == -INFINITY ? 0.f : top;
        s *= exp2_fast(m - ref);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(u[e].y, exp2_fast(u[e].x - ref), s);
        m = top;
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const float um = __shfl_xor(m, o), us = __shfl_xor(s, o);
        const float top = fmaxf(m, um), ref = top == -INFINITY ? 0.f : top;
        s = s * exp2_fast(m - ref) + us * exp2_fast(um - ref);
        m = top;
    }
    if (lane == 0) {
        const float ls = logf(s), low = m * kLn2Low;
        lse[map[j]] = fmaf(m, kLn2, ls) + low;
        loss[map[j]] = tgt[j] < 0 ? __uint_as_float(0x7fc00000u) : fmaf(m, kLn2, -zt[j]) + (ls + low);
    }
}

struct OutArgs {
    mm::Operand a, b;
    mm::Segments seg;
    const int* cnt;
    int d, dp;             // output columns (the matrix core's rows), and rounded up to four
    int rows;              // output rows, or -1: the gathered tokens
    int k;                 // reduction length, or -1: the gathered tokens
    int split, k_per;      // slices of the reduction and their length
    float* acc;            // fp32 [split][acc_rows][dp], or null: straight to out
    int64_t acc_rows;
    int add;               // add to acc
    void* out;
    const int* map;        // output row of a gathered token, or null
    int out_bf16, accumulate;
    const float* factor;   // of the outputs, or null
    const float* wtop;     // D and W were scaled: multiply by *wtop 2^-14 (each piece's own) and by the row's scale; or null
    const float* row_scale;
    // dH in bf16: what the rounding of D left of the target's element, times the target's row of W
    const float* rest;     // or null
    const int* tgt;
    const uint16_t* w;     // bf16 [vocab][d]
    // dW in bf16: the same for its rows, summed over the tokens by sum_weighted_rows
    const int* slot;       // [rows], or null
    const float* extra;
};

// the row of extra for output row r, or null
__device__ __forceinline__ const float* extra_row(const OutArgs& a, int64_t r) {
    const int s = a.slot ? a.slot[r] : 0;
    return s > 0 ? a.extra + (s - 1) * (int64_t)a.dp : nullptr;
}

// n elements of the output from column c of row r of the reduction's result: four, fewer at a ragged end
__device__ __forceinline__ void store_out(const OutArgs& a, int64_t r, int c, int n, float (&v)[4]) {
    if (a.rest && a.tgt[r] >= 0) {
        const float left = a.rest[r];
        const uint16_t* w = a.w + (int64_t)a.tgt[r] * a.d + c;
        if (n == 4) {
            const u32x2 x = *(const u32x2_any*)w;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(left, up16((x[e / 2] >> (16 * (e % 2))) & 0xffffu), v[e]);
        } else {
            for (int e = 0; e < n; ++e) v[e] = fmaf(left, up16(w[e]), v[e]);
        }
    }
    if (a.row_scale) {
        const float f = a.row_scale[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= f;
    }
    if (a.factor) {
        const float f = *a.factor;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= f;
    }
    const int64_t at = (a.map ? a.map[r] : r) * (int64_t)a.d + c;
    if (n == 4) {
        float o[4];
        if (a.out_bf16) {
            u32x2_any* p = (u32x2_any*)((uint16_t*)a.out + at);
            u32x2 w{0, 0};
            if (a.accumulate) w = *p;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = v[e] + (a.accumulate ? up16((w[e / 2] >> (16 * (e % 2))) & 0xffffu) : 0.f);
            *p = u32x2{down16(o[0]) | (down16(o[1]) << 16), down16(o[2]) | (down16(o[3]) << 16)};
        } else {
            f32x4_any* p = (f32x4_any*)((float*)a.out + at);
            f32x4 w{0.f, 0.f, 0.f, 0.f};
            if (a.accumulate) w = *p;
            *p = f32x4{w[0] + v[0], w[1] + v[1], w[2] + v[2], w[3] + v[3]};
        }
    } else {
        for (int e = 0; e < n; ++e) {
            if (a.out_bf16) {
                uint16_t* p = (uint16_t*)a.out + at + e;
                *p = (uint16_t)down16(v[e] + (a.accumulate ? up16(*p) : 0.f));
            } else {
                float* p = (float*)a.out + at + e;
                *p = v[e] + (a.accumulate ? *p : 0.f);
            }
        }
    }
}

template <class C>
__global__ __launch_bounds__(C::THREADS) void out_kernel(OutArgs a) {
    __shared__ __attribute__((aligned(1024))) uint16_t lds[C::kLds];
    const int count = a.cnt[0], rows = a.rows < 0 ? count : a.rows, k = a.k < 0 ? (count + 63) / 64 * 64 : a.k;
    Walk walk((a.d + C::BM - 1) / C::BM, (rows + C::BN - 1) / C::BN, a.split);
    if (walk.done()) return;
    if (a.k < 0) a.a.rows = count;   // dW reduces over the tokens
    a.b.rows = count;
    typename mm::ProductOf<C>::type mul(lds);
    int mt, nt, slice;
    auto start = [&]() {   // false: a slice without any k
        walk.tile(mt, nt, slice);
        const int k0 = slice * a.k_per, k1 = k0 + a.k_per < k ? k0 + a.k_per : k;
        mul.m0 = mt * C::BM;
        mul.n0 = nt * C::BN;
        if (k0 < k1) mul.start(a.a, a.b, mul.m0, mul.n0, k0, k1, a.seg);
        return k0 < k1;
    };
    bool any = start();
    for (;;) {
        const int m0 = mul.m0, n0 = mul.n0, sl = slice;
        typename C::Acc acc = {};
        if (any) mul.finish(a.a, a.b, acc);
        walk.next();
        const bool more = !walk.done();
        if (more) any = start();
        if (a.wtop) {
            const float f = a.wtop[0] * (1.f / 16384.f);
#pragma unroll
            for (int i = 0; i < C::MI; ++i)
#pragma unroll
                for (int j = 0; j < C::NI; ++j) acc[i][j] *= f;
        }
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const int n = n0 + mul.xb + 16 * j + mul.lane % 16;
            if (n >= rows) continue;
            if constexpr (C::TA && C::TB) {   // dW
                if (const float* extra = a.acc ? nullptr : extra_row(a, n)) {   // all of a row before its stores, which they cannot pass
#pragma unroll
                    for (int i = 0; i < C::MI; ++i) {
                        const int m = m0 + mul.xa + 16 * i + 4 * (mul.lane / 16);
                        if (m < a.d) acc[i][j] += *(const f32x4*)(extra + m);   // (rows of a multiple of four)
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < C::MI; ++i) {
                const int m = m0 + mul.xa + 16 * i + 4 * (mul.lane / 16);
                if (m >= a.d) continue;
                float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                if (!a.acc) {
                    store_out(a, n, m, a.d - m < 4 ? a.d - m : 4, v);
                } else {
                    f32x4* p = (f32x4*)(a.acc + (sl * a.acc_rows + n) * a.dp + m);
                    *p = a.add ? *p + acc[i][j] : acc[i][j];
                }
            }
        }
        if (!more) return;
    }
}

// dW of up to N tokens, a stream of writes: four columns of H's rows per thread in registers, D's columns in LDS, fp32 sums.
// D and H come from the parts that the other products use.
template <int N>
__global__ __launch_bounds__(256) void rank_out_kernel(OutArgs a, int hparts, int dparts) {
    constexpr int R = 64;
    __shared__ __attribute__((aligned(16))) float d[R][N];
    const int count = a.cnt[0], c = (int)(blockIdx.y * 256 + threadIdx.x) * 4, n = a.d - c < 4 ? a.d - c : 4;
    f32x4 h[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        h[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (j < count && n > 0)   // (H's planes have columns up to a multiple of 64)
            for (int q = hparts - 1; q >= 0; --q) {
                const u32x2 w = *(const u32x2*)(a.a.p + q * a.a.plane + j * a.a.ld + c);
                h[j] += f32x4{up16(w[0] & 0xffffu), up16(w[0] >> 16), up16(w[1] & 0xffffu), up16(w[1] >> 16)};
            }
    }
    for (int r0 = blockIdx.x * R; r0 < a.rows; r0 += gridDim.x * R) {
        __syncthreads();
        for (int i = threadIdx.x; i < R * N; i += 256) {
            const int r = i % R, j = i / R;
            float x = 0.f;
            if (j < count && r0 + r < a.rows)
                for (int q = dparts - 1; q >= 0; --q) x += up16(a.b.p[q * a.b.plane + j * a.b.ld + r0 + r]);
            d[r][j] = x;
        }
        __syncthreads();
        if (n <= 0) continue;
        const int rows = a.rows - r0 < R ? a.rows - r0 : R;
#pragma unroll 2
        for (int r = 0; r < rows; ++r) {
            f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float x = d[r][j];
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = fmaf(x, h[j][e], sum[e]);
            }
            float v[4] = {sum[0], sum[1], sum[2], sum[3]};
            store_out(a, r0 + r, c, n, v);
        }
    }
}

// The slices' sums, rounded to the output: four columns per group of G lanes, which share the slices (many slices come
// with few outputs).
template <int G>
__global__ __launch_bounds__(256) void join_kernel(OutArgs a) {
    const int rows = a.rows < 0 ? a.cnt[0] : a.rows, nc = a.dp / 4;
    const int lane = threadIdx.x % G;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G; i < (int64_t)rows * nc; i += (int64_t)gridDim.x * (256 / G)) {
        const int64_t r = i / nc;
        const int c = (int)(i - r * nc) * 4, n = a.d - c < 4 ? a.d - c : 4;
        f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = lane; s < a.split; s += G) sum += *(const f32x4*)(a.acc + (s * a.acc_rows + r) * a.dp + c);
        float v[4] = {sum[0], sum[1], sum[2], sum[3]};
#pragma unroll
        for (int o = G / 2; o; o >>= 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], o);
        if (lane == 0) {
            if (const float* extra = extra_row(a, r)) {
                const f32x4 x = *(const f32x4*)(extra + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += x[e];
            }
            store_out(a, r, c, n, v);
        }
    }
}

// Logits whose reduction was sliced: partial sums [split][n][piece], and the scales of fp16 parts (or null).
struct SliceArgs {
    const float* z;
    int64_t n, piece;
    int split, v;
    const int* cnt;
    const float* hinv;
    const float* winv;
    // D
    const int* tgt;
    const float2* lg;
    const float* gscale;
    const float* wtop;
    uint16_t* dl;
    uint16_t* dl16;
    float* rest;
    int64_t np;
};

// logits v .. v + 3 of gathered token j, -inf behind the vocabulary
__device__ __forceinline__ f32x4 sum_slices(const SliceArgs& a, int64_t j, int v) {
    f32x4 z{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.split; ++s) z += *(const f32x4*)(a.z + (s * a.n + j) * a.piece + v);
    if (a.winv) {
        const f32x4 w = *(const f32x4*)(a.winv + v);
        const float h = a.hinv[j];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = z[e] * h * w[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (v + e >= a.v) z[e] = -INFINITY;
    return z;
}

// loss and lse from sliced logits, T threads (64 or 256) per gathered token
template <int T>
__global__ __launch_bounds__(256) void slice_loss_kernel(SliceArgs a, const int* map, float* loss, float* lse) {
    __shared__ float2 red[4];
    __shared__ float target[4];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, team = threadIdx.x / T, at = threadIdx.x % T;
    const int64_t j = (int64_t)blockIdx.x * (256 / T) + team;
    const bool row = j < a.cnt[0];
    float m = -INFINITY, s = 0.f;
    if (row) {
        const int y = a.tgt[j];
        for (int v = at * 4; v < a.v; v += T * 4) {
            const f32x4 z = sum_slices(a, j, v);
            float top = m;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, z[e] * kLog2e);
            const float ref = top == -INFINITY ? 0.f : top;
            s *= exp2_fast(m - ref);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s += exp2_fast(fmaf(z[e], kLog2e, -ref));
                if (v + e == y) target[team] = z[e];
            }
            m = top;
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const float um = __shfl_xor(m, o), us = __shfl_xor(s, o);
        const float top = fmaxf(m, um), ref = top == -INFINITY ? 0.f : top;
        s = s * exp2_fast(m - ref) + us * exp2_fast(um - ref);
        m = top;
    }
    if (lane == 0) red[w] = float2{m, s};
    __syncthreads();
    if (at != 0 || !row) return;
    if (T == 256) {
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const float top = fmaxf(m, red[i].x), ref = top == -INFINITY ? 0.f : top;
            s = s * exp2_fast(m - ref) + red[i].y * exp2_fast(red[i].x - ref);
            m = top;
        }
    }
    const float ls = logf(s), low = m * kLn2Low;
    lse[map[j]] = fmaf(m, kLn2, ls) + low;
    loss[map[j]] = a.tgt[j] < 0 ? __uint_as_float(0x7fc00000u) : fmaf(m, kLn2, -target[team]) + (ls + low);
}

// D from sliced logits as logit_kernel forms it, eight of a token's per thread, zeros up to a multiple of 64.
template <int EPI>
__global__ __launch_bounds__(256) void slice_grad_kernel(SliceArgs a) {
    constexpr int PD = EPI == EPI_D3 ? 3 : EPI == EPI_D2 ? 2 : 1;
    const int64_t j = blockIdx.y;
    const int v = (int)(blockIdx.x * 256 + threadIdx.x) * 8;
    if (j >= a.cnt[0] || v >= (a.v + 63) / 64 * 64) return;
    const int y = a.tgt[j];
    const float2 lg = a.lg[j];
    const f32x4 z0 = sum_slices(a, j, v), z1 = sum_slices(a, j, v + 4);
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float z = e < 4 ? z0[e & 3] : z1[e & 3];
        p[e] = PD == 3 ? exp_exact(z, lg.x) : exp2_fast(fmaf(z, kLog2e, -(lg.x * kLog2e)));
        if (v + e == y) {
            p[e] -= 1.f;
            const float d = p[e] * lg.y;
            a.rest[j] = d - up16(down16(d));
        }
    }
    if (a.dl) {
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = p[e] * lg.y;
        store8<PD>(a.dl, a.np * a.piece, j * a.piece + v, d);
    }
    if (a.dl16) {
        const float unit = lg.y / a.gscale[j] * (16384.f / a.wtop[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = v + e < a.v ? p[e] * (unit * a.winv[v + e]) : 0.f;
        store8_f16(a.dl16, a.np * a.piece, j * a.piece + v, p, 1.f);
    }
}

// plane pairs (A's part, B's part), smallest products first
mm::Segments segments(int pa, int pb) {
    auto list = [](std::initializer_list<int> e) {
        mm::Segments s{0, 0};
        for (int x : e) s.list |= (uint32_t)x << (4 * s.n++);
        return s;
    };
    if (pa == 3 && pb == 3) return list({1 | 1 << 2, 0 | 2 << 2, 2 | 0 << 2, 0 | 1 << 2, 1 | 0 << 2, 0});
    if (pa == 2) return list({1, 1 << 2, 0});   // fp16 parts h, l: l h, h l, h h
    if (pb == 3) return list({2 << 2, 1 << 2, 0});
    if (pb == 2) return list({1 << 2, 0});
    return list({0});
}

using Z256 = mm::Config<256, 256, 2, 4, 2, false, false>;
using Z128 = mm::Config<128, 128, 2, 2, 4, false, false>;
using Z32 = mm::Config<128, 32, 4, 1, 4, false, false>;
using Z64 = mm::Config<64, 64, 2, 2, 8, false, false>;
using F64 = mm::Config<64, 64, 2, 2, 8, false, false, true>;
using F256 = mm::Config<256, 256, 2, 4, 2, false, false, true>;
using F128 = mm::Config<128, 128, 2, 2, 4, false, false, true>;
template <bool V4> using P32 = mm::FewConfig<32, 3, false, V4>;
template <bool V4> using P64 = mm::FewConfig<64, 2, false, V4>;
template <bool V4> using Q32 = mm::FewConfig<32, 3, true, V4>;
template <bool V4> using Q64 = mm::FewConfig<64, 2, true, V4>;
using E256 = mm::Config<256, 256, 2, 4, 2, true, false, true>;
using E128 = mm::Config<128, 128, 2, 2, 4, true, false, true>;
using E64 = mm::Config<64, 64, 2, 2, 8, true, false, true>;
using H256 = mm::Config<256, 256, 2, 4, 2, true, false>;
using H128 = mm::Config<128, 128, 2, 2, 4, true, false>;
using H32 = mm::Config<128, 32, 4, 1, 4, true, false>;
using H64 = mm::Config<64, 64, 2, 2, 8, true, false>;
using W64 = mm::Config<64, 64, 2, 2, 8, true, true>;
using W256 = mm::Config<256, 256, 2, 4, 2, true, true>;
using Ws = mm::Config<128, 64, 2, 2, 2, true, true>;
using W128 = mm::Config<128, 128, 2, 2, 4, true, true>;

// One workgroup per tile, or as many as the chip holds, which then walk the tiles.
template <class C>
dim3 walkers(int64_t tiles) {
    return dim3((unsigned)(tiles < kCUs * C::kPerCU ? tiles : kCUs * C::kPerCU));
}

template <class C, int EPI>
void launch_logits(const LogitArgs& a, int64_t n, hipStream_t s) {
    const int64_t t = ceil_div64(a.w.rows, C::BM) * ceil_div64(n, C::BN);
    hipLaunchKernelGGL((logit_kernel<C, EPI>), walkers<C>(t), dim3(C::THREADS), 0, s, a);
}

template <bool V4, int EPI>
void launch_few_logits(const LogitArgs& a, int64_t n, hipStream_t s) {
    if (n <= 32) launch_logits<P32<V4>, EPI>(a, n, s);
    else launch_logits<P64<V4>, EPI>(a, n, s);
}

template <int EPI>
void launch_logits(const LogitArgs& a, const XentPlan& p, hipStream_t s) {
    if (p.parts == 1) {
        if (p.tile_z == TILE_256) launch_logits<Z256, EPI>(a, p.n, s);
        else if (p.tile_z == TILE_128) launch_logits<Z128, EPI>(a, p.n, s);
        else if (p.tile_z == TILE_64) launch_logits<Z64, EPI>(a, p.n, s);
        else launch_logits<Z32, EPI>(a, p.n, s);
    } else if constexpr (EPI == EPI_LOSS || EPI == EPI_D3) {   // fp32: D in three parts; more than kFewTokens tokens where W goes through planes
        if (p.few && p.d % 4 == 0) launch_few_logits<true, EPI>(a, p.n, s);
        else if (p.few) launch_few_logits<false, EPI>(a, p.n, s);
        else if (p.tile_z == TILE_256) launch_logits<F256, EPI>(a, p.n, s);
        else if (p.tile_z == TILE_128) launch_logits<F128, EPI>(a, p.n, s);
        else launch_logits<F64, EPI>(a, p.n, s);
    }
}

template <bool GRAD>
void launch_pack(const PackArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div64(a.n, kPackRows));
    if (a.blocks) hipLaunchKernelGGL(count_kernel, dim3((unsigned)ceil_div64(a.n, kCountBlock)), dim3(512), 0, s, a);
    if (a.x.bf16) hipLaunchKernelGGL((pack_kernel<true, GRAD>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((pack_kernel<false, GRAD>), grid, dim3(512), 0, s, a);
}

// W's rows [v0, v0 + rows) as an operand of both products over W: in place (bf16, or fp32 for few tokens), or as planes in
// the workspace, fp16 ones of fp32 rows, with the largest inverse scale if `top`.
mm::Operand weights(const XentArgs& x, const XentPlan& p, char* ws, int64_t v0, int64_t rows, bool top, hipStream_t s) {
    if (!p.wpack)
        return mm::Operand{(const uint16_t*)((const char*)x.W + v0 * p.d * (x.bf16 ? 2 : 4)), 0, p.d, (int)rows};
    uint16_t* w = (uint16_t*)(ws + p.w);
    uint16_t* w16 = x.bf16 ? nullptr : w;
    if (!x.bf16) w = nullptr;
    float* inv = (float*)(ws + p.winv);
    const int64_t plane = p.piece * p.kp;
    const dim3 grid((unsigned)ceil_div64(rows, 4));
    if (x.bf16) {
        hipLaunchKernelGGL((plane_kernel<true>), grid, dim3(256), 0, s, x.W, v0, rows, p.d, p.kp, w, w16, plane, inv);
    } else {
        hipLaunchKernelGGL((plane_kernel<false>), grid, dim3(256), 0, s, x.W, v0, rows, p.d, p.kp, w, w16, plane, inv);
        if (top) hipLaunchKernelGGL(top_kernel, dim3(1), dim3(1024), 0, s, inv, (int)rows, (float*)(ws + p.wtop));
    }
    return mm::Operand{(uint16_t*)(ws + p.w), plane, p.kp, (int)rows};
}

PackArgs pack_args(const XentArgs& x, const XentPlan& p, char* ws, bool exact) {
    return PackArgs{x, p.n, p.v, p.d, p.kp, p.np, exact || x.bf16 || p.few ? (uint16_t*)(ws + p.h) : nullptr,
                    x.bf16 || p.few ? nullptr : (uint16_t*)(ws + p.h16), (float*)(ws + p.hinv), (int*)(ws + p.map),
                    (int*)(ws + p.tgt), exact && p.exact_targets && x.dW ? (int*)(ws + p.pos) : nullptr, (float2*)(ws + p.lg),
                    x.bf16 || p.few ? nullptr : (float*)(ws + p.gscale), (int*)(ws + p.cnt), (float*)(ws + p.cnt) + 1,
                    p.n > kCountDirect ? (int*)(ws + p.cnt) + 64 : nullptr};
}

LogitArgs logit_args(const XentPlan& p, const PackArgs& pk, char* ws) {
    LogitArgs a{};
    a.h = mm::Operand{pk.h16 ? pk.h16 : pk.h, p.np * p.kp, p.kp, 0};
    a.seg = p.parts == 1 ? segments(1, 1) : segments(2, 2);
    a.kp = (int)p.kp; a.cnt = pk.cnt; a.tgt = pk.tgt;
    a.hinv = pk.inv; a.winv = (float*)(ws + p.winv); a.wtop = (float*)(ws + p.wtop); a.gscale = pk.gscale;
    return a;
}

template <class C>
void launch_out(const OutArgs& a, int64_t rows, hipStream_t s) {
    const int64_t t = ceil_div64(a.d, C::BM) * ceil_div64(rows, C::BN) * a.split;
    hipLaunchKernelGGL((out_kernel<C>), walkers<C>(t), dim3(C::THREADS), 0, s, a);
}

template <bool V4>
void launch_few_out(const OutArgs& a, int64_t n, hipStream_t s) {
    if (n <= 32) launch_out<Q32<V4>>(a, n, s);
    else launch_out<Q64<V4>>(a, n, s);
}

void launch_join(const OutArgs& a, int64_t rows, hipStream_t s) {
    const dim3 grid((unsigned)join_blocks(rows, a.dp, a.split));
    if (join_lanes(a.split) == 8) hipLaunchKernelGGL((join_kernel<8>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((join_kernel<1>), grid, dim3(256), 0, s, a);
}

template <int N>
void launch_rank(const OutArgs& a, const XentPlan& p, hipStream_t s) {
    const int64_t across = ceil_div64(a.d, 1024), down = ceil_div64(a.rows, 64), most = ceil_div64(kCUs * 8, across);
    hipLaunchKernelGGL((rank_out_kernel<N>), dim3((unsigned)(down < most ? down : most), (unsigned)across), dim3(256), 0, s, a,
                       p.parts, p.dparts);
}

// The logits with their reduction in slices, as partial sums of an output of p.n rows of p.piece columns.
template <bool V4>
void launch_few_slices(const OutArgs& a, int64_t n, hipStream_t s) {
    if (n <= 32) launch_out<P32<V4>>(a, n, s);
    else launch_out<P64<V4>>(a, n, s);
}

SliceArgs launch_slices(const LogitArgs& z, const XentPlan& p, char* ws, hipStream_t s) {
    OutArgs o{};
    o.a = z.w; o.b = z.h; o.seg = z.seg; o.cnt = z.cnt; o.d = z.w.rows; o.dp = (int)p.piece; o.rows = -1; o.k = z.kp;
    o.split = (int)p.split_z; o.k_per = (int)(ceil_div64(p.kp / 64, p.split_z) * 64);
    o.acc = (float*)(ws + p.z); o.acc_rows = p.n;
    if (p.few && p.d % 4 == 0) launch_few_slices<true>(o, p.n, s);
    else if (p.few) launch_few_slices<false>(o, p.n, s);
    else if (p.parts == 1 && p.tile_z == TILE_256) launch_out<Z256>(o, p.n, s);
    else if (p.parts == 1 && p.tile_z == TILE_128) launch_out<Z128>(o, p.n, s);
    else if (p.parts == 1 && p.tile_z == TILE_64) launch_out<Z64>(o, p.n, s);
    else if (p.parts == 1) launch_out<Z32>(o, p.n, s);
    else if (p.tile_z == TILE_256) launch_out<F256>(o, p.n, s);
    else if (p.tile_z == TILE_128) launch_out<F128>(o, p.n, s);
    else launch_out<F64>(o, p.n, s);
    const bool scaled = p.parts > 1 && !p.few;
    return SliceArgs{o.acc, p.n, p.piece, o.split, (int)p.v, z.cnt, scaled ? z.hinv : nullptr, scaled ? z.winv : nullptr,
                     z.tgt, z.lg, z.gscale, z.wtop, z.dl, z.dl16, z.rest, p.np};
}

}  // namespace

int run_xent(const XentArgs& x, const XentPlan& p, char* ws, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    const PackArgs pk = pack_args(x, p, ws, false);
    launch_pack<false>(pk, s);
    LogitArgs a = logit_args(p, pk, ws);
    if (p.split_z > 1) {
        a.w = weights(x, p, ws, 0, p.v, false, s);
        const SliceArgs z = launch_slices(a, p, ws, s);
        // a wave per token where 256 threads would not all have logits (a wave and four: 4000 x 100 x 4096 bf16 45 and 48 us, 4000 x
        // 200 x 4096 fp32 83 and 85; 300 x 1000 x 2100 fp32 39 and 35)
        if (p.v <= 256) hipLaunchKernelGGL((slice_loss_kernel<64>), dim3((unsigned)ceil_div64(p.n, 4)), dim3(256), 0, s, z, pk.map, x.loss, x.lse_out);
        else hipLaunchKernelGGL((slice_loss_kernel<256>), dim3((unsigned)p.n), dim3(256), 0, s, z, pk.map, x.loss, x.lse_out);
        return (int)hipGetLastError();
    }
    a.part = (float2*)(ws + p.part); a.zt = (float*)(ws + p.zt); a.nvt = (int)p.nvt;
    for (int64_t v0 = 0; v0 < p.v; v0 += p.piece) {
        a.w = weights(x, p, ws, v0, p.v - v0 < p.piece ? p.v - v0 : p.piece, false, s);
        a.v0 = (int)v0;
        launch_logits<EPI_LOSS>(a, p, s);
    }
    hipLaunchKernelGGL(loss_kernel, dim3((unsigned)ceil_div64(p.n, 4)), dim3(256), 0, s, a.part, a.zt, a.tgt, pk.map, pk.cnt,
                       a.nvt, x.loss, x.lse_out);
    return (int)hipGetLastError();
}

__global__ __launch_bounds__(256) void clear_kernel(uint16_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

int run_xent_grad(const XentArgs& x, const XentPlan& p, char* ws, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    if (p.n == 0) {   // no tokens: dW is zero
        const int64_t n = p.v * p.d * (x.dw_bf16 ? 1 : 2);
        hipLaunchKernelGGL(clear_kernel, dim3((unsigned)stride_blocks(ceil_div64(n, 256 * 8))), dim3(256), 0, s, (uint16_t*)x.dW, n);
        return (int)hipGetLastError();
    }
    const PackArgs pk = pack_args(x, p, ws, true);
    launch_pack<true>(pk, s);
    LogitArgs z = logit_args(p, pk, ws);
    z.lg = pk.lg;
    const bool scaled = !x.bf16 && !p.few;   // dH from fp16 parts of scaled D and W
    z.dl = x.dW || !scaled ? (uint16_t*)(ws + p.dl) : nullptr;
    z.dl16 = scaled && x.dH ? (uint16_t*)(ws + p.dl16) : nullptr;
    z.rest = (float*)(ws + p.rest); z.np = p.np; z.piece = p.piece;
    const mm::Operand dl{z.dl, p.np * p.piece, p.piece, 0};
    OutArgs h{};
    const float* factor = x.grad_n == 1 ? pk.factor : nullptr;
    h.cnt = pk.cnt; h.d = (int)p.d; h.dp = (int)p.dp; h.factor = factor; h.rows = -1; h.split = (int)p.split_h; h.map = pk.map; h.out = x.dH; h.out_bf16 = x.bf16;
    h.acc = p.pieces > 1 || p.split_h > 1 ? (float*)(ws + p.acc_h) : nullptr;
    h.acc_rows = p.np;
    if (scaled) { h.wtop = z.wtop; h.row_scale = pk.gscale; }
    if (x.bf16) { h.rest = z.rest; h.tgt = pk.tgt; h.w = (const uint16_t*)x.W; }
    OutArgs w{};
    w.cnt = pk.cnt; w.d = (int)p.d; w.dp = (int)p.dp; w.factor = factor; w.k = -1; w.split = (int)p.split_w; w.out_bf16 = x.dw_bf16; w.accumulate = x.accumulate;
    w.acc = p.split_w > 1 ? (float*)(ws + p.acc_w) : nullptr;
    w.acc_rows = p.piece;
    const bool exact_targets = x.dW && p.exact_targets;
    const EmbedArgs rows_of{x.targets, x.H, nullptr, p.n, p.v, p.d, 1.f, x.ignore, x.t64, 1, 0, 0};
    if (exact_targets) {
        const int e = sort_weighted_rows(rows_of, p.sorted, (int*)(ws + p.slot), ws + p.sort, stream);
        if (e) return e;
        w.extra = (const float*)(ws + p.extra);
    }
    for (int64_t v0 = 0; v0 < p.v; v0 += p.piece) {
        const int64_t rows = p.v - v0 < p.piece ? p.v - v0 : p.piece;
        z.w = weights(x, p, ws, v0, rows, x.dH != nullptr, s);
        z.v0 = (int)v0;
        if (p.split_z > 1) {
            const SliceArgs a = launch_slices(z, p, ws, s);
            const dim3 grid((unsigned)ceil_div64(p.v, 256 * 8), (unsigned)p.n);
            if (p.dparts == 1) hipLaunchKernelGGL((slice_grad_kernel<EPI_D1>), grid, dim3(256), 0, s, a);
            else if (p.dparts == 2) hipLaunchKernelGGL((slice_grad_kernel<EPI_D2>), grid, dim3(256), 0, s, a);
            else hipLaunchKernelGGL((slice_grad_kernel<EPI_D3>), grid, dim3(256), 0, s, a);
        } else if (p.dparts == 1) launch_logits<EPI_D1>(z, p, s);
        else if (p.dparts == 2) launch_logits<EPI_D2>(z, p, s);
        else launch_logits<EPI_D3>(z, p, s);
        if (x.dH) {
            h.a = z.w;
            h.b = scaled ? mm::Operand{z.dl16, p.np * p.piece, p.piece, 0} : dl;
            h.seg = scaled ? segments(2, 2) : segments(p.parts, x.bf16 ? 1 : 3);
            h.k = (int)(ceil_div64(rows, 64) * 64);
            h.k_per = (int)(ceil_div64(ceil_div64(h.k, p.split_h), 64) * 64);
            h.add = v0 > 0;
            if (p.few && p.d % 4 == 0) launch_few_out<true>(h, p.n, s);
            else if (p.few) launch_few_out<false>(h, p.n, s);
            else if (scaled && p.tile_h == TILE_256) launch_out<E256>(h, p.n, s);
            else if (scaled && p.tile_h == TILE_128) launch_out<E128>(h, p.n, s);
            else if (scaled) launch_out<E64>(h, p.n, s);
            else if (p.tile_h == TILE_256) launch_out<H256>(h, p.n, s);
            else if (p.tile_h == TILE_128) launch_out<H128>(h, p.n, s);
            else if (p.tile_h == TILE_64) launch_out<H64>(h, p.n, s);
            else launch_out<H32>(h, p.n, s);
        }
        if (x.dW) {
            w.a = mm::Operand{pk.h, p.np * p.kp, p.kp, 0}; w.b = dl;
            w.seg = segments(p.parts, p.dparts);
            w.rows = (int)rows;
            w.k_per = (int)(ceil_div64(ceil_div64(p.np, p.split_w), 64) * 64);
            w.out = (char*)x.dW + v0 * p.d * (x.dw_bf16 ? 2 : 4);
            if (exact_targets) {
                const WeightedRows sums{z.rest, pk.pos, (int*)(ws + p.slot), (float*)(ws + p.extra), p.dp, v0, v0 + rows,
                                        p.extra_by_row};
                const int e = sum_weighted_rows(rows_of, p.sorted, sums, ws + p.sort, stream);
                if (e) return e;
                w.slot = (const int*)(ws + p.slot) + v0;
            }
            if (p.n <= 8) launch_rank<8>(w, p, s);
            else if (p.n <= kRankTokens) launch_rank<16>(w, p, s);
            else if (p.tile_w == TILE_256) launch_out<W256>(w, rows, s);
            else if (p.tile_w == TILE_64) launch_out<W64>(w, rows, s);
            else if (p.n <= kShortTokens) launch_out<Ws>(w, rows, s);
            else launch_out<W128>(w, rows, s);
            if (w.acc) launch_join(w, rows, s);
        }
    }
    if (x.dH && h.acc) launch_join(h, p.n, s);
    return (int)hipGetLastError();
}

}  // namespace dion
