// Dropout from a counter-based generator, and the root-mean-square norm with the residual's addition, its output in the
// activations' type or in 8 bits, and its gradients.
//
//   h = residual + keep x / (1 - p);  rstd = (mean h^2 + eps)^(-1/2);  y = h rstd w
//   n = h rstd;  g = dY w;  dh = rstd (g - n mean(g n)) + dsum;  dx = keep dh / (1 - p);  dw = sum over the rows of dY n
//
// One pass over the data: a team of threads (a wave, four or sixteen) holds a row in registers between the row's sum and
// its output.  (Above 16384 elements a row outgrows them in part: 10 to 450 vector registers spill, and the gradient reads its
// rows twice.  2^26 elements in rows of 65536: norm 181 us, to 8 bits 400.)  dw is summed per thread over the rows that its workgroup strides over, then over the workgroups in a fixed
// order.
//
// The mask is Philox4x32-10 over the elements' numbers: a call yields the words of four elements in a row, so the eight of
// a vector take two calls, or three where the row does not start at a multiple of four.
//
// Bound by HBM: dropout of 65536 x 4096 bf16 with a residual 312 us (5.2 TB/s), norm of 16384 x 2048 bf16 to 8 bits with dropout 71 us
// (3.3 TB/s: fp64 arithmetic and the mask; 61 where calls follow one another), gradient of 65536 x 4096 with an fp32 stream 839 us (5.1 TB/s); small ones by the launch (one row
// of 2048: 2.7 us).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "block_plan.h"
#include "rows.hpp"

namespace dion {

namespace {

// The same with the type known when it runs (the norm's weight).
struct RawAny8 {
    u32x4 a, b;
    __device__ __forceinline__ void load(const void* p, int c, int d, int bf16) {
        if (bf16) {
            Raw8<true> r;
            r.load(p, 0, c, d);
            a = r.w[0];
        } else {
            Raw8<false> r;
            r.load(p, 0, c, d);
            a = r.w[0];
            b = r.w[1];
        }
    }
    __device__ __forceinline__ void get(int bf16, float (&v)[8]) const {
        if (bf16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[2 * e] = up16(a[e] & 0xffffu); v[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u); }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[e] = __uint_as_float(a[e]); v[4 + e] = __uint_as_float(b[e]); }
        }
    }
};

// ---------------------------------------------------------------------------
// The mask
// ---------------------------------------------------------------------------
__device__ __forceinline__ void philox(uint64_t block, uint64_t site, uint64_t key, uint32_t (&w)[4]) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)site, c3 = (uint32_t)(site >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
}

// v[e] = keep v[e] scale for the elements at .. at + 7; at % 4 must be the same for the wave
template <class F>
__device__ __forceinline__ void drop8(const Mask& m, uint64_t key, int64_t at, F scale, F (&v)[8]) {
    uint32_t w[12];
    const int off = __builtin_amdgcn_readfirstlane((int)(at & 3));
    const uint64_t block = (uint64_t)at >> 2;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i == 2 && off == 0) break;
        uint32_t q[4];
        philox(block + i, (uint64_t)m.site, key, q);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = q[e];
    }
    auto apply = [&](auto o) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = w[decltype(o)::value + e] >= m.threshold ? v[e] * scale : (F)0;
    };
    struct C0 { enum { value = 0 }; };
    struct C1 { enum { value = 1 }; };
    struct C2 { enum { value = 2 }; };
    struct C3 { enum { value = 3 }; };
    if (off == 0) apply(C0());
    else if (off == 1) apply(C1());
    else if (off == 2) apply(C2());
    else apply(C3());
}

template <bool XB, bool OB>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a) {
    const uint64_t key = a.mask.on ? (uint64_t)*a.mask.seed : 0;
    const float scale = (float)a.mask.scale;
    const int64_t vecs = (a.n + 7) / 8;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < vecs; q += (int64_t)gridDim.x * 256) {
        const int64_t at = q * 8;
        const int left = a.n - at < 8 ? (int)(a.n - at) : 8;
        Raw8<XB> x;
        Raw8<OB> r;
        x.load(a.x, at, 0, left);
        if (a.residual) r.load(a.residual, at, 0, left);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x.get(e);
        if (a.mask.on) drop8(a.mask, key, at, scale, v);
        if (a.residual) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r.get(e);
        }
        put8<OB>(a.out, at, 0, left, v);
    }
}

// ---------------------------------------------------------------------------
// Norm
// ---------------------------------------------------------------------------
struct Sum {
    template <class F>
    static __device__ __forceinline__ F of(F a, F b) { return a + b; }
};
struct Max {
    template <class F>
    static __device__ __forceinline__ F of(F a, F b) { return a > b ? a : b; }
};

// Over the team's threads, the same value for all of them.  red: 16 values of LDS; calls alternate between two of them.
template <int TEAM, class OP, class F>
__device__ __forceinline__ F team(F v, F* red) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = OP::of(v, __shfl_xor(v, o));
    if constexpr (TEAM > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < TEAM / 64; ++i) v = OP::of(v, red[i]);
    }
    return v;
}

// x to fp32 with the lowest bit set where it is not exact (rounded to odd): rounding that to fewer bits is rounding x once,
// and it is above or below a number of fewer bits as x is.
__device__ __forceinline__ float to_odd(double x) {
    const float f = (float)x;
    const double rest = x - (double)f;
    const uint32_t b = __float_as_uint(f);
    if (rest == 0.0 || rest != rest || (b & 1u)) return f;   // (x infinite or NaN: so is rest's difference)
    return __uint_as_float((rest > 0.0) == (x > 0.0) ? b + 1 : b - 1);
}

// The same to 20 bits of fraction in two instructions and the conversion, for bf16's seven (subnormal numbers of fp32 may still be
// rounded twice).  16384 rows of 2048, the stream rounded to fp32 first 45 us, so 46, with to_odd 51.
__device__ __forceinline__ float to_20_odd(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint32_t low = (uint32_t)b;
    return (float)__longlong_as_double((long long)((b & 0xffffffff00000000u) | (uint64_t)(low != 0 ? 1u : 0u) << 32));
}
__device__ __forceinline__ float to_20_odd(float x) { return x; }

// Q8: in fp64, y in 8 bits.
template <bool XB, bool SB, int TEAM, int VECS, bool Q8>
__global__ __launch_bounds__(TEAM == 64 ? 256 : TEAM) void norm_kernel(NormArgs a) {
    using F = typename std::conditional<Q8, double, float>::type;
    __shared__ F red[2][16];   // (Q8: two times 16 floats in the second)
    const int t = TEAM == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = TEAM == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= a.rows) return;   // (a whole team)
    const int64_t at = row * a.d;
    Raw8<XB> x[VECS];
    Raw8<SB> r[VECS];
    RawAny8 w[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * TEAM + t) * 8;
        x[i].load(a.x, at, c, a.d);
        if (a.residual) r[i].load(a.residual, at, c, a.d);
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) w[i].load(a.w, (i * TEAM + t) * 8, a.d, a.w_bf16);
    const uint64_t key = a.mask.on ? (uint64_t)*a.mask.seed : 0;
    F h[VECS][8], sum = 0;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * TEAM + t) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = (F)x[i].get(e);
        if (a.mask.on) drop8(a.mask, key, at + c, (F)a.mask.scale, h[i]);
        if (a.residual) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] += (F)r[i].get(e);
        }
        if (a.h) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = SB ? to_20_odd(h[i][e]) : (float)h[i][e];   // (rounded once)
            put8<SB>(a.h, at, c, a.d, o);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += h[i][e] * h[i][e];   // zeros behind column d (where a mask may keep them)
    }
    sum = team<TEAM, Sum>(sum, red[0]);
    F rstd = (F)1 / sqrt(sum / (F)a.d + (F)a.eps), seen = rstd;
    if constexpr (!Q8) {
        // Squares that leave fp32's range: the row again, times a power of two that brings them back (the same for the team).
        // With eps at least 2^-100 nothing that underflows counts.  (The code alone costs 2^26 elements in
        // rows of 65536, bf16, 174 -> 181 us and of 32768, fp32, 228 -> 240; shorter rows nothing.)
        if (sum == INFINITY || (sum < 0x1p-70f && a.eps < 0x1p-100)) {
            const bool large = sum == INFINITY;
            const float f = large ? 0x1p-80f : 0x1p90f;
            sum = 0;
#pragma unroll
            for (int i = 0; i < VECS; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    h[i][e] *= f;
                    sum += h[i][e] * h[i][e];
                }
            sum = team<TEAM, Sum>(sum, red[1]);
            const double exact = 1.0 / sqrt((double)sum / a.d * (large ? 0x1p160 : 0x1p-180) + a.eps);
            seen = (float)exact;
            rstd = (float)(exact * (large ? 0x1p80 : 0x1p-90));
        }
    }
    if (a.rstd && t == 0) a.rstd[row] = (float)seen;
    float y[VECS][8], top = 0.f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        float wv[8];
        w[i].get(a.w_bf16, wv);
        if constexpr (Q8) {   // from here on in fp32, rounded to odd: comparisons with the numbers of fewer bits stay as they are
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[i][e] = to_odd(h[i][e] * rstd * (F)wv[e]);
                top = fmaxf(top, fabsf(y[i][e]));
            }
        } else {
            const int c = (i * TEAM + t) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = h[i][e] * rstd * wv[e];
            if (a.y_bf16) put8<true>(a.y, at, c, a.d, y[i]);
            else put8<false>(a.y, at, c, a.d, y[i]);
        }
    }
    if constexpr (Q8) {
        float* red32 = (float*)red[1];
        top = team<TEAM, Max>(top, red32);
        if (top == INFINITY) {   // (the same for the team) the largest of the finite ones
            top = 0.f;
#pragma unroll
            for (int i = 0; i < VECS; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fabsf(y[i][e]) < INFINITY ? fmaxf(top, fabsf(y[i][e])) : top;
            top = team<TEAM, Max>(top, red32 + 16);
        }
        // top = m 2^e, 1 <= m < 2, and 448 = 1.75 2^8
        const uint32_t bits = __float_as_uint(top);
        int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
        e = e < -126 ? -126 : e;
        if (top == 0.f) e = 0;
        const float inverse = __uint_as_float((uint32_t)(127 - e) << 23);
        if (t == 0) a.scale[row] = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * TEAM + t) * 8;
            uint32_t q[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const float v0 = y[i][k] * inverse, v1 = y[i][k + 1] * inverse;
                const uint32_t p = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v0, v1, 0, false) & 0xffffu;
                const uint32_t b0 = fabsf(v0) <= 448.f ? p & 0xffu : 0x7fu, b1 = fabsf(v1) <= 448.f ? p >> 8 : 0x7fu;
                q[k / 4] |= (b0 | (b1 << 8)) << (8 * (k % 4));
            }
            uint8_t* out = (uint8_t*)a.y + at + c;
            if (c + 8 <= a.d) {
                *(u32x2_bytes*)out = u32x2_bytes{q[0], q[1]};
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < a.d) out[k] = (uint8_t)(q[k / 4] >> (8 * (k % 4)));
            }
        }
    }
}

__device__ __forceinline__ void put_dw(const NormGradArgs& a, int c, float v) {
    if (a.dw_bf16) {
        uint16_t* p = (uint16_t*)a.dw + c;
        *p = (uint16_t)down16(v + (a.accumulate ? up16(*p) : 0.f));
    } else {
        float* p = (float*)a.dw + c;
        *p = v + (a.accumulate ? *p : 0.f);
    }
}

// KEEP: dY and h of a row stay in registers between its sum and its output, else they are read again.
template <bool YB, bool SB, int TEAM, int VECS, bool KEEP>
__global__ __launch_bounds__(TEAM == 64 ? 256 : TEAM) void norm_grad_kernel(NormGradArgs a) {
    constexpr int TEAMS = TEAM == 64 ? 4 : 1;
    __shared__ float red[2][16];
    __shared__ __attribute__((aligned(16))) float dws[TEAM == 64 ? 4 * 64 * VECS * 8 : 1];
    const int t = TEAM == 64 ? threadIdx.x & 63 : threadIdx.x, me = TEAM == 64 ? threadIdx.x >> 6 : 0;
    const uint64_t key = a.mask.on && a.dx ? (uint64_t)*a.mask.seed : 0;
    const float scale = (float)a.mask.scale, over = 1.f / (float)a.d;
    float dw[VECS][8];
    RawAny8 w[KEEP ? VECS : 1];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
        if (KEEP) w[KEEP ? i : 0].load(a.w, (i * TEAM + t) * 8, a.d, a.w_bf16);
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * TEAMS + me; row < a.rows; row += (int64_t)gridDim.x * TEAMS, turn ^= 1) {
        const int64_t at = row * a.d;
        Raw8<YB> y[KEEP ? VECS : 1];
        Raw8<SB> h[KEEP ? VECS : 1], s[KEEP ? VECS : 1];
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const int c = (i * TEAM + t) * 8;
                y[KEEP ? i : 0].load(a.dy, at, c, a.d);
                h[KEEP ? i : 0].load(a.h, at, c, a.d);
                if (a.dsum) s[KEEP ? i : 0].load(a.dsum, at, c, a.d);
            }
        }
        const float rstd = a.rstd[row];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int k = KEEP ? i : 0, c = (i * TEAM + t) * 8;
            if (!KEEP) {
                y[k].load(a.dy, at, c, a.d);
                h[k].load(a.h, at, c, a.d);
                w[k].load(a.w, c, a.d, a.w_bf16);
            }
            float wv[8];
            w[k].get(a.w_bf16, wv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = h[k].get(e) * rstd, dy = y[k].get(e);
                dw[i][e] = fmaf(dy, n, dw[i][e]);
                dot = fmaf(dy * wv[e], n, dot);
            }
        }
        const float mean = team<TEAM, Sum>(dot, red[turn]) * over;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int k = KEEP ? i : 0, c = (i * TEAM + t) * 8;
            if (!KEEP) {
                y[k].load(a.dy, at, c, a.d);
                h[k].load(a.h, at, c, a.d);
                w[k].load(a.w, c, a.d, a.w_bf16);
                if (a.dsum) s[k].load(a.dsum, at, c, a.d);
            }
            float wv[8], o[8];
            w[k].get(a.w_bf16, wv);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = rstd * (y[k].get(e) * wv[e] - h[k].get(e) * rstd * mean);
            if (a.dsum) {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] += s[k].get(e);
            }
            put8<SB>(a.dh, at, c, a.d, o);
            if (a.dx) {
                if (a.mask.on) drop8(a.mask, key, at + c, scale, o);
                put8<YB>(a.dx, at, c, a.d, o);
            }
        }
    }
    if (!a.dw) return;
    if constexpr (TEAM == 64) {
        constexpr int D = 64 * VECS * 8;
#pragma unroll
        for (int i = 0; i < VECS; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *(f32x4*)&dws[me * D + (i * 64 + t) * 8 + e] = f32x4{dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]};
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += 256) {
            const float v = (dws[c] + dws[D + c]) + (dws[2 * D + c] + dws[3 * D + c]);
            if (gridDim.x == 1) put_dw(a, c, v);
            else a.part[(int64_t)blockIdx.x * a.d + c] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * TEAM + t) * 8;
            if (gridDim.x == 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < a.d) put_dw(a, c + e, dw[i][e]);
            } else {
                put8<false>(a.part, (int64_t)blockIdx.x * a.d, c, a.d, dw[i]);
            }
        }
    }
}

// dw from the workgroups' sums: 32 columns a workgroup, 32 threads to a column.
__global__ __launch_bounds__(1024) void norm_join_kernel(NormGradArgs a, int blocks) {
    __shared__ float part[32][33];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32, c = (int)blockIdx.x * 32 + x;
    float v = 0.f;
    if (c < a.d) {
#pragma unroll 8
        for (int b = y; b < blocks; b += 32) v += a.part[(int64_t)b * a.d + c];
    }
    part[y][x] = v;
    __syncthreads();
    v = part[x][y];   // (a wave now has two columns' 32 sums)
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor(v, o);
    const int col = (int)blockIdx.x * 32 + y;
    if (x == 0 && col < a.d) put_dw(a, col, v);
}

template <class F>
void of_types(int first, int second, F f) {
    if (first) {
        if (second) f(std::true_type(), std::true_type());
        else f(std::true_type(), std::false_type());
    } else {
        if (second) f(std::false_type(), std::true_type());
        else f(std::false_type(), std::false_type());
    }
}

template <int TEAM, int VECS>
void launch_norm(const NormArgs& a, hipStream_t s) {
    of_types(a.x_bf16, a.s_bf16, [&](auto x, auto r) {
        constexpr bool XB = decltype(x)::value, SB = decltype(r)::value;
        const dim3 grid((unsigned)(TEAM == 64 ? ceil_div64(a.rows, 4) : a.rows)), block(TEAM == 64 ? 256 : TEAM);
        if (a.scale) hipLaunchKernelGGL((norm_kernel<XB, SB, TEAM, VECS, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((norm_kernel<XB, SB, TEAM, VECS, false>), grid, block, 0, s, a);
    });
}

template <int TEAM, int VECS>
void launch_norm_grad(const NormGradArgs& a, const NormPlan& p, hipStream_t s) {
    of_types(a.y_bf16, a.s_bf16, [&](auto y, auto r) {
        constexpr bool YB = decltype(y)::value, SB = decltype(r)::value;
        // 1024 threads have 128 registers each: not enough for four vectors of three rows, the weight and dw
        hipLaunchKernelGGL((norm_grad_kernel<YB, SB, TEAM, VECS, TEAM != 1024>), dim3((unsigned)p.blocks),
                           dim3(TEAM == 64 ? 256 : TEAM), 0, s, a);
    });
}

template <class F>
void of_plan(const NormPlan& p, F f) {
    struct T64 { enum { value = 64 }; };
    struct T256 { enum { value = 256 }; };
    struct T1024 { enum { value = 1024 }; };
    struct V1 { enum { value = 1 }; };
    struct V2 { enum { value = 2 }; };
    struct V4 { enum { value = 4 }; };
    struct V8 { enum { value = 8 }; };
    if (p.team == 64) {
        if (p.vecs == 1) f(T64(), V1());
        else f(T64(), V2());
    } else if (p.team == 256) {
        if (p.vecs == 1) f(T256(), V1());
        else if (p.vecs == 2) f(T256(), V2());
        else if (p.vecs == 4) f(T256(), V4());
        else f(T256(), V8());
    } else {
        if (p.vecs == 4) f(T1024(), V4());
        else f(T1024(), V8());
    }
}

}  // namespace

int run_dropout(const DropoutArgs& a, void* stream) {
    const int64_t blocks = ceil_div64(ceil_div64(a.n, 8), 256);
    const dim3 grid((unsigned)stride_blocks(blocks));
    of_types(a.x_bf16, a.out_bf16, [&](auto x, auto o) {
        hipLaunchKernelGGL((dropout_kernel<decltype(x)::value, decltype(o)::value>), grid, dim3(256), 0, (hipStream_t)stream, a);
    });
    return (int)hipGetLastError();
}

int run_rms_norm(const NormArgs& a, void* stream) {
    const NormPlan p = make_norm_plan(a.rows, a.d, a.scale && a.x_bf16);
    if (p.team == 64 && p.vecs == 4) {   // (bf16 rows to 8 bits alone)
        const dim3 grid((unsigned)ceil_div64(a.rows, 4));
        if (a.s_bf16) hipLaunchKernelGGL((norm_kernel<true, true, 64, 4, true>), grid, dim3(256), 0, (hipStream_t)stream, a);
        else hipLaunchKernelGGL((norm_kernel<true, false, 64, 4, true>), grid, dim3(256), 0, (hipStream_t)stream, a);
        return (int)hipGetLastError();
    }
    of_plan(p, [&](auto t, auto v) { launch_norm<decltype(t)::value, decltype(v)::value>(a, (hipStream_t)stream); });
    return (int)hipGetLastError();
}

int run_rms_norm_grad(const NormGradArgs& a, const NormPlan& p, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    if (a.rows > 0)
        of_plan(p, [&](auto t, auto v) { launch_norm_grad<decltype(t)::value, decltype(v)::value>(a, p, s); });
    if (a.dw && p.blocks != 1)   // (no rows: sums of nothing)
        hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)ceil_div64(a.d, 32)), dim3(1024), 0, s, a, (int)p.blocks);
    return (int)hipGetLastError();
}

}  // namespace dion
