// The feed-forward block's activations and the form in which its two projections are kept for the gradient.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dion_block.h"

namespace dion {

namespace {

// 1 / (1 + exp(-z)), zero below -87.  EXACT: to a few ulp (the rounding of -z log2(e) is carried into the result, and the
// reciprocal is refined once); else that rounding's |z| 2^-24 stays, which is far below bf16's.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z) {
    const float h = z * -1.44269504f;
    float e = __builtin_amdgcn_exp2f(h);
    if constexpr (!EXACT) return __builtin_amdgcn_rcpf(1.f + e);
    const float l = fmaf(z, -1.44269504f, -h) - z * 1.92596299e-8f;   // log2(e) - 1.44269504f
    e = 1.f + fmaf(e, l * 0.693147181f, e);
    const float r = __builtin_amdgcn_rcpf(e);
    return z < -87.f ? 0.f : fmaf(r, fmaf(-e, r, 1.f), r);
}

// act(a) and its derivative: a r and r + a r (1 - r) z' with r = 1 / (1 + exp(-z)) and
//   silu  z = a;  gelu  z = 2 sqrt(2 / pi) (x + 0.044715 x^3), as (1 + tanh(z / 2)) / 2 = r, and z is past every border at |a| = 30
template <bool EXACT>
__device__ __forceinline__ float activate(int act, float a, float& slope) {
    float x = a, z = a, dz = 1.f;
    if (act != DION_SILU) {
        x = fminf(fmaxf(a, -30.f), 30.f);   // (of a NaN: -30)
        const float q = x * x;
        z = 1.59576912f * x * fmaf(0.044715f, q, 1.f);
        dz = 1.59576912f * fmaf(0.134145f, q, 1.f);
    }
    const float r = sigmoid<EXACT>(z);
    const float v = a * r;   // (where x is not a, r (1 - r) is zero; a NaN is one again)
    slope = fmaf(v * (1.f - r), dz, r);
    return v;
}

// a and b as the gradient is handed them, for bf16 operands: 16 bits, a sign and either, for magnitudes in [2^-8, 2^8), a set
// bit, four of exponent and ten of fraction, or a clear bit and 14 for the others, rounded to nearest, ties away from zero.  In
// bf16 (seven of fraction) da, db and u would carry its rounding twice more: dW of 8192 x 2048 x 5632 against 64 bits 3.5e-3, with
// this form 2.4e-3, where the rounding of da and of dW to bf16 alone leaves 2.3e-3.
// The others.  EVEN: the 128 binades from 2^-80 to 2^-8 and from 2^8 to 2^64 with seven bits of fraction each, as bf16 has;
// smaller ones are zero, larger ones NaN, which is the last number.  Else the upper 14 bits of the magnitude's fp32 form: all of
// its range, but six bits of fraction.
constexpr uint32_t kEvenBelow = 72u << 7, kEvenNan = 0x3fffu;   // numbers of the binades below the window; the last one
template <bool EVEN>
__device__ __forceinline__ uint32_t keep32(float x0, float x1) {   // two of them
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t m = __float_as_uint(h ? x1 : x0) & 0x7fffffffu;
        const uint32_t fine = m - ((119u << 23) - 0x1000u);
        uint32_t far;
        if constexpr (EVEN) {
            const int n = (int)((m + 0x8000u) >> 16) - (47 << 7);   // 127 - 80 = 47
            // (a magnitude just below the window that rounds up to it is at its first number, in `fine`'s bits)
            far = n < (int)kEvenBelow ? (uint32_t)(n < 0 ? 0 : n)
                  : n < (int)kEvenBelow + (16 << 7) ? 0x4000u
                  : n - (16 << 7) < (int)kEvenNan ? (uint32_t)n - (16u << 7) : kEvenNan;
        } else {
            far = m + 0x10000u;
            far = (far > 0x7fffffffu ? 0x7fffffffu : far) >> 17;   // (a NaN stays one)
        }
        c[h] = fine < (16u << 23) ? (fine >> 13) | 0x4000u : far;
    }
    const uint32_t signs = __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302u);
    return ((c[0] | (c[1] << 16)) & 0x7fff7fffu) | (signs & 0x80008000u);
}
template <bool EVEN>
__device__ __forceinline__ float kept16(uint32_t c) {
    const uint32_t v = c & 0x3fffu;
    uint32_t far;
    if constexpr (EVEN) {
        far = (v + (v < kEvenBelow ? 47u << 7 : 63u << 7)) << 16;
        far = v == 0 ? 0 : v == kEvenNan ? 0x7fc00000u : far;
    } else {
        far = v << 17;
    }
    return __uint_as_float((c & 0x4000u ? (v + (119u << 10)) << 13 : far) | ((c & 0x8000u) << 16));
}

}  // namespace

}  // namespace dion
