// What the kernels around the tile products of mm16.hpp share: parts of fp32 values, rows packed into planes, the walk of a
// workgroup over its tiles, the store of a lane's pieces.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

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

// A lane's 4-row pieces of two neighbouring blocks of 16 rows: the lane quarters trade their four rows of one
// against the other's (v_permlane32_swap, v_permlane16_swap), so that a lane has eight consecutive rows and four lanes
// 64 bytes.  a, b: the four values of each block, packed in two words.
__device__ __forceinline__ u32x4 trade(const uint32_t (&a)[2], const uint32_t (&b)[2]) {
    u32x4 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto x = __builtin_amdgcn_permlane32_swap(a[h], b[h], false, false);
        const auto z = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
        w[h] = z[0];
        w[2 + h] = z[1];
    }
    return w;
}

// And back: the two blocks' words from eight consecutive rows.
__device__ __forceinline__ void untrade(const u32x4& w, uint32_t (&a)[2], uint32_t (&b)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto x = __builtin_amdgcn_permlane16_swap(w[h], w[2 + h], false, false);
        const auto z = __builtin_amdgcn_permlane32_swap(x[0], x[1], false, false);
        a[h] = z[0];
        b[h] = z[1];
    }
}

// Stores such pieces; to: the address for this lane's quarter.
__device__ __forceinline__ void store_pair(uint16_t* to, const uint32_t (&a)[2], const uint32_t (&b)[2], bool in) {
    const u32x4 w = trade(a, b);
    if (in) *(u32x4*)to = w;
}

// plane pairs (A's part, B's part), smallest products first
inline mm::Segments segments(int pa, int pb) {
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

// One workgroup per tile, or as many as the chip holds, which then walk the tiles.
template <class C>
dim3 walkers(int64_t tiles) {
    return dim3((unsigned)(tiles < kCUs * C::kPerCU ? tiles : kCUs * C::kPerCU));
}

}  // namespace

}  // namespace dion
