// Eight elements of a row of any length and type, in registers.
#pragma once
#include "vocab/tiles.hpp"

namespace dion {

namespace {

typedef uint32_t __attribute__((ext_vector_type(2), aligned(1))) u32x2_bytes;   // eight of a row of 8-bit numbers

// Eight elements of a row as they are in memory, so that all loads of a row can be on their way before the first is used.
template <bool BF16>
struct Raw8 {
    u32x4 w[BF16 ? 1 : 2];
    // columns c .. c + 7 of the row at p + row, zeros behind column d
    __device__ __forceinline__ void load(const void* p, int64_t row, int c, int d) {
        if (c + 8 <= d) {
            if constexpr (BF16) {
                w[0] = *(const u32x4_any*)((const uint16_t*)p + row + c);
            } else {
                const u32x4_any* q = (const u32x4_any*)((const float*)p + row + c);
                w[0] = q[0];
                w[1] = q[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (c + e >= d) continue;
                if constexpr (BF16) w[0][e / 2] |= (uint32_t)((const uint16_t*)p)[row + c + e] << (16 * (e % 2));
                else w[e / 4][e % 4] = ((const uint32_t*)p)[row + c + e];
            }
        }
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (BF16) return e % 2 ? __uint_as_float(w[0][e / 2] & 0xffff0000u) : up16(w[0][e / 2] & 0xffffu);
        else return __uint_as_float(w[e / 4][e % 4]);
    }
};

template <bool BF16>
__device__ __forceinline__ void put8(void* p, int64_t row, int c, int d, const float (&v)[8]) {
    if (c + 8 <= d) {
        if constexpr (BF16) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = down16(v[2 * e]) | (down16(v[2 * e + 1]) << 16);
            *(u32x4_any*)((uint16_t*)p + row + c) = w;
        } else {
            f32x4_any* q = (f32x4_any*)((float*)p + row + c);
            q[0] = f32x4{v[0], v[1], v[2], v[3]};
            q[1] = f32x4{v[4], v[5], v[6], v[7]};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c + e >= d) continue;
            if constexpr (BF16) ((uint16_t*)p)[row + c + e] = (uint16_t)down16(v[e]);
            else ((float*)p)[row + c + e] = v[e];
        }
    }
}

// Four columns of a row of `d` elements at any element's address: bf16 or fp32.
template <bool BF16>
__device__ __forceinline__ void put4(void* p, int64_t row, int c, int d, const float (&v)[4]) {
    if (c + 4 <= d) {
        if constexpr (BF16)
            *(u32x2_any*)((uint16_t*)p + row + c) = u32x2{down16(v[0]) | (down16(v[1]) << 16), down16(v[2]) | (down16(v[3]) << 16)};
        else
            *(f32x4_any*)((float*)p + row + c) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (c + e >= d) continue;
            if constexpr (BF16) ((uint16_t*)p)[row + c + e] = (uint16_t)down16(v[e]);
            else ((float*)p)[row + c + e] = v[e];
        }
    }
}

// N (4 or 8) 8-bit numbers (e4m3) of a row from column c, times s; zeros from column d on
template <int N>
__device__ __forceinline__ void load_e4m3(const void* in, int64_t row, int c, int d, float s, float (&v)[N]) {
    const uint8_t* p = (const uint8_t*)in + row + c;
    uint32_t w[2] = {0, 0};
    if (c + N <= d) {
        if constexpr (N == 8) {
            const u32x2_bytes q = *(const u32x2_bytes*)p;
            w[0] = q[0];
            w[1] = q[1];
        } else {
            __builtin_memcpy(w, p, 4);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (c + e < d) w[e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
    }
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true);
        v[4 * h] = lo[0] * s;
        v[4 * h + 1] = lo[1] * s;
        v[4 * h + 2] = hi[0] * s;
        v[4 * h + 3] = hi[1] * s;
    }
}

}  // namespace

}  // namespace dion
