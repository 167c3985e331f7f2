// Tile products on the bf16 matrix cores of gfx950 (v_mfma_f32_16x16x32_bf16) for the vocabulary
// operators: C[m][n] = sum over segments and k of A[m][k] B[n][k], fp32 accumulation.
//
// Operands are bf16 planes in memory.  An operand is read either along its rows ([x][k], k
// contiguous) or transposed ([k][x], x contiguous); a transposed one is turned around by the LDS
// read itself (ds_read_b64_tr_b16), so that D, H and W serve several products in one layout.
// fp32 operands come as three planes h + m + l (an exact split); a segment list then names the
// plane pairs to multiply, smallest first, and the k loop runs over all of them.
//
// A workgroup owns a BM x BN tile, its waves WM x WN parts of it.  Slabs of 64 k go from memory
// straight to LDS (buffer loads with an LDS destination, 16 bytes per lane), STAGES - 1 slabs
// ahead; one barrier per slab.  The LDS image is swizzled by permuting which 16 bytes a lane
// fetches: chunk c of row x of an [x][64] tile sits at c ^ (x & 7), so that the 16 rows of a
// fragment read fall on different banks; a [64][x] tile moves its 32-byte units by the row's
// position in the fragment.
//
// Lane layout of v_mfma_f32_16x16x32_bf16: A[l % 16][8 (l / 16) + i], B likewise, D element v of
// lane l is D[4 (l / 16) + v][l % 16].  ds_read_b64_tr_b16 on 16 lanes: lane j fetches four
// elements of row j / 4, columns 4 (j % 4).. + 3; lane i gets column i of the four rows.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dion {
namespace mm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kBK = 64;   // k per slab

struct Operand {
    const uint16_t* p;
    int64_t plane;   // elements between part planes
    int64_t ld;      // elements between rows, a multiple of 8
    int rows;        // rows: of x for a k-contiguous operand, of k for a transposed one; reads are clamped to them
};

// Plane pairs of a product: entry s in bits 4s..: A's plane in two bits, B's in the next two.
struct Segments {
    uint32_t n;
    uint32_t list;
};

template <int X>   // rows of 16-byte chunks per [64][X] row
__device__ __forceinline__ int tr_swz(int k) {
    constexpr int units = X / 16;   // 32-byte units per row
    if constexpr (units >= 16) return ((k & 3) | ((k >> 1) & 12)) << 1;
    else return ((((k & 3) | ((k >> 1) & 12)) & (units - 1))) << 1;
}

// One operand's tile of X rows of x by 64 k in LDS.
template <int X, bool TR, int WAVES>
struct Tile {
    static constexpr int kElems = X * kBK;
    static constexpr int kLoads = X / 8 / WAVES;   // 1 KB wave loads per slab and wave
    static_assert(X / 8 % WAVES == 0, "whole wave loads");
    uint32_t off[kLoads];   // byte offset of this lane's chunk from the slab's base
    int krow[TR ? kLoads : 1];

    // x0: first row of x of the tile (k-contiguous: the slab base is row x0; transposed: column x0)
    __device__ __forceinline__ void init(const Operand& o, int x0, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = wave * kLoads + i;
            if constexpr (!TR) {
                const int x = q * 8 + lane / 8, c = (lane % 8) ^ (x & 7);
                const int row = x0 + x < o.rows ? x : o.rows - 1 - x0;
                off[i] = (uint32_t)(row * o.ld + c * 8) * 2u;
            } else {
                constexpr int NC = X / 8;   // chunks per row of k
                const int k = q * (64 / NC) + lane / NC, c = (lane % NC) ^ tr_swz<X>(k);
                krow[i] = k;
                int64_t col = x0 + c * 8;
                if (col > o.ld - 8) col = o.ld - 8;   // past the row: unused columns, any valid address
                off[i] = (uint32_t)((k * o.ld + col) * 2);
            }
        }
    }
    // Starts the loads of the slab at k0 of plane `part` into lds (this tile's image).
    __device__ __forceinline__ void load(const Operand& o, int x0, int part, int k0, uint16_t* lds, int wave) const {
        const uint16_t* base = o.p + part * o.plane + (TR ? (int64_t)k0 * o.ld : (int64_t)x0 * o.ld + k0);
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 0x7fffffff, 0x00027000);
        if (TR && k0 + kBK > o.rows) {   // the last slab: rows of k past the end re-read the last row
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int over = k0 + krow[TR ? i : 0] - (o.rows - 1);
                const uint32_t at = off[i] - (over > 0 ? (uint32_t)(over * o.ld * 2) : 0u);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (wave * kLoads + i) * 512), 16, at, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (wave * kLoads + i) * 512), 16, off[i], 0, 0, 0);
        }
    }
    // Fragment of the 16 rows from x (a multiple of 16, relative to the tile), k step ks (0 or 1).
    static __device__ __forceinline__ u32x4 frag(uint16_t* lds, int x, int ks, int lane) {
        if constexpr (!TR) {
            const int row = x + lane % 16;
            return *(const u32x4*)&lds[row * kBK + (((ks * 4 + lane / 16) ^ (row & 7)) << 3)];
        } else {
            const int j = lane % 16, k = ks * 32 + 8 * (lane / 16) + j / 4;
            uint16_t* at = lds + k * X + ((((x >> 3) + ((j >> 1) & 1)) ^ tr_swz<X>(k)) << 3) + 4 * (j & 1);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * X));
            const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
            return u32x4{a[0], a[1], b[0], b[1]};
        }
    }
};

template <int N>
__device__ __forceinline__ void wait_slab() {   // all but the newest N loads of this wave landed, and every wave is here
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int BM_, int BN_, int WM_, int WN_, int STAGES_, bool TA_, bool TB_>
struct Config {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr bool TA = TA_, TB = TB_;
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;   // 16 x 16 blocks per wave
    static constexpr int kStage = (BM + BN) * kBK;               // elements of one slab's tiles
    static constexpr int kLds = STAGES * kStage;                 // elements
    typedef f32x4 Acc[MI][NI];
};

// acc += the product over k in [k0, k1) (multiples of 64) of every segment.  The caller's tile starts at
// (m0, n0).  Every thread of the workgroup calls it.
template <class C>
struct Product {
static __device__ __forceinline__ void run(const Operand& a, const Operand& b, int m0, int n0, int k0, int k1,
                                           Segments seg, uint16_t* lds, typename C::Acc& acc) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % C::WM, wn = wave / C::WM;
    Tile<C::BM, C::TA, C::WAVES> ta;
    Tile<C::BN, C::TB, C::WAVES> tb;
    constexpr int kPer = Tile<C::BM, C::TA, C::WAVES>::kLoads + Tile<C::BN, C::TB, C::WAVES>::kLoads;
    ta.init(a, m0, wave, lane);
    tb.init(b, n0, wave, lane);
    const int nk = (k1 - k0) / kBK, total = nk * (int)seg.n;
    int ls = 0, lk = 0, lslot = 0;   // the next slab to load: segment, slab within it, LDS stage
    auto load = [&]() {
        const uint32_t e = seg.list >> (4 * ls);
        uint16_t* t = lds + lslot * C::kStage;
        ta.load(a, m0, e & 3, k0 + lk * kBK, t, wave);
        tb.load(b, n0, (e >> 2) & 3, k0 + lk * kBK, t + C::BM * kBK, wave);
        if (++lk == nk) { lk = 0; ++ls; }
        if (++lslot == C::STAGES) lslot = 0;
    };
    const int ahead = C::STAGES - 1 < total ? C::STAGES - 1 : total;
    for (int i = 0; i < ahead; ++i) load();
    int slot = 0;
    for (int it = 0; it < total; ++it) {
        // slabs it + 1 .. it + STAGES - 2 may still be in flight, and near the end fewer are
        if (it + C::STAGES - 2 < total) wait_slab<(C::STAGES - 2) * kPer>();
        else wait_slab<0>();
        if (it + C::STAGES - 1 < total) load();
        uint16_t* la = lds + slot * C::kStage;
        uint16_t* lb = la + C::BM * kBK;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            u32x4 fa[C::MI], fb[C::NI];
#pragma unroll
            for (int i = 0; i < C::MI; ++i) fa[i] = ta.frag(la, wm * (C::BM / C::WM) + 16 * i, ks, lane);
#pragma unroll
            for (int j = 0; j < C::NI; ++j) fb[j] = tb.frag(lb, wn * (C::BN / C::WN) + 16 * j, ks, lane);
#pragma unroll
            for (int i = 0; i < C::MI; ++i)
#pragma unroll
                for (int j = 0; j < C::NI; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fa[i]),
                                                                        __builtin_bit_cast(bf16x8, fb[j]), acc[i][j], 0, 0, 0);
        }
        if (++slot == C::STAGES) slot = 0;
    }
}
};

}  // namespace mm
}  // namespace dion
