// Tile products on the 16-bit matrix cores of gfx950 (v_mfma_f32_16x16x32_bf16 and _f16) for the vocabulary
// operators: C[m][n] = sum over segments and k of A[m][k] B[n][k], fp32 accumulation.
//
// Operands are planes of 16-bit values in memory.  An operand is read either along its rows ([x][k], k
// contiguous) or transposed ([k][x], x contiguous); a transposed one is turned around by the LDS
// read itself (ds_read_b64_tr_b16), so that D, H and W serve several products in one layout.
// fp32 operands come as three planes h + m + l (an exact split); a segment list then names the
// plane pairs to multiply, smallest first, and every 64 k run over all of them.  Where the caller knows a
// scale per row, two fp16 planes (11 + 11 bits) and three pairs do (F16).
//
// A workgroup owns a BM x BN tile, its waves WM x WN parts of it.  Slabs of 64 k go from memory
// straight to LDS (buffer loads with an LDS destination, 16 bytes per lane) into a ring of STAGES
// stages; one barrier per slab.  The LDS image is swizzled by permuting which 16 bytes a lane
// fetches: chunk c of row x of an [x][64] tile sits at c ^ (x / 2 % 8), so that the 16 rows of a
// fragment read (128 bytes apart) fall on different banks of 64; a [64][x] tile moves its 32-byte units by the row's
// position in the fragment.
//
// Measured (8192 tokens x 32000 x 2048, bf16, 256 x 256 tiles, two stages): 32 x 32 x 16 products instead of 16 x 16 x 32 ran
// 5 to 9% slower, slabs of 32 k in four or five stages 10 to 30% (a barrier costs more than the deeper ring gains), raised
// wave priority and earlier LDS reads the same.  No LDS bank conflicts.
//
// Lane layout of v_mfma_f32_16x16x32_bf16: A[l % 16][8 (l / 16) + i], B likewise, D element v of
// lane l is D[4 (l / 16) + v][l % 16].  ds_read_b64_tr_b16 on 16 lanes: lane j fetches four
// elements of row j / 4, columns 4 (j % 4).. + 3; lane i gets column i of the four rows.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace dion {
namespace mm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
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
    int rows;        // of x for a k-contiguous operand (reads are clamped to them), of k for a transposed one (zeros behind them)
    int64_t pair = 0;   // PairTile: elements from the first matrix to the second
};

// Plane pairs of a product: entry s in bits 4s..: A's plane in two bits, B's in the next two.
struct Segments {
    uint32_t n;
    uint32_t list;
};

constexpr uint32_t kOutside = 0x80000000u;   // an offset outside every descriptor's range

// WORDS (1 or 4) words per lane from the descriptor's range (zeros outside it) to 256 WORDS bytes of LDS at byte address
// lds, which must be the same for all lanes.  Written as assembly because the compiler waits for every load in flight before
// a transposed LDS read that follows the builtin of this load, wherever it reads; it names no output register, and
// wait_slab() is what waits for it.  (m0 is the compiler's only for instructions that do not occur here.)
template <int WORDS>
__device__ __forceinline__ void load_to_lds(u32x4 desc, uint32_t off, uint32_t lds) {
    if constexpr (WORDS == 4)
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(desc),
                     "s"(__builtin_amdgcn_readfirstlane(lds)));
    else
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(off), "s"(desc),
                     "s"(__builtin_amdgcn_readfirstlane(lds)));
}

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

    // x0: first row of x of the tile (k-contiguous: the slab base is row x0; transposed: column x0)
    __device__ __forceinline__ void init(const Operand& o, int x0, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = wave * kLoads + i;
            if constexpr (!TR) {
                const int x = q * 8 + lane / 8, c = (lane % 8) ^ ((x >> 1) & 7);
                const int row = x0 + x < o.rows ? x : o.rows - 1 - x0;
                off[i] = (uint32_t)(row * o.ld + c * 8) * 2u;
            } else {
                constexpr int NC = X / 8;   // chunks per row of k
                const int k = q * (64 / NC) + lane / NC, c = (lane % NC) ^ tr_swz<X>(k);
                int64_t col = x0 + c * 8;
                if (col > o.ld - 8) col = o.ld - 8;   // past the row: unused columns, any valid address
                off[i] = (uint32_t)((k * o.ld + col) * 2);
            }
        }
    }
    // The slab at k0 of plane `part`, as the descriptor its loads go through.
    static __device__ __forceinline__ u32x4 slab(const Operand& o, int x0, int part, int k0) {
        const uint16_t* base = o.p + part * o.plane + (TR ? (int64_t)k0 * o.ld : (int64_t)x0 * o.ld + k0);
        // a transposed operand ends at its last row of k: the descriptor's range makes the rows behind it read as zeros
        const int64_t left = TR ? (o.rows - k0) * o.ld * 2 : 0x7fffffff;
        const uint64_t at = (uint64_t)base;
        return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, (uint32_t)(left < 0x7fffffff ? left : 0x7fffffff), 0x00027000u};
    }
    // Starts the i-th of this wave's loads of a slab into lds (this tile's image).
    __device__ __forceinline__ void load(u32x4 r, int i, uint32_t lds, int wave) const {
        load_to_lds<4>(r, off[i], lds + (wave * kLoads + i) * 1024);
    }
    // Fragment of the 16 rows from x (a multiple of 16, relative to the tile), k step ks (0 or 1).
    static __device__ __forceinline__ u32x4 frag(uint16_t* lds, int x, int ks, int lane) {
        if constexpr (!TR) {
            const int row = x + lane % 16;
            return *(const u32x4*)&lds[row * kBK + (((ks * 4 + lane / 16) ^ ((row >> 1) & 7)) << 3)];
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

// A tile whose rows come from two k-contiguous matrices of the same shape, o.pair elements apart, 16 of each in turn: X / 2
// rows of either, from row x0 / 2.  A wave then has the same rows of both products in the same lanes.
template <int X, int WAVES>
struct PairTile : Tile<X, false, WAVES> {
    using Base = Tile<X, false, WAVES>;
    static_assert(Base::kLoads % 2 == 0, "a wave load of eight rows belongs to one matrix, and so do two in a row");
    // of the i-th load of a wave
    static __device__ __forceinline__ int matrix(int i, int wave) {
        return Base::kLoads % 4 == 0 ? (i >> 1) & 1 : ((wave * Base::kLoads + i) >> 1) & 1;
    }
    __device__ __forceinline__ void init(const Operand& o, int x0, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < Base::kLoads; ++i) {
            const int q = wave * Base::kLoads + i, x = q * 8 + lane / 8, c = (lane % 8) ^ ((x >> 1) & 7);
            const int r = x / 32 * 16 + x % 16, row = x0 / 2 + r < o.rows ? r : o.rows - 1 - x0 / 2;
            this->off[i] = (uint32_t)(row * o.ld + c * 8) * 2u;
        }
    }
    static __device__ __forceinline__ u32x4 slab(const Operand& o, int x0, int part, int k0, int matrix) {
        const uint64_t at = (uint64_t)(o.p + part * o.plane + matrix * o.pair + (int64_t)(x0 / 2) * o.ld + k0);
        return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, 0x7fffffffu, 0x00027000u};
    }
};

// All but the newest N loads of this wave landed, its LDS reads are done, and every wave is here.
template <int N>
__device__ __forceinline__ void wait_slab() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <int BM_, int BN_, int WM_, int WN_, int STAGES_, bool TA_, bool TB_, bool F16_ = false, bool PAIR_ = false>
struct Config {
    static constexpr bool F16 = F16_, FEW = false;   // fp16 planes
    static constexpr bool PAIR = PAIR_;              // A is a PairTile
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr bool TA = TA_, TB = TB_;
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;   // 16 x 16 blocks per wave
    static constexpr int kStage = (BM + BN) * kBK;               // elements of one slab's tiles
    static constexpr int kLds = STAGES * kStage;                 // elements
    static constexpr int kPerCU = 163840 / (kLds * 2 + 4096) < 1 ? 1 : 163840 / (kLds * 2 + 4096);   // workgroups that LDS leaves room for
    typedef f32x4 Acc[MI][NI];
};

// One tile product: start() sets out on the tile at (m0, n0) over k in [k0, k1) (multiples of 64, k0 < k1) of every
// segment and starts its first loads, finish() adds the product to acc.  Every thread of the workgroup calls them.
// Between finish() and the next start() no barrier is needed: the last barrier of finish() comes after the last LDS
// read that counts, and start() only writes the stages.
//
// A slab is two steps of 32 k.  While the matrix cores work on one step, the fragments of the next
// one are read: a block row's A fragment as soon as that row's products are issued, so that one set
// of A registers is enough.  The one barrier of a slab stands between its two steps: by then every
// wave has read the whole slab, its stage is loaded again, and the next slab is there.
template <class C>
struct Product {
    using TileA = typename std::conditional<C::PAIR, PairTile<C::BM, C::WAVES>, Tile<C::BM, C::TA, C::WAVES>>::type;
    using TileB = Tile<C::BN, C::TB, C::WAVES>;
    static constexpr int kPer = TileA::kLoads + TileB::kLoads;

    int lane, wave, xa, xb, total, m0, n0;
    uint16_t* lds;

    __device__ __forceinline__ explicit Product(uint16_t* lds_) : lds(lds_) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        xa = (wave % C::WM) * (C::BM / C::WM);
        xb = (wave / C::WM) * (C::BN / C::WN);
    }

    __device__ __forceinline__ void start(const Operand& a, const Operand& b, int m0_, int n0_, int k0, int k1,
                                          Segments seg) {
        m0 = m0_;
        n0 = n0_;
        ta.init(a, m0, wave, lane);
        tb.init(b, n0, wave, lane);
        total = (k1 - k0) / kBK * (int)seg.n;
        ld = Loads(k0, seg);
        const int ahead = C::STAGES < total ? C::STAGES : total;
        for (int i = 0; i < ahead; ++i) {
            ld.begin(a, b, m0, n0, lds);
#pragma unroll
            for (int q = 0; q < kPer; ++q) ld.one(ta, tb, q, wave);
        }
    }

    __device__ __forceinline__ void finish(const Operand& a, const Operand& b, typename C::Acc& acc) {
        // loads end in order, so that what the caller stored since start() can only make this wait longer
        if (total >= C::STAGES) wait_slab<(C::STAGES - 1) * kPer>();
        else wait_slab<0>();
        u32x4 fa[C::MI], fb[C::NI];
        uint16_t* la = lds;
#pragma unroll
        for (int i = 0; i < C::MI; ++i) fa[i] = TileA::frag(la, xa + 16 * i, 0, lane);
#pragma unroll
        for (int j = 0; j < C::NI; ++j) fb[j] = TileB::frag(la + C::BM * kBK, xb + 16 * j, 0, lane);
        int slot = 0;
        auto next = [&]() {
            if (++slot == C::STAGES) slot = 0;
            la = lds + slot * C::kStage;
        };
        int it = 0;
        for (; it + C::STAGES < total; ++it) {
            step<0>(la, 1, fa, fb, acc, [](int) {});
            ld.begin(a, b, m0, n0, lds);
            next();
            wait_slab<(C::STAGES - 2) * kPer>();
            step<kPer>(la, 0, fa, fb, acc, [&](int i) { ld.one(ta, tb, i, wave); });
            __builtin_amdgcn_sched_barrier(0);
        }
        for (; it < total; ++it) {   // nothing left to load
            step<0>(la, 1, fa, fb, acc, [](int) {});
            wait_slab<0>();
            next();
            step<0>(la, 0, fa, fb, acc, [](int) {});   // (behind the last slab it reads a stage whose values are not used)
        }
    }

private:
    // The loads of one slab: which is next, and its descriptors.  All segments of 64 k come before the next 64, so that
    // the planes they share are still in L2.
    struct Loads {
        int k = 0, slot = 0, left = 0;
        Segments all{0, 0};
        uint32_t list = 0;
        u32x4 ra, rb, ra2;
        uint32_t to;
        Loads() = default;
        __device__ __forceinline__ Loads(int k0, Segments seg) : k(k0), left((int)seg.n), all(seg), list(seg.list) {}
        __device__ __forceinline__ void begin(const Operand& a, const Operand& b, int m0, int n0, uint16_t* lds) {
            if constexpr (C::PAIR) {
                ra = TileA::slab(a, m0, list & 3, k, 0);
                ra2 = TileA::slab(a, m0, list & 3, k, 1);
            } else {
                ra = TileA::slab(a, m0, list & 3, k);
            }
            rb = TileB::slab(b, n0, (list >> 2) & 3, k);
            to = (uint32_t)(uintptr_t)(lds_void*)lds + slot * (C::kStage * 2);
            list >>= 4;
            if (--left == 0) { left = (int)all.n; list = all.list; k += kBK; }
            if (++slot == C::STAGES) slot = 0;
        }
        __device__ __forceinline__ void one(const TileA& ta, const TileB& tb, int i, int wave) const {
            if constexpr (C::PAIR) {
                if (i < TileA::kLoads) {
                    ta.load(TileA::matrix(i, wave) ? ra2 : ra, i, to, wave);
                    return;
                }
            }
            if (i < TileA::kLoads) ta.load(ra, i, to, wave);
            else tb.load(rb, i - TileA::kLoads, to + C::BM * kBK * 2, wave);
        }
    };

    TileA ta;
    TileB tb;
    Loads ld;

    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        if constexpr (C::F16)
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }

    // The products of the fragments at hand, and the fragments of step ks of the stage la in their place;
    // load(0 .. LOADS - 1) starts the loads that go along.
    template <int LOADS, class F>
    __device__ __forceinline__ void step(uint16_t* la, int ks, u32x4 (&fa)[C::MI], u32x4 (&fb)[C::NI],
                                         typename C::Acc& acc, F load) const {
        constexpr int per_row = (LOADS + C::MI - 1) / C::MI;
        constexpr int da = C::TA ? 2 : 1, db = C::TB ? 2 : 1;   // LDS reads per fragment
        constexpr int gap = C::MI * C::NI * 3 / 4 / (C::MI * da + C::NI * db) > 1
                                ? C::MI * C::NI * 3 / 4 / (C::MI * da + C::NI * db) : 1;   // products per LDS read
        u32x4 nb[C::NI];
#pragma unroll
        for (int j = 0; j < C::NI; ++j) nb[j] = TileB::frag(la + C::BM * kBK, xb + 16 * j, ks, lane);
#pragma unroll
        for (int i = 0; i < C::MI; ++i) {
#pragma unroll
            for (int j = 0; j < C::NI; ++j)
                acc[i][j] = mma(fa[i], fb[j], acc[i][j]);
#pragma unroll
            for (int q = 0; q < per_row; ++q)
                if (i * per_row + q < LOADS) load(i * per_row + q);
            fa[i] = TileA::frag(la, xa + 16 * i, ks, lane);
        }
#pragma unroll
        for (int j = 0; j < C::NI; ++j) fb[j] = nb[j];
        // keep the reads spread over the first three quarters of the products
#pragma unroll
        for (int r = 0; r < C::NI * db; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x008, gap, 0);   // matrix products
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // LDS read
        }
#pragma unroll
        for (int i = 0; i < C::MI; ++i) {
#pragma unroll
            for (int r = 0; r < da; ++r) {
                __builtin_amdgcn_sched_group_barrier(0x008, gap, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
    }
};

// ---------------------------------------------------------------------------
// Products of few columns with an fp32 matrix read in place: A is fp32 ([x][k] or transposed [k][x]; V4: rows of a multiple
// of four elements, loaded 16 bytes per lane, else four), B three bf16 planes.  Such a product is a stream of A: its tiles go to LDS as they are, and a wave splits
// its fragments into the three parts in registers, all six part products of a slab at once.  (Planes of A in the workspace
// would be written and read again: 4 + 6 bytes per element and more.)  A tile of 128 rows, eight waves of 16 rows each.
//
// LDS image of a [128][64] fp32 tile: 16-byte chunk c of row x at c ^ (x & 15); of a transposed [64][128] one: chunk c of
// row k at c ^ 4 (k / 8 % 4), so that the four rows that a read takes together fall on different banks.
template <int BN_, int STAGES_, bool TA_, bool V4_>
struct FewConfig {
    static constexpr int BM = 128, BN = BN_, WM = 8, WN = 1, STAGES = STAGES_;
    static constexpr bool TA = TA_, TB = false, F16 = false, FEW = true, V4 = V4_;
    static constexpr int WAVES = 8, THREADS = 512, MI = 1, NI = BN / 16;
    static constexpr int kA = BM * kBK * 2, kStage = kA + 3 * BN * kBK;   // in 16-bit elements
    static constexpr int kLds = STAGES * kStage;
    static constexpr int kPerCU = 1;
    typedef f32x4 Acc[MI][NI];
};

template <class C>
struct FewProduct {
    using TileB = Tile<C::BN, false, 4>;   // the planes are loaded by four waves each, two at a time
    static constexpr int kVec = C::V4 ? 4 : 1;   // elements of A per lane and load
    static constexpr int kLoadsA = C::BM * kBK / (64 * kVec) / 8, kLoadsB = 3 * C::BN * kBK * 2 / 1024;   // per wave; per workgroup

    int lane, wave, xa, xb, total, m0, n0;
    uint16_t* lds;

    __device__ __forceinline__ explicit FewProduct(uint16_t* lds_) : lds(lds_) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        xa = wave * 16;
        xb = 0;
    }

    __device__ __forceinline__ void start(const Operand& a, const Operand& b, int m0_, int n0_, int k0_, int k1, Segments) {
        m0 = m0_;
        n0 = n0_;
        k = k0_;
        total = (k1 - k0_) / kBK;
        slot = 0;
        const int ahead = C::STAGES < total ? C::STAGES : total;
        for (int i = 0; i < ahead; ++i) load(a, b);
    }

    __device__ __forceinline__ void finish(const Operand& a, const Operand& b, typename C::Acc& acc) {
        int at = 0;
        for (int it = 0; it < total; ++it) {
            // each later slab under way has at least this many loads in every wave
            if (it + C::STAGES <= total) wait_slab<(C::STAGES - 1) * (kLoadsA + kLoadsB / 8)>();
            else wait_slab<0>();
            const uint16_t* la = lds + at * C::kStage;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u32x4 fa[3];
                split(la, ks, fa);
#pragma unroll
                for (int j = 0; j < C::NI; ++j) {
                    u32x4 fb[3];
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        fb[q] = TileB::frag((uint16_t*)la + C::kA + q * C::BN * kBK, 16 * j, ks, lane);
                    constexpr int ta[6] = {1, 0, 2, 0, 1, 0}, tb[6] = {1, 2, 0, 1, 0, 0};   // smallest first
#pragma unroll
                    for (int t = 0; t < 6; ++t)
                        acc[0][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, fa[ta[t]]), __builtin_bit_cast(bf16x8, fb[tb[t]]), acc[0][j], 0, 0, 0);
                }
            }
            if (++at == C::STAGES) at = 0;
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // every wave has read the slab
            if (it + C::STAGES < total) load(a, b);
        }
    }

private:
    int k, slot;

    __device__ __forceinline__ void load(const Operand& a, const Operand& b) {
        const uint32_t to = (uint32_t)(uintptr_t)(lds_void*)lds + slot * (C::kStage * 2);
        const float* A = (const float*)a.p;
        const int width = (int)a.ld;   // elements of a row, whose last slab or tile ends inside the row
        // offsets outside the descriptor's range (columns behind the row, rows behind the matrix) read as zeros
        const float* base = C::TA ? A + (int64_t)k * a.ld : A + (int64_t)m0 * a.ld + k;
        const int64_t left = (C::TA ? (int64_t)(a.rows - k) * a.ld : (int64_t)(a.rows - m0) * a.ld - k) * 4;
        const uint64_t p = (uint64_t)base;
        const u32x4 ra{(uint32_t)p, (uint32_t)(p >> 32) & 0xffffu, (uint32_t)(left < 0x7fffffff ? left : 0x7fffffff), 0x00027000u};
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            const int q = wave * kLoadsA + i;
            const int at = (q * 64 + lane) * kVec, chunk = at / 4, e = at % 4;   // this lane's element of the image
            uint32_t off;
            if constexpr (!C::TA) {
                const int x = chunk / 16, c = ((chunk % 16) ^ (x & 15)) * 4 + e;
                off = k + c < width ? (uint32_t)(x * width + c) * 4u : kOutside;
            } else {
                const int r = chunk / 32, col = m0 + ((chunk % 32) ^ (((r >> 3) & 3) << 2)) * 4 + e;
                off = col < width ? (uint32_t)(r * width + col) * 4u : kOutside;
            }
            load_to_lds<kVec>(ra, off, to + q * 256 * kVec);
        }
        for (int q = wave; q < kLoadsB; q += 8) {   // eight rows of a plane each
            const int plane = q / (C::BN / 8), x = q % (C::BN / 8) * 8 + lane / 8, c = (lane % 8) ^ ((x >> 1) & 7);
            const uint64_t pb = (uint64_t)(b.p + plane * b.plane + (int64_t)n0 * b.ld + k);
            const u32x4 rb{(uint32_t)__builtin_amdgcn_readfirstlane((int)pb),
                           (uint32_t)__builtin_amdgcn_readfirstlane((int)(pb >> 32)) & 0xffffu, 0x7fffffffu, 0x00027000u};
            const int row = n0 + x < b.rows ? x : b.rows - 1 - n0;
            load_to_lds<4>(rb, (uint32_t)(row * b.ld + c * 8) * 2u, to + C::kA * 2 + q * 1024);
        }
        k += kBK;
        if (++slot == C::STAGES) slot = 0;
    }

    // this wave's fragment of the slab's step ks in three parts
    __device__ __forceinline__ void split(const uint16_t* la, int ks, u32x4 (&f)[3]) const {
        const float* t = (const float*)la;
        float v[8];
        const int g = lane / 16, x = xa + lane % 16;
        if constexpr (!C::TA) {
            const f32x4 lo = *(const f32x4*)&t[x * kBK + (((ks * 8 + 2 * g) ^ (x & 15)) << 2)];
            const f32x4 hi = *(const f32x4*)&t[x * kBK + (((ks * 8 + 2 * g + 1) ^ (x & 15)) << 2)];
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[e] = lo[e]; v[4 + e] = hi[e]; }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = t[(ks * 32 + 8 * g + e) * C::BM + (((x >> 2) ^ (g << 2)) << 2) + (x & 3)];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t w[2][3];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float a = v[2 * e + h];
                w[h][0] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a);
                const float r = a - __uint_as_float(w[h][0] << 16);
                w[h][1] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)r);
                w[h][2] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)(r - __uint_as_float(w[h][1] << 16)));
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) f[q][e] = w[0][q] | (w[1][q] << 16);
        }
    }
};

template <class C, bool FEW = C::FEW>
struct ProductOf { using type = Product<C>; };
template <class C>
struct ProductOf<C, true> { using type = FewProduct<C>; };

}  // namespace mm
}  // namespace dion
