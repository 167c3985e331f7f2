// Gated feed-forward block and its gradients.
//
//   a = X Wg^T;  b = X Wu^T;  u = act(a) b;  Y = u Wd^T
//   du = dY Wd;  da = du b act'(a);  db = du act(a);  dX = da Wg + db Wu;  dWg = da^T X;  dWu = db^T X;  dWd = dY^T u
//
// a and b are one product whose tiles take 16 rows of Wg and of Wu in turn, so that a lane holds both for the same elements
// and the epilogue forms u; du's epilogue reads a and b and forms da, db (side by side, one operand of 2 hidden columns)
// and u.  Then dX is one product over both, and so are dWg and dWu.  Every product runs along the contiguous dimension of
// its output in the matrix core's rows, as in cross_entropy.hip.
//
// bf16 operands multiply as they are, in place where rows are a multiple of 64 elements.  fp32 operands go through planes in
// the workspace: a, b and du as two fp16 parts of each row scaled by a power of two (three products; Wd's rows run along du's
// reduction, so their scales go into dY), the other products as three bf16 parts (six products), since the rows of u, da and db
// that they would be scaled by are not known when they are formed.  Where tiles are left over that do not fill the chip, their
// reductions are sliced: the partial sums are stored, and a pass over them takes the epilogue's place.
//
// Bound by the matrix cores, whose clocks fall under this load.  8192 x 2048 x 5632 bf16 (rows, width, hidden): a, b and u 362 us
// (1.04 PFLOP/s, a library product of that shape 1.07), Y 156 (1.21), du, da, db and u 283 (0.67; a and b are read and three
// outputs written; in the even form 294), dX 297 (1.27), the three weights' gradients 485 (1.17).  4096 x 1024 x 4096 fp32, part products: a, b and u 197
// us (1.05 PFLOP/s), Y 154 and 16 (1.21), du 188 (0.55), dX 317 and 15 (1.25), gradients 569 (1.09), planes 3 x 30.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "block_plan.h"
#include "dion_block.h"
#include "gate.hpp"
#include "rows.hpp"

namespace dion {

namespace {

// ---------------------------------------------------------------------------
// Planes
// ---------------------------------------------------------------------------
// Rows [rows][d] of a matrix to planes with `all` rows of kp elements, zeros behind the matrix; kind: 0 fp32, 1 bf16, 2 e4m3
// with a scale per row.  out: PARTS bf16 planes, or null.  out16: two fp16 ones of the row times a power of two, whose inverse
// goes to inv, and times fold[column] first where that is given; or null.
struct PackJob {
    const void* in;
    const float* scale;
    const float* fold;
    uint16_t* out;
    uint16_t* out16;
    float* inv;
    int64_t rows, all, plane;
    int kind, d, kp;
    unsigned first;   // its first workgroup
};
constexpr int kPackJobs = 5;   // X, Wg, Wu, Wd, dY
struct PackJobs {
    PackJob job[kPackJobs];
    int n;
    unsigned blocks;
};

__device__ __forceinline__ void load_any8(const PackJob& job, int64_t row, int c, int d, float s, float (&v)[8]) {
    if (job.kind == 0) {
        load8<false>(job.in, row, c, d, v);
    } else if (job.kind == 1) {
        load8<true>(job.in, row, c, d, v);
    } else {
        load_e4m3<8>(job.in, row, c, d, s, v);
    }
}

__device__ __forceinline__ void fold8(const PackJob& job, int c, int d, float (&v)[8]) {
    if (!job.fold) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < d) v[e] *= job.fold[c + e];
}

// A wave per row, four of a matrix to a workgroup.
template <int PARTS>
__global__ __launch_bounds__(256) void planes_kernel(PackJobs jobs) {
    int at = 0;
    while (at + 1 < jobs.n && blockIdx.x >= jobs.job[at + 1].first) ++at;
    const PackJob& job = jobs.job[at];
    const int64_t r = (int64_t)(blockIdx.x - job.first) * 4 + (threadIdx.x >> 6);
    if (r >= job.all) return;
    const int d = r < job.rows ? job.d : 0, kp = job.kp, lane = threadIdx.x & 63;
    const float s = job.scale && r < job.rows ? job.scale[r] : 1.f;
    const int64_t row = r * job.d;
    float scale = 1.f;
    if (PARTS == 3 && job.out16) {
        float top = 0.f;
#pragma unroll 4
        for (int c = lane * 8; c < d; c += 512) {
            float v[8];
            load_any8(job, row, c, d, s, v);
            fold8(job, c, d, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fabsf(v[e]) < INFINITY ? fmaxf(top, fabsf(v[e])) : top;   // (others reach no scale)
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        float inverse;
        scale = row_scale(top, inverse);
        if (lane == 0) job.inv[r] = inverse;
    }
#pragma unroll 4
    for (int c = lane * 8; c < kp; c += 512) {
        float v[8];
        load_any8(job, row, c, d, s, v);
        if (job.out) store8<PARTS>(job.out, job.plane, r * kp + c, v);
        if (PARTS == 3 && job.out16) {
            fold8(job, c, d, v);
            store8_f16(job.out16, job.plane, r * kp + c, v, scale);
        }
    }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// A workgroup's share of `total` items.  Workgroups go to the eight XCDs in turn; each XCD takes a contiguous range, which its
// workgroups walk side by side.
struct Turn {
    int at, end, by;
    __device__ __forceinline__ explicit Turn(int total) {
        const int q = total / 8, r = total % 8, x = blockIdx.x % 8;
        by = ((int)gridDim.x - x + 7) / 8;
        const int start = x * q + (x < r ? x : r);
        at = start + blockIdx.x / 8;
        end = start + q + (x < r ? 1 : 0);
    }
    __device__ __forceinline__ bool done() const { return at >= end; }
};

// Tile `t` of a grid of tm rows, in bands of eight tile rows, so that an XCD's L2 serves the operands' re-reads.
__device__ __forceinline__ void place(int t, int tm, int tn, int& mt, int& nt) {
    constexpr int G = 8;
    const int band = t / (G * tn), m0 = band * G, g = tm - m0 < G ? tm - m0 : G, in = t - band * G * tn;
    mt = m0 + in % g;
    nt = in / g;
}

// One product, or two whose reductions have the same length: the second one's tiles come behind the first one's.
struct Operands {
    mm::Operand a, b;
    int64_t m, n;   // rows of a and b that the tiles cover
};

// A lane's place in a tile: column block j's row, the first block's column.
struct Lane {
    int xa, row, quarter;
};

// The tiles of P, whole ones first, then those whose reduction is cut into slices, which leave their sums in `acc` as the lanes
// hold them.  The next tile's loads start before the epilogue of this one.
template <class C, class P>
__global__ __launch_bounds__(C::THREADS) void product_kernel(P p, Cut cut, mm::Segments seg, float* acc) {
    __shared__ __attribute__((aligned(1024))) uint16_t lds[C::kLds];
    mm::Product<C> mul(lds);
    Turn turn(cut.full);
    bool sliced = false;
    auto seek = [&]() {
        if (turn.done() && !sliced) {
            sliced = true;
            turn = Turn(cut.rem * cut.slices);
        }
        return !turn.done();
    };
    if (!seek()) return;
    Operands o;
    int which, unit;
    auto start = [&]() {
        const int slice = sliced ? turn.at / cut.rem : 0, in = sliced ? turn.at - slice * cut.rem : 0;
        int tile = sliced ? cut.full + in : turn.at, mt, nt;
        unit = sliced ? in * cut.slices + slice : -1;
        which = P::kProducts == 2 && tile >= p.template tiles<C>(0);
        if (which) tile -= p.template tiles<C>(0);
        o = p.operands(which);
        place(tile, ((int)o.m + C::BM - 1) / C::BM, ((int)o.n + C::BN - 1) / C::BN, mt, nt);
        const int k0 = slice * cut.k_per, k1 = sliced && k0 + cut.k_per < cut.k ? k0 + cut.k_per : cut.k;
        mul.start(o.a, o.b, mt * C::BM, nt * C::BN, k0, k1, seg);
    };
    start();
    for (;;) {
        const int m0 = mul.m0, n0 = mul.n0, was = which, u = unit;
        typename C::Acc sum = {};
        mul.finish(o.a, o.b, sum);
        turn.at += turn.by;
        const bool more = seek();
        if (more) start();
        if (u >= 0) {
            f32x4* to = (f32x4*)acc + (int64_t)u * C::MI * C::NI * C::THREADS + threadIdx.x;
#pragma unroll
            for (int i = 0; i < C::MI; ++i)
#pragma unroll
                for (int j = 0; j < C::NI; ++j) to[(i * C::NI + j) * C::THREADS] = sum[i][j];
        } else {
            const auto store = [&](auto edge) {
#pragma unroll
                for (int j = 0; j < C::NI; ++j) {
                    f32x4 v[C::MI];
#pragma unroll
                    for (int i = 0; i < C::MI; ++i) v[i] = sum[i][j];
                    p.template column<C, decltype(edge)::value>(
                        was, m0, n0, Lane{mul.xa, mul.xb + 16 * j + mul.lane % 16, mul.lane / 16}, v);
                    __builtin_amdgcn_sched_barrier(0);   // a column's values die before the next one's are formed
                }
            };
            if (p.template inside<C>(was, m0)) store(std::false_type());
            else store(std::true_type());
        }
        if (!more) return;
    }
}

// The epilogue of the sliced tiles, a workgroup for each of a tile's NI columns of blocks.
template <class C, class P>
__global__ __launch_bounds__(C::THREADS) void join_kernel(P p, Cut cut, const float* acc) {
    const int in = blockIdx.x / C::NI, j = blockIdx.x % C::NI;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int tile = cut.full + in, mt, nt;
    const int which = P::kProducts == 2 && tile >= p.template tiles<C>(0);
    if (which) tile -= p.template tiles<C>(0);
    const Operands o = p.operands(which);
    place(tile, ((int)o.m + C::BM - 1) / C::BM, ((int)o.n + C::BN - 1) / C::BN, mt, nt);
    const f32x4* from = (const f32x4*)acc + ((int64_t)in * cut.slices * C::MI * C::NI + j) * C::THREADS + threadIdx.x;
    f32x4 v[C::MI];
#pragma unroll
    for (int i = 0; i < C::MI; ++i) v[i] = from[i * C::NI * C::THREADS];
#pragma unroll 2
    for (int s = 1; s < cut.slices; ++s)
#pragma unroll
        for (int i = 0; i < C::MI; ++i) v[i] += from[((int64_t)s * C::MI + i) * C::NI * C::THREADS];
    p.template column<C, true>(which, mt * C::BM, nt * C::BN,
                               Lane{wave % C::WM * (C::BM / C::WM), wave / C::WM * (C::BN / C::WN) + 16 * j + lane % 16, lane / 16}, v);
}

struct GatedArgs {
    Operands o;            // Wg and Wu (a PairTile) and X, or Wd and dY
    int64_t rows;
    int f, fk, act;
    void* gate;            // [rows][f], or null
    void* up;
    uint16_t* u;           // planes [PARTS][rows][fk], or null (du)
    uint16_t* dab;         // du: planes [PARTS][rows][2 fk], or for two parts [rows][2][2 fk], or null
    const float* xinv;     // fp32: what the sums of a row are multiplied by,
    const float* winv;     // and those of a column (a, and `winv_b` on b), du: null
    int winv_b;
};

// Rows of a matrix from one of them on, read and written through a descriptor: offsets are 32 bits, what lies behind the last
// row reads as zero and is not written.
struct Rows {
    __amdgpu_buffer_rsrc_t to;
    int ld;   // elements
    template <int BYTES>
    static __device__ __forceinline__ Rows of(const void* p, int64_t row, int64_t rows, int ld) {
        const int64_t left = row < rows ? (rows - row) * ld * BYTES : 0;
        return Rows{__builtin_amdgcn_make_buffer_rsrc((void*)((const char*)p + row * ld * BYTES), 0,
                                                      (int)(left < 0x7fffffff ? left : 0x7fffffff), 0x00027000), ld};
    }
};

// A tile's values as a lane has them: H (1 or 2) neighbouring blocks of 16 columns, of which its quarter has four each.  Two
// blocks of 16-bit values are traded, so that the lane stores eight in a row.
struct Spot {
    int row;       // from the first of Rows
    int c0;        // the first block's first column, the same for the wave
    int quarter;
    __device__ __forceinline__ int own(int h) const { return c0 + 16 * h + 4 * quarter; }                     // of four
    __device__ __forceinline__ int traded() const { return c0 + 16 * (quarter / 2) + 8 * (quarter % 2); }     // of eight
};

// 16-bit words to columns below d.  EDGE: the tile may reach behind them (else nothing is checked).  ROUND: rows of a multiple
// of eight elements, which end with a lane's.
template <int H, bool EDGE, bool ROUND>
__device__ __forceinline__ void put_words(const Rows& to, const Spot& s, int d, const uint32_t (&w)[H][2]) {
    constexpr int N = 4 * H;
    const int c = H == 2 ? s.traded() : s.own(0);
    const uint32_t off = (uint32_t)(s.row * to.ld + c) * 2u;
    u32x4 t;
    if constexpr (H == 2) t = trade(w[0], w[1]);
    else t = u32x4{w[0][0], w[0][1], 0, 0};
    if (!EDGE || ROUND || s.c0 + 16 * H <= d) {
        const uint32_t at = EDGE && ROUND && c >= d ? mm::kOutside : off;
        if constexpr (H == 2) __builtin_amdgcn_raw_buffer_store_b128(t, to.to, at, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b64(u32x2{t[0], t[1]}, to.to, at, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(t[e / 2] >> (16 * (e % 2))), to.to,
                                                  c + e < d ? off + 2u * e : mm::kOutside, 0, 0);
    }
}

// Two blocks' words as this lane stores them, columns below d (the others may be anything).  A ragged end is read one by
// one: a vector whose last word is half behind the last row reads as zero there.
template <bool EDGE>
__device__ __forceinline__ u32x4 load_words(const Rows& from, const Spot& s, int d) {
    const int c = s.traded();
    const uint32_t off = (uint32_t)(s.row * from.ld + c) * 2u;
    if (!EDGE || s.c0 + 32 <= d) return __builtin_amdgcn_raw_buffer_load_b128(from.to, off, 0, 0);
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = __builtin_amdgcn_raw_buffer_load_b16(from.to, c + e < d ? off + 2u * e : mm::kOutside, 0, 0);
    u32x4 t;
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = h[2 * e] | (h[2 * e + 1] << 16);
    return t;
}

template <bool EDGE>
__device__ __forceinline__ void put_floats(const Rows& to, const Spot& s, int h, int d, const float (&v)[4]) {
    const int c = s.own(h);
    const uint32_t off = (uint32_t)(s.row * to.ld + c) * 4u;
    if (!EDGE || s.c0 + 16 * h + 16 <= d) {
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                     __float_as_uint(v[3])}, to.to, off, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), to.to, c + e < d ? off + 4u * e : mm::kOutside, 0, 0);
    }
}

__device__ __forceinline__ void get_floats(const Rows& from, const Spot& s, int h, float (&v)[4]) {
    const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(from.to, (uint32_t)(s.row * from.ld + s.own(h)) * 4u, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(t[e]);
}

// Parts of the values to planes whose rows end at `kp` columns, a multiple of 64: each the rounding of what the ones before it
// leave, an exact split.
template <int PARTS, int H, bool EDGE>
__device__ __forceinline__ void put_parts(const Rows (&to)[PARTS], const Spot& s, int kp, float (&v)[H][4]) {
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
        uint32_t w[H][2];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const uint32_t a = down16(v[h][e]), b = down16(v[h][e + 1]);
                w[h][e / 2] = a | (b << 16);
                v[h][e] -= up16(a);
                v[h][e + 1] -= up16(b);
            }
        put_words<H, EDGE, true>(to[q], s, kp, w);
    }
}

// a or b to its buffer, rows of d elements
template <int PARTS, bool EVEN, int H, bool EDGE>
__device__ __forceinline__ void put_kept(const Rows& to, const Spot& s, int d, const float (&v)[H][4]) {
    if constexpr (PARTS != 3) {
        uint32_t w[H][2];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int e = 0; e < 4; e += 2) w[h][e / 2] = keep32<EVEN>(v[h][e], v[h][e + 1]);
        put_words<H, EDGE, false>(to, s, d, w);
    } else {
#pragma unroll
        for (int h = 0; h < H; ++h) put_floats<EDGE>(to, s, h, d, v[h]);
    }
}

// Two blocks of a or b as they are in memory.
template <int PARTS, bool EVEN>
struct Raw {
    u32x4 w[PARTS != 3 ? 1 : 2];
    template <bool EDGE>
    __device__ __forceinline__ void load(const Rows& from, const Spot& s, int d) {
        if constexpr (PARTS != 3) {
            w[0] = load_words<EDGE>(from, s, d);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[h] = __builtin_amdgcn_raw_buffer_load_b128(from.to, (uint32_t)(s.row * from.ld + s.own(h)) * 4u, 0, 0);
        }
    }
    __device__ __forceinline__ void get(float (&v)[2][4]) const {
        if constexpr (PARTS != 3) {
            uint32_t t[2][2];
            untrade(w[0], t[0], t[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[h][e] = kept16<EVEN>(t[h][e / 2] >> (16 * (e % 2)) & 0xffffu);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[h][e] = __uint_as_float(w[h][e]);
        }
    }
};

// What the epilogues write and read, from row n on.
template <int PARTS>
struct GatedRows {
    Rows gate, up, u[PARTS], da[PARTS], db[PARTS];
    __device__ __forceinline__ GatedRows(const GatedArgs& g, int64_t n) {
        constexpr int B = PARTS != 3 ? 2 : 4;
        gate = Rows::of<B>(g.gate, n, g.gate ? g.rows : 0, g.f);
        up = Rows::of<B>(g.up, n, g.up ? g.rows : 0, g.f);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            u[q] = Rows::of<2>(g.u + q * g.rows * g.fk, n, g.u ? g.rows : 0, g.fk);
            const int64_t at = PARTS == 2 ? (int64_t)q * 2 * g.fk : q * g.rows * 2 * g.fk;
            constexpr int WIDE = PARTS == 2 ? 4 : 2;
            da[q] = Rows::of<2>(g.dab + at, n, g.dab ? g.rows : 0, WIDE * g.fk);
            db[q] = da[q];
            db[q].to = Rows::of<2>(g.dab + at + g.fk, n, g.dab ? g.rows : 0, WIDE * g.fk).to;
        }
    }
};

// u of H blocks from a and b, which are kept where asked for.
template <int PARTS, bool EVEN, int H, bool EDGE>
__device__ __forceinline__ void gated(const GatedArgs& g, const GatedRows<PARTS>& to, const Spot& s, const float (&a)[H][4],
                                      const float (&b)[H][4]) {
    if (g.gate) {
        put_kept<PARTS, EVEN, H, EDGE>(to.gate, s, g.f, a);
        put_kept<PARTS, EVEN, H, EDGE>(to.up, s, g.f, b);
    }
    if (!g.u) return;
    float u[H][4];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float slope;
            u[h][e] = activate<PARTS == 3>(g.act, a[h][e], slope) * b[h][e];
            if (EDGE && s.own(h) + e >= g.f) u[h][e] = 0.f;
        }
    put_parts<PARTS, H, EDGE>(to.u, s, g.fk, u);
}

// da, db and u of two blocks from du, a and b.
template <int PARTS, bool EDGE>
__device__ __forceinline__ void dgated(const GatedArgs& g, const GatedRows<PARTS>& to, const Spot& s, const float (&du)[2][4],
                                       const float (&a)[2][4], const float (&b)[2][4]) {
    float da[2][4], db[2][4], u[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float slope;
            const float v = activate<PARTS == 3>(g.act, a[h][e], slope);
            da[h][e] = du[h][e] * b[h][e] * slope;
            db[h][e] = du[h][e] * v;
            u[h][e] = v * b[h][e];
            if (EDGE && s.own(h) + e >= g.f) da[h][e] = db[h][e] = u[h][e] = 0.f;   // (made of anything there)
        }
    if (g.dab) {
        put_parts<PARTS, 2, EDGE>(to.da, s, g.fk, da);
        put_parts<PARTS, 2, EDGE>(to.db, s, g.fk, db);
    }
    if (g.u) put_parts<PARTS, 2, EDGE>(to.u, s, g.fk, u);
}

struct Single {
    static constexpr int kProducts = 1;
    template <class C>
    __device__ __forceinline__ int tiles(int) const { return 0; }
};

// a and b: blocks 2 i and 2 i + 1 of a tile are a and b of the same 16 columns
template <int PARTS, bool EVEN>
struct Gated : Single {
    GatedArgs g;
    explicit Gated(const GatedArgs& a) : g(a) {}
    __device__ __forceinline__ const Operands& operands(int) const { return g.o; }
    template <class C>
    __device__ __forceinline__ bool inside(int, int m0) const { return m0 + C::BM <= 2 * g.f; }
    template <class C, bool EDGE>
    __device__ __forceinline__ void column(int, int m0, int n0, const Lane& l, const f32x4 (&v)[C::MI]) const {
        constexpr int H = C::MI % 4 == 0 ? 2 : 1;
        const GatedRows<PARTS> to(g, n0);
        const int c0 = (m0 + l.xa) / 2;
        const float x = PARTS != 3 ? 1.f : g.xinv[n0 + l.row];
#pragma unroll
        for (int i = 0; i < C::MI; i += 2 * H) {
            float a[H][4], b[H][4];
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) { a[h][e] = v[i + 2 * h][e]; b[h][e] = v[i + 2 * h + 1][e]; }
            if constexpr (PARTS == 3) {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float* w = g.winv + c0 + 8 * i + 16 * h + 4 * l.quarter;
                    const f32x4 wa = *(const f32x4*)w, wb = *(const f32x4*)(w + g.winv_b);
#pragma unroll
                    for (int e = 0; e < 4; ++e) { a[h][e] = a[h][e] * x * wa[e]; b[h][e] = b[h][e] * x * wb[e]; }
                }
            }
            gated<PARTS, EVEN, H, EDGE>(g, to, Spot{l.row, c0 + 8 * i, l.quarter}, a, b);
        }
    }
};

// du.  A column's a and b are all on their way before the first is used.
template <int PARTS, bool EVEN>
struct Dgated : Single {
    GatedArgs g;
    explicit Dgated(const GatedArgs& a) : g(a) {}
    __device__ __forceinline__ const Operands& operands(int) const { return g.o; }
    template <class C>
    __device__ __forceinline__ bool inside(int, int m0) const { return m0 + C::BM <= g.f; }
    template <class C, bool EDGE>
    __device__ __forceinline__ void column(int, int m0, int n0, const Lane& l, const f32x4 (&v)[C::MI]) const {
        const GatedRows<PARTS> to(g, n0);
        const float x = PARTS != 3 ? 1.f : g.xinv[n0 + l.row];
        // fp32 ones, which are twice as wide, half a column at a time: 4096 x 1024 x 4096 234 us, so 188.  (25 vector registers still
        // spill, and 30 of the bf16 ones, which go by whole columns; both spill scalar ones, mostly the rows' descriptors.)
        constexpr int N = PARTS == 3 && C::MI >= 8 ? C::MI / 2 : C::MI;
#pragma unroll
        for (int i0 = 0; i0 < C::MI; i0 += N) {
            Raw<PARTS, EVEN> ra[N / 2], rb[N / 2];
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const Spot s{l.row, m0 + l.xa + 16 * (i0 + i), l.quarter};
                ra[i / 2].template load<EDGE>(to.gate, s, g.f);
                rb[i / 2].template load<EDGE>(to.up, s, g.f);
            }
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float du[2][4], a[2][4], b[2][4];
                ra[i / 2].get(a);
                rb[i / 2].get(b);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) du[h][e] = PARTS != 3 ? v[i0 + i + h][e] : v[i0 + i + h][e] * x;
                dgated<PARTS, EDGE>(g, to, Spot{l.row, m0 + l.xa + 16 * (i0 + i), l.quarter}, du, a, b);
            }
            if (N < C::MI) __builtin_amdgcn_sched_barrier(0);
        }
    }
};

struct OutArgs {
    Operands o;
    int cols;               // of the output
    int64_t second, valid;  // rows of the product from which they are the second output's (all where there is one), rows of each
    void* out;
    void* out2;
    int bf16, accumulate;
};

// Rows n .. n + 15 of the product (n a multiple of 16) in their output.
__device__ __forceinline__ Rows out_rows(const OutArgs& a, int64_t n) {
    const bool two = n >= a.second;   // (a multiple of 64 where there are two outputs)
    void* out = two ? a.out2 : a.out;
    const int64_t row = two ? n - a.second : n, rows = two && !a.out2 ? 0 : a.valid;
    return a.bf16 ? Rows::of<2>(out, row, rows, a.cols) : Rows::of<4>(out, row, rows, a.cols);
}

template <bool EDGE>
__device__ __forceinline__ void put_out(const OutArgs& a, const Rows& to, const Spot& s, float (&v)[2][4]) {
    if (a.bf16) {
        uint32_t w[2][2];
        if (a.accumulate) {
            untrade(load_words<EDGE>(to, s, a.cols), w[0], w[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[h][e] += up16(w[h][e / 2] >> (16 * (e % 2)) & 0xffffu);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; e += 2) w[h][e / 2] = down16(v[h][e]) | (down16(v[h][e + 1]) << 16);
        put_words<2, EDGE, false>(to, s, a.cols, w);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (a.accumulate) {
                float old[4];
                get_floats(to, s, h, old);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[h][e] += old[e];
            }
            put_floats<EDGE>(to, s, h, a.cols, v[h]);
        }
    }
}

// Products into outputs: one, or dWg | dWu and dWd at once.
template <int N>
struct Out {
    static constexpr int kProducts = N;
    OutArgs p[N];
    explicit Out(const OutArgs& a) : p{a} {}
    Out(const OutArgs& a, const OutArgs& b) : p{a, b} {}
    template <class C>
    __device__ __forceinline__ int tiles(int i) const {
        return (((int)p[i].o.m + C::BM - 1) / C::BM) * (((int)p[i].o.n + C::BN - 1) / C::BN);
    }
    __device__ __forceinline__ const Operands& operands(int which) const { return p[N == 2 ? which : 0].o; }
    template <class C>
    __device__ __forceinline__ bool inside(int which, int m0) const { return m0 + C::BM <= p[N == 2 ? which : 0].cols; }
    template <class C, bool EDGE>
    __device__ __forceinline__ void column(int which, int m0, int n0, const Lane& l, const f32x4 (&v)[C::MI]) const {
        const OutArgs& a = p[N == 2 ? which : 0];
        const int n = __builtin_amdgcn_readfirstlane(l.row) & ~15;   // the block's first row
        const Rows to = out_rows(a, n0 + n);
#pragma unroll
        for (int i = 0; i < C::MI; i += 2) {
            float w[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[h][e] = v[i + h][e];
            put_out<EDGE>(a, to, Spot{l.row - n, m0 + l.xa + 16 * i, l.quarter}, w);
        }
    }
};

__global__ __launch_bounds__(256) void zeros_kernel(uint16_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <bool TA, bool TB, bool F16, bool PAIR, class F>
void of_tile(int tile, F f) {
    if (tile == TILE_256) f(mm::Config<256, 256, 2, 4, 2, TA, TB, F16, PAIR>());
    else if (tile == TILE_128) f(mm::Config<128, 128, 2, 2, 2, TA, TB, F16, PAIR>());   // two workgroups to a CU
    else if (tile == TILE_64) f(mm::Config<64, 64, 2, 2, 8, TA, TB, F16, PAIR>());
    else if constexpr (!TB) f(mm::Config<128, 32, 4, 1, 4, TA, TB, F16, PAIR>());
}

template <class C, class P>
void launch(const P& p, const Product& r, mm::Segments seg, float* acc, hipStream_t s) {
    const Cut& c = r.cut;
    const int64_t items = c.full > (int64_t)c.rem * c.slices ? c.full : (int64_t)c.rem * c.slices;
    hipLaunchKernelGGL((product_kernel<C, P>), walkers<C>(items), dim3(C::THREADS), 0, s, p, c, seg, acc);
    if (c.rem) hipLaunchKernelGGL((join_kernel<C, P>), dim3((unsigned)(c.rem * C::NI)), dim3(C::THREADS), 0, s, p, c, acc);
}

template <bool GRAD, int PARTS, bool EVEN>
void launch_gated(const GatedArgs& g, const Product& r, mm::Segments seg, float* acc, hipStream_t s) {
    using P = typename std::conditional<GRAD, Dgated<PARTS, EVEN>, Gated<PARTS, EVEN>>::type;
    if constexpr (GRAD && PARTS == 2) launch<mm::Config<128, 32, 4, 1, 4, true, false, false, false>>(P(g), r, seg, acc, s);   // so few rows
    else of_tile<GRAD, false, PARTS == 3, !GRAD>(r.tile, [&](auto c) { launch<decltype(c)>(P(g), r, seg, acc, s); });
}

// even: the form of gate and up, for bf16 operands.  (One that is known when the kernel runs cost du of 8192 x 2048 x 5632 30 us.)
template <bool GRAD>
void launch_gated(const GatedArgs& g, const Product& r, int parts, int even, float* acc, hipStream_t s) {
    if (parts == 3) launch_gated<GRAD, 3, false>(g, r, segments(2, 2), acc, s);
    else if (parts == 1 && even) launch_gated<GRAD, 1, true>(g, r, segments(1, 1), acc, s);
    else if (parts == 1) launch_gated<GRAD, 1, false>(g, r, segments(1, 1), acc, s);
    else if (even) launch_gated<GRAD, 2, true>(g, r, segments(1, 1), acc, s);
    else launch_gated<GRAD, 2, false>(g, r, segments(1, 1), acc, s);
}

template <bool TA, bool TB, int N>
void launch_out(const Out<N>& o, const Product& r, mm::Segments seg, float* acc, hipStream_t s) {
    of_tile<TA, TB, false, false>(r.tile, [&](auto c) { launch<decltype(c)>(o, r, seg, acc, s); });
}

// Planes that a job fills: bf16 ones, fp16 ones, or both.
void pack(PackJobs& jobs, PackJob job) {
    if (job.all == 0) job.all = job.rows;
    job.kp = (job.d + 63) / 64 * 64;
    job.first = jobs.blocks;
    jobs.job[jobs.n++] = job;
    jobs.blocks += (unsigned)ceil_div64(job.all, 4);
}

void launch_pack(const PackJobs& jobs, int parts, hipStream_t s) {
    if (jobs.n == 0) return;
    if (parts == 1) hipLaunchKernelGGL((planes_kernel<1>), dim3(jobs.blocks), dim3(256), 0, s, jobs);
    else hipLaunchKernelGGL((planes_kernel<3>), dim3(jobs.blocks), dim3(256), 0, s, jobs);
}

struct Inputs {
    mm::Operand x, w, wd, dy;           // parts of X, of Wg and, `pair` elements on, Wu, of Wd, of dY
    mm::Operand x16, w16, wd16, dy16;   // what a, b and du are formed from: fp16 planes for fp32, else the same
};

// The operands of the products that are asked for: forms: a and b, out: Y, dx, dgu and dd: the gradients.
Inputs inputs(const FfnArgs& a, const FfnPlan& p, char* ws, bool forms, bool out, hipStream_t s) {
    Inputs in{};
    PackJobs jobs{};
    const int kind = a.bf16 ? 1 : 0, t = (int)p.t, d = (int)p.d, f = (int)p.f;
    auto at = [&](size_t off) { return (uint16_t*)(ws + off); };
    auto inverse = [&](size_t off) { return (float*)(ws + off); };
    const int64_t wplane = 2 * p.fk * p.dk, wpair = p.fk * p.dk;
    const int xkind = a.x_scale ? 2 : kind;
    if (a.bf16) {
        in.x = mm::Operand{(const uint16_t*)a.X, 0, p.d, t};
        if (p.xpack && (forms || a.dWg)) {
            pack(jobs, {a.X, a.x_scale, nullptr, at(p.x), nullptr, nullptr, t, 0, p.t * p.dk, xkind, d});
            in.x = mm::Operand{at(p.x), 0, p.dk, t};
        }
        in.w = mm::Operand{(const uint16_t*)a.Wg, 0, p.d, f, ((intptr_t)a.Wu - (intptr_t)a.Wg) / 2};
        if (p.wpack && (forms || a.dX)) {
            pack(jobs, {a.Wg, nullptr, nullptr, at(p.w), nullptr, nullptr, f, p.fk, wplane, kind, d});
            pack(jobs, {a.Wu, nullptr, nullptr, at(p.w) + wpair, nullptr, nullptr, f, p.fk, wplane, kind, d});
            in.w = mm::Operand{at(p.w), 0, p.dk, f, wpair};
        }
        in.wd = mm::Operand{(const uint16_t*)a.Wd, 0, p.f, d};
        if (p.dpack) {
            pack(jobs, {a.Wd, nullptr, nullptr, at(p.wd), nullptr, nullptr, d, 0, p.d * p.fk, kind, f});
            in.wd = mm::Operand{at(p.wd), 0, p.fk, d};
        }
        in.dy = mm::Operand{(const uint16_t*)a.dY, 0, p.d, t};
        if (p.ypack && a.dY) {
            pack(jobs, {a.dY, nullptr, nullptr, at(p.dy), nullptr, nullptr, t, 0, p.t * p.dk, kind, d});
            in.dy = mm::Operand{at(p.dy), 0, p.dk, t};
        }
        in.x16 = in.x; in.w16 = in.w; in.wd16 = in.wd; in.dy16 = in.dy;
        launch_pack(jobs, 1, s);
        return in;
    }
    if (forms || a.dWg)
        pack(jobs, {a.X, a.x_scale, nullptr, a.dWg ? at(p.x) : nullptr, forms ? at(p.x16) : nullptr, inverse(p.xinv), t, 0,
                    p.t * p.dk, xkind, d});
    if (forms || a.dX)
        for (int i = 0; i < 2; ++i)
            pack(jobs, {i ? a.Wu : a.Wg, nullptr, nullptr, a.dX ? at(p.w) + i * wpair : nullptr, forms ? at(p.w16) + i * wpair : nullptr,
                        inverse(p.winv) + i * scale_rows(p.fk), f, p.fk, wplane, kind, d});
    pack(jobs, {a.Wd, nullptr, nullptr, out ? at(p.wd) : nullptr, out ? nullptr : at(p.wd16), inverse(p.dinv), d, 0, p.d * p.fk, kind, f});
    launch_pack(jobs, 3, s);
    if (a.dY) {   // du = (dY / scale of Wd's row) (Wd scaled): behind Wd's scales
        PackJobs last{};
        pack(last, {a.dY, nullptr, inverse(p.dinv), a.dWd ? at(p.dy) : nullptr, at(p.dy16), inverse(p.yinv), t, 0, p.t * p.dk, kind, d});
        launch_pack(last, 3, s);
    }
    in.x = mm::Operand{at(p.x), p.t * p.dk, p.dk, t};
    in.w = mm::Operand{at(p.w), wplane, p.dk, f, wpair};
    in.wd = mm::Operand{at(p.wd), p.d * p.fk, p.fk, d};
    in.dy = mm::Operand{at(p.dy), p.t * p.dk, p.dk, t};
    in.x16 = in.x; in.w16 = in.w; in.wd16 = in.wd; in.dy16 = in.dy;
    in.x16.p = at(p.x16); in.w16.p = at(p.w16); in.wd16.p = at(p.wd16); in.dy16.p = at(p.dy16);
    return in;
}

// Planes of the rows alone, of X and of dY.
Inputs rows_in_planes(const FfnArgs& a, const FfnPlan& p, char* ws, bool x, hipStream_t s) {
    Inputs in{};
    PackJobs jobs{};
    const int t = (int)p.t, d = (int)p.d;
    in.x = mm::Operand{(uint16_t*)(ws + p.x), p.t * p.dk, p.dk, t};
    in.dy = mm::Operand{(uint16_t*)(ws + p.dy), p.t * p.dk, p.dk, t};
    if (x) pack(jobs, {a.X, a.x_scale, nullptr, (uint16_t*)(ws + p.x), nullptr, nullptr, t, 0, p.t * p.dk, a.x_scale ? 2 : 0, d});
    if (a.dY) pack(jobs, {a.dY, nullptr, nullptr, (uint16_t*)(ws + p.dy), nullptr, nullptr, t, 0, p.t * p.dk, 0, d});
    launch_pack(jobs, 3, s);
    return in;
}

// The products of u, da and db: of bf16 operands, whose planes are all the same, with one part or two of them.
mm::Segments part_products(const FfnPlan& p) {
    if (p.parts == 3) return segments(3, 3);
    return p.uparts == 2 ? mm::Segments{2, 1 | 1 << 2} : segments(1, 1);   // the second parts first
}

GatedArgs gated_args(const FfnArgs& a, const FfnPlan& p, const mm::Operand& w, const mm::Operand& x, int64_t m, char* ws) {
    GatedArgs g{};
    g.o = Operands{w, x, m, p.t};
    g.rows = p.t; g.f = (int)p.f; g.fk = (int)p.fk; g.act = a.act;
    g.gate = a.gate; g.up = a.up;
    g.u = (uint16_t*)(ws + p.u);
    g.xinv = (const float*)(ws + p.xinv); g.winv = (const float*)(ws + p.winv);
    g.winv_b = (int)scale_rows(p.fk);
    return g;
}

OutArgs out_args(const mm::Operand& x, const mm::Operand& y, int64_t cols, int64_t rows, void* out, int bf16, int accumulate) {
    return OutArgs{{x, y, cols, rows}, (int)cols, rows, rows, out, nullptr, bf16, accumulate};
}

}  // namespace

int run_zeros(void* out, int64_t n, void* stream) {
    hipLaunchKernelGGL(zeros_kernel, dim3((unsigned)stride_blocks(ceil_div64(n, 256 * 8))), dim3(256), 0, (hipStream_t)stream,
                       (uint16_t*)out, n);
    return (int)hipGetLastError();
}

int run_ffn(const FfnArgs& a, const FfnPlan& p, char* ws, void* stream) {
    if (p.few) return run_ffn_few(a, p, ws, stream);
    const hipStream_t s = (hipStream_t)stream;
    if (p.mid) {
        rows_in_planes(a, p, ws, true, s);
        const int e = run_mid_gate(a, p, true, ws, stream);
        return e ? e : run_mid_out(a, p, ws, stream);
    }
    const Inputs in = inputs(a, p, ws, true, true, s);
    const mm::Segments seg = part_products(p);
    float* acc = (float*)(ws + p.acc);
    launch_gated<false>(gated_args(a, p, in.w16, in.x16, 2 * p.fk, ws), p.gu, p.uparts, a.even, acc, s);
    const mm::Operand u{(uint16_t*)(ws + p.u), p.t * p.fk, p.fk, (int)p.t};
    launch_out<false, false>(Out<1>(out_args(in.wd, u, p.d, p.t, a.Y, a.bf16, 0)), p.y, seg, acc, s);
    return (int)hipGetLastError();
}

int run_ffn_grad(const FfnArgs& args, const FfnPlan& p, char* ws, void* stream) {
    if (p.few) return run_ffn_few_grad(args, p, ws, stream);
    const hipStream_t s = (hipStream_t)stream;
    FfnArgs a = args;
    const bool form = !a.gate;
    const Inputs in = p.mid ? rows_in_planes(a, p, ws, form || a.dWg, s) : inputs(a, p, ws, form, false, s);
    const mm::Segments seg = part_products(p);
    float* acc = (float*)(ws + p.acc);
    if (form) {
        a.gate = ws + p.gate;
        a.up = ws + p.up;
        a.even = 1;
    }
    const mm::Operand dab{(uint16_t*)(ws + p.dab), p.uparts == 2 ? 2 * p.fk : p.t * 2 * p.fk, (p.uparts == 2 ? 4 : 2) * p.fk, (int)p.t};
    const mm::Operand u{(uint16_t*)(ws + p.u), p.t * p.fk, p.fk, (int)p.t};
    if (p.mid) {
        int e = form ? run_mid_gate(a, p, false, ws, stream) : 0;
        if (!e) e = run_mid_du(a, p, ws, stream);
        if (!e && a.dX) e = run_mid_dx(a, p, ws, stream);
        if (e) return e;
    } else {
        if (form) {
            GatedArgs g = gated_args(a, p, in.w16, in.x16, 2 * p.fk, ws);
            g.u = nullptr;
            launch_gated<false>(g, p.gu, p.uparts, a.even, acc, s);
        }
        GatedArgs g = gated_args(a, p, in.wd16, in.dy16, p.fk, ws);
        g.xinv = (const float*)(ws + p.yinv);
        g.dab = a.dX || a.dWg ? (uint16_t*)(ws + p.dab) : nullptr;
        if (!a.dWd) g.u = nullptr;
        launch_gated<true>(g, p.du, p.uparts, a.even, acc, s);
        if (a.dX) {   // over da and Wg, db and Wu: two planes of one part each in place, one matrix of 2 fk rows where packed
            OutArgs o = out_args(in.w, dab, p.d, p.t, a.dX, a.bf16, 0);
            mm::Segments pairs = seg;
            if (p.wpack) {
                o.o.a.rows = (int)(2 * p.fk);
            } else {
                o.o.a.plane = in.w.pair;
                o.o.b.plane = p.fk;
                pairs = p.uparts == 2 ? mm::Segments{4, 2 << 2 | (1 | 3 << 2) << 4 | 0 << 8 | (1 | 1 << 2) << 12}
                                      : mm::Segments{2, 0 | (1 | 1 << 2) << 4};
            }
            launch_out<true, false>(Out<1>(o), p.dx, pairs, acc, s);
        }
    }
    OutArgs gu = out_args(in.x, dab, p.d, 2 * p.fk, a.dWg, a.dw_bf16, a.accumulate);
    gu.second = p.fk; gu.valid = p.f; gu.out2 = a.dWu;
    const OutArgs d = out_args(u, in.dy, p.f, p.d, a.dWd, a.dw_bf16, a.accumulate);
    if (a.dWg && a.dWd) launch_out<true, true>(Out<2>(gu, d), p.dw, seg, acc, s);
    else if (a.dWg) launch_out<true, true>(Out<1>(gu), p.dgu, seg, acc, s);
    else if (a.dWd) launch_out<true, true>(Out<1>(d), p.dd, seg, acc, s);
    return (int)hipGetLastError();
}

}  // namespace dion
