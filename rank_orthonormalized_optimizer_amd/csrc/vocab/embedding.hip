// Embedding lookup with a scale, and the gradient of its table by sorted tokens.
//
//   Y[t] = scale * W[ids[t]]                        one gather, bound by HBM (read and write d elements per token)
//   dW[v] (+)= scale * sum over ids[t] = v of dY[t]
//
// The gradient sorts the tokens by id, in their order where ids are equal, and cuts the sorted list into chunks of equal
// length, so that frequent ids load no workgroup more than others.  A team of threads walks one chunk, adding rows of dY in fp32 registers; a run
// of one id that lies inside the chunk is written to its row, the part of a run that crosses a
// border goes to a partial row, and a second pass adds the partial rows of a run in chunk order.
// No floating-point atomics: the order of additions depends on the tokens alone.
//
// Bound by HBM, small calls by their launches.  Measured: 65536 rows of 4096 bf16 looked up in 181 us (5.9 TB/s, where a
// copy of 2 GiB reaches 4.9); gradient of 16384 tokens, 32000 x 2048 bf16, 62 us in three launches (29 sorting beside the
// clearing of the table, whose 131 MB take 19; 18 adding rows, 5.2 TB/s; 7 joining); 65536 tokens added to a 65536 x 4096
// fp32 table 298 us (256 of them at 4.5 TB/s of rows read, added to and written).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dion_vocab.h"
#include "vocab_plan.h"

namespace dion {

namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float up16(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ uint32_t down16(float f) { return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f); }

// Vectors at any element's address: the memory unit takes such accesses whole.
typedef f32x4_t __attribute__((aligned(4))) f32x4_any;
typedef u32x4_t __attribute__((aligned(2))) u32x4_any;
typedef u32x2_t __attribute__((aligned(2))) u32x2_any;

// VEC consecutive elements (8, 4 or 1) of an fp32 or bf16 array as floats
template <bool BF16, int VEC>
struct Row {
    static __device__ __forceinline__ void load(const void* p, int64_t i, float* v) {
        if constexpr (BF16) {
            const uint16_t* s = (const uint16_t*)p + i;
            if constexpr (VEC == 8) {
                const u32x4_t w = *(const u32x4_any*)s;
#pragma unroll
                for (int e = 0; e < 4; ++e) { v[2 * e] = up16(w[e]); v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u); }
            } else if constexpr (VEC == 4) {
                const u32x2_t w = *(const u32x2_any*)s;
#pragma unroll
                for (int e = 0; e < 2; ++e) { v[2 * e] = up16(w[e]); v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u); }
            } else {
                v[0] = up16(*s);
            }
        } else {
            const float* s = (const float*)p + i;
            if constexpr (VEC == 1) {
                v[0] = *s;
            } else {
#pragma unroll
                for (int q = 0; q < VEC / 4; ++q) {
                    const f32x4_t w = *(const f32x4_any*)(s + 4 * q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * q + e] = w[e];
                }
            }
        }
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float* v) {
        if constexpr (BF16) {
            uint16_t* s = (uint16_t*)p + i;
            if constexpr (VEC == 8) {
                u32x4_t w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = down16(v[2 * e]) | (down16(v[2 * e + 1]) << 16);
                *(u32x4_any*)s = w;
            } else if constexpr (VEC == 4) {
                u32x2_t w;
#pragma unroll
                for (int e = 0; e < 2; ++e) w[e] = down16(v[2 * e]) | (down16(v[2 * e + 1]) << 16);
                *(u32x2_any*)s = w;
            } else {
                *s = (uint16_t)down16(v[0]);
            }
        } else {
            float* s = (float*)p + i;
            if constexpr (VEC == 1) {
                *s = v[0];
            } else {
#pragma unroll
                for (int q = 0; q < VEC / 4; ++q)
                    *(f32x4_any*)(s + 4 * q) = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            }
        }
    }
};

__device__ __forceinline__ int64_t load_id(const void* ids, int64_t i, int ids64) {
    return ids64 ? ((const int64_t*)ids)[i] : (int64_t)((const int32_t*)ids)[i];
}

// ---------------------------------------------------------------------------
// Lookup.  A team of tx threads (a power of two) covers the columns of a row in steps of
// tx * VEC; 256 / tx rows per workgroup and pass.  Rows may start at any element and end inside a vector, whose elements
// then go one by one (20000 fp32 rows of 1250: 50 us all one by one, 25 this way; 50000 bf16 rows of 333: 41 and 19).
// ---------------------------------------------------------------------------
template <bool W16, bool O16, int VEC>
__global__ __launch_bounds__(256) void lookup_kernel(EmbedArgs a, int tx_log2) {
    const int tx = threadIdx.x & ((1 << tx_log2) - 1), ty = threadIdx.x >> tx_log2;
    const int64_t t = (int64_t)blockIdx.x * (256 >> tx_log2) + ty;
    if (t >= a.tokens) return;
    const int64_t id = load_id(a.ids, t, a.ids64);
    const bool ok = id >= 0 && id < a.vocab;
    const int64_t src = (ok ? id : 0) * a.width, dst = t * a.width;
    const int64_t step = (int64_t)VEC << tx_log2;
    for (int64_t c = (int64_t)tx * VEC + (int64_t)blockIdx.y * step; c < a.width; c += step * gridDim.y) {
        float v[VEC];
        if (c + VEC <= a.width) {
            Row<W16, VEC>::load(a.in, src + c, v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = ok ? v[e] * a.scale : __uint_as_float(0x7fc00000u);
            Row<O16, VEC>::store(a.out, dst + c, v);
        } else {
            for (int e = 0; e < (int)(a.width - c); ++e) {
                Row<W16, 1>::load(a.in, src + c + e, v);
                v[0] = ok ? v[0] * a.scale : __uint_as_float(0x7fc00000u);
                Row<O16, 1>::store(a.out, dst + c + e, v);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Sorting
// ---------------------------------------------------------------------------
// The sort key of token i: its id, or vocab (sorted behind every row) where the token leaves no gradient.
__device__ __forceinline__ uint32_t token_key(const EmbedArgs& a, int64_t i) {
    const int64_t id = load_id(a.ids, i, a.ids64);
    return (uint32_t)(id >= 0 && id < a.vocab && id != a.padding_id ? id : a.vocab);
}

// Position of this lane's key among the keys of equal digit met so far by its wave, which are
// counted in cnt[]: all lanes of a digit read its count, then the first of them raises it.
// The wave's LDS accesses stay in order (volatile).
__device__ __forceinline__ uint32_t wave_rank(uint32_t digit, volatile uint32_t* cnt) {
    uint64_t same = ~0ull;
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
        const bool bit = (digit >> b) & 1;
        const uint64_t bal = __ballot(bit);
        same &= bit ? bal : ~bal;
    }
    const uint64_t below = same & ((1ull << (threadIdx.x & 63)) - 1);
    const uint32_t rank = (uint32_t)__popcll(below), seen = cnt[digit];
    if (rank == 0) cnt[digit] = seen + (uint32_t)__popcll(same);
    return seen + rank;
}

// Zeros over the table by workgroups first..gridDim.x - 1 (base 16-byte aligned).
__device__ void zero_fill(void* p, int64_t bytes, int first) {
    const int64_t n16 = bytes / 16, stride = (int64_t)(gridDim.x - first) * blockDim.x;
    const int64_t i0 = (int64_t)(blockIdx.x - first) * blockDim.x + threadIdx.x;
    for (int64_t i = i0; i < n16; i += stride) ((u32x4_t*)p)[i] = u32x4_t{0, 0, 0, 0};
    for (int64_t i = 16 * n16 / 2 + i0; i < bytes / 2; i += stride) ((uint16_t*)p)[i] = 0;   // elements are 2 or 4 bytes
}

// Few tokens: a token's place is the number of tokens that sort before it, counted by comparing it with all of them.
// Each workgroup places 64 tokens, its sixteen waves each going through a sixteenth of a piece of the keys in LDS; the
// workgroups from `sorters` on clear the table meanwhile.  Keys are whole numbers below 2^24 and go as floats: a comparison
// is a subtraction clamped to [0, 1] and an addition, exact, and nothing waits for a carry bit.
__global__ __launch_bounds__(1024) void rank_kernel(EmbedArgs a, uint32_t* keys, uint32_t* idx, int sorters,
                                                    int64_t zero_bytes) {
    if ((int)blockIdx.x >= sorters) {
        zero_fill(a.out, zero_bytes, sorters);
        return;
    }
    constexpr int PIECE = 8192;
    __shared__ __attribute__((aligned(16))) float sk[PIECE];
    __shared__ float sum[16][64];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n = (int)a.tokens;
    const int t0 = blockIdx.x * 64, t = t0 + lane;
    const uint32_t key = t < n ? token_key(a, t) : 0;
    float before = 0.f;
    const float below = (float)key, upto = below + 1.f;   // key < below, key < upto
    float ahead[PIECE / 1024];   // the next piece's keys, fetched while this one is gone through
    auto fetch = [&](int p0) {
#pragma unroll
        for (int i = 0; i < PIECE / 1024; ++i) {
            const int p = p0 + i * 1024 + tid;
            ahead[i] = p < n ? (float)token_key(a, p) : 3e7f;   // behind every key
        }
    };
    fetch(0);
    for (int p0 = 0; p0 < n; p0 += PIECE) {
        const int part = ((n - p0 < PIECE ? n - p0 : PIECE) + 63) / 64 * 4;   // keys per wave, a multiple of four
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PIECE / 1024; ++i) sk[i * 1024 + tid] = ahead[i];
        __syncthreads();
        if (p0 + PIECE < n) fetch(p0 + PIECE);
        const float* mine = sk + w * part;   // keys of the tokens q0 .. q0 + part - 1
        const int q0 = p0 + w * part;
        if (q0 + part <= t0) {              // all before this workgroup's tokens: equal ids come first
#pragma unroll 4
            for (int i = 0; i < part; i += 4) {
                const f32x4_t k = *(const f32x4_t*)&mine[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) before += __builtin_amdgcn_fmed3f(upto - k[e], 0.f, 1.f);
            }
        } else if (q0 >= t0 + 64) {         // all behind them
#pragma unroll 4
            for (int i = 0; i < part; i += 4) {
                const f32x4_t k = *(const f32x4_t*)&mine[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) before += __builtin_amdgcn_fmed3f(below - k[e], 0.f, 1.f);
            }
        } else {
#pragma unroll 4
            for (int i = 0; i < part; i += 4) {
                const f32x4_t k = *(const f32x4_t*)&mine[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) before += __builtin_amdgcn_fmed3f((q0 + i + e < t ? upto : below) - k[e], 0.f, 1.f);
            }
        }
    }
    sum[w][lane] = before;
    __syncthreads();
    if (w == 0 && t < n) {
        float place = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) place += sum[i][lane];
        keys[(int)place] = key;
        idx[(int)place] = (uint32_t)t;
    }
}

// Many tokens: a stable radix sort, kDigitBits a pass, by workgroups of 256 ITEMS tokens: digit counts per
// workgroup ([digit][workgroup]), then the scatter, which adds up the counts before its own by itself (reading all of
// them from L2 took 3 us where a prefix kernel between the two took 21).  The first pass reads the ids.
template <int ITEMS>
__global__ __launch_bounds__(256) void radix_count_kernel(EmbedArgs a, int shift, const uint32_t* keys, uint32_t* counts,
                                                          int nblk, int64_t zero_bytes) {
    if ((int)blockIdx.x >= nblk) {
        zero_fill(a.out, zero_bytes, nblk);
        return;
    }
    __shared__ uint32_t h[kDigits];
    for (int i = threadIdx.x; i < kDigits; i += 256) h[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int64_t pos = ((int64_t)blockIdx.x * ITEMS + i) * 256 + threadIdx.x;
        if (pos < a.tokens) atomicAdd(&h[((keys ? keys[pos] : token_key(a, pos)) >> shift) & (kDigits - 1)], 1u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kDigits; i += 256) counts[(int64_t)i * nblk + blockIdx.x] = h[i];
}

template <int ITEMS>
__global__ __launch_bounds__(256) void radix_scatter_kernel(EmbedArgs a, int shift, const uint32_t* keys,
                                                            const uint32_t* idx, const uint32_t* counts, int nblk,
                                                            uint32_t* keys_out, uint32_t* idx_out) {
    static_assert(kDigits == 512, "two digits per thread");
    __shared__ uint32_t cnt[4 * kDigits], tmp[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int i = tid; i < 4 * kDigits; i += 256) cnt[i] = 0;
    uint32_t key[ITEMS], rk[ITEMS], tok[ITEMS];
    const int64_t p0 = (int64_t)blockIdx.x * 256 * ITEMS + w * 64 * ITEMS + lane;   // a wave's tokens in order: stable
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int64_t pos = p0 + 64 * i;
        key[i] = pos < a.tokens ? (keys ? keys[pos] : token_key(a, pos)) : 0xffffffffu;
        tok[i] = pos < a.tokens && keys ? idx[pos] : (uint32_t)pos;
    }
    // this thread's digits 2 tid and 2 tid + 1: tokens of lower workgroups, and of all
    uint32_t low[2] = {0, 0}, all[2] = {0, 0};
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const uint32_t* c = counts + (int64_t)(2 * tid + d) * nblk;
#pragma unroll 16
        for (int b = 0; b < nblk; ++b) {
            const uint32_t v = c[b];
            all[d] += v;
            low[d] += b < (int)blockIdx.x ? v : 0;
        }
    }
    const uint32_t sum = all[0] + all[1];   // exclusive prefix over the digits
    uint32_t s = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t u = __shfl_up(s, o);
        if (lane >= o) s += u;
    }
    if (lane == 63) tmp[w] = s;
    __syncthreads();
    uint32_t first = s - sum;
    for (int i = 0; i < w; ++i) first += tmp[i];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) rk[i] = wave_rank((key[i] >> shift) & (kDigits - 1), cnt + kDigits * w);
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        uint32_t run = first + (d ? all[0] : 0) + low[d];
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = cnt[kDigits * i + 2 * tid + d];
            cnt[kDigits * i + 2 * tid + d] = run;
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int64_t pos = p0 + 64 * i;
        if (pos >= a.tokens) continue;   // (past the end: the last positions of the last workgroup)
        const uint32_t to = cnt[kDigits * w + ((key[i] >> shift) & (kDigits - 1))] + rk[i];
        keys_out[to] = key[i];
        idx_out[to] = tok[i];
    }
}

template <int ITEMS>
void launch_radix(const EmbedArgs& a, int d, const uint32_t* kin, const uint32_t* iin, uint32_t* counts, int nblk,
                  uint32_t* kout, uint32_t* iout, int64_t zero, unsigned fill, hipStream_t s) {
    hipLaunchKernelGGL((radix_count_kernel<ITEMS>), dim3(nblk + fill), dim3(256), 0, s, a, kDigitBits * d, kin, counts, nblk, zero);
    hipLaunchKernelGGL((radix_scatter_kernel<ITEMS>), dim3(nblk), dim3(256), 0, s, a, kDigitBits * d, kin, iin, counts, nblk,
                       kout, iout);
}

// ---------------------------------------------------------------------------
// Sums over runs of equal ids
// ---------------------------------------------------------------------------
struct RunArgs {
    EmbedArgs e;
    const uint32_t* keys;   // sorted
    const uint32_t* idx;
    float* part;            // [nchunk][2][pitch]: head and tail partial rows of each chunk
    int64_t chunk, nchunk, pitch;
    int tx_log2;
    WeightedRows w;         // kernels with WEIGHTED
};

// A thread's columns: VEC > 1: one vector; VEC == 1: four columns tx apart.
template <int VEC>
struct Cols {
    static constexpr int W = VEC > 1 ? VEC : 4;
    int64_t c[VEC > 1 ? 1 : 4];
    int n;   // how many of them lie inside the row
    __device__ __forceinline__ Cols(int tx, int tx_log2, int64_t slab, int64_t width) {
        if constexpr (VEC > 1) {
            c[0] = (slab * (1 << tx_log2) + tx) * VEC;
            n = c[0] < width;
        } else {
            n = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[j] = ((slab * 4 + j) << tx_log2) + tx;
                n += c[j] < width;
            }
        }
    }
    template <bool BF16>
    __device__ __forceinline__ void load(const void* p, int64_t row, float* v) const {
        if constexpr (VEC > 1) {
            Row<BF16, VEC>::load(p, row + c[0], v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = 0.f;
                if (j < n) Row<BF16, 1>::load(p, row + c[j], v + j);
            }
        }
    }
    template <bool BF16>
    __device__ __forceinline__ void store(void* p, int64_t row, const float* v) const {
        if constexpr (VEC > 1) {
            Row<BF16, VEC>::store(p, row + c[0], v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) Row<BF16, 1>::store(p, row + c[j], v + j);
        }
    }
};

template <bool O16, bool ADD, int VEC>
__device__ __forceinline__ void write_row(const RunArgs& a, const Cols<VEC>& cols, uint32_t key, const float* acc, const float* old) {
    constexpr int W = Cols<VEC>::W;
    float v[W];
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = ADD ? old[e] + a.e.scale * acc[e] : a.e.scale * acc[e];
    cols.template store<O16>(a.e.out, (int64_t)key * a.e.width, v);
}

// WEIGHTED: the sum of a run, for the row of extra that sorted position `at` of the run, or its id, names
template <int VEC>
__device__ __forceinline__ void write_extra(const RunArgs& a, const Cols<VEC>& cols, uint32_t key, int64_t at, const float* acc) {
    if (key < a.w.lo || key >= a.w.hi) return;
    const int64_t row = a.w.by_row ? key - a.w.lo : at;
    cols.template store<false>(a.w.extra, row * a.w.pitch, acc);
    if (cols.c[0] == 0) a.w.slot[key] = (int)row + 1;
}

// Whether the run of `key` is one to sum: WEIGHTED kernels take the tokens a range of ids at a time.
template <bool WEIGHTED>
__device__ __forceinline__ bool outside(const RunArgs& a, uint32_t first, uint32_t last) {
    return WEIGHTED && (last < a.w.lo || first >= a.w.hi);
}

// ADD: the rows to add to are fetched with the tokens' rows whose runs end there, not when they are written: most runs
// are of one token, and each would wait for its own row.
template <bool Y16, bool O16, bool ADD, int VEC, bool WEIGHTED>
__global__ __launch_bounds__(256) void run_sum_kernel(RunArgs a) {
    constexpr int W = Cols<VEC>::W, U = ADD ? 4 : 8;
    const int tx = threadIdx.x & ((1 << a.tx_log2) - 1), ty = threadIdx.x >> a.tx_log2;
    const int64_t ch = (int64_t)blockIdx.x * (256 >> a.tx_log2) + ty;
    const Cols<VEC> cols(tx, a.tx_log2, blockIdx.y, a.e.width);
    if (ch >= a.nchunk || cols.n == 0) return;
    const int64_t n = a.e.tokens, p0 = ch * a.chunk, p1 = p0 + a.chunk < n ? p0 + a.chunk : n;
    const uint32_t none = (uint32_t)a.e.vocab;
    uint32_t key = a.keys[p0];
    if (outside<WEIGHTED>(a, key, a.keys[p1 - 1])) return;
    bool open = p0 > 0 && a.keys[p0 - 1] == key;   // the run began before this chunk
    float acc[W];
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = 0.f;
    for (int64_t p = p0; p < p1 && key != none; p += U) {
        uint32_t next[U], tok[U];
        float v[U][W], old[ADD ? U : 1][W], weight[WEIGHTED ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t q = p + u < p1 ? p + u : p1 - 1;
            tok[u] = a.idx[q];
            next[u] = q + 1 < n ? a.keys[q + 1] : none;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            cols.template load<Y16>(a.e.in, (int64_t)tok[u] * a.e.width, v[u]);
            if (WEIGHTED) weight[u] = a.w.weight[a.w.pos[tok[u]]];
            if (ADD) {
                const uint32_t here = u ? next[u - 1] : key;
                if (here != none && next[u] != here) cols.template load<O16>(a.e.out, (int64_t)here * a.e.width, old[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p + u >= p1 || key == none) break;
#pragma unroll
            for (int e = 0; e < W; ++e) acc[e] = WEIGHTED ? fmaf(weight[WEIGHTED ? u : 0], v[u][e], acc[e]) : acc[e] + v[u][e];
            if (next[u] != key) {
                if (open) cols.template store<false>(a.part, ch * 2 * a.pitch, acc);
                else if constexpr (WEIGHTED) write_extra(a, cols, key, p + u, acc);
                else write_row<O16, ADD, VEC>(a, cols, key, acc, old[ADD ? u : 0]);
                open = false;
#pragma unroll
                for (int e = 0; e < W; ++e) acc[e] = 0.f;
                key = next[u];
            } else if (p + u == p1 - 1) {   // the run goes on in the next chunk
                cols.template store<false>(a.part, (ch * 2 + (open ? 0 : 1)) * a.pitch, acc);
            }
        }
    }
}

// Adds up the runs that begin in a chunk and go on behind it: its tail partial row, then the head
// partial rows of the chunks that the run reaches.  Eight teams of 32 threads share 32 accesses of the row's columns,
// each adding every eighth chunk; their sums are added in order.
template <bool O16, bool ADD, int VEC, bool WEIGHTED>
__global__ __launch_bounds__(256) void run_join_kernel(RunArgs a) {
    constexpr int W = Cols<VEC>::W, U = 4;
    const int tx = threadIdx.x & 31, team = threadIdx.x >> 5;
    const int64_t ch = blockIdx.x, p0 = ch * a.chunk, p1 = p0 + a.chunk;
    const uint32_t key = a.keys[p1];
    if (key == (uint32_t)a.e.vocab || a.keys[p1 - 1] != key || (p0 > 0 && a.keys[p0 - 1] == key)) return;
    if (outside<WEIGHTED>(a, key, key)) return;
    const Cols<VEC> cols(tx, 5, blockIdx.y, a.e.width);
    __shared__ float sums[8][32][W + 1];
    float acc[W], old[W];
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = 0.f;
    if (cols.n > 0) {
        if (team == 0) {
            cols.template load<false>(a.part, (ch * 2 + 1) * a.pitch, acc);
            if (ADD) cols.template load<O16>(a.e.out, (int64_t)key * a.e.width, old);
        }
        for (int64_t c = ch + 1 + team;; c += 8 * U) {   // this team's chunks that start with the id
            float v[U][W];
            bool goes[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = c + 8 * u < a.nchunk ? c + 8 * u : a.nchunk - 1;
                goes[u] = c + 8 * u < a.nchunk && a.keys[at * a.chunk] == key;
                if (goes[u]) cols.template load<false>(a.part, at * 2 * a.pitch, v[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (goes[u]) {
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[e] += v[u][e];
                }
            if (!goes[U - 1]) break;
        }
    }
#pragma unroll
    for (int e = 0; e < W; ++e) sums[team][tx][e] = acc[e];
    __syncthreads();
    if (team > 0 || cols.n == 0) return;
#pragma unroll
    for (int i = 1; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < W; ++e) acc[e] += sums[i][tx][e];
    if constexpr (WEIGHTED) write_extra(a, cols, key, p1 - 1, acc);
    else write_row<O16, ADD, VEC>(a, cols, key, acc, old);
}

// Elements per access of the gradient: eight where rows start at 16 bytes for bf16 and 32 for fp32, four, or single ones.
int row_vec(int64_t width) { return width % 8 == 0 ? 8 : width % 4 == 0 ? 4 : 1; }

// log2 of the threads that share a row of `chunks` accesses: enough for the row, at most 256
int team_log2(int64_t chunks) {
    int l = 0;
    while (l < 8 && ((int64_t)1 << l) < chunks) ++l;
    return l;
}

template <bool W16, bool O16, int VEC>
void launch_lookup(const EmbedArgs& a, hipStream_t s) {
    const int64_t chunks = ceil_div64(a.width, VEC);
    const int l = team_log2(chunks);
    const int64_t steps = ceil_div64(chunks, (int64_t)1 << l);
    const dim3 grid((unsigned)ceil_div64(a.tokens, 256 >> l), (unsigned)steps);
    hipLaunchKernelGGL((lookup_kernel<W16, O16, VEC>), grid, dim3(256), 0, s, a, l);
}

// Eight elements per access; four where an fp32 row fits a workgroup that way (fp32, 20000 rows of 1024: 21 us by eights, 20
// by fours; of 1250: 25 and 28).
template <bool W16, bool O16>
void launch_lookup(const EmbedArgs& a, hipStream_t s) {
    if (!(W16 && O16) && a.width <= 1024) launch_lookup<W16, O16, W16 && O16 ? 8 : 4>(a, s);
    else launch_lookup<W16, O16, 8>(a, s);
}

template <bool Y16, bool O16, bool ADD, int VEC, bool WEIGHTED>
void launch_runs(RunArgs r, hipStream_t s) {
    const int64_t chunks = ceil_div64(r.e.width, Cols<VEC>::W);
    r.tx_log2 = team_log2(chunks);
    const dim3 grid((unsigned)ceil_div64(r.nchunk, 256 >> r.tx_log2),
                    (unsigned)ceil_div64(chunks, (int64_t)1 << r.tx_log2));
    hipLaunchKernelGGL((run_sum_kernel<Y16, O16, ADD, VEC, WEIGHTED>), grid, dim3(256), 0, s, r);
    if (r.nchunk > 1)
        hipLaunchKernelGGL((run_join_kernel<O16, ADD, VEC, WEIGHTED>), dim3((unsigned)(r.nchunk - 1), (unsigned)ceil_div64(chunks, 32)),
                           dim3(256), 0, s, r);
}

template <bool Y16, bool O16, bool ADD, bool WEIGHTED = false>
void launch_runs(const RunArgs& r, hipStream_t s) {
    switch (row_vec(r.e.width)) {
        case 8: launch_runs<Y16, O16, ADD, 8, WEIGHTED>(r, s); break;
        case 4: launch_runs<Y16, O16, ADD, 4, WEIGHTED>(r, s); break;
        default: launch_runs<Y16, O16, ADD, 1, WEIGHTED>(r, s); break;
    }
}

template <bool Y16, bool O16>
void launch_runs(const RunArgs& r, hipStream_t s) {
    if (r.e.accumulate) launch_runs<Y16, O16, true>(r, s);
    else launch_runs<Y16, O16, false>(r, s);
}

// Which of the two buffers the sorted tokens end in.
int sorted_buffer(const EmbedGradPlan& p) { return p.sort_blocks == 0 ? 0 : (p.digits - 1) & 1; }

// Sorts the tokens into the buffers sorted_buffer() names, and clears `zero` bytes at a.out meanwhile.
void sort_tokens(const EmbedArgs& a, const EmbedGradPlan& p, int64_t zero, char* ws, hipStream_t s) {
    const int64_t want = ceil_div64(zero, 1024 * 16 * 4);   // four 16-byte stores per thread
    const unsigned fill = (unsigned)(want < 2048 ? want : 2048);
    uint32_t* keys[2] = {(uint32_t*)(ws + p.keys[0]), (uint32_t*)(ws + p.keys[1])};
    uint32_t* idx[2] = {(uint32_t*)(ws + p.idx[0]), (uint32_t*)(ws + p.idx[1])};
    if (p.sort_blocks == 0) {
        const unsigned sorters = (unsigned)ceil_div64(a.tokens, 64);
        if (sorters + fill > 0)
            hipLaunchKernelGGL(rank_kernel, dim3(sorters + fill), dim3(1024), 0, s, a, keys[0], idx[0], (int)sorters, zero);
        return;
    }
    const int nblk = (int)p.sort_blocks;
    uint32_t* counts = (uint32_t*)(ws + p.counts);
    for (int d = 0; d < p.digits; ++d) {
        const uint32_t* kin = d ? keys[(d - 1) & 1] : nullptr;
        const uint32_t* iin = d ? idx[(d - 1) & 1] : nullptr;
        const int at = d & 1;
        if (p.sort_items == 4) launch_radix<4>(a, d, kin, iin, counts, nblk, keys[at], idx[at], d ? 0 : zero, d ? 0 : 4 * fill, s);
        else launch_radix<16>(a, d, kin, iin, counts, nblk, keys[at], idx[at], d ? 0 : zero, d ? 0 : 4 * fill, s);
    }
}

RunArgs run_args(const EmbedArgs& a, const EmbedGradPlan& p, char* ws) {
    const int at = sorted_buffer(p);
    return RunArgs{a, (uint32_t*)(ws + p.keys[at]), (uint32_t*)(ws + p.idx[at]), (float*)(ws + p.part), p.chunk, p.nchunk,
                   (a.width + 7) / 8 * 8, 0, {}};
}

}  // namespace

int run_embedding(const EmbedArgs& a, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    if (a.in_bf16) a.out_bf16 ? launch_lookup<true, true>(a, s) : launch_lookup<true, false>(a, s);
    else a.out_bf16 ? launch_lookup<false, true>(a, s) : launch_lookup<false, false>(a, s);
    return (int)hipGetLastError();
}

int run_embedding_grad(const EmbedArgs& a, const EmbedGradPlan& p, char* ws, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    sort_tokens(a, p, a.accumulate ? 0 : a.vocab * a.width * (a.out_bf16 ? 2 : 4), ws, s);
    if (a.tokens > 0) {
        const RunArgs r = run_args(a, p, ws);
        if (a.in_bf16) a.out_bf16 ? launch_runs<true, true>(r, s) : launch_runs<true, false>(r, s);
        else a.out_bf16 ? launch_runs<false, true>(r, s) : launch_runs<false, false>(r, s);
    }
    return (int)hipGetLastError();
}

int sort_weighted_rows(const EmbedArgs& a, const EmbedGradPlan& p, int* slot, char* ws, void* stream) {
    EmbedArgs clear = a;
    clear.out = slot;
    sort_tokens(clear, p, a.vocab * 4, ws, (hipStream_t)stream);
    return (int)hipGetLastError();
}

int sum_weighted_rows(const EmbedArgs& a, const EmbedGradPlan& p, const WeightedRows& w, char* ws, void* stream) {
    RunArgs r = run_args(a, p, ws);
    r.w = w;
    launch_runs<true, false, false, true>(r, (hipStream_t)stream);
    return (int)hipGetLastError();
}

}  // namespace dion
