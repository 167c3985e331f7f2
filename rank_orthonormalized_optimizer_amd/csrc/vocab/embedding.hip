// Embedding lookup with a scale, and the gradient of its table by sorted tokens.
//
//   Y[t] = scale * W[ids[t]]                        one gather, bound by HBM (read and write d elements per token)
//   dW[v] (+)= scale * sum over ids[t] = v of dY[t]
//
// The gradient sorts the tokens by id (stable radix sort of (id, token) pairs, eight bits a pass)
// and cuts the sorted list into chunks of equal length, so that frequent ids load no workgroup
// more than others.  A team of threads walks one chunk, adding rows of dY in fp32 registers; a run
// of one id that lies inside the chunk is written to its row, the part of a run that crosses a
// border goes to a partial row, and a second pass adds the partial rows of a run in chunk order.
// No atomics: the order of additions depends on the tokens alone.
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

// VEC consecutive elements (8, 4 or 1) of an fp32 or bf16 array as floats; the address is
// aligned to VEC elements (16 bytes at most)
template <bool BF16, int VEC>
struct Row {
    static __device__ __forceinline__ void load(const void* p, int64_t i, float* v) {
        if constexpr (BF16) {
            const uint16_t* s = (const uint16_t*)p + i;
            if constexpr (VEC == 8) {
                const u32x4_t w = *(const u32x4_t*)s;
#pragma unroll
                for (int e = 0; e < 4; ++e) { v[2 * e] = up16(w[e]); v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u); }
            } else if constexpr (VEC == 4) {
                const u32x2_t w = *(const u32x2_t*)s;
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
                    const f32x4_t w = *(const f32x4_t*)(s + 4 * q);
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
                *(u32x4_t*)s = w;
            } else if constexpr (VEC == 4) {
                u32x2_t w;
#pragma unroll
                for (int e = 0; e < 2; ++e) w[e] = down16(v[2 * e]) | (down16(v[2 * e + 1]) << 16);
                *(u32x2_t*)s = w;
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
                    *(f32x4_t*)(s + 4 * q) = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            }
        }
    }
};

__device__ __forceinline__ int64_t load_id(const void* ids, int64_t i, int ids64) {
    return ids64 ? ((const int64_t*)ids)[i] : (int64_t)((const int32_t*)ids)[i];
}

// ---------------------------------------------------------------------------
// Lookup.  A team of tx threads (a power of two) covers the columns of a row in steps of
// tx * VEC; 256 / tx rows per workgroup and pass.
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
        Row<W16, VEC>::load(a.in, src + c, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = ok ? v[e] * a.scale : __uint_as_float(0x7fc00000u);
        Row<O16, VEC>::store(a.out, dst + c, v);
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
// counted in cnt[256]: all lanes of a digit read its count, then the first of them raises it.
// The wave's LDS accesses stay in order (volatile).
__device__ __forceinline__ uint32_t wave_rank(uint32_t digit, volatile uint32_t* cnt) {
    uint64_t same = ~0ull;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const bool bit = (digit >> b) & 1;
        const uint64_t bal = __ballot(bit);
        same &= bit ? bal : ~bal;
    }
    const uint64_t below = same & ((1ull << (threadIdx.x & 63)) - 1);
    const uint32_t rank = (uint32_t)__popcll(below), seen = cnt[digit];
    if (rank == 0) cnt[digit] = seen + (uint32_t)__popcll(same);
    return seen + rank;
}

// Exclusive prefix over 256 values, one per thread of the first four waves; every thread of the
// workgroup calls it.  tmp: four words of LDS.
__device__ __forceinline__ uint32_t scan256(uint32_t v, uint32_t* tmp) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint32_t s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t u = __shfl_up(s, o);
        if (lane >= o) s += u;
    }
    if (w < 4 && lane == 63) tmp[w] = s;
    __syncthreads();
    uint32_t base = 0;
    for (int i = 0; i < 4; ++i) base += i < w ? tmp[i] : 0;
    return base + s - v;
}

// Zeros over the table by workgroups first..gridDim.x - 1 (base 16-byte aligned).
__device__ void zero_fill(void* p, int64_t bytes, int first) {
    const int64_t n16 = bytes / 16, stride = (int64_t)(gridDim.x - first) * blockDim.x;
    const int64_t i0 = (int64_t)(blockIdx.x - first) * blockDim.x + threadIdx.x;
    for (int64_t i = i0; i < n16; i += stride) ((u32x4_t*)p)[i] = u32x4_t{0, 0, 0, 0};
    for (int64_t i = 16 * n16 / 2 + i0; i < bytes / 2; i += stride) ((uint16_t*)p)[i] = 0;   // elements are 2 or 4 bytes
}

// Workgroup 0 sorts all tokens (at most 1024 * ITEMS), the others clear the table meanwhile.
// Wave w ranks the positions [64 ITEMS w, 64 ITEMS (w + 1)) in order, which keeps the sort stable.
template <int ITEMS>
__global__ __launch_bounds__(1024) void sort1_kernel(EmbedArgs a, int digits, uint32_t* keys, uint32_t* idx,
                                                     int64_t zero_bytes) {
    if (blockIdx.x > 0) {
        zero_fill(a.out, zero_bytes, 1);
        return;
    }
    __shared__ uint32_t sk[1024 * ITEMS], si[1024 * ITEMS], cnt[16 * 256], base[256], tmp[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n = (int)a.tokens;
    uint32_t key[ITEMS], tok[ITEMS], rk[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int pos = (w * ITEMS + i) * 64 + lane;
        key[i] = pos < n ? token_key(a, pos) : 0xffffffffu;   // positions past the end stay last
        tok[i] = (uint32_t)pos;
    }
    for (int d = 0; d < digits; ++d) {
        for (int i = tid; i < 16 * 256; i += 1024) cnt[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) rk[i] = wave_rank((key[i] >> (8 * d)) & 255u, cnt + 256 * w);
        __syncthreads();
        uint32_t run = 0;
        if (tid < 256)
            for (int i = 0; i < 16; ++i) {
                const uint32_t c = cnt[256 * i + tid];
                cnt[256 * i + tid] = run;
                run += c;
            }
        const uint32_t b = scan256(run, tmp);
        if (tid < 256) base[tid] = b;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t g = (key[i] >> (8 * d)) & 255u, to = base[g] + cnt[256 * w + g] + rk[i];
            sk[to] = key[i];
            si[to] = tok[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int pos = (w * ITEMS + i) * 64 + lane;
            key[i] = sk[pos];
            tok[i] = si[pos];
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int pos = (w * ITEMS + i) * 64 + lane;
        if (pos < n) {
            keys[pos] = key[i];
            idx[pos] = tok[i];
        }
    }
}

// One radix pass over many workgroups of kSortBlock tokens: digit counts per workgroup, their
// prefix (digit-major), and the stable scatter.  The first pass reads the ids.
__global__ __launch_bounds__(256) void radix_count_kernel(EmbedArgs a, int shift, const uint32_t* keys, uint32_t* counts,
                                                          int nblk, int64_t zero_bytes) {
    if ((int)blockIdx.x >= nblk) {
        zero_fill(a.out, zero_bytes, nblk);
        return;
    }
    __shared__ uint32_t h[256];
    h[threadIdx.x] = 0;
    __syncthreads();
    for (int i = 0; i < kSortBlock / 256; ++i) {
        const int64_t pos = (int64_t)blockIdx.x * kSortBlock + i * 256 + threadIdx.x;
        if (pos < a.tokens) atomicAdd(&h[((keys ? keys[pos] : token_key(a, pos)) >> shift) & 255u], 1u);
    }
    __syncthreads();
    counts[(int64_t)threadIdx.x * nblk + blockIdx.x] = h[threadIdx.x];
}

__global__ __launch_bounds__(1024) void radix_scan_kernel(uint32_t* counts, int64_t n) {
    __shared__ uint32_t tmp[16], carry_s;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    uint32_t carry = 0;
    for (int64_t i0 = 0; i0 < n; i0 += 4096) {
        uint32_t v[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = i0 + 4 * tid + e;
            v[e] = i < n ? counts[i] : 0;
            sum += v[e];
        }
        uint32_t s = sum;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t u = __shfl_up(s, o);
            if (lane >= o) s += u;
        }
        if (lane == 63) tmp[w] = s;
        __syncthreads();
        uint32_t at = carry + s - sum;
        for (int i = 0; i < w; ++i) at += tmp[i];
        if (tid == 1023) carry_s = at + sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = i0 + 4 * tid + e;
            if (i < n) counts[i] = at;
            at += v[e];
        }
        __syncthreads();
        carry = carry_s;
    }
}

__global__ __launch_bounds__(256) void radix_scatter_kernel(EmbedArgs a, int shift, const uint32_t* keys,
                                                            const uint32_t* idx, const uint32_t* counts, int nblk,
                                                            uint32_t* keys_out, uint32_t* idx_out) {
    constexpr int ITEMS = kSortBlock / 256;
    __shared__ uint32_t cnt[4 * 256];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int i = tid; i < 4 * 256; i += 256) cnt[i] = 0;
    uint32_t key[ITEMS], rk[ITEMS];
    const int64_t p0 = (int64_t)blockIdx.x * kSortBlock + w * 64 * ITEMS + lane;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int64_t pos = p0 + 64 * i;
        key[i] = pos < a.tokens ? (keys ? keys[pos] : token_key(a, pos)) : 0xffffffffu;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) rk[i] = wave_rank((key[i] >> shift) & 255u, cnt + 256 * w);
    __syncthreads();
    uint32_t run = counts[(int64_t)tid * nblk + blockIdx.x];
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = cnt[256 * i + tid];
        cnt[256 * i + tid] = run;
        run += c;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int64_t pos = p0 + 64 * i;
        if (pos >= a.tokens) continue;   // (past the end: the last positions of the last workgroup)
        const uint32_t to = cnt[256 * w + ((key[i] >> shift) & 255u)] + rk[i];
        keys_out[to] = key[i];
        idx_out[to] = keys ? idx[pos] : (uint32_t)pos;
    }
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

template <bool O16, int VEC>
__device__ __forceinline__ void write_row(const RunArgs& a, const Cols<VEC>& cols, uint32_t key, const float* acc) {
    constexpr int W = Cols<VEC>::W;
    float v[W];
    const int64_t row = (int64_t)key * a.e.width;
    if (a.e.accumulate) {
        cols.template load<O16>(a.e.out, row, v);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] += a.e.scale * acc[e];
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = a.e.scale * acc[e];
    }
    cols.template store<O16>(a.e.out, row, v);
}

template <bool Y16, bool O16, int VEC>
__global__ __launch_bounds__(256) void run_sum_kernel(RunArgs a) {
    constexpr int W = Cols<VEC>::W, U = 8;
    const int tx = threadIdx.x & ((1 << a.tx_log2) - 1), ty = threadIdx.x >> a.tx_log2;
    const int64_t ch = (int64_t)blockIdx.x * (256 >> a.tx_log2) + ty;
    const Cols<VEC> cols(tx, a.tx_log2, blockIdx.y, a.e.width);
    if (ch >= a.nchunk || cols.n == 0) return;
    const int64_t n = a.e.tokens, p0 = ch * a.chunk, p1 = p0 + a.chunk < n ? p0 + a.chunk : n;
    const uint32_t none = (uint32_t)a.e.vocab;
    uint32_t key = a.keys[p0];
    bool open = p0 > 0 && a.keys[p0 - 1] == key;   // the run began before this chunk
    float acc[W];
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = 0.f;
    for (int64_t p = p0; p < p1 && key != none; p += U) {
        uint32_t next[U], tok[U];
        float v[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t q = p + u < p1 ? p + u : p1 - 1;
            tok[u] = a.idx[q];
            next[u] = q + 1 < n ? a.keys[q + 1] : none;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) cols.template load<Y16>(a.e.in, (int64_t)tok[u] * a.e.width, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p + u >= p1 || key == none) break;
#pragma unroll
            for (int e = 0; e < W; ++e) acc[e] += v[u][e];
            if (next[u] != key) {
                if (open) cols.template store<false>(a.part, ch * 2 * a.pitch, acc);
                else write_row<O16, VEC>(a, cols, key, acc);
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
// partial rows of the chunks that the run reaches.
template <bool O16, int VEC>
__global__ __launch_bounds__(256) void run_join_kernel(RunArgs a) {
    constexpr int W = Cols<VEC>::W, U = 8;
    const int tx = threadIdx.x & ((1 << a.tx_log2) - 1), ty = threadIdx.x >> a.tx_log2;
    const int64_t ch = (int64_t)blockIdx.x * (256 >> a.tx_log2) + ty;
    const Cols<VEC> cols(tx, a.tx_log2, blockIdx.y, a.e.width);
    if (ch + 1 >= a.nchunk || cols.n == 0) return;
    const int64_t p0 = ch * a.chunk, p1 = p0 + a.chunk;
    const uint32_t key = a.keys[p1];
    if (key == (uint32_t)a.e.vocab || a.keys[p1 - 1] != key || (p0 > 0 && a.keys[p0 - 1] == key)) return;
    int64_t lo = ch + 1, hi = a.nchunk;   // the last chunk that starts with this id
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (a.keys[mid * a.chunk] == key) lo = mid;
        else hi = mid;
    }
    float acc[W];
    cols.template load<false>(a.part, (ch * 2 + 1) * a.pitch, acc);
    for (int64_t c = ch + 1; c <= lo; c += U) {
        float v[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u) cols.template load<false>(a.part, (c + u <= lo ? c + u : lo) * 2 * a.pitch, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u <= lo) {
#pragma unroll
                for (int e = 0; e < W; ++e) acc[e] += v[u][e];
            }
    }
    write_row<O16, VEC>(a, cols, key, acc);
}

// Elements per access: eight where rows start at 16 bytes for bf16 and 32 for fp32, four, or single ones.
int row_vec(int64_t width) { return width % 8 == 0 ? 8 : width % 4 == 0 ? 4 : 1; }

// log2 of the threads that share a row of `chunks` accesses: enough for the row, at most 256
int team_log2(int64_t chunks) {
    int l = 0;
    while (l < 8 && ((int64_t)1 << l) < chunks) ++l;
    return l;
}

template <bool W16, bool O16>
void launch_lookup(const EmbedArgs& a, hipStream_t s) {
    const int vec = row_vec(a.width);
    const int64_t chunks = ceil_div64(a.width, vec);
    const int l = team_log2(chunks);
    const int64_t steps = ceil_div64(chunks, (int64_t)1 << l);
    const dim3 grid((unsigned)ceil_div64(a.tokens, 256 >> l), (unsigned)steps);
    if (vec == 8) hipLaunchKernelGGL((lookup_kernel<W16, O16, 8>), grid, dim3(256), 0, s, a, l);
    else if (vec == 4) hipLaunchKernelGGL((lookup_kernel<W16, O16, 4>), grid, dim3(256), 0, s, a, l);
    else hipLaunchKernelGGL((lookup_kernel<W16, O16, 1>), grid, dim3(256), 0, s, a, l);
}

template <bool Y16, bool O16, int VEC>
void launch_runs(RunArgs r, hipStream_t s) {
    const int64_t chunks = ceil_div64(r.e.width, Cols<VEC>::W);
    r.tx_log2 = team_log2(chunks);
    const dim3 grid((unsigned)ceil_div64(r.nchunk, 256 >> r.tx_log2),
                    (unsigned)ceil_div64(chunks, (int64_t)1 << r.tx_log2));
    hipLaunchKernelGGL((run_sum_kernel<Y16, O16, VEC>), grid, dim3(256), 0, s, r);
    if (r.nchunk > 1) hipLaunchKernelGGL((run_join_kernel<O16, VEC>), grid, dim3(256), 0, s, r);
}

template <bool Y16, bool O16>
void launch_runs(const RunArgs& r, hipStream_t s) {
    switch (row_vec(r.e.width)) {
        case 8: launch_runs<Y16, O16, 8>(r, s); break;
        case 4: launch_runs<Y16, O16, 4>(r, s); break;
        default: launch_runs<Y16, O16, 1>(r, s); break;
    }
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
    const int64_t zero = a.accumulate ? 0 : a.vocab * a.width * (a.out_bf16 ? 2 : 4);
    const int64_t want = ceil_div64(zero, 1024 * 16 * 4);   // four 16-byte stores per thread
    const unsigned fill = (unsigned)(want < 2048 ? want : 2048);
    uint32_t* keys[2] = {(uint32_t*)(ws + p.keys[0]), (uint32_t*)(ws + p.keys[1])};
    uint32_t* idx[2] = {(uint32_t*)(ws + p.idx[0]), (uint32_t*)(ws + p.idx[1])};
    int at = 0;
    if (p.sort_blocks == 0) {
        const dim3 grid(1 + fill), block(1024);
        if (a.tokens <= 1024) hipLaunchKernelGGL((sort1_kernel<1>), grid, block, 0, s, a, p.digits, keys[0], idx[0], zero);
        else if (a.tokens <= 4096) hipLaunchKernelGGL((sort1_kernel<4>), grid, block, 0, s, a, p.digits, keys[0], idx[0], zero);
        else hipLaunchKernelGGL((sort1_kernel<kSort1Items>), grid, block, 0, s, a, p.digits, keys[0], idx[0], zero);
    } else {
        const int nblk = (int)p.sort_blocks;
        uint32_t* counts = (uint32_t*)(ws + p.counts);
        for (int d = 0; d < p.digits; ++d) {
            const uint32_t* kin = d ? keys[(d - 1) & 1] : nullptr;
            const uint32_t* iin = d ? idx[(d - 1) & 1] : nullptr;
            at = d & 1;
            hipLaunchKernelGGL(radix_count_kernel, dim3(nblk + (d ? 0 : 4 * fill)), dim3(256), 0, s, a, 8 * d, kin, counts,
                               nblk, d ? 0 : zero);
            hipLaunchKernelGGL(radix_scan_kernel, dim3(1), dim3(1024), 0, s, counts, (int64_t)256 * nblk);
            hipLaunchKernelGGL(radix_scatter_kernel, dim3(nblk), dim3(256), 0, s, a, 8 * d, kin, iin, counts, nblk,
                               keys[at], idx[at]);
        }
    }
    if (a.tokens > 0) {
        const RunArgs r{a, keys[at], idx[at], (float*)(ws + p.part), p.chunk, p.nchunk, (a.width + 7) / 8 * 8, 0};
        if (a.in_bf16) a.out_bf16 ? launch_runs<true, true>(r, s) : launch_runs<true, false>(r, s);
        else a.out_bf16 ? launch_runs<false, true>(r, s) : launch_runs<false, false>(r, s);
    }
    return (int)hipGetLastError();
}

}  // namespace dion
