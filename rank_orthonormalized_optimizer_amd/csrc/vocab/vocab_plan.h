// Host-side sizes and launch entry points of the vocabulary operators (arguments validated in
// vocab_api.cpp).  Every run_* returns a hipError_t value.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace dion {

constexpr int64_t kVocabMax = ((int64_t)1 << 24) - 1, kWidthMax = (int64_t)1 << 16;

inline int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Workgroups for a pass that strides over its items where `blocks` are more: HIP takes fewer than 2^32 threads per grid
// dimension, which a pass over tokens x width of the largest sizes would reach.
inline int64_t stride_blocks(int64_t blocks) { return blocks < 65536 ? blocks : 65536; }
inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }

struct EmbedArgs {
    const void* ids;
    const void* in;      // W or dY
    void* out;           // Y or dW
    int64_t tokens, vocab, width;
    float scale;
    int64_t padding_id;
    int ids64, in_bf16, out_bf16, accumulate;
};
int run_embedding(const EmbedArgs& a, void* stream);

// Layout of the table gradient's workspace: two (key, token) buffers, the radix counters, and the
// fp32 partial rows of runs that cross chunk borders.
struct EmbedGradPlan {
    int64_t chunk;            // sorted tokens per chunk
    int64_t nchunk;
    int64_t sort_blocks;      // 0: the tokens are sorted by counting
    int sort_items;           // radix sort: tokens per thread (256 threads a workgroup)
    int digits;               // radix passes
    size_t keys[2], idx[2], counts, part, total;
};

// Up to so many tokens are sorted by counting (rank_kernel, every key against every other), more by radix (table gradient of
// 32000 x 2048 bf16 by counting and by radix: 8192 tokens 35 and 52 us, 16384 52 and 58, 32768 99 and 80; 16384 tokens added
// to 65536 x 256 41 and 39)
constexpr int kRankMax = 16384;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;   // two passes up to a vocabulary of 2^18 - 1

inline bool make_embed_grad_plan(int64_t tokens, int64_t vocab, int64_t width, EmbedGradPlan* p) {
    EmbedGradPlan q{};
    // At most 512 chunks of at least 16 tokens: with wide rows short enough to fill the chip (a workgroup takes a chunk where
    // a row has 2048 bf16 elements or more) and long enough that the partial rows at the chunk borders stay a fraction of the
    // rows read.  Against 256, 1024 and 2048 chunks: 16384 tokens x 2048 bf16 52 us and 57, 54, 54; 65536 x 4096 added to
    // fp32 286 and 357, 308, 291.  Narrow rows, many chunks to a workgroup, would gain from more: 65536 x 1024 82 and 119, 71, 73;
    // 65536 x 255 fp32 88 and 138, 64, 59; 65536 x 64 bf16 71 and 111, 53, 47.
    q.chunk = 16;
    while (q.chunk * 512 < tokens) q.chunk *= 2;
    q.nchunk = ceil_div64(tokens, q.chunk);
    q.sort_items = tokens <= 1 << 17 ? 4 : 16;   // at most 256 workgroups, whose counts every one of them reads
    q.sort_blocks = tokens <= kRankMax ? 0 : ceil_div64(tokens, 256 * q.sort_items);
    q.digits = 1;
    while (q.digits < 4 && (vocab >> (kDigitBits * q.digits)) != 0) ++q.digits;   // keys 0..vocab
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t at = off; off += align256(bytes); return at; };
    for (int i = 0; i < 2; ++i) {
        q.keys[i] = take((size_t)tokens * 4);
        q.idx[i] = take((size_t)tokens * 4);
    }
    q.counts = take((size_t)q.sort_blocks * kDigits * 4);
    q.part = take((size_t)q.nchunk * 2 * (size_t)((width + 7) / 8 * 8) * 4);
    q.total = off;
    *p = q;
    return true;
}
int run_embedding_grad(const EmbedArgs& a, const EmbedGradPlan& p, char* ws, void* stream);

// Sums of a few weighted rows per id, for the output of another kernel to add: extra[slot[v] - 1] = the sum over ids[t] = v of
// weight[pos[t]] in[t], for the rows v in [lo, hi) that some token has; slot is 0 elsewhere.  A row of extra belongs to a row
// of [lo, hi) (by_row), or to a sorted token.
struct WeightedRows {
    const float* weight;
    const int* pos;
    int* slot;           // [vocab]
    float* extra;        // [rows][pitch]
    int64_t pitch;
    int64_t lo, hi;
    int by_row;
};
// sorts the tokens by id (a.in unused) and clears slot; then any number of ranges
int sort_weighted_rows(const EmbedArgs& a, const EmbedGradPlan& p, int* slot, char* ws, void* stream);
int sum_weighted_rows(const EmbedArgs& a, const EmbedGradPlan& p, const WeightedRows& w, char* ws, void* stream);

// Layout of a cross entropy call.  parts: bf16 parts of an operand (1 for bf16, 3 for fp32, whose logits take two fp16 parts);
// dparts: parts of D (1 or 2 for bf16 alone, see kTwoParts; 3).  The vocabulary goes in `pieces` of `piece` rows (a multiple of
// 256).
struct XentPlan {
    int64_t n, v, d, kp, dp;  // tokens, vocab, width, width rounded up to 64 and to 4
    int64_t np;               // tokens rounded up to 256
    int parts, dparts;
    bool few;                 // fp32 and few tokens: the products over W read it in place
    bool wpack;               // W goes through packed planes (fp32, or a width that is no multiple of 64)
    int64_t piece, pieces;
    int64_t nvt;              // softmax partials per token (forward)
    int tile_z, tile_h, tile_w;   // tile shapes of the logits, dH and dW (TILE_*)
    bool exact_targets;       // dW gets what the one part of D leaves of each target's element, by rows summed beside the product
    bool extra_by_row;        // those sums: one row per row of the piece, or per token, whichever are fewer
    EmbedGradPlan sorted;     // the tokens by target
    int64_t split_z, split_h, split_w;   // slices of the reductions of the logits (over the width), dH (the piece), dW (the tokens)
    size_t h, h16, hinv, map, tgt, lg, cnt, part, zt, z, w, winv, wtop, gscale, dl, dl16, rest, pos, slot, extra, sort, acc_h, acc_w;
    size_t total;
};

enum { TILE_256 = 0, TILE_128 = 1, TILE_32 = 2, TILE_64 = 3 };   // 256 x 256, 128 x 128, 128 x 32 (few tokens), 64 x 64
// Elements of D per piece of the vocabulary: 512 MiB per bf16 part.  Four times as many gave -1 to +5% on 8192 tokens,
// a fifth as many +14% (fp32, 4096 x 32000 x 1024: the products over a piece no longer fill the chip).
constexpr int64_t kPieceElems = (int64_t)1 << 28;
// but for many tokens as many as give the piece kPieceRows rows, up to kPieceMost: each piece adds to dH, a pass over
// tokens x width in fp32 (131072 tokens x 32000 x 2048, bf16, with gradients: pieces of 2048 rows 60.9 ms, 4096 55.8, 8192
// 53.0, 16384 53.7; fp32, 65536 tokens: 4096 rows 102.0 ms, 8192 95.9)
constexpr int64_t kPieceRows = 8192, kPieceMost = (int64_t)1 << 30;
// of W's planes per piece, a bound of the workspace alone: 512 MiB, this and 8 GiB are within 1% (fp32 loss 1024 x 131072 x 4096
// 3.33, 3.29 and 3.30 ms, with gradients 4096 x 65536 x 4096 25.7, 25.7 and 25.8; bf16 loss 2048 x 131072 x 1000 534, 535 and 531 us)
constexpr int64_t kPlaneBytes = (int64_t)2048 << 20;
constexpr int kCUs = 256;
constexpr int kCountBlock = 4096;          // tokens per count of gathered rows,
// which up to so many tokens do without, each workgroup of the gathering counting from the first token (with counts and without,
// bf16 loss over 1000 x 128: 8192 tokens 26.6 and 24.6 us, 16384 32.8 and 35.4, 32768 54 and 73, 65536 94 and 185)
constexpr int64_t kCountDirect = 16384;
// dW of so few tokens is a stream of writes: three workgroups per CU with tiles of 128 x 64 (128 x 128 and two: 22 tokens x
// 111040 x 1024 bf16 with gradients 297 us instead of 275, 64 x 64 and four 272, but fp32 4 x 115186 x 636 441 us, not 414)
constexpr int64_t kShortTokens = 128;
// and of so few, with fp32 sums in the vector units (with gradients, matrix cores against that: fp32 2 x 82297 x 2232 949 and
// 780 us, 8 x 32000 x 2048 316 and 267; bf16 9 x 40448 x 1024 113 and 107; 17 and more tokens 5 to 24% slower that way)
constexpr int64_t kRankTokens = 16;
// bf16 gradients: up to so many tokens x vocab x width dW is made of two parts of D, beyond of one and the exact sums for the
// targets' elements, three launches beside a second product (two parts and sums: 257 x 1013 x 255 32 and 51 us, 22 x 111040 x
// 1024 240 and 254, 300 x 32000 x 1024 167 and 176; 4096 x 8192 x 512 210 and 193, 1024 x 32000 x 768 280 and 239, 128 x 131072
// x 4096 1410 and 1259)
constexpr double kTwoParts = 1.25e10;
// fp32: up to so many tokens the products over W read it in place (see FewProduct).  With gradients, against planes of W in
// the workspace: 32000 x 1024, 65 tokens 232 us and 404, 128 tokens 330 and 446, 180 tokens 423 and 432; 100544 x 2624, 164
// tokens 3.2 ms and 2.9.
constexpr int64_t kFewTokens = 128;

inline int64_t tile_m(int t) { return t == TILE_256 ? 256 : t == TILE_64 ? 64 : 128; }
inline int64_t tile_n(int t) { return t == TILE_256 ? 256 : t == TILE_128 ? 128 : t == TILE_64 ? 64 : 32; }
inline int64_t tiles(int64_t m, int64_t n, int t) { return ceil_div64(m, tile_m(t)) * ceil_div64(n, tile_n(t)); }
// Slices of a reduction of length k (`terms` part products of it) so that an output of m x n fills the chip, each of
// 24 slabs of 64 at least (8 for the small tiles, whose slabs are shorter): a slice costs a pass over the output.  Against
// half and twice as many: fp32 with gradients 257 x 1013 x 255 66 us and 69, 71, 300 x 5000 x 1024 191 and 200, 197; bf16 1024 x
// 8192 x 1024 170 and 176, 189; fp32 loss 1198 x 1640 x 3923 95 and 95, 145; bf16 loss 64 x 8192 x 2048 23 and 29, 23.
inline int64_t pick_split(int64_t m, int64_t n, int64_t k, int64_t terms, int tile) {
    int64_t s = kCUs / tiles(m, n, tile);
    const int64_t most = ceil_div64(k, 64) * terms / (tile == TILE_32 || tile == TILE_64 ? 8 : 24);
    if (s > most) s = most;
    if (s > ceil_div64(k, 64)) s = ceil_div64(k, 64);
    return s < 1 ? 1 : s;
}
// The largest tile, which reads each operand least often, that still gives half the CUs a workgroup, if the
// reduction is long enough by slices of it.  Against a quarter and all of the CUs: fp32 with gradients 300 x 5000 x 1024 191 us
// and 234, 197; bf16 700 x 2048 x 2048 114 and 147, 114, 1024 x 8192 x 1024 170 and 184, 176; fp32 loss 1198 x 1640 x 3923 95 and
// 94, 139.
inline int pick_tile(int64_t m, int64_t n, int64_t k, int64_t terms) {
    if (n <= 32) return TILE_32;
    if (tiles(m, n, TILE_256) * pick_split(m, n, k, terms, TILE_256) >= kCUs / 2) return TILE_256;
    return tiles(m, n, TILE_128) * pick_split(m, n, k, terms, TILE_128) >= kCUs / 2 ? TILE_128 : TILE_64;
}
// The logits' tile where their reduction is not sliced.  Where even 128 x 128 tiles leave half the CUs idle, 64 x 64 ones
// serve, whose ring of eight slabs also hides more of the loads' latency (fp32 257 x 1013 x 255: logits 31 -> 7 us).
inline int pick_logit_tile(int64_t m, int64_t n) {
    if (n <= 32) return TILE_32;
    return tiles(m, n, TILE_256) >= kCUs / 2 ? TILE_256 : tiles(m, n, TILE_128) >= kCUs / 2 ? TILE_128 : TILE_64;
}

inline bool make_xent_plan(int64_t tokens, int64_t vocab, int64_t width, int bf16, int dw_bf16, int for_grad,
                           XentPlan* p) {
    XentPlan q{};
    q.n = tokens; q.v = vocab; q.d = width;
    q.kp = ceil_div64(width, 64) * 64;
    q.dp = ceil_div64(width, 4) * 4;
    q.np = ceil_div64(tokens < 1 ? 1 : tokens, 256) * 256;
    q.parts = bf16 ? 1 : 3;
    q.dparts = !bf16 || !dw_bf16 ? 3 : tokens <= kRankTokens || (double)tokens * vocab * width <= kTwoParts ? 2 : 1;
    q.few = !bf16 && tokens <= kFewTokens;
    q.wpack = !q.few && (!bf16 || width % 64 != 0);
    const bool scaled = !bf16 && !q.few;   // products over W from two fp16 parts of scaled rows
    const int64_t plane_row = !q.wpack ? 0 : q.kp * (bf16 ? 2 : 4);   // bytes of W's planes per row
    const int64_t all = ceil_div64(vocab, 256) * 256;
    int64_t most = all;
    if (plane_row > 0 && kPlaneBytes / plane_row < most) most = kPlaneBytes / plane_row;
    if (for_grad) {
        const int64_t fit = kPieceMost / q.np, few = fit < kPieceRows ? fit : kPieceRows;
        const int64_t rows = kPieceElems / q.np > few ? kPieceElems / q.np : few;
        if (rows < most) most = rows;
    }
    most = most < 256 ? 256 : most / 256 * 256;
    q.piece = ceil_div64(ceil_div64(all, ceil_div64(all, most)), 256) * 256;   // equal pieces
    q.pieces = ceil_div64(all, q.piece);
    q.tile_z = q.few ? TILE_32 : pick_logit_tile(q.piece, tokens);
    // Too few tiles for the chip and a long reduction: it is sliced, and a pass over the partial logits, which are few, takes
    // the epilogue's place (fp32 loss, one slice and more: 1 x 12347 x 3582 105 and 73 us, 15 x 2304 x 4032 98 and 32,
    // 1198 x 1640 x 3923 189 and 96).
    q.split_z = 1;
    const int64_t zn = q.few && tokens > 32 ? ceil_div64(tokens, 2) : tokens;   // few: 64 columns a tile
    if (q.pieces == 1 && tokens > 0 && tiles(q.piece, zn, q.few ? TILE_32 : TILE_128) < kCUs) {
        const int64_t terms = bf16 ? 1 : q.few ? 6 : 3;
        const int t = q.few ? TILE_32 : pick_tile(q.piece, zn, width, terms);
        const int64_t slabs = ceil_div64(width, 64), s = pick_split(q.piece, zn, width, terms, t);
        if (s > 1) {
            q.tile_z = t;
            q.split_z = ceil_div64(slabs, ceil_div64(slabs, s));   // none without any k
        }
    }
    q.nvt = ceil_div64(vocab, tile_m(q.tile_z));
    size_t off = 0;
    auto take = [&](int64_t bytes) { const size_t at = off; off += align256((size_t)bytes); return at; };
    q.cnt = take(256 + ceil_div64(q.np, kCountBlock) * 4);
    if (bf16 || for_grad || q.few) q.h = take(q.parts * q.np * q.kp * 2);
    if (scaled) {
        q.h16 = take(2 * q.np * q.kp * 2);
        q.hinv = take(q.np * 4);
        q.winv = take(q.piece * 4);
        q.wtop = take(4);
    }
    q.map = take(q.np * 4);
    q.tgt = take(q.np * 4);
    if (q.wpack) q.w = take(q.piece * plane_row);
    if (q.split_z > 1) q.z = take(q.split_z * tokens * q.piece * 4);
    if (!for_grad) {
        if (q.split_z == 1) {
            q.part = take(q.np * q.nvt * 8);
            q.zt = take(q.np * 4);
        }
    } else {
        const int64_t n = tokens < 1 ? 1 : tokens;
        const int64_t terms_h = bf16 ? 1 : scaled ? 3 : 6, terms_w = bf16 ? q.dparts : 6;
        q.tile_h = q.few ? TILE_32 : pick_tile(width, n, q.piece, terms_h);
        q.tile_w = n <= kShortTokens ? TILE_128 : pick_tile(width, q.piece, n, terms_w);
        // (the products of few columns take 64 at a time where there are more than 32)
        q.split_h = pick_split(width, q.few && n > 32 ? ceil_div64(n, 2) : n, q.piece, terms_h, q.tile_h);
        q.split_w = pick_split(width, q.piece, n, terms_w, q.tile_w);
        q.lg = take(q.np * 8);
        q.rest = take(q.np * 4);
        q.dl = take(q.dparts * q.np * q.piece * 2);
        if (scaled) {
            q.dl16 = take(2 * q.np * q.piece * 2);
            q.gscale = take(q.np * 4);
        }
        q.exact_targets = q.dparts == 1;
        if (q.exact_targets) {
            q.extra_by_row = q.piece <= q.np;
            make_embed_grad_plan(tokens, vocab, width, &q.sorted);
            q.pos = take(q.np * 4);
            q.slot = take(vocab * 4);
            q.extra = take((q.extra_by_row ? q.piece : q.np) * q.dp * 4);
            q.sort = take((int64_t)q.sorted.total);
        }
        if (q.pieces > 1 || q.split_h > 1) q.acc_h = take(q.split_h * q.np * q.dp * 4);
        if (q.split_w > 1) q.acc_w = take(q.split_w * q.piece * q.dp * 4);
    }
    q.total = off;
    *p = q;
    return off < ((size_t)1 << 46);
}

// Lanes that share the slices of four columns of the output, and the workgroups of 256 that join them.  Eight lanes and one, with
// gradients: fp32 1 x 100000 x 64 61 and 76 us, 64 x 131072 x 255 182 and 190; bf16 32 x 131072 x 256 87 and 96, 512 x 32000 x 2048
// (eight slices) 317 and 310.
inline int join_lanes(int64_t split) { return split >= 8 ? 8 : 1; }
inline int64_t join_blocks(int64_t rows, int64_t dp, int64_t split) {
    return stride_blocks(ceil_div64(rows * (dp / 4) * join_lanes(split), 256));
}

struct XentArgs {
    const void* H;
    const void* W;
    const void* targets;
    float* loss;         // forward
    float* lse_out;      // forward
    const float* lse;    // gradient
    const float* grad;
    int64_t grad_n;
    void* dH;
    void* dW;
    int64_t ignore;
    int t64, bf16, dw_bf16, accumulate;
};
int run_xent(const XentArgs& a, const XentPlan& p, char* ws, void* stream);
int run_xent_grad(const XentArgs& a, const XentPlan& p, char* ws, void* stream);

}  // namespace dion
