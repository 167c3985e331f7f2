// extern "C" entry points of the vocabulary operators: argument validation (pure host code, no
// HIP call before every check has passed) and workspace sizes.
#include <math.h>
#include <stdint.h>

#include "dion_vocab.h"
#include "vocab_plan.h"

namespace {

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

bool overlap(const Range& a, const Range& b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

// sizes are bounded by check_sizes, so the byte counts are exact in 64 bits
Range span(const void* p, int64_t count, int64_t bytes) {
    const uintptr_t lo = (uintptr_t)p;
    return Range{lo, lo + (uintptr_t)(p ? count * bytes : 0)};
}

bool check_sizes(int64_t tokens, int64_t vocab, int64_t width) {
    return tokens >= 0 && tokens <= DION_VOCAB_MAX_TOKENS && vocab >= 1 && vocab <= dion::kVocabMax && width >= 1 &&
           width <= dion::kWidthMax;
}

bool is_dtype(int t) { return t == DION_F32 || t == DION_BF16; }
bool is_index(int t) { return t == DION_I32 || t == DION_I64; }
int64_t size_of(int t) { return t == DION_BF16 ? 2 : 4; }
int64_t size_of_index(int t) { return t == DION_I64 ? 8 : 4; }
bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// the first `written` ranges must overlap nothing else
bool any_overlap(const Range* r, int written, int n) {
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(r[i], r[j])) return true;
    return false;
}

}  // namespace

extern "C" {

int dion_embedding(const void* ids, const void* W, void* out, int64_t tokens, int64_t vocab, int64_t width,
                   float scale, int id_dtype, int w_dtype, int out_dtype, void* stream) {
    if (!check_sizes(tokens, vocab, width)) return DION_ERR_SHAPE;
    if (!isfinite(scale)) return DION_ERR_HYPER;
    if (!is_index(id_dtype) || !is_dtype(w_dtype) || !is_dtype(out_dtype)) return DION_ERR_DTYPE;
    if (tokens == 0) return DION_OK;
    if (!ids || !W || !out) return DION_ERR_NULL;
    if (misaligned(ids, size_of_index(id_dtype)) || misaligned(W, 16) || misaligned(out, 16)) return DION_ERR_ALIGN;
    const Range rs[3] = {span(out, tokens * width, size_of(out_dtype)), span(ids, tokens, size_of_index(id_dtype)),
                         span(W, vocab * width, size_of(w_dtype))};
    if (any_overlap(rs, 1, 3)) return DION_ERR_OVERLAP;
    const dion::EmbedArgs a{ids, W, out, tokens, vocab, width, scale, -1, id_dtype == DION_I64, w_dtype == DION_BF16,
                            out_dtype == DION_BF16, 0};
    const int e = dion::run_embedding(a, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

size_t dion_embedding_grad_workspace_size(int64_t tokens, int64_t vocab, int64_t width) {
    dion::EmbedGradPlan p;
    if (!check_sizes(tokens, vocab, width) || !dion::make_embed_grad_plan(tokens, vocab, width, &p)) return 0;
    return p.total;
}

int dion_embedding_grad(const void* ids, const void* dY, void* dW, int64_t tokens, int64_t vocab, int64_t width,
                        float scale, int64_t padding_id, int id_dtype, int y_dtype, int w_dtype, int accumulate,
                        void* workspace, size_t workspace_bytes, void* stream) {
    if (!check_sizes(tokens, vocab, width)) return DION_ERR_SHAPE;
    if (!isfinite(scale)) return DION_ERR_HYPER;
    if (!is_index(id_dtype) || !is_dtype(y_dtype) || !is_dtype(w_dtype)) return DION_ERR_DTYPE;
    if (accumulate != 0 && accumulate != 1) return DION_ERR_OPTION;
    dion::EmbedGradPlan p;
    if (!dion::make_embed_grad_plan(tokens, vocab, width, &p)) return DION_ERR_SHAPE;
    if (tokens == 0 && accumulate) return DION_OK;
    if (!dW || (tokens > 0 && (!ids || !dY || !workspace))) return DION_ERR_NULL;
    if (misaligned(ids, size_of_index(id_dtype)) || misaligned(dY, 16) || misaligned(dW, 16) ||
        misaligned(workspace, 256))
        return DION_ERR_ALIGN;
    if (workspace_bytes < p.total) return DION_ERR_WORKSPACE;
    const Range rs[4] = {span(dW, vocab * width, size_of(w_dtype)), span(workspace, (int64_t)p.total, 1),
                         span(ids, tokens, size_of_index(id_dtype)), span(dY, tokens * width, size_of(y_dtype))};
    if (any_overlap(rs, 2, 4)) return DION_ERR_OVERLAP;
    const dion::EmbedArgs a{ids, dY, dW, tokens, vocab, width, scale, padding_id, id_dtype == DION_I64,
                            y_dtype == DION_BF16, w_dtype == DION_BF16, accumulate};
    const int e = dion::run_embedding_grad(a, p, (char*)workspace, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

size_t dion_linear_xent_workspace_size(int64_t tokens, int64_t vocab, int64_t width, int dtype, int dw_dtype,
                                       int for_grad) {
    dion::XentPlan p;
    if (!check_sizes(tokens, vocab, width) || !is_dtype(dtype) || !is_dtype(dw_dtype)) return 0;
    if (!dion::make_xent_plan(tokens, vocab, width, dtype == DION_BF16, dw_dtype == DION_BF16, for_grad != 0, &p)) return 0;
    return p.total;
}

int dion_linear_xent(const void* H, const void* W, const void* targets, float* loss, float* lse, int64_t tokens,
                     int64_t vocab, int64_t width, int64_t ignore_index, int t_dtype, int dtype, void* workspace,
                     size_t workspace_bytes, void* stream) {
    if (!check_sizes(tokens, vocab, width)) return DION_ERR_SHAPE;
    if (!is_index(t_dtype) || !is_dtype(dtype)) return DION_ERR_DTYPE;
    dion::XentPlan p;
    if (!dion::make_xent_plan(tokens, vocab, width, dtype == DION_BF16, 1, 0, &p)) return DION_ERR_SHAPE;
    if (tokens == 0) return DION_OK;
    if (!H || !W || !targets || !loss || !lse || !workspace) return DION_ERR_NULL;
    if (misaligned(targets, size_of_index(t_dtype)) || misaligned(H, 16) || misaligned(W, 16) ||
        misaligned(loss, 4) || misaligned(lse, 4) || misaligned(workspace, 256))
        return DION_ERR_ALIGN;
    if (workspace_bytes < p.total) return DION_ERR_WORKSPACE;
    const Range rs[6] = {span(loss, tokens, 4), span(lse, tokens, 4), span(workspace, (int64_t)p.total, 1),
                         span(H, tokens * width, size_of(dtype)), span(W, vocab * width, size_of(dtype)),
                         span(targets, tokens, size_of_index(t_dtype))};
    if (any_overlap(rs, 3, 6)) return DION_ERR_OVERLAP;
    dion::XentArgs a{};
    a.H = H; a.W = W; a.targets = targets; a.loss = loss; a.lse_out = lse; a.ignore = ignore_index;
    a.t64 = t_dtype == DION_I64; a.bf16 = dtype == DION_BF16;
    const int e = dion::run_xent(a, p, (char*)workspace, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

int dion_linear_xent_grad(const void* H, const void* W, const void* targets, const float* lse, const float* grad,
                          int64_t grad_n, void* dH, void* dW, int64_t tokens, int64_t vocab, int64_t width,
                          int64_t ignore_index, int t_dtype, int dtype, int dw_dtype, int accumulate,
                          void* workspace, size_t workspace_bytes, void* stream) {
    if (!check_sizes(tokens, vocab, width) || (grad_n != 1 && grad_n != tokens)) return DION_ERR_SHAPE;
    if (!is_index(t_dtype) || !is_dtype(dtype) || !is_dtype(dw_dtype)) return DION_ERR_DTYPE;
    if (accumulate != 0 && accumulate != 1) return DION_ERR_OPTION;
    dion::XentPlan p;
    if (!dion::make_xent_plan(tokens, vocab, width, dtype == DION_BF16, dw_dtype == DION_BF16, 1, &p))
        return DION_ERR_SHAPE;
    if (!dH && !dW) return DION_ERR_NULL;
    if (tokens == 0 && (!dW || accumulate)) return DION_OK;
    if (tokens > 0 && (!H || !W || !targets || !lse || !grad || !workspace)) return DION_ERR_NULL;
    if (misaligned(targets, size_of_index(t_dtype)) || misaligned(H, 16) || misaligned(W, 16) ||
        misaligned(dH, 16) || misaligned(dW, 16) || misaligned(lse, 4) || misaligned(grad, 4) ||
        misaligned(workspace, 256))
        return DION_ERR_ALIGN;
    if (workspace_bytes < p.total) return DION_ERR_WORKSPACE;
    const Range rs[8] = {span(dH, tokens * width, size_of(dtype)), span(dW, vocab * width, size_of(dw_dtype)),
                         span(workspace, (int64_t)p.total, 1), span(H, tokens * width, size_of(dtype)),
                         span(W, vocab * width, size_of(dtype)), span(targets, tokens, size_of_index(t_dtype)),
                         span(lse, tokens, 4), span(grad, grad_n, 4)};
    if (any_overlap(rs, 3, 8)) return DION_ERR_OVERLAP;
    dion::XentArgs a{};
    a.H = H; a.W = W; a.targets = targets; a.lse = lse; a.grad = grad; a.grad_n = grad_n; a.dH = dH; a.dW = dW;
    a.ignore = ignore_index; a.t64 = t_dtype == DION_I64; a.bf16 = dtype == DION_BF16;
    a.dw_bf16 = dw_dtype == DION_BF16; a.accumulate = accumulate;
    const int e = dion::run_xent_grad(a, p, (char*)workspace, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

}  // extern "C"
