// extern "C" entry points of the residual blocks' operators: argument validation (pure host code, no
// HIP call before every check has passed) and workspace sizes.
#include <math.h>
#include <stdint.h>

#include "block_plan.h"
#include "dion_block.h"

namespace {

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

bool overlap(const Range& a, const Range& b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

// sizes are bounded before any span is formed, so the byte counts are exact in 64 bits
Range span(const void* p, int64_t count, int64_t bytes) {
    const uintptr_t lo = (uintptr_t)p;
    return Range{lo, lo + (uintptr_t)(p ? count * bytes : 0)};
}

// the first `written` ranges must overlap nothing else; range `alias` may be range `of` itself (in place)
bool any_overlap(const Range* r, int written, int n, int alias = -1, int of = -1) {
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < n; ++j) {
            if (i == alias && j == of && r[i].lo == r[j].lo) continue;
            if (overlap(r[i], r[j])) return true;
        }
    return false;
}

bool check_rows(int64_t rows, int64_t width) {
    return rows >= 0 && rows <= DION_BLOCK_MAX_ROWS && width >= 1 && width <= dion::kWidthMax;
}

bool is_dtype(int t) { return t == DION_F32 || t == DION_BF16; }
int64_t size_of(int t) { return t == DION_E4M3 ? 1 : t == DION_BF16 ? 2 : 4; }
bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// false: no activation, or a form of gate and up that the type does not have
bool split_act(int& act, int dtype, int* even) {
    *even = (act & DION_KEEP_EVEN) != 0;
    act &= ~DION_KEEP_EVEN;
    return (act == DION_SILU || act == DION_GELU) && (!*even || dtype == DION_BF16);
}

// false: p is no probability of dropping
bool make_mask(double p, const int64_t* seed, int64_t site, dion::Mask* m) {
    if (!(p >= 0 && p < 1)) return false;
    const double t = rint(p * 4294967296.0);
    *m = dion::Mask{seed, site, t < 4294967295.0 ? (uint32_t)t : 4294967295u, 1.0 / (1.0 - p), p > 0};
    return true;
}

}  // namespace

extern "C" {

int dion_dropout(const void* x, const void* residual, void* out, int64_t n, double p, const int64_t* seed, int64_t site,
                 int x_dtype, int out_dtype, void* stream) {
    if (n < 0 || n > (int64_t)1 << 36) return DION_ERR_SHAPE;
    dion::DropoutArgs a{x, residual, out, n, {}, x_dtype == DION_BF16, out_dtype == DION_BF16};
    if (!make_mask(p, seed, site, &a.mask)) return DION_ERR_HYPER;
    if (!is_dtype(x_dtype) || !is_dtype(out_dtype)) return DION_ERR_DTYPE;
    if (n == 0) return DION_OK;
    if (!x || !out || (a.mask.on && !seed)) return DION_ERR_NULL;
    if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(out, 16) || misaligned(seed, 8)) return DION_ERR_ALIGN;
    const Range rs[4] = {span(out, n, size_of(out_dtype)), span(x, n, size_of(x_dtype)), span(residual, n, size_of(out_dtype)),
                         span(seed, 1, 8)};
    if (any_overlap(rs, 1, 4, 0, 2)) return DION_ERR_OVERLAP;
    const int e = dion::run_dropout(a, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

int dion_rms_norm(const void* x, const void* residual, const void* w, void* h, void* y, float* scale, float* rstd,
                  int64_t rows, int64_t width, double eps, double p, const int64_t* seed, int64_t site, int x_dtype,
                  int s_dtype, int w_dtype, int y_dtype, void* stream) {
    if (!check_rows(rows, width)) return DION_ERR_SHAPE;
    dion::NormArgs a{x, residual, w, h, y, scale, rstd, rows, (int)width, eps, {}, x_dtype == DION_BF16, s_dtype == DION_BF16,
                     w_dtype == DION_BF16, y_dtype == DION_BF16};
    if (!(eps >= 0) || !isfinite(eps) || !make_mask(p, seed, site, &a.mask)) return DION_ERR_HYPER;
    if (!is_dtype(x_dtype) || !is_dtype(s_dtype) || !is_dtype(w_dtype) || (!is_dtype(y_dtype) && y_dtype != DION_E4M3))
        return DION_ERR_DTYPE;
    if (rows == 0) return DION_OK;
    if (!x || !w || !y || (a.mask.on && !seed) || (y_dtype == DION_E4M3) != (scale != nullptr)) return DION_ERR_NULL;
    if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(w, 16) || misaligned(h, 16) || misaligned(y, 16) ||
        misaligned(scale, 4) || misaligned(rstd, 4) || misaligned(seed, 8))
        return DION_ERR_ALIGN;
    const int64_t n = rows * width;
    const Range rs[8] = {span(h, n, size_of(s_dtype)), span(y, n, size_of(y_dtype)), span(scale, rows, 4), span(rstd, rows, 4),
                         span(x, n, size_of(x_dtype)), span(residual, n, size_of(s_dtype)), span(w, width, size_of(w_dtype)),
                         span(seed, 1, 8)};
    if (any_overlap(rs, 4, 8, 0, 5)) return DION_ERR_OVERLAP;
    const int e = dion::run_rms_norm(a, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

size_t dion_rms_norm_grad_workspace_size(int64_t rows, int64_t width) {
    return check_rows(rows, width) ? dion::make_norm_plan(rows, width).total : 0;
}

int dion_rms_norm_grad(const void* dY, const void* h, const void* w, const float* rstd, const void* dsum, void* dh, void* dx,
                       void* dw, int64_t rows, int64_t width, double p, const int64_t* seed, int64_t site, int y_dtype,
                       int s_dtype, int w_dtype, int dw_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                       void* stream) {
    if (!check_rows(rows, width)) return DION_ERR_SHAPE;
    dion::NormGradArgs a{dY, h, w, rstd, dsum, dh, dx, dw, (float*)workspace, rows, (int)width, {}, y_dtype == DION_BF16,
                         s_dtype == DION_BF16, w_dtype == DION_BF16, dw_dtype == DION_BF16, accumulate};
    if (!make_mask(p, seed, site, &a.mask)) return DION_ERR_HYPER;
    if (!is_dtype(y_dtype) || !is_dtype(s_dtype) || !is_dtype(w_dtype) || !is_dtype(dw_dtype)) return DION_ERR_DTYPE;
    if (accumulate != 0 && accumulate != 1) return DION_ERR_OPTION;
    if (rows == 0 && (!dw || accumulate)) return DION_OK;
    const dion::NormPlan plan = dion::make_norm_plan(rows, width);
    if (rows > 0 && (!dY || !h || !w || !rstd || !dh || (a.mask.on && dx && !seed) || (dw && plan.total && !workspace)))
        return DION_ERR_NULL;
    if (misaligned(dY, 16) || misaligned(h, 16) || misaligned(w, 16) || misaligned(rstd, 4) || misaligned(dsum, 16) ||
        misaligned(dh, 16) || misaligned(dx, 16) || misaligned(dw, 16) || misaligned(seed, 8) || misaligned(workspace, 256))
        return DION_ERR_ALIGN;
    if (dw && workspace_bytes < plan.total) return DION_ERR_WORKSPACE;
    const int64_t n = rows * width;
    const Range rs[10] = {span(dh, n, size_of(s_dtype)), span(dx, n, size_of(y_dtype)), span(dw, width, size_of(dw_dtype)),
                          span(workspace, dw ? (int64_t)plan.total : 0, 1), span(dY, n, size_of(y_dtype)),
                          span(h, n, size_of(s_dtype)), span(dsum, n, size_of(s_dtype)), span(w, width, size_of(w_dtype)),
                          span(rstd, rows, 4), span(seed, 1, 8)};
    if (any_overlap(rs, 4, 10, 0, 6)) return DION_ERR_OVERLAP;
    const int e = dion::run_rms_norm_grad(a, plan, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

static bool make_plan(int64_t rows, int64_t width, int64_t hidden, int dtype, int x_dtype, int for_grad, int saved,
                      dion::FfnPlan* p) {
    return check_rows(rows, width) && hidden >= 1 && hidden <= dion::kHiddenMax &&
           dion::make_ffn_plan(rows, width, hidden, dtype == DION_BF16, x_dtype == DION_E4M3, for_grad, saved, p);
}

size_t dion_gated_ffn_workspace_size(int64_t rows, int64_t width, int64_t hidden, int dtype, int x_dtype, int for_grad) {
    dion::FfnPlan p;
    if (!is_dtype(dtype) || (x_dtype != dtype && x_dtype != DION_E4M3) || for_grad < 0 || for_grad > 2) return 0;
    return make_plan(rows, width, hidden, dtype, x_dtype, for_grad > 0, for_grad == 1, &p) ? p.total : 0;
}

int dion_gated_ffn(const void* X, const float* x_scale, const void* Wg, const void* Wu, const void* Wd, void* gate, void* up,
                   void* Y, int64_t rows, int64_t width, int64_t hidden, int act, int x_dtype, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
    if (!is_dtype(dtype) || (x_dtype != dtype && x_dtype != DION_E4M3)) return DION_ERR_DTYPE;
    dion::FfnPlan p;
    if (!make_plan(rows, width, hidden, dtype, x_dtype, 0, 0, &p)) return DION_ERR_SHAPE;
    int even;
    if (!split_act(act, dtype, &even)) return DION_ERR_OPTION;
    if (rows == 0) return DION_OK;
    if (!X || !Wg || !Wu || !Wd || !Y || !workspace || !gate != !up || (x_dtype == DION_E4M3) != (x_scale != nullptr))
        return DION_ERR_NULL;
    if (misaligned(X, 16) || misaligned(x_scale, 4) || misaligned(Wg, 16) || misaligned(Wu, 16) || misaligned(Wd, 16) ||
        misaligned(gate, 16) || misaligned(up, 16) || misaligned(Y, 16) || misaligned(workspace, 256))
        return DION_ERR_ALIGN;
    if (workspace_bytes < p.total) return DION_ERR_WORKSPACE;
    const int64_t b = size_of(dtype);
    const Range rs[9] = {span(Y, rows * width, b), span(gate, rows * hidden, b), span(up, rows * hidden, b),
                         span(workspace, (int64_t)p.total, 1), span(X, rows * width, size_of(x_dtype)), span(x_scale, rows, 4),
                         span(Wg, hidden * width, b), span(Wu, hidden * width, b), span(Wd, hidden * width, b)};
    if (any_overlap(rs, 4, 9)) return DION_ERR_OVERLAP;
    dion::FfnArgs a{};
    a.X = X; a.x_scale = x_scale; a.Wg = Wg; a.Wu = Wu; a.Wd = Wd; a.Y = Y; a.gate = gate; a.up = up;
    a.act = act; a.bf16 = dtype == DION_BF16; a.even = even;
    const int e = dion::run_ffn(a, p, (char*)workspace, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

int dion_gated_ffn_grad(const void* X, const float* x_scale, const void* Wg, const void* Wu, const void* Wd, const void* dY,
                        const void* gate, const void* up, void* dX, void* dWg, void* dWu, void* dWd, int64_t rows,
                        int64_t width, int64_t hidden, int act, int x_dtype, int dtype, int dw_dtype, int accumulate,
                        void* workspace, size_t workspace_bytes, void* stream) {
    if (!is_dtype(dtype) || !is_dtype(dw_dtype) || (x_dtype != dtype && x_dtype != DION_E4M3)) return DION_ERR_DTYPE;
    dion::FfnPlan p;
    if (!make_plan(rows, width, hidden, dtype, x_dtype, 1, gate != nullptr, &p)) return DION_ERR_SHAPE;
    int even;
    if (!split_act(act, dtype, &even) || (accumulate != 0 && accumulate != 1)) return DION_ERR_OPTION;
    // (no rows: dX has no elements, and an array without any may be NULL)
    if ((rows > 0 && !dX && !dWg && !dWd) || !dWg != !dWu || !gate != !up) return DION_ERR_NULL;
    if (rows == 0 && (accumulate || (!dWg && !dWd))) return DION_OK;
    if (rows > 0 && (!X || !Wg || !Wu || !Wd || !dY || !workspace || (x_dtype == DION_E4M3) != (x_scale != nullptr)))
        return DION_ERR_NULL;
    if (misaligned(X, 16) || misaligned(x_scale, 4) || misaligned(Wg, 16) || misaligned(Wu, 16) || misaligned(Wd, 16) ||
        misaligned(dY, 16) || misaligned(gate, 16) || misaligned(up, 16) || misaligned(dX, 16) || misaligned(dWg, 16) ||
        misaligned(dWu, 16) || misaligned(dWd, 16) || misaligned(workspace, 256))
        return DION_ERR_ALIGN;
    if (rows > 0 && workspace_bytes < p.total) return DION_ERR_WORKSPACE;
    const int64_t b = size_of(dtype), wb = size_of(dw_dtype);
    const Range rs[13] = {span(dX, rows * width, b), span(dWg, hidden * width, wb), span(dWu, hidden * width, wb),
                          span(dWd, hidden * width, wb), span(workspace, rows > 0 ? (int64_t)p.total : 0, 1),
                          span(X, rows * width, size_of(x_dtype)), span(x_scale, rows, 4), span(Wg, hidden * width, b),
                          span(Wu, hidden * width, b), span(Wd, hidden * width, b), span(dY, rows * width, b),
                          span(gate, rows * hidden, b), span(up, rows * hidden, b)};
    if (any_overlap(rs, 5, 13)) return DION_ERR_OVERLAP;
    int e = 0;
    if (rows == 0) {   // no rows: the weights' gradients are zero
        void* out[3] = {dWg, dWu, dWd};
        for (int i = 0; i < 3 && !e; ++i)
            if (out[i]) e = dion::run_zeros(out[i], hidden * width * wb / 2, stream);
        return e ? DION_ERR_HIP - e : DION_OK;
    }
    dion::FfnArgs a{};
    a.X = X; a.x_scale = x_scale; a.Wg = Wg; a.Wu = Wu; a.Wd = Wd; a.dY = dY; a.gate = (void*)gate; a.up = (void*)up;
    a.dX = dX; a.dWg = dWg; a.dWu = dWu; a.dWd = dWd;
    a.act = act; a.bf16 = dtype == DION_BF16; a.dw_bf16 = dw_dtype == DION_BF16; a.accumulate = accumulate; a.even = even;
    e = dion::run_ffn_grad(a, p, (char*)workspace, stream);
    return e ? DION_ERR_HIP - e : DION_OK;
}

}  // extern "C"
