/*
 * dion_block.h — C ABI of the operators of a model's residual blocks: dropout whose mask is never stored, the
 * root-mean-square norm with the residual's addition in front of it (and dropout, and an output in 8 bits), the gated
 * feed-forward block, and their gradients.  They stand between the vocabulary operators of dion_vocab.h at the two ends of
 * the model; the weight gradients go where the optimizer steps of dion.h read them.
 *
 *   dion_dropout         out = residual + keep x / (1 - p)
 *   dion_rms_norm        h = residual + keep x / (1 - p);  rstd = (mean h^2 + eps)^(-1/2);  y = h rstd w
 *                        in 8 bits: q = e4m3(y / scale), scale the least power of two with max |y| <= 448 scale
 *   dion_rms_norm_grad   n = h rstd;  g = dY w;  dh = rstd (g - n mean(g n)) + dsum;  dx = keep dh / (1 - p);  dw (+)= sum dY n
 *   dion_gated_ffn       a = X Wg^T;  b = X Wu^T;  u = act(a) b;  Y = u Wd^T
 *   dion_gated_ffn_grad  du = dY Wd;  da = du b act'(a);  db = du act(a);  dX = da Wg + db Wu;
 *                        dWg (+)= da^T X;  dWu (+)= db^T X;  dWd (+)= dY^T u
 *
 * The mask.  keep of element i of an array (row-major, of any shape) is: word i % 4 of Philox4x32-10 (Salmon, Moraes, Dror
 * and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with the counter (i / 4, site), 64 bits each, and the key
 * `seed` is at least p 2^32 (rounded, and at most 2^32 - 1).  It depends on the seed, the site and the element's number alone, so that the gradient
 * forms it again: dion_dropout without residual of the output's gradient, or dx of dion_rms_norm_grad.  The seed is read
 * from device memory when the kernel runs; a captured graph draws another mask on each replay if the program changes it.
 * Sites keep the masks of different layers apart.
 *
 * Memory, execution and errors are those of dion.h: caller-owned device memory, row-major and contiguous, nothing allocated
 * and nothing kept between calls; asynchronous on `stream` (NULL = default stream) with no host synchronization, safe to
 * capture in a HIP graph; results bitwise reproducible (no floating-point atomics); status codes of dion.h, checked on the
 * host before anything is enqueued.  Matrices and vectors must be 16-byte aligned, workspaces 256-byte, fp32 per-row arrays
 * as their elements, the seed 8-byte; any width is taken.  Written arrays must not overlap anything else, but for what is
 * said below.  Calls that share a workspace must be ordered on one stream.  Sums, norms and products accumulate in fp32
 * or more; each output is rounded once to its type.
 *
 * Limits: rows <= DION_BLOCK_MAX_ROWS, 1 <= width <= 2^16, 1 <= hidden <= 2^17; beyond them DION_ERR_SHAPE.
 */
#ifndef DION_BLOCK_MI355X_H
#define DION_BLOCK_MI355X_H

#include "dion.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a third element type where it is named: OCP e4m3 (no infinities, largest 448) with an fp32 scale per row */
#define DION_E4M3 2

typedef enum { DION_SILU = 0, DION_GELU = 1 } dion_activation;   /* a / (1 + exp(-a)); the tanh form of gelu */
/* added to the activation, in both calls of a block: bf16's gate and up are kept in the even form */
#define DION_KEEP_EVEN 16

#define DION_BLOCK_MAX_ROWS ((int64_t)1 << 20)

/*
 * Dropout with an optional addition, formed in fp32 and rounded once.
 *   x         device, [n], x_dtype (DION_F32 or DION_BF16), read only.  0 <= n <= 2^36
 *   residual  device, [n], out_dtype, or NULL
 *   out       device, [n], out_dtype, written; may be residual itself (added to in place)
 *   p         probability of dropping an element, in [0, 1)
 *   seed      device, one int64; may be NULL where p is 0
 */
int dion_dropout(const void* x, const void* residual, void* out, int64_t n, double p, const int64_t* seed, int64_t site,
                 int x_dtype, int out_dtype, void* stream);

/*
 * Root-mean-square norm of each row.
 *   x         device, [rows][width], x_dtype, read only
 *   residual  device, [rows][width], s_dtype (of the residual stream), or NULL
 *   w         device, [width], w_dtype
 *   h         device, [rows][width], s_dtype, written; may be residual itself; or NULL: not written
 *   y         device, [rows][width], y_dtype (DION_F32, DION_BF16 or DION_E4M3), written
 *   scale     device fp32 [rows], written where y_dtype is DION_E4M3 (1 for a row of zeros), else NULL
 *   rstd      device fp32 [rows], written, or NULL
 *   eps       >= 0, finite.  p, seed, site as above, over rows x width elements
 * Arithmetic: in fp32; y is formed from h before its rounding; rows whose squares leave fp32's range are scaled first (rstd
 * itself may then be subnormal, or infinite above 2^128).  With DION_E4M3 in fp64, so that no rounding on the way moves
 * a value across a border of its 8-bit numbers.  Elements that are not finite become NaN in 8 bits and do not count for scale.
 */
int dion_rms_norm(const void* x, const void* residual, const void* w, void* h, void* y, float* scale, float* rstd,
                  int64_t rows, int64_t width, double eps, double p, const int64_t* seed, int64_t site, int x_dtype,
                  int s_dtype, int w_dtype, int y_dtype, void* stream);

/*
 * Gradients of the norm, its dropout and its addition.
 *   dY         device, [rows][width], y_dtype (DION_F32 or DION_BF16)
 *   h, rstd    from dion_rms_norm (h is x itself where there was neither residual nor dropout); h has s_dtype
 *   dsum       device, [rows][width], s_dtype: the gradient that reaches h by other ways (the stream behind it), or NULL
 *   dh         device, [rows][width], s_dtype, written: h's gradient, which is the residual's; may be dsum itself
 *   dx         device, [rows][width], y_dtype, written: the gradient of x; or NULL
 *   dw         device, [width], dw_dtype, written, or added to with accumulate 1; or NULL
 *   workspace  device, >= dion_rms_norm_grad_workspace_size(rows, width) bytes, 256-byte aligned; may be NULL where that is 0
 */
size_t dion_rms_norm_grad_workspace_size(int64_t rows, int64_t width);
int dion_rms_norm_grad(const void* dY, const void* h, const void* w, const float* rstd, const void* dsum, void* dh, void* dx,
                       void* dw, int64_t rows, int64_t width, double p, const int64_t* seed, int64_t site, int y_dtype,
                       int s_dtype, int w_dtype, int dw_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Gated feed-forward block.
 *   X         device, [rows][width], x_dtype: dtype, or DION_E4M3 with x_scale, fp32 [rows] (else NULL)
 *   Wg, Wu    device, [hidden][width], dtype (DION_F32 or DION_BF16)
 *   Wd        device, [width][hidden], dtype
 *   gate, up  device, [rows][hidden], elements of dtype's size: a and b, written for the gradient; both or neither NULL.  In
 *             fp32 for fp32.  For bf16 in 16 bits of their own, more exact than bf16 at the usual sizes: bit 15 the sign; bit 14
 *             set for magnitudes in [2^-8, 2^8), with 4 bits of exponent (from 2^-8) and 10 of fraction below it; else clear.
 *             Then with DION_KEEP_EVEN 7 bits of exponent n (2^(n - 80) below 72, else 2^(n - 64)) and 7 of fraction, as exact as
 *             bf16; all zeros is 0, for what rounds to 2^-80 or less, and all ones NaN, for what rounds to 2^64 - 2^56 or more
 *             and what is not finite.  Without it the upper 14 bits of the magnitude's fp32 form (8 of exponent, 6 of fraction):
 *             any magnitude, at half of bf16's exactness, so twice its rounding in the gradients of blocks whose projections are
 *             far from 1.  Rounded to nearest, ties away from zero
 *   Y         device, [rows][width], dtype, written
 *   act       dion_activation, and for bf16 DION_KEEP_EVEN or not (which counts where gate and up are given)
 * Arithmetic: bf16 operands multiply exactly and add up in fp32 on the matrix cores; u is rounded to bf16 for the second
 * product, or for up to 64 rows to two bf16 parts.  fp32 operands give fp32-accurate products: a, b and du from two fp16 parts of each row scaled by a power of two
 * (2^-23 of an element and 2^-38 of its row's largest left out, or 2^-125 where that is more, three part products, terms below
 * 2^-22 dropped; rows up to 2^100; for du dY's elements count times 2^-13 of the largest of Wd's row that they meet), the others from three bf16 parts (an exact split, six part products, terms below 2^-24 dropped), and all of few
 * rows in fp32 (how many rows are few is a matter of the sizes).  8-bit rows go as bf16, which holds x scale exactly where
 * scale is a power of two, as dion_rms_norm leaves it, and is rounded else.  Operands are taken to be finite; others make what they reach NaN or infinite.
 * Workspace size: for_grad 0 for dion_gated_ffn, 1 for dion_gated_ffn_grad given gate and up, 2 without them; 0 for invalid
 * sizes.  It does not only grow with the rows, since few and many go different ways: a workspace for several numbers of rows
 * has the largest of their sizes.
 */
size_t dion_gated_ffn_workspace_size(int64_t rows, int64_t width, int64_t hidden, int dtype, int x_dtype, int for_grad);
int dion_gated_ffn(const void* X, const float* x_scale, const void* Wg, const void* Wu, const void* Wd, void* gate, void* up,
                   void* Y, int64_t rows, int64_t width, int64_t hidden, int act, int x_dtype, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * Its gradients.
 *   dY             device, [rows][width], dtype
 *   gate, up       from dion_gated_ffn on the same X, Wg, Wu, with the same act, read only; or both NULL: formed again (for bf16
 *                  in the even form)
 *   dX             device, [rows][width], dtype, written (of the values that X stands for), or NULL
 *   dWg, dWu, dWd  device, shaped as the weights, dw_dtype, written, or added to with accumulate 1; dWg and dWu both or
 *                  neither NULL, dWd or NULL.  One output at least is given, where there are rows
 * Arithmetic: as above; da, db and u are rounded to bf16 where dtype is bf16 (for up to 16 rows to two bf16 parts), and a and b to the form in which they are kept.
 */
int dion_gated_ffn_grad(const void* X, const float* x_scale, const void* Wg, const void* Wu, const void* Wd, const void* dY,
                        const void* gate, const void* up, void* dX, void* dWg, void* dWu, void* dWd, int64_t rows,
                        int64_t width, int64_t hidden, int act, int x_dtype, int dtype, int dw_dtype, int accumulate,
                        void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DION_BLOCK_MI355X_H */
