/*
 * dion_vocab.h — C ABI of the operators over a language model's two vocabulary matrices, the
 * embedding table and the output head: W, vocab x width.  They stand at the two ends of the model
 * whose weights dion.h updates, and leave W's gradient where its optimizer steps read it.
 *
 *   dion_embedding         Y[t] = scale * W[ids[t]]
 *   dion_embedding_grad    dW[v] (+)= scale * (sum of dY[t] over the tokens t with ids[t] = v)
 *   dion_linear_xent       z[t] = W H[t];  lse[t] = log sum_v exp z[t][v];  loss[t] = lse[t] - z[t][target[t]]
 *   dion_linear_xent_grad  D[t][v] = grad[t] (exp(z[t][v] - lse[t]) - [v = target[t]]);
 *                          dH = D W;  dW (+)= D^T H
 *
 * The logits z (tokens x vocab) are not kept from the loss to the gradient.  The loss keeps a running maximum and sum per
 * tile of the vocabulary (where the tiles do not fill the chip, it stores partial logits, few then, in its workspace).  The
 * gradient forms them again, a piece of the vocabulary at a time, and holds D of that piece in its workspace: 16-bit parts
 * of 2^28 elements each, or of as many as 8192 rows of the vocabulary need, at most 2^30.  Up to 2^28 elements that is D of
 * the whole vocabulary, which is as large as logits.  Workspaces of 8192 tokens x 32000 x 2048: loss 40 MiB, gradient
 * 604 MiB for bf16 outputs (one part) and 1532 MiB for an fp32 dW (three), where bf16 logits are 500; 8192 x 131072 x 4096:
 * 96, 849 and 1728 MiB (2048); 4096 x 32000 x 1024 in fp32: 145 and 1479 MiB (fp32 logits 500).
 *
 * Memory, execution and errors are those of dion.h: caller-owned device memory, row-major and
 * contiguous, nothing allocated and nothing kept between calls; asynchronous on `stream` (NULL =
 * default stream) with no host synchronization, safe to capture in a HIP graph; results bitwise
 * reproducible (no floating-point atomics); status codes of dion.h, checked on the host before
 * anything is enqueued.  Matrices must be 16-byte aligned, workspaces 256-byte, ids, targets and
 * the fp32 per-token arrays as their elements; any width is taken.  Written arrays must not
 * overlap anything else.  Calls that share a workspace must be ordered on one stream.  Sums,
 * softmax statistics and products accumulate in fp32; each output is rounded once to its type.
 *
 * Limits: tokens <= DION_VOCAB_MAX_TOKENS, 1 <= vocab < 2^24, 1 <= width <= 2^16; beyond them DION_ERR_SHAPE.
 */
#ifndef DION_VOCAB_MI355X_H
#define DION_VOCAB_MI355X_H

#include "dion.h"

#ifdef __cplusplus
extern "C" {
#endif

/* type of token ids and targets */
typedef enum { DION_I32 = 0, DION_I64 = 1 } dion_index_dtype;

#define DION_VOCAB_MAX_TOKENS ((int64_t)1 << 20)

/*
 * Embedding lookup: out[t][:] = scale * W[ids[t]][:], formed in fp32 and rounded once.
 *   ids    device, [tokens], id_dtype (DION_I32 or DION_I64); an id outside [0, vocab) gives a row of NaN
 *   W      device, [vocab][width], w_dtype (DION_F32 or DION_BF16), read only
 *   out    device, [tokens][width], out_dtype, written
 *   scale  finite.  tokens >= 0 (0 is a no-op)
 */
int dion_embedding(const void* ids, const void* W, void* out, int64_t tokens, int64_t vocab, int64_t width,
                   float scale, int id_dtype, int w_dtype, int out_dtype, void* stream);

/*
 * Gradient of the table: dW[v] (+)= scale * sum of dY[t] over ids[t] = v, the tokens sorted by id
 * (stable), each row's tokens added in a fixed order in fp32 and rounded once.
 *   ids         as above; ids equal to padding_id and ids outside [0, vocab) leave no gradient
 *               (a padding_id outside [0, vocab) excludes none)
 *   dY          device, [tokens][width], y_dtype, read only
 *   dW          device, [vocab][width], w_dtype.  accumulate 0: every row is written, zeros where no
 *               token has that id; accumulate 1: added to what is there (rows without tokens untouched)
 *   workspace   device, >= dion_embedding_grad_workspace_size(tokens, vocab, width) bytes, 256-byte
 *               aligned (contents on entry ignored); may be NULL where that size is 0
 */
size_t dion_embedding_grad_workspace_size(int64_t tokens, int64_t vocab, int64_t width);
int dion_embedding_grad(const void* ids, const void* dY, void* dW, int64_t tokens, int64_t vocab, int64_t width,
                        float scale, int64_t padding_id, int id_dtype, int y_dtype, int w_dtype, int accumulate,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Softmax cross entropy of a linear head, per token.
 *   H        device, [tokens][width], dtype (DION_F32 or DION_BF16; W has the same), read only
 *   W        device, [vocab][width], dtype, read only
 *   targets  device, [tokens], t_dtype (DION_I32 or DION_I64).  A target equal to ignore_index leaves
 *            its token out: loss and lse 0, and H's row is not used (it may hold anything).  Any other
 *            target outside [0, vocab) gives that token a NaN loss
 *   loss     device fp32 [tokens], written
 *   lse      device fp32 [tokens], written: log sum_v exp z[t][v], for dion_linear_xent_grad
 * Arithmetic: bf16 operands multiply exactly and add up in fp32 on the matrix cores.  fp32 operands give fp32-accurate
 * logits from 16-bit parts, whichever is cheaper for the sizes: three bf16 parts (an exact split, six part products, terms
 * below 2^-24 dropped), or two fp16 parts of each row scaled by a power of two (2^-23 of an element and 2^-38 of its row's
 * largest left out, or 2^-125 where that is more, three part products, terms below 2^-22 dropped).
 * Operands are taken to be finite and logits below 2^127; others make what they reach NaN or infinite.
 * Workspace size for both calls: dion_linear_xent_workspace_size (for_grad 0 or 1; 0 for invalid sizes).
 */
size_t dion_linear_xent_workspace_size(int64_t tokens, int64_t vocab, int64_t width, int dtype, int dw_dtype,
                                       int for_grad);
int dion_linear_xent(const void* H, const void* W, const void* targets, float* loss, float* lse, int64_t tokens,
                     int64_t vocab, int64_t width, int64_t ignore_index, int t_dtype, int dtype, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * Gradients of sum_t grad[t] loss[t].
 *   lse      from dion_linear_xent on the same H, W and targets
 *   grad     device fp32 [grad_n], grad_n = tokens, or 1 for the same factor on every token
 *   dH       device, [tokens][width], dtype, written (zeros where the target is ignored), or NULL
 *   dW       device, [vocab][width], dw_dtype (DION_F32 or DION_BF16), or NULL; accumulate 1 adds to
 *            what is there.  At least one of dH and dW is given
 * A token whose target is neither ignored nor in [0, vocab) makes its dH row and dW NaN.
 * Arithmetic: for bf16 outputs of bf16 operands D is rounded once to bf16 (without grad where grad_n is 1: that factor is
 * applied to the fp32 sums), and what the rounding left of the target's element is added to dH and dW in fp32; small dW come
 * from two bf16 parts of D.  Where the output or the operands are fp32, the products are fp32-accurate, from 16-bit parts as
 * in dion_linear_xent: dW from three bf16 parts of D and H, dH from three bf16 parts, or from two fp16 parts of D (per token)
 * and of W (per row) scaled by powers of two, which leaves out vocab 2^-38 of |grad[t]| times the largest |W| besides.
 * Products below fp32's normal numbers may count as zeros.
 * Where no target counts, grad is not used (1 / count may be infinite then).
 */
int dion_linear_xent_grad(const void* H, const void* W, const void* targets, const float* lse, const float* grad,
                          int64_t grad_n, void* dH, void* dW, int64_t tokens, int64_t vocab, int64_t width,
                          int64_t ignore_index, int t_dtype, int dtype, int dw_dtype, int accumulate,
                          void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DION_VOCAB_MI355X_H */
