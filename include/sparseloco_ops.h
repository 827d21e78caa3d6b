/*
 * sparseloco_ops.h -- C ABI of libsparseloco.so, continued: the operators on
 * either side of a round's records, hand-written HIP for AMD MI355X (gfx950).
 *
 *   sl_orthogonalize, sl_muon_step   the matrix update that turns a gradient,
 *       or the aggregated pseudo-gradient, into a weight update
 *   sl_token_logprobs                the score of given tokens that says
 *       whether a received update lowers the loss
 *
 * Conventions as in sparseloco.h: device pointers owned by the caller, work
 * enqueued on `stream` and not waited for, argument errors returned as a status
 * before anything is enqueued, no allocation, no state between calls, repeated
 * calls bitwise identical.  The _workspace functions return -1 for arguments
 * that their operator refuses.  Where a call needs scratch memory the caller passes
 * `workspace` (256-byte aligned, at least the bytes that the matching
 * _workspace function returns; contents undefined before and after).  Calls
 * that overlap in time need a workspace each, and so do two captured graphs
 * that may run at once.
 */
#ifndef SPARSELOCO_OPS_H
#define SPARSELOCO_OPS_H

#include "sparseloco.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SL_F32 = 0,
    SL_BF16 = 1,
    SL_F16 = 2
} sl_dtype;

/* How sl_orthogonalize and sl_muon_step form their matrix products. */
typedef enum {
    SL_PRODUCTS_F16 = 0,  /* operands rounded to fp16, sums in fp32: the result is
                             within about 1e-3 of the exact one (2-norm of the
                             difference over 2-norm), finer than bf16 holds */
    SL_PRODUCTS_SPLIT = 1 /* each operand the sum of two fp16 values (22 bits), three
                             products: within about what fp32 arithmetic leaves
                             (1e-6 to 3e-6, and more where singular values span
                             decades: 2e-5 if one outweighs the others a hundred
                             times), at three times the work.  sl_muon_step on
                             matrices of some thousand rows and columns that are
                             not square: about 1e-5 */
} sl_products;

#define SL_MAX_STEPS 16
#define SL_MAX_SIDE (1 << 20)    /* rows and cols of one matrix */
#define SL_MAX_ALTERNATIVES 32   /* n_top of sl_token_logprobs */
#define SL_MAX_VOCAB (1 << 22)   /* vocab of sl_token_logprobs */

/*
 * sl_orthogonalize -- Newton-Schulz orthogonalisation of count matrices.
 *
 * For each matrix x (rows x cols): X <- x / (|x|_F + eps), then for each
 * (a, b, c) of coefficients
 *     A = X X^T,  X <- a X + (b A + c A A) X
 * (with X^T in X's place when rows > cols; the result is the same), which
 * drives the singular values towards 1 and keeps the singular vectors.  The
 * norm is summed in fp64.  A zero matrix gives zeros.
 *
 * x, x_type      in  element (i, r, c) at x + (i * x_stride + r * x_ld + c); not written
 * out, out_type  out likewise, fully overwritten; must not overlap x
 * x_ld, out_ld       row strides in elements, >= cols
 * x_stride, out_stride  matrix strides in elements; out's at least (rows - 1) *
 *                out_ld + cols when count > 1 (x's may be anything >= 0)
 * rows, cols     0..SL_MAX_SIDE; count 0..65535 (any of them 0: nothing is done);
 *                rows * cols * count and min(rows, cols)^2 * count at most 2^40
 * coefficients   HOST float[n_steps][3].  Refused (SL_ERR_INVALID_ARG) if not
 *                finite, or if with singular values in [0, 1] to start from some
 *                iterate's (the last step's result apart) would pass 3.8, some
 *                b s^2 + c s^4 30 or some a + b s^2 + c s^4 10^4 in magnitude:
 *                beyond that the fp16 operands could overflow
 * n_steps        1..SL_MAX_STEPS
 * eps            finite, >= 0
 * products       an sl_products
 * Buffers are aligned to their element size.
 */
int64_t sl_orthogonalize_workspace(int64_t rows, int64_t cols, int64_t count, int32_t products);
sl_status sl_orthogonalize(const void* x, int32_t x_type, int64_t x_ld, int64_t x_stride, void* out,
                           int32_t out_type, int64_t out_ld, int64_t out_stride, int64_t rows, int64_t cols,
                           int64_t count, const float* coefficients, int32_t n_steps, float eps, int32_t products,
                           void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sl_muon_step -- momentum, orthogonalisation and weight update in one call,
 * for count contiguous matrices of rows x cols each, back to back.
 *
 *     g = grad_scale * grad
 *     momentum <- decay * momentum + g        (one rounding of the product g,
 *                                              one of the fused multiply-add)
 *     u = g + decay * momentum if nesterov, else momentum
 *     O = the result of sl_orthogonalize(u)   (never written to memory)
 *     theta <- theta * (1 - lr * weight_decay) - lr * update_scale * O
 *
 * As an inner step grad is the gradient; as an outer update it is the sum that
 * sl_aggregate wrote, with grad_scale = 1 / n_peers (its sign is that of
 * sl_apply_mean: theta moves against it).
 *
 * theta, theta_type   in/out SL_F32 or SL_BF16
 * momentum            in/out float32
 * grad, grad_type     in  SL_F32 or SL_BF16
 * lr, weight_decay, update_scale, grad_scale, decay   finite
 * rows, cols, count, coefficients, n_steps, eps, products   as for sl_orthogonalize
 * theta, momentum and grad are aligned to 16 bytes and must not overlap.
 */
int64_t sl_muon_step_workspace(int64_t rows, int64_t cols, int64_t count, int32_t products);
sl_status sl_muon_step(void* theta, int32_t theta_type, float* momentum, const void* grad, int32_t grad_type,
                       int64_t rows, int64_t cols, int64_t count, float grad_scale, float decay, int32_t nesterov,
                       float lr, float weight_decay, float update_scale, const float* coefficients, int32_t n_steps,
                       float eps, int32_t products, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * sl_token_logprobs -- log probabilities of given tokens under a row of logits
 * each, the rows' entropies and their n_top likeliest tokens, in one pass.
 *
 * The gate that the pages put before aggregation ([CV], the Gauntlet
 * paragraph) scores a peer by the loss drop that its update brings on given
 * text; the loss of a token is -logprob.  For each row x[0..vocab):
 *     lse = log(sum_j exp(x_j))
 *     logprob        = x[target] - lse
 *     entropy        = -sum_j p_j log p_j,  p_j = exp(x_j - lse)
 *     top_index[k]   = the token of the k-th largest x; equal ones lower token first
 *     top_logprob[k] = x[top_index[k]] - lse
 * Sums and exponentials are fp32, taken relative to the row's maximum.
 * A logit of -inf bans its token: it counts as probability 0, and is not an
 * alternative.  Alternatives beyond the last token that is not banned have
 * top_index -1 and top_logprob -inf.  A row of banned tokens only has logprob
 * -inf and entropy 0.  A row with a NaN or +inf has NaN for logprob, entropy
 * and every top_logprob, and top_index -1.  A target outside 0..vocab-1 marks
 * a position without a token: logprob is 0 there, the rest as usual.
 *
 * logits, type  in  any sl_dtype; row r at logits + r * ld elements, aligned to
 *               the element size
 * ld            row stride in elements, >= vocab
 * targets       in  int64[rows], or NULL (then logprob must be NULL)
 * rows          0..2^31-1 (0: nothing is done); vocab 1..SL_MAX_VOCAB
 * n_top         0..SL_MAX_ALTERNATIVES
 * logprob       out float32[rows], or NULL
 * entropy       out float32[rows], or NULL
 * top_logprob   out float32[rows][n_top], or NULL if n_top is 0
 * top_index     out int32[rows][n_top], or NULL if n_top is 0
 * No output may overlap an input or another output.
 */
int64_t sl_token_logprobs_workspace(int64_t rows, int64_t vocab, int32_t type, int32_t n_top);
sl_status sl_token_logprobs(const void* logits, int32_t type, int64_t ld, const int64_t* targets, int64_t rows,
                            int64_t vocab, int32_t n_top, float* logprob, float* entropy, float* top_logprob,
                            int32_t* top_index, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSELOCO_OPS_H */
