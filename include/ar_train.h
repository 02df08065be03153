/*
 * ar_train.h -- the two ends of the data-parallel step around the all-reduce
 * of ar.h, on one GPU:
 *
 *   before it, the losses that make the gradients: the log-probability of a
 *   token under a policy, the clipped policy loss with a KL term and the
 *   preference loss over pairs of sequences, each with the gradient of the
 *   logits;
 *   the products of expert layers and their gradients, between the two;
 *   after it, the global norm of the reduced gradients, clipping by it, and
 *   updates of matrices orthogonalised by Newton-Schulz products.
 *
 * Same conventions as ar.h: status codes, data types, plain device pointers
 * owned by the caller, one cudaStream_t per call (NULL = legacy default
 * stream), every call asynchronous, argument errors returned before anything
 * is enqueued.  No call allocates device memory, keeps anything between calls
 * or needs a communicator; calls on different streams may overlap as long as
 * their outputs and workspaces differ.  Every call may be captured in a CUDA
 * graph.  Kernels are launched with programmatic dependent launch, as the
 * all-reduce's are (ar.h, "Launch order"): stream order holds.
 * Results do not depend on timing: there are no floating-point atomics, and a
 * call repeated on the same device gives the same bits.  (The one wait inside a
 * kernel, of a cluster's blocks for one another in the policy loss, is bounded to
 * about a second.  Where one ran out, the cluster's rows, of which there are at most
 * 32, would give NaN in gradient and log-probability, and so would the statistics.
 * AR_LATE_BLOCK=<rank> in the environment of the process lets that block of
 * every cluster give up its first wait, and the block of that number of the
 * products below give up at once: for tests.)
 *
 * Logits.  A matrix of `rows` tokens by `vocab` columns, AR_FLOAT32 or
 * AR_BFLOAT16; row t starts at logits + t * row_stride elements
 * (row_stride >= vocab).  Pointers need element alignment only.  All
 * arithmetic, statistics and sums are fp32; a bf16 gradient is rounded once, to
 * nearest even.  A logit of -infinity is a column of probability zero; a row
 * with no finite logit, with +infinity or with NaN gives NaN.
 * Targets.  rows indices of `target_bytes` (4 or 8) bytes each, signed.  An
 * index outside [0, vocab) is not followed: its row gives NaN.
 * Weights.  One fp32 per row, or NULL for 1.  A row of weight 0 is masked:
 * nothing else of that row is read, its log-probability is 0, its gradient is
 * 0 and it adds nothing to any sum, whatever its inputs hold (NaN included).
 */
#ifndef AR_TRAIN_H_
#define AR_TRAIN_H_

#include <stddef.h>

#include "ar.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest matrix of logits: rows and columns. */
#define AR_MAX_TOKENS ((size_t)1 << 28)
#define AR_MAX_VOCAB ((size_t)1 << 30)

/*
 * logprobs[t] = x[t, y_t] - log sum_j exp(x[t, j]), fp32, for each row.
 *   logprobs  device array of `rows` floats
 * rows == 0 is a no-op.  Errors: AR_ERR_INVALID_ARG (NULL or misaligned
 * pointer, vocab == 0, row_stride < vocab, enum), AR_ERR_UNSUPPORTED
 * (AR_INT32, or more than AR_MAX_TOKENS rows or AR_MAX_VOCAB columns),
 * AR_ERR_CUDA (launch failed).
 */
ar_status_t ar_token_logprobs(const void* logits, size_t rows, size_t vocab, size_t row_stride,
                              ar_dtype_t dtype, const void* targets, int target_bytes,
                              const float* weights, float* logprobs, void* stream);

/*
 * Clipped policy loss with a KL term, and the gradient of the logits.  With
 * lp the token's log-probability, r = exp(lp - old), d = ref - lp:
 *
 *   term  = -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
 *           + kl_coef (exp(d) - 1 - d)
 *   loss  = scale * sum_t w_t term_t
 *   dterm = -A r where the unclipped side is taken, else 0
 *           (clipped: A > 0 and r > 1 + clip_high, or A < 0 and r < 1 - clip_low),
 *           + kl_coef (1 - exp(d))
 *   grad[t, j] = scale w_t dterm_t ([j == y_t] - p[t, j]),  p = softmax of the row
 *
 *   old_logprobs, advantages   rows floats
 *   ref_logprobs  rows floats; NULL leaves the KL term out (kl_coef is then ignored);
 *                 with kl_coef == 0 it makes the statistic alone
 *   grad          rows by vocab, the logits' type, row stride grad_stride; may be
 *                 the logits themselves (same address and stride), any other
 *                 overlap with them is rejected
 *   logprobs      rows floats: lp (0 for masked rows)
 *   stats         4 floats: loss, scale * sum w (exp(d) - 1 - d),
 *                 scale * sum w [clipped], scale * sum w
 *   workspace     at least ar_policy_loss_workspace(rows) bytes, 16-byte aligned;
 *                 its contents on entry do not matter
 * rows == 0 writes zero stats.  Errors as for ar_token_logprobs;
 * AR_ERR_INVALID_ARG also for a NaN parameter, a negative clip bound, a
 * workspace that is too small or an overlap.
 */
size_t ar_policy_loss_workspace(size_t rows);
ar_status_t ar_policy_loss(const void* logits, size_t rows, size_t vocab, size_t row_stride,
                           ar_dtype_t dtype, const void* targets, int target_bytes,
                           const float* weights, const float* old_logprobs,
                           const float* advantages, const float* ref_logprobs, float clip_low,
                           float clip_high, float kl_coef, float scale, void* grad,
                           size_t grad_stride, float* logprobs, float* stats, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Preference loss over pairs of sequences, and the gradient of the logits.
 * Sequence k is rows [offsets[k], offsets[k+1]); sequences 2i and 2i + 1 are
 * the chosen and the rejected answer of pair i.  With R_k the sum over the
 * sequence's rows of w_t (lp_t - ref_t):
 *
 *   z_i  = beta (R_2i - R_2i+1)
 *   loss = scale * sum_i (1 - ls) softplus(-z_i) + ls softplus(z_i)
 *   grad[t, j] = scale dz_i (+-beta) w_t ([j == y_t] - p[t, j]),
 *                dz = ls sigmoid(z) - (1 - ls) sigmoid(-z), + for chosen rows
 *
 *   offsets       2 * pairs + 1 device indices of offset_bytes (4 or 8) bytes,
 *                 non-decreasing, in [0, rows] (values outside are clamped);
 *                 a sequence may be empty.  Rows of no sequence get
 *                 gradient 0
 *   ref_logprobs  rows floats; NULL: no reference (ref = 0)
 *   label_smoothing  ls, in [0, 1]
 *   loss          1 float
 *   margins       pairs floats: z
 *   workspace     at least ar_preference_loss_workspace(rows, pairs) bytes,
 *                 16-byte aligned
 * grad, logprobs, weights and errors as for ar_policy_loss.
 */
size_t ar_preference_loss_workspace(size_t rows, size_t pairs);
ar_status_t ar_preference_loss(const void* logits, size_t rows, size_t vocab, size_t row_stride,
                               ar_dtype_t dtype, const void* targets, int target_bytes,
                               const float* weights, const void* offsets, int offset_bytes,
                               size_t pairs, const float* ref_logprobs, float beta,
                               float label_smoothing, float scale, void* grad, size_t grad_stride,
                               float* logprobs, float* loss, float* margins, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Global norm of `ntensors` gradient tensors: norm = sqrt(sum of squares of
 * all elements), squares and sums in fp32 or wider (a square above the fp32
 * range makes the norm infinite).
 *   grads    host array of device pointers (element alignment)
 *   counts   host array of element counts (0 allowed; the pointer is then ignored)
 *   dtypes   host array: AR_FLOAT32 or AR_BFLOAT16 for each tensor
 *   norm     device float
 *   workspace  at least ar_grad_norm_workspace() bytes, 16-byte aligned
 * The host arrays are read during the call only.
 */
size_t ar_grad_norm_workspace(void);
ar_status_t ar_grad_norm(size_t ntensors, const void* const* grads, const size_t* counts,
                         const ar_dtype_t* dtypes, float* norm, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Clipping by the global norm: norm as above, coef = min(1, max_norm /
 * (norm + eps)), outs[i] = grads[i] * coef rounded once to the tensor's type.
 *   outs     host array of device pointers; outs[i] may equal grads[i], a part
 *            of it is rejected; an overlap with another tensor or output is the
 *            caller's error (it is not checked).  NULL: in place for all
 * With coef == 1 an output in place is left untouched.  An infinite norm
 * gives coef 0 and a NaN norm coef NaN, and the products follow (0 * infinity
 * is NaN).  max_norm and eps must be >= 0.
 */
ar_status_t ar_clip_grads(size_t ntensors, const void* const* grads, void* const* outs,
                          const size_t* counts, const ar_dtype_t* dtypes, float max_norm, float eps,
                          float* norm, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Products with the weights of each row's expert.  Rows are sorted by expert:
 * expert e has rows [offsets[e], offsets[e + 1]) of x and y.
 *
 *   y[t, f] = sum_k W_e[f, k] x[t, k]
 *
 *   x         rows by `in`, AR_BFLOAT16; row t at x + t * x_stride elements
 *             (x_stride >= in)
 *   weights   experts matrices of `out` by `in`, AR_BFLOAT16; element (e, f, k) at
 *             e * expert_stride + f * out_stride + k * in_stride elements.  One of
 *             out_stride and in_stride is 1, the other at least the contiguous
 *             side's length, and expert_stride at least a whole matrix
 *   offsets   experts + 1 device indices of offset_bytes (4 or 8) bytes.  Values
 *             outside [0, rows] are clamped, a smaller one than one before it
 *             counts as that; an expert may have no rows
 *   y         rows by `out`, y_dtype (AR_FLOAT32 or AR_BFLOAT16), row stride
 *             y_stride; no part of the inputs.  Rows of no expert (in front of
 *             offsets[0], behind offsets[experts]) are left as they are, or with
 *             zero_rest != 0 made 0; rows of x outside the experts' are not read
 *             into any result
 *   workspace 16-byte aligned, at least the sum of ar_expert_workspace() of x and
 *             of weights bytes: operands that are not 16-byte aligned, or whose
 *             strides are not whole 16 bytes, are laid out there first.  NULL when
 *             that is 0.  With ar_expert_parts_workspace() bytes more, where that is not 0, long
 *             sums that make few tiles are split into parts, which takes less time; they are
 *             added up in a fixed order, but another one than without
 * The same call gives the gradient of x: dx = ar_expert_product(dy, weights with
 * `in` and `out` and their strides exchanged).  Sums are fp32, rounded once.
 * (The tensor cores cut what an addition loses: 960 products lose up to 2e-6 of their sum.  fp32 results add
 * such runs up, rounded; of a bf16 result a sum over k products is short by about k * 2e-9 of it, an eighth
 * of a half step at 2^18.  For longer ones ask for fp32.  Where fp32 runs are added up, values below 2^-126 may
 * become 0.)
 * rows == 0 or out == 0 is a no-op; in == 0 gives zeros for the experts' rows.
 * Errors: AR_ERR_INVALID_ARG (NULL or misaligned pointer, strides, enum, workspace
 * too small, overlap of y with x or weights), AR_ERR_UNSUPPORTED (another data type, more than
 * AR_MAX_TOKENS rows, AR_MAX_EXPERTS experts, AR_MAX_FEATURES columns or 2^30 tiles
 * of 128 x 128), AR_ERR_CUDA.  Waits inside the kernel are bounded (two seconds);
 * what a block has not computed when one runs out is NaN.
 */
#define AR_MAX_EXPERTS 1024
#define AR_MAX_FEATURES ((size_t)1 << 24)

/* Workspace of an operand of `count` matrices of `rows` rows of `cols` contiguous
 * bf16 elements, with the rows and the matrices at these strides (elements). */
size_t ar_expert_workspace(const void* at, size_t cols, size_t rows, size_t count, size_t row_stride,
                           size_t matrix_stride);
/* What the products of these sizes can use besides; 0 where nothing is won.  of_weights: of the gradient of the
 * weights.  Asks the current device for its number of multiprocessors. */
size_t ar_expert_parts_workspace(size_t rows, size_t experts, size_t out, size_t in, int of_weights);
ar_status_t ar_expert_product(const void* x, size_t rows, size_t x_stride, const void* weights, size_t experts,
                              size_t out, size_t in, size_t expert_stride, size_t out_stride, size_t in_stride,
                              const void* offsets, int offset_bytes, void* y, size_t y_stride, ar_dtype_t y_dtype,
                              int zero_rest, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of the weights: dW_e[f, k] = sum over expert e's rows of dy[t, f] x[t, k],
 * 0 for an expert without rows; with accumulate != 0 added to what dW holds (of an expert that has rows; in fp32
 * what lies below 2^-126, of dW or of the sum, may become 0).
 *   dy        rows by `out`, x rows by `in`, AR_BFLOAT16
 *   dw        dw_dtype (AR_FLOAT32 or AR_BFLOAT16), laid out by its three strides as
 *             the weights are; no part of dy or x
 *   workspace the sum of ar_expert_workspace() of dy and of x, or more, as above
 * Everything else as for ar_expert_product.
 */
ar_status_t ar_expert_weight_gradient(const void* dy, size_t dy_stride, const void* x, size_t x_stride, size_t rows,
                                      size_t experts, size_t out, size_t in, const void* offsets, int offset_bytes,
                                      void* dw, size_t expert_stride, size_t out_stride, size_t in_stride,
                                      ar_dtype_t dw_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * Orthogonalised updates.  Stack i holds counts[i] matrices of rows[i] by cols[i],
 * contiguous, one behind the other.  For each matrix g:
 *
 *   m   <- beta m + g;  u = g + beta m with nesterov != 0, else m   (no momentum: u = g)
 *   X    = u / (|u| + eps)                                          (|u|: Frobenius norm)
 *   steps times, with (a, b, c) = coefficients:
 *          A = X X^T,  X <- a X + (b A + c A^2) X    (rows <= cols; else A = X^T X, from the right)
 *   out  = scale X
 *
 *   grads     host array of device pointers, AR_FLOAT32 or AR_BFLOAT16 by dtypes
 *   momentum  host array of device pointers, fp32, updated; NULL: no momentum
 *   outs      host array of device pointers, bf16.  outs[i] may be grads[i] where that is bf16; any
 *             other overlap of the tensors is the caller's error
 *   scales    host array of a factor for each stack, NULL: 1
 *   steps     1 to AR_MAX_ORTHOGONAL_STEPS
 *   workspace at least ar_orthogonalize_workspace() bytes, 16-byte aligned; its contents on
 *             entry do not matter
 * Momentum, norms and all sums are fp32; X, A and b A + c A^2 are held between the products in fp16 times
 * powers of two that follow from bounds of the singular values; the result is rounded once to bf16.  So a
 * direction whose singular value is s of the norm is known to about 3e-4 / (s sqrt(min(rows, cols))) of itself
 * (of 4096 matrices of 2 x 2 normal values 99% are off by less than 0.65% of their 2-norm, the worst by 7%): next to
 * nothing for a matrix of rank one in the directions that it lacks.  Elements whose squares are below fp32's
 * range do not count in the norm.
 * A matrix of zeros gives zeros; one whose norm is not finite (a square above the fp32 range makes
 * it infinite) gives NaN.  Empty stacks are left out.  Pointers need element alignment only.
 * The host arrays are read during the call only.  Errors: AR_ERR_INVALID_ARG (NULL or misaligned pointer, enum,
 * steps, a parameter that is not finite, eps < 0, coefficients under which the singular values of a matrix of
 * norm 1 exceed 10^6, workspace too small), AR_ERR_UNSUPPORTED (AR_INT32, a side above AR_MAX_SIDE, more than
 * AR_MAX_MATRICES matrices in a stack), AR_ERR_CUDA.  Waits inside the kernels are bounded (two seconds);
 * what a block has not computed when one runs out is NaN.
 */
#define AR_MAX_ORTHOGONAL_STEPS 16
#define AR_MAX_SIDE ((size_t)1 << 16)
#define AR_MAX_MATRICES ((size_t)1 << 12)

size_t ar_orthogonalize_workspace(size_t nstacks, const size_t* counts, const size_t* rows, const size_t* cols,
                                  int steps);
ar_status_t ar_orthogonalize(size_t nstacks, const void* const* grads, float* const* momentum, void* const* outs,
                             const size_t* counts, const size_t* rows, const size_t* cols, const ar_dtype_t* dtypes,
                             const float* scales, float beta, int nesterov, int steps, const float* coefficients,
                             float eps, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* AR_TRAIN_H_ */
