/*
 * ar_train.h -- the two ends of the data-parallel step around the all-reduce
 * of ar.h, on one GPU:
 *
 *   before it, the losses that make the gradients: the log-probability of a
 *   token under a policy, the clipped policy loss with a KL term and the
 *   preference loss over pairs of sequences, each with the gradient of the
 *   logits;
 *   after it, the global norm of the reduced gradients and clipping by it.
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
 * every cluster give up its first wait: for tests.)
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

#ifdef __cplusplus
}
#endif

#endif /* AR_TRAIN_H_ */
