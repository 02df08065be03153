// ar_train_launch.h -- internal interface between the C ABI of the training
// operators (ar_train_api.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

#include "../../include/ar.h"
#include "../../include/ar_train.h"
#include "ar_launch.h"

namespace ar {

// One operator's logits matrix and its per-row arrays.
struct LogitsCall {
  const void* logits;
  void* grad;                      // NULL for log-probabilities alone
  size_t rows, vocab, row_stride, grad_stride;
  int dtype;                       // ar_dtype_t: fp32 or bf16
  const void* targets;
  int target_bytes;                // 4 or 8
  const float* weights;            // NULL: all 1
  float* logprobs;
  cudaStream_t stream;
  int sms;                         // multiprocessors of the device
};

struct PolicyCall {
  const float *old_logprobs, *advantages, *ref_logprobs;
  float lo, hi, kl_coef, scale;
  float* stats;
  void* workspace;
};

struct PreferenceCall {
  const void* offsets;
  int offset_bytes;
  size_t pairs;
  const float* ref_logprobs;
  float beta, label_smoothing, scale;
  float *loss, *margins;
  void* workspace;
};

// Most blocks of a kernel whose rows are strided over its blocks.
constexpr unsigned kMaxLossBlocks = 1216;

cudaError_t launch_logprobs(const LogitsCall& c);
cudaError_t launch_policy(const LogitsCall& c, const PolicyCall& p);
cudaError_t launch_preference(const LogitsCall& c, const PreferenceCall& p);
size_t policy_workspace(size_t rows);
size_t preference_workspace(size_t rows, size_t pairs);

// One call over many gradient tensors (host arrays, read during the call).
struct GradsCall {
  size_t ntensors;
  const void* const* grads;
  void* const* outs;               // NULL: in place
  const size_t* counts;
  const ar_dtype_t* dtypes;        // fp32 or bf16 each
  float max_norm, eps;
  float* norm;
  void* workspace;
  int sms;
  cudaStream_t stream;
};

cudaError_t launch_grad_norm(const GradsCall& c);
cudaError_t launch_clip_grads(const GradsCall& c);
size_t grad_norm_workspace();

// Rows of 16-bit elements: nz matrices of ny rows of nx elements (strides in elements).
struct ExpertMatrix {
  const void* at;
  size_t nx, ny, nz, y_stride, z_stride;
};

constexpr int kMaxExperts = AR_MAX_EXPERTS;

// One call of the expert products.
struct ExpertsCall {
  size_t rows, experts, in, out;
  ExpertMatrix x, dy;              // rows by in, rows by out (dy: of the weight gradient)
  ExpertMatrix w;                  // the weights, or the strides of their gradient: its contiguous side is nx
  bool w_in_contiguous;
  const void* offsets;
  int offset_bytes;
  void* y;                         // rows by out, or the weights' gradient
  size_t y_stride;
  int dtype;                       // of y: fp32 or bf16
  bool zero_rest, accumulate;
  void* workspace;
  size_t spare;                    // bytes of it behind the operands'
  int sms;
  cudaStream_t stream;
};

// One call of the orthogonalisation (host arrays, read during the call).
struct OrthogonalCall {
  size_t nstacks;
  const void* const* grads;
  float* const* momentum;          // NULL: none
  void* const* outs;
  const size_t *counts, *rows, *cols;
  const ar_dtype_t* dtypes;        // of the gradients: fp32 or bf16
  const float* scales;             // NULL: 1
  float beta;
  bool nesterov;
  int steps;
  float a, b, c, eps;
  void* workspace;
  int sms;
  cudaStream_t stream;
};

size_t orthogonal_workspace(const OrthogonalCall& c);
bool orthogonal_bounded(const OrthogonalCall& c);
cudaError_t launch_orthogonal(const OrthogonalCall& c);

size_t expert_matrix_workspace(const ExpertMatrix& m);
size_t expert_parts_workspace(const ExpertsCall& c, bool of_weights);  // of c its sizes and sms
cudaError_t launch_expert_product(const ExpertsCall& c);
cudaError_t launch_expert_weight_gradient(const ExpertsCall& c);

}  // namespace ar
