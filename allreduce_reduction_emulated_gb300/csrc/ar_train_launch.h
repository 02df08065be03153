// ar_train_launch.h -- internal interface between the C ABI of the training
// operators (ar_train_api.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

#include "../../include/ar.h"
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

}  // namespace ar
