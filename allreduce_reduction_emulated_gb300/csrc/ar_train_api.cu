// ar_train_api.cu -- the C ABI of the training operators (declared in
// include/ar_train.h): argument checks and dispatch.  Host code only; the
// kernels live in ar_logits.cu and ar_clip.cu.  Nothing here allocates or throws.
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include <nvtx3/nvToolsExt.h>

#include "../../include/ar_train.h"
#include "ar_train_launch.h"

namespace {

// One NVTX range per call in the library's domain (a no-op unless a profiler
// is attached).
struct Range {
  explicit Range(const char* name) {
    static const nvtxDomainHandle_t d = nvtxDomainCreateA("allreduce_emulated");
    domain = d;
    nvtxEventAttributes_t a = {};
    a.version = NVTX_VERSION;
    a.size = NVTX_EVENT_ATTRIB_STRUCT_SIZE;
    a.messageType = NVTX_MESSAGE_TYPE_ASCII;
    a.message.ascii = name;
    nvtxDomainRangePushEx(domain, &a);
  }
  ~Range() { nvtxDomainRangePop(domain); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
  nvtxDomainHandle_t domain;
};

// AR_DEBUG=1: one line per call, as for the all-reduce
bool debug() {
  static const bool on = [] {
    const char* s = std::getenv("AR_DEBUG");
    return s && std::atoi(s) != 0;
  }();
  return on;
}

bool aligned(const void* p, size_t n) { return p && ((uintptr_t)p & (n - 1)) == 0; }
bool aligned_or_null(const void* p, size_t n) { return !p || aligned(p, n); }
bool index_bytes(int n) { return n == 4 || n == 8; }
bool nan(float x) { return !(x == x); }

ar_status_t finish(cudaError_t e, const char* what, size_t a, size_t b) {
  if (debug()) std::fprintf(stderr, "[ar] %s %zu x %zu status=%s\n", what, a, b, cudaGetErrorString(e));
  if (e == cudaSuccess) return AR_SUCCESS;
  cudaGetLastError();
  return AR_ERR_CUDA;
}

// Bytes from the first to past the last element of a matrix, or 0 when that
// does not fit an address.
size_t span(size_t rows, size_t vocab, size_t stride, size_t es) {
  const size_t most = (size_t)1 << 62;
  if (stride > most / es / rows) return 0;
  return ((rows - 1) * stride + vocab) * es;
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + bn && y < x + an;
}

// What every operator on logits checks; rows > 0.
ar_status_t check_logits(const ar::LogitsCall& c, bool grad) {
  if (c.dtype == AR_INT32) return AR_ERR_UNSUPPORTED;
  if (c.dtype != AR_FLOAT32 && c.dtype != AR_BFLOAT16) return AR_ERR_INVALID_ARG;
  if (!index_bytes(c.target_bytes)) return AR_ERR_INVALID_ARG;
  if (c.rows == 0) return AR_SUCCESS;
  if (c.rows > AR_MAX_TOKENS || c.vocab > AR_MAX_VOCAB) return AR_ERR_UNSUPPORTED;
  const size_t es = ar::elem_bytes(c.dtype);
  if (c.vocab == 0 || c.row_stride < c.vocab || !aligned(c.logits, es)) return AR_ERR_INVALID_ARG;
  if (!aligned(c.targets, (size_t)c.target_bytes) || !aligned(c.logprobs, 4) || !aligned_or_null(c.weights, 4))
    return AR_ERR_INVALID_ARG;
  const size_t in = span(c.rows, c.vocab, c.row_stride, es);
  if (!in) return AR_ERR_INVALID_ARG;
  if (!grad) return AR_SUCCESS;
  if (c.grad_stride < c.vocab || !aligned(c.grad, es)) return AR_ERR_INVALID_ARG;
  const size_t out = span(c.rows, c.vocab, c.grad_stride, es);
  if (!out) return AR_ERR_INVALID_ARG;
  const bool in_place = c.grad == c.logits && (c.grad_stride == c.row_stride || c.rows == 1);
  if (!in_place && overlap(c.logits, in, c.grad, out)) return AR_ERR_INVALID_ARG;
  return AR_SUCCESS;
}

ar_status_t check_grads(size_t n, const void* const* grads, void* const* outs, const size_t* counts,
                        const ar_dtype_t* dtypes) {
  if (n == 0) return AR_SUCCESS;
  if (!grads || !counts || !dtypes) return AR_ERR_INVALID_ARG;
  for (size_t i = 0; i < n; ++i) {
    if (dtypes[i] == AR_INT32) return AR_ERR_UNSUPPORTED;
    if (dtypes[i] != AR_FLOAT32 && dtypes[i] != AR_BFLOAT16) return AR_ERR_INVALID_ARG;
    if (counts[i] == 0) continue;
    const size_t es = ar::elem_bytes(dtypes[i]);
    if (counts[i] > ((size_t)1 << 62) / es || !aligned(grads[i], es)) return AR_ERR_INVALID_ARG;
    if (!outs) continue;
    if (!aligned(outs[i], es)) return AR_ERR_INVALID_ARG;
    if (outs[i] != grads[i] && overlap(grads[i], counts[i] * es, outs[i], counts[i] * es)) return AR_ERR_INVALID_ARG;
  }
  return AR_SUCCESS;
}

// Of the current device; asked once per device.
bool multiprocessors(int* sms) {
  static std::atomic<int> known[64];
  int dev = -1;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0) {
    if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return true;
    if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
      if (dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
      return true;
    }
  }
  cudaGetLastError();
  return false;
}

}  // namespace

extern "C" {

ar_status_t ar_token_logprobs(const void* logits, size_t rows, size_t vocab, size_t row_stride, ar_dtype_t dtype,
                              const void* targets, int target_bytes, const float* weights, float* logprobs,
                              void* stream) {
  ar::LogitsCall c{logits, nullptr, rows, vocab, row_stride, 0, (int)dtype, targets, target_bytes, weights,
                         logprobs, static_cast<cudaStream_t>(stream), 0};
  const ar_status_t st = check_logits(c, false);
  if (st != AR_SUCCESS || rows == 0) return st;
  if (!multiprocessors(&c.sms)) return AR_ERR_CUDA;
  Range range("ar_token_logprobs");
  return finish(ar::launch_logprobs(c), "token_logprobs", rows, vocab);
}

size_t ar_policy_loss_workspace(size_t rows) {
  return rows > (size_t)1 << 56 ? SIZE_MAX : ar::policy_workspace(rows);
}

ar_status_t ar_policy_loss(const void* logits, size_t rows, size_t vocab, size_t row_stride, ar_dtype_t dtype,
                           const void* targets, int target_bytes, const float* weights, const float* old_logprobs,
                           const float* advantages, const float* ref_logprobs, float clip_low, float clip_high,
                           float kl_coef, float scale, void* grad, size_t grad_stride, float* logprobs, float* stats,
                           void* workspace, size_t workspace_bytes, void* stream) {
  ar::LogitsCall c{logits, grad, rows, vocab, row_stride, grad_stride, (int)dtype, targets, target_bytes, weights,
                         logprobs, static_cast<cudaStream_t>(stream), 0};
  const ar_status_t st = check_logits(c, true);
  if (st != AR_SUCCESS) return st;
  if (!(clip_low >= 0.0f) || !(clip_high >= 0.0f) || nan(kl_coef) || nan(scale)) return AR_ERR_INVALID_ARG;
  if (!aligned(stats, 4) || !aligned(workspace, 16) || workspace_bytes < ar_policy_loss_workspace(rows))
    return AR_ERR_INVALID_ARG;
  if (rows && (!aligned(old_logprobs, 4) || !aligned(advantages, 4) || !aligned_or_null(ref_logprobs, 4)))
    return AR_ERR_INVALID_ARG;
  const ar::PolicyCall p{old_logprobs, advantages, ref_logprobs, (float)(1.0 - (double)clip_low),
                         (float)(1.0 + (double)clip_high), kl_coef, scale, stats, workspace};
  if (!multiprocessors(&c.sms)) return AR_ERR_CUDA;
  Range range("ar_policy_loss");
  return finish(ar::launch_policy(c, p), "policy_loss", rows, vocab);
}

size_t ar_preference_loss_workspace(size_t rows, size_t pairs) {
  const size_t most = (size_t)1 << 56;
  return rows > most || pairs > most ? SIZE_MAX : ar::preference_workspace(rows, pairs);
}

ar_status_t ar_preference_loss(const void* logits, size_t rows, size_t vocab, size_t row_stride, ar_dtype_t dtype,
                               const void* targets, int target_bytes, const float* weights, const void* offsets,
                               int offset_bytes, size_t pairs, const float* ref_logprobs, float beta,
                               float label_smoothing, float scale, void* grad, size_t grad_stride, float* logprobs,
                               float* loss, float* margins, void* workspace, size_t workspace_bytes, void* stream) {
  ar::LogitsCall c{logits, grad, rows, vocab, row_stride, grad_stride, (int)dtype, targets, target_bytes, weights,
                         logprobs, static_cast<cudaStream_t>(stream), 0};
  const ar_status_t st = check_logits(c, true);
  if (st != AR_SUCCESS) return st;
  if (nan(beta) || nan(scale) || !(label_smoothing >= 0.0f && label_smoothing <= 1.0f)) return AR_ERR_INVALID_ARG;
  if (!index_bytes(offset_bytes) || !aligned(loss, 4)) return AR_ERR_INVALID_ARG;
  if (pairs && (!aligned(offsets, (size_t)offset_bytes) || !aligned(margins, 4))) return AR_ERR_INVALID_ARG;
  if (rows && !aligned_or_null(ref_logprobs, 4)) return AR_ERR_INVALID_ARG;
  const size_t need = ar_preference_loss_workspace(rows, pairs);
  if (workspace_bytes < need || (need && !aligned(workspace, 16))) return AR_ERR_INVALID_ARG;
  const ar::PreferenceCall p{offsets, offset_bytes, pairs, ref_logprobs, beta, label_smoothing, scale, loss, margins,
                             workspace};
  if (!multiprocessors(&c.sms)) return AR_ERR_CUDA;
  Range range("ar_preference_loss");
  return finish(ar::launch_preference(c, p), "preference_loss", rows, vocab);
}

size_t ar_grad_norm_workspace(void) { return ar::grad_norm_workspace(); }

ar_status_t ar_grad_norm(size_t ntensors, const void* const* grads, const size_t* counts, const ar_dtype_t* dtypes,
                         float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  const ar_status_t st = check_grads(ntensors, grads, nullptr, counts, dtypes);
  if (st != AR_SUCCESS) return st;
  if (!aligned(norm, 4) || !aligned(workspace, 16) || workspace_bytes < ar_grad_norm_workspace())
    return AR_ERR_INVALID_ARG;
  ar::GradsCall c{ntensors, grads, nullptr, counts, dtypes, 0.0f, 0.0f, norm, workspace,
                  0, static_cast<cudaStream_t>(stream)};
  if (!multiprocessors(&c.sms)) return AR_ERR_CUDA;
  Range range("ar_grad_norm");
  return finish(ar::launch_grad_norm(c), "grad_norm", ntensors, 1);
}

ar_status_t ar_clip_grads(size_t ntensors, const void* const* grads, void* const* outs, const size_t* counts,
                          const ar_dtype_t* dtypes, float max_norm, float eps, float* norm, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const ar_status_t st = check_grads(ntensors, grads, outs, counts, dtypes);
  if (st != AR_SUCCESS) return st;
  if (!(max_norm >= 0.0f) || !(eps >= 0.0f)) return AR_ERR_INVALID_ARG;
  if (!aligned(norm, 4) || !aligned(workspace, 16) || workspace_bytes < ar_grad_norm_workspace())
    return AR_ERR_INVALID_ARG;
  ar::GradsCall c{ntensors, grads, outs, counts, dtypes, max_norm, eps, norm, workspace,
                  0, static_cast<cudaStream_t>(stream)};
  if (!multiprocessors(&c.sms)) return AR_ERR_CUDA;
  Range range("ar_clip_grads");
  return finish(ar::launch_clip_grads(c), "clip_grads", ntensors, 1);
}

}  // extern "C"
