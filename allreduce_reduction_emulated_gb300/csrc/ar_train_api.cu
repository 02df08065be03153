// ar_train_api.cu -- the C ABI of the training operators (declared in
// include/ar_train.h): argument checks and dispatch.  Host code only; the
// kernels live in ar_logits.cu, ar_clip.cu, ar_experts.cu and ar_orthogonal.cu.
// Nothing here allocates or throws.
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
bool finite(float x) { return x - x == 0.0f; }

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

// A matrix of 16-bit rows that a product reads: element alignment, rows at least as far apart as they are long.
ar_status_t check_rows(const ar::ExpertMatrix& m) {
  if (!m.nx || !m.ny || !m.nz) return AR_SUCCESS;
  if (!aligned(m.at, 2) || (m.ny > 1 && m.y_stride < m.nx)) return AR_ERR_INVALID_ARG;
  return span(m.ny, m.nx, m.ny > 1 ? m.y_stride : m.nx, 2) ? AR_SUCCESS : AR_ERR_INVALID_ARG;
}

// Bytes from the first to past the last element of matrices of any size above 0.
size_t span_of(const ar::ExpertMatrix& m, size_t es) {
  return ((m.nz - 1) * m.z_stride + (m.ny - 1) * m.y_stride + m.nx) * es;
}

// Whether two matrices of `rows` > 0 rows share memory; columns and strides in bytes.  Columns of one
// wider matrix do not.
bool rows_overlap(const void* a, size_t a_cols, size_t a_stride, const void* b, size_t b_cols, size_t b_stride, size_t rows) {
  if (!overlap(a, (rows - 1) * a_stride + a_cols, b, (rows - 1) * b_stride + b_cols)) return false;
  if (a_stride != b_stride) return true;
  const bool behind = (uintptr_t)b > (uintptr_t)a;
  const size_t way = (behind ? (uintptr_t)b - (uintptr_t)a : (uintptr_t)a - (uintptr_t)b) % a_stride;
  return behind ? way < a_cols || way + b_cols > a_stride : way < b_cols || way + a_cols > a_stride;
}

// Sizes, offsets, the layout of the weights (or of their gradient) and the workspace of the expert products.
// Fills in c.w and c.w_in_contiguous.
ar_status_t check_experts(ar::ExpertsCall& c, const void* w, size_t es, size_t expert_stride, size_t out_stride,
                          size_t in_stride) {
  if (c.dtype == AR_INT32) return AR_ERR_UNSUPPORTED;
  if (c.dtype != AR_FLOAT32 && c.dtype != AR_BFLOAT16) return AR_ERR_INVALID_ARG;
  if (!index_bytes(c.offset_bytes)) return AR_ERR_INVALID_ARG;
  if (c.rows > AR_MAX_TOKENS || c.experts > AR_MAX_EXPERTS || c.in > AR_MAX_FEATURES || c.out > AR_MAX_FEATURES)
    return AR_ERR_UNSUPPORTED;
  if (!aligned(c.offsets, (size_t)c.offset_bytes)) return AR_ERR_INVALID_ARG;
  if (!c.experts || !c.in || !c.out) return AR_SUCCESS;
  const size_t most = (size_t)1 << 40;
  c.w_in_contiguous = in_stride == 1 && (out_stride >= c.in || c.out == 1);
  if (!c.w_in_contiguous && !(out_stride == 1 && (in_stride >= c.out || c.in == 1))) return AR_ERR_INVALID_ARG;
  size_t nx = c.in, ny = c.out, pitch = out_stride;
  if (!c.w_in_contiguous) nx = c.out, ny = c.in, pitch = in_stride;
  if (ny == 1) pitch = nx;
  if (pitch > most || expert_stride > most || !aligned(w, es)) return AR_ERR_INVALID_ARG;
  if (c.experts > 1 && expert_stride < (ny - 1) * pitch + nx) return AR_ERR_INVALID_ARG;
  c.w = ar::ExpertMatrix{w, nx, ny, c.experts, pitch, expert_stride};
  return AR_SUCCESS;
}

bool too_many_tiles(size_t a, size_t b, size_t n) {
  const double tiles = ((double)a / 128 + 1) * ((double)b / 128 + (double)n);
  return tiles > (double)(1 << 30);
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

size_t ar_expert_workspace(const void* at, size_t cols, size_t rows, size_t count, size_t row_stride,
                           size_t matrix_stride) {
  const size_t most = (size_t)1 << 40;
  if (cols > AR_MAX_FEATURES || rows > AR_MAX_TOKENS || count > AR_MAX_EXPERTS || row_stride > most ||
      matrix_stride > most)
    return SIZE_MAX;
  return ar::expert_matrix_workspace(ar::ExpertMatrix{at, cols, rows, count, row_stride, matrix_stride});
}

size_t ar_expert_parts_workspace(size_t rows, size_t experts, size_t out, size_t in, int of_weights) {
  if (rows > AR_MAX_TOKENS || experts > AR_MAX_EXPERTS || in > AR_MAX_FEATURES || out > AR_MAX_FEATURES) return SIZE_MAX;
  ar::ExpertsCall c = {};
  c.rows = rows, c.experts = experts, c.in = in, c.out = out;
  if (!rows || !experts || !in || !out || !multiprocessors(&c.sms)) return 0;
  return ar::expert_parts_workspace(c, of_weights != 0);
}

ar_status_t ar_expert_product(const void* x, size_t rows, size_t x_stride, const void* weights, size_t experts,
                              size_t out, size_t in, size_t expert_stride, size_t out_stride, size_t in_stride,
                              const void* offsets, int offset_bytes, void* y, size_t y_stride, ar_dtype_t y_dtype,
                              int zero_rest, void* workspace, size_t workspace_bytes, void* stream) {
  ar::ExpertsCall c = {};
  c.rows = rows, c.experts = experts, c.in = in, c.out = out;
  c.offsets = offsets, c.offset_bytes = offset_bytes;
  c.x = ar::ExpertMatrix{x, in, rows, 1, rows > 1 ? x_stride : in, 0};
  c.y = y, c.y_stride = rows > 1 ? y_stride : out, c.dtype = (int)y_dtype;
  c.zero_rest = zero_rest != 0;
  c.workspace = workspace, c.stream = static_cast<cudaStream_t>(stream);
  if (too_many_tiles(out, rows, experts + 2)) return AR_ERR_UNSUPPORTED;
  ar_status_t st = check_experts(c, weights, 2, expert_stride, out_stride, in_stride);
  if (st == AR_SUCCESS) st = check_rows(c.x);
  if (st != AR_SUCCESS) return st;
  if (rows == 0 || out == 0) return AR_SUCCESS;
  const size_t es = ar::elem_bytes(c.dtype);
  const size_t there = c.y_stride < out ? 0 : span(rows, out, c.y_stride, es);
  if (!aligned(y, es) || !there) return AR_ERR_INVALID_ARG;
  if (in && rows_overlap(x, in * 2, c.x.y_stride * 2, y, out * es, c.y_stride * es, rows)) return AR_ERR_INVALID_ARG;
  if (in && experts && overlap(weights, span_of(c.w, 2), y, there)) return AR_ERR_INVALID_ARG;
  const size_t need = ar::expert_matrix_workspace(c.x) + ar::expert_matrix_workspace(c.w);
  if (workspace_bytes < need || (need && !aligned(workspace, 16))) return AR_ERR_INVALID_ARG;
  c.spare = aligned(workspace, 16) ? workspace_bytes - need : 0;
  if (!multiprocessors(&c.sms)) return AR_ERR_CUDA;
  Range range("ar_expert_product");
  return finish(ar::launch_expert_product(c), "expert_product", rows, out);
}

ar_status_t ar_expert_weight_gradient(const void* dy, size_t dy_stride, const void* x, size_t x_stride, size_t rows,
                                      size_t experts, size_t out, size_t in, const void* offsets, int offset_bytes,
                                      void* dw, size_t expert_stride, size_t out_stride, size_t in_stride,
                                      ar_dtype_t dw_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  ar::ExpertsCall c = {};
  c.rows = rows, c.experts = experts, c.in = in, c.out = out;
  c.offsets = offsets, c.offset_bytes = offset_bytes;
  c.x = ar::ExpertMatrix{x, in, rows, 1, rows > 1 ? x_stride : in, 0};
  c.dy = ar::ExpertMatrix{dy, out, rows, 1, rows > 1 ? dy_stride : out, 0};
  c.y = dw, c.dtype = (int)dw_dtype;
  c.accumulate = accumulate != 0;
  c.workspace = workspace, c.stream = static_cast<cudaStream_t>(stream);
  ar_status_t st = check_experts(c, dw, ar::elem_bytes(c.dtype), expert_stride, out_stride, in_stride);
  if (st == AR_SUCCESS) st = check_rows(c.x);
  if (st == AR_SUCCESS) st = check_rows(c.dy);
  if (st != AR_SUCCESS) return st;
  if ((double)experts * ((double)in / 128 + 1) * ((double)out / 128 + 1) > (double)(1 << 30)) return AR_ERR_UNSUPPORTED;
  if (experts == 0 || in == 0 || out == 0) return AR_SUCCESS;
  const size_t there = span_of(c.w, ar::elem_bytes(c.dtype));
  if (rows && (overlap(x, span_of(c.x, 2), dw, there) || overlap(dy, span_of(c.dy, 2), dw, there)))
    return AR_ERR_INVALID_ARG;
  const size_t need = ar::expert_matrix_workspace(c.x) + ar::expert_matrix_workspace(c.dy);
  if (workspace_bytes < need || (need && !aligned(workspace, 16))) return AR_ERR_INVALID_ARG;
  c.spare = aligned(workspace, 16) ? workspace_bytes - need : 0;
  if (!multiprocessors(&c.sms)) return AR_ERR_CUDA;
  Range range("ar_expert_weight_gradient");
  return finish(ar::launch_expert_weight_gradient(c), "expert_weight_gradient", out, in);
}

size_t ar_orthogonalize_workspace(size_t nstacks, const size_t* counts, const size_t* rows, const size_t* cols,
                                  int steps) {
  if (nstacks && (!counts || !rows || !cols)) return SIZE_MAX;
  for (size_t i = 0; i < nstacks; ++i)
    if (counts[i] > AR_MAX_MATRICES || rows[i] > AR_MAX_SIDE || cols[i] > AR_MAX_SIDE) return SIZE_MAX;
  if (steps < 1 || steps > AR_MAX_ORTHOGONAL_STEPS) return SIZE_MAX;
  ar::OrthogonalCall c = {};
  c.nstacks = nstacks, c.counts = counts, c.rows = rows, c.cols = cols, c.steps = steps;
  return ar::orthogonal_workspace(c);
}

ar_status_t ar_orthogonalize(size_t nstacks, const void* const* grads, float* const* momentum, void* const* outs,
                             const size_t* counts, const size_t* rows, const size_t* cols, const ar_dtype_t* dtypes,
                             const float* scales, float beta, int nesterov, int steps, const float* coefficients,
                             float eps, void* workspace, size_t workspace_bytes, void* stream) {
  if (!coefficients || steps < 1 || steps > AR_MAX_ORTHOGONAL_STEPS) return AR_ERR_INVALID_ARG;
  if (!finite(beta) || !finite(eps) || eps < 0.0f) return AR_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (!finite(coefficients[i])) return AR_ERR_INVALID_ARG;
  if (nstacks && (!grads || !outs || !counts || !rows || !cols || !dtypes)) return AR_ERR_INVALID_ARG;
  for (size_t i = 0; i < nstacks; ++i) {
    if (dtypes[i] == AR_INT32) return AR_ERR_UNSUPPORTED;
    if (dtypes[i] != AR_FLOAT32 && dtypes[i] != AR_BFLOAT16) return AR_ERR_INVALID_ARG;
    if (counts[i] > AR_MAX_MATRICES || rows[i] > AR_MAX_SIDE || cols[i] > AR_MAX_SIDE) return AR_ERR_UNSUPPORTED;
    if (scales && !finite(scales[i])) return AR_ERR_INVALID_ARG;
    if (!counts[i] || !rows[i] || !cols[i]) continue;
    if (!aligned(grads[i], ar::elem_bytes(dtypes[i])) || !aligned(outs[i], 2)) return AR_ERR_INVALID_ARG;
    if (momentum && !aligned(momentum[i], 4)) return AR_ERR_INVALID_ARG;
  }
  ar::OrthogonalCall c = {nstacks, grads, momentum, outs, counts, rows, cols, dtypes, scales, beta, nesterov != 0,
                          steps, coefficients[0], coefficients[1], coefficients[2], eps, workspace, 0,
                          static_cast<cudaStream_t>(stream)};
  if (!ar::orthogonal_bounded(c)) return AR_ERR_INVALID_ARG;
  const size_t need = ar::orthogonal_workspace(c);
  if (workspace_bytes < need || (need && !aligned(workspace, 16))) return AR_ERR_INVALID_ARG;
  if (!multiprocessors(&c.sms)) return AR_ERR_CUDA;
  Range range("ar_orthogonalize");
  return finish(ar::launch_orthogonal(c), "orthogonalize", nstacks, (size_t)steps);
}

}  // extern "C"
