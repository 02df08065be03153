// ar_logits.cu -- kernels of the operators on a logits matrix (ar_train.h):
// token log-probabilities, the policy loss and the preference loss with the
// gradient of the logits.
//
// softmax statistics in one pass over a row: each thread keeps a running
// maximum m and the sum of e^(x - m), rescaled when m grows; a block joins the
// threads' pairs.
#include <algorithm>

#include "ar_logits.cuh"
#include "ar_train.h"
#include "ar_train_launch.h"

namespace ar {

namespace {

constexpr int kThreads = 256;

template <int DT>
struct Matrix {
  const typename ElemOf<DT>::T* logits;
  typename ElemOf<DT>::T* grad;
  unsigned long long rows, vocab, stride, grad_stride;
  const void* targets;
  int target_bytes;
  const float* weights;
  float* logprobs;

  explicit Matrix(const LogitsCall& c)
      : logits(static_cast<const typename ElemOf<DT>::T*>(c.logits)),
        grad(static_cast<typename ElemOf<DT>::T*>(c.grad)),
        rows(c.rows), vocab(c.vocab), stride(c.row_stride), grad_stride(c.grad_stride), targets(c.targets),
        target_bytes(c.target_bytes), weights(c.weights), logprobs(c.logprobs) {}
};

template <int DT>
__device__ __forceinline__ MaxSum row_stats(const typename ElemOf<DT>::T* row, long long vocab, float2* sh) {
  const Slots<DT> in(row, vocab);
  MaxSum a;
  const long long n = in.count();
  for (long long s = threadIdx.x; s < n; s += kThreads) {
    float x[Lanes<DT>::N];
    in.load(s, x, -INFINITY);
    a.add(x);
  }
  return block_join<kThreads>(a, sh);
}

// grad[j] = c * ([j == y] - p[j]).  The target's 1 - p is -expm1(log p).
template <int DT>
__device__ __forceinline__ void row_grad(const typename ElemOf<DT>::T* row, typename ElemOf<DT>::T* grad,
                                         long long vocab, long long y, float lp, MaxSum st, float c) {
  constexpr int N = Lanes<DT>::N;
  const Slots<DT> in(row, vocab);
  const bool same = (((uintptr_t)row ^ (uintptr_t)grad) & 15) == 0;
  const float f = -c / st.s;
  const long long n = in.count();
  for (long long s = threadIdx.x; s < n; s += kThreads) {
    float x[N];
    in.load(s, x, -INFINITY);
    const long long j = in.first(s);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = j + i == y ? -c * expm1f(lp) : f * exp_diff(x[i], st.m);
    store_slot<DT>(in, grad, same, s, x);
  }
}

template <int DT>
__device__ __forceinline__ void row_zero(typename ElemOf<DT>::T* grad, long long vocab) {
  const Slots<DT> out(grad, vocab);
  const long long n = out.count();
  const float zero[Lanes<DT>::N] = {};
  for (long long s = threadIdx.x; s < n; s += kThreads) store_slot<DT>(out, grad, true, s, zero);
}

// ----------------------------------------------------------- log-probabilities

// stats != NULL: {m, s} of every row for the gradient that follows
template <int DT>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const Matrix<DT> a, float2* stats) {
  pdl_enter();
  __shared__ float2 sh[kThreads / 32];
  for (unsigned long long t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const float w = a.weights ? a.weights[t] : 1.0f;
    if (w == 0.0f) {
      if (threadIdx.x == 0) a.logprobs[t] = 0.0f;
      continue;
    }
    const typename ElemOf<DT>::T* row = a.logits + t * a.stride;
    const MaxSum st = row_stats<DT>(row, (long long)a.vocab, sh);
    if (threadIdx.x == 0) {
      const long long y = load_index(a.targets, a.target_bytes, t);
      a.logprobs[t] = target_logprob(row, (long long)a.vocab, y, st.m, st.s);
      if (stats) stats[t] = make_float2(st.m, st.s);
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------- policy loss

template <int DT>
__global__ void __launch_bounds__(kThreads) policy_kernel(const Matrix<DT> a, const PolicyParams p, float4* partial) {
  pdl_enter();
  __shared__ float2 sh[kThreads / 32];
  __shared__ float sh_c[2];
  PolicySums sum;
  for (unsigned long long t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const float w = a.weights ? a.weights[t] : 1.0f;
    typename ElemOf<DT>::T* grad = a.grad + t * a.grad_stride;
    if (w == 0.0f) {
      row_zero<DT>(grad, (long long)a.vocab);
      if (threadIdx.x == 0) a.logprobs[t] = 0.0f;
      continue;
    }
    const typename ElemOf<DT>::T* row = a.logits + t * a.stride;
    const long long y = load_index(a.targets, a.target_bytes, t);
    const MaxSum st = row_stats<DT>(row, (long long)a.vocab, sh);
    if (threadIdx.x == 0) {
      const float lp = target_logprob(row, (long long)a.vocab, y, st.m, st.s);
      a.logprobs[t] = lp;
      sh_c[0] = policy_token(p, t, w, lp, sum);
      sh_c[1] = lp;
    }
    __syncthreads();  // also: the target's logit is read before an in-place gradient is written
    row_grad<DT>(row, grad, (long long)a.vocab, y, sh_c[1], st, sh_c[0]);
    __syncthreads();
  }
  if (threadIdx.x == 0) partial[blockIdx.x] = make_float4(sum.loss, sum.kl, sum.clipped, sum.weight);
}

// The blocks' sums in a fixed order.
__global__ void __launch_bounds__(kThreads) policy_sum_kernel(const float4* partial, int n, float scale, float* stats) {
  pdl_enter();
  __shared__ float sh[4][kThreads / 32];
  float v[4] = {};
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float4 q = partial[i];
    v[0] += q.x; v[1] += q.y; v[2] += q.z; v[3] += q.w;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float r = block_sum<kThreads>(v[k], sh[k]);
    if (threadIdx.x == 0) stats[k] = scale * r;
  }
}

// ------------------------------------------------------------ preference loss

struct PairParams {
  const void* offsets;
  int offset_bytes;
  unsigned long long pairs, rows;
  const float* weights;
  const float* logprobs;
  const float* ref_logprobs;
  float beta, ls, scale;
  float* margins;
  float* pair_loss;  // pairs
  float* side;       // 2 * pairs: d(loss)/d(R_k)
  float* loss;
};

__device__ __forceinline__ unsigned long long offset_at(const PairParams& p, unsigned long long k) {
  const long long v = load_index(p.offsets, p.offset_bytes, k);
  return v < 0 ? 0ull : min((unsigned long long)v, p.rows);
}

// One block per pair: the two sequences' sums, the pair's loss and the two
// factors of the gradient.
__global__ void __launch_bounds__(kThreads) pair_kernel(const PairParams p) {
  pdl_enter();
  __shared__ float sh[2][kThreads / 32];
  for (unsigned long long i = blockIdx.x; i < p.pairs; i += gridDim.x) {
    float R[2];
    for (int k = 0; k < 2; ++k) {
      const unsigned long long b = offset_at(p, 2 * i + k), e = offset_at(p, 2 * i + k + 1);
      float v = 0.0f;
      for (unsigned long long t = b + threadIdx.x; t < e; t += kThreads) {
        const float w = p.weights ? p.weights[t] : 1.0f;
        if (w != 0.0f) v += w * (p.ref_logprobs ? p.logprobs[t] - p.ref_logprobs[t] : p.logprobs[t]);
      }
      R[k] = block_sum<kThreads>(v, sh[k]);
    }
    if (threadIdx.x == 0) {
      const float z = p.beta * (R[0] - R[1]);
      // softplus(-z) = max(-z, 0) + log1p(e^-|z|); softplus(z) = softplus(-z) + z
      const float e = expf(-fabsf(z));
      const float sp = fmaxf(-z, 0.0f) + log1pf(e);
      p.margins[i] = z;
      p.pair_loss[i] = z != z ? z : (1.0f - p.ls) * sp + p.ls * (sp + z);
      // sigmoid(-z) and sigmoid(z), the smaller one without cancellation
      const float small = e / (1.0f + e), big = 1.0f / (1.0f + e);
      const float neg = z >= 0.0f ? small : big, pos = z >= 0.0f ? big : small;
      const float dz = z != z ? z : p.ls * pos - (1.0f - p.ls) * neg;
      p.side[2 * i] = p.scale * p.beta * dz;
      p.side[2 * i + 1] = -p.scale * p.beta * dz;
    }
    __syncthreads();
  }
}

// The sequence of row t (offsets are non-decreasing): the last k with
// offsets[k] <= t, or -1 when t lies in none.
__device__ __forceinline__ long long sequence_of(const PairParams& p, unsigned long long t) {
  unsigned long long lo = 0, hi = 2 * p.pairs + 1;  // offsets[lo] <= t < offsets[hi]
  if (hi == 1 || offset_at(p, 0) > t) return -1;
  while (hi - lo > 1) {
    const unsigned long long mid = (lo + hi) / 2;
    if (offset_at(p, mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo < 2 * p.pairs ? (long long)lo : -1;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) preference_grad_kernel(const Matrix<DT> a, const PairParams p,
                                                                   const float2* stats) {
  pdl_enter();
  __shared__ float sh[kThreads / 32];
  if (blockIdx.x == 0) {
    float v = 0.0f;
    for (unsigned long long i = threadIdx.x; i < p.pairs; i += kThreads) v += p.pair_loss[i];
    v = block_sum<kThreads>(v, sh);
    if (threadIdx.x == 0) *p.loss = p.scale * v;
  }
  for (unsigned long long t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const float w = a.weights ? a.weights[t] : 1.0f;
    typename ElemOf<DT>::T* grad = a.grad + t * a.grad_stride;
    const long long k = w == 0.0f ? -1 : sequence_of(p, t);
    if (k < 0) {
      row_zero<DT>(grad, (long long)a.vocab);
      continue;
    }
    MaxSum st;
    st.m = stats[t].x;
    st.s = stats[t].y;
    row_grad<DT>(a.logits + t * a.stride, grad, (long long)a.vocab, load_index(a.targets, a.target_bytes, t),
                 a.logprobs[t], st, w * p.side[k]);
  }
}

inline unsigned grid_of(unsigned long long work, unsigned most) {
  return (unsigned)std::max(1ull, std::min<unsigned long long>(work, most));
}

template <int DT>
cudaError_t run_logprobs(const LogitsCall& c) {
  return launch_kernel(logprob_kernel<DT>, grid_of(c.rows, kMaxLossBlocks), kThreads, 0, c.stream, true,
                       Matrix<DT>(c), (float2*)nullptr);
}

template <int DT>
cudaError_t run_policy(const LogitsCall& c, const PolicyParams& p, float* stats, float4* partial) {
  const unsigned grid = grid_of(c.rows, kMaxLossBlocks);
  cudaError_t e = launch_kernel(policy_kernel<DT>, grid, kThreads, 0, c.stream, true, Matrix<DT>(c), p, partial);
  if (e == cudaSuccess)
    e = launch_kernel(policy_sum_kernel, 1, kThreads, 0, c.stream, true, (const float4*)partial, (int)grid, p.scale,
                      stats);
  return e;
}

template <int DT>
cudaError_t run_preference(const LogitsCall& c, const PairParams& p, float2* stats) {
  cudaError_t e = cudaSuccess;
  if (c.rows)
    e = launch_kernel(logprob_kernel<DT>, grid_of(c.rows, kMaxLossBlocks), kThreads, 0, c.stream, true, Matrix<DT>(c),
                      stats);
  if (e == cudaSuccess && p.pairs)
    e = launch_kernel(pair_kernel, grid_of(p.pairs, kMaxLossBlocks), kThreads, 0, c.stream, true, p);
  if (e == cudaSuccess)
    e = launch_kernel(preference_grad_kernel<DT>, grid_of(c.rows, kMaxLossBlocks), kThreads, 0, c.stream, true,
                      Matrix<DT>(c), p, (const float2*)stats);
  return e;
}

}  // namespace

cudaError_t launch_logprobs(const LogitsCall& c) {
  return c.dtype == kF32 ? run_logprobs<kF32>(c) : run_logprobs<kBF16>(c);
}

cudaError_t launch_policy(const LogitsCall& c, const PolicyCall& q) {
  const PolicyParams p{q.old_logprobs, q.advantages, q.ref_logprobs, q.lo, q.hi, q.kl_coef, q.scale};
  float4* partial = static_cast<float4*>(q.workspace);
  return c.dtype == kF32 ? run_policy<kF32>(c, p, q.stats, partial) : run_policy<kBF16>(c, p, q.stats, partial);
}

// workspace: {m, s} per row, then the pairs' losses and the sequences' factors
size_t preference_workspace(size_t rows, size_t pairs) { return rows * sizeof(float2) + 3 * pairs * sizeof(float); }

cudaError_t launch_preference(const LogitsCall& c, const PreferenceCall& q) {
  float2* stats = static_cast<float2*>(q.workspace);
  float* pair_loss = reinterpret_cast<float*>(stats + c.rows);
  const PairParams p{q.offsets, q.offset_bytes, q.pairs, c.rows, c.weights, c.logprobs, q.ref_logprobs,
                     q.beta, q.label_smoothing, q.scale, q.margins, pair_loss, pair_loss + q.pairs, q.loss};
  return c.dtype == kF32 ? run_preference<kF32>(c, p, stats) : run_preference<kBF16>(c, p, stats);
}

}  // namespace ar
