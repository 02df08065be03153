// ar_clip.cu -- the global norm over many gradient tensors and clipping by it
// (ar_train.h).
//
// norm = sqrt(sum g^2), out = g * min(1, max_norm / (norm + eps)).
// The tensors are cut into chunks of kChunkSlots 16-byte slots, numbered over
// all tensors, so that the blocks get equal work whatever the tensors' sizes:
// block b takes chunks b, b + grid, ...  Each block leaves one partial sum of
// squares; the clipping kernel's blocks each add all partials, in the same
// order and in fp64, and scale their chunks.  No atomics: the bits of the
// norm depend on the sizes and the device alone.
// The clipping kernel takes the chunks from the last to the first, so that it
// starts with the data that the norm kernel has left in L2.
#include <algorithm>

#include "ar_logits.cuh"
#include "ar_train.h"
#include "ar_train_launch.h"

namespace ar {

namespace {

constexpr int kThreads = 256;
constexpr int kSlotsPerThread = 8;
constexpr int kChunkSlots = kThreads * kSlotsPerThread;  // 32 KiB
constexpr int kBlocksPerSm = 8;
constexpr int kMaxPartials = 8192;
constexpr int kSmallTable = 64, kLargeTable = 1000;      // tensors per launch (kernel parameters: 32 bytes each)

struct Tensor {
  const void* grad;
  void* out;                  // NULL in the norm kernel
  unsigned long long count;
  unsigned int first_chunk;   // of this launch
  int dtype;
};

template <int CAP>
struct Table {
  Tensor t[CAP];
  int n;
  unsigned int chunks;
};

// tensor of a chunk: the last one whose first chunk is not after it
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& tab, unsigned int chunk) {
  int lo = 0, hi = tab.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.t[mid].first_chunk <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// f(slot, whole, x) for this thread's slots of a chunk; partial slots are
// filled with zeros.  All loads of a full chunk are issued before the first use.
template <int DT, class F>
__device__ __forceinline__ void for_chunk(const Tensor& t, unsigned int chunk, F&& f) {
  constexpr int N = Lanes<DT>::N;
  const Slots<DT> in(static_cast<const typename ElemOf<DT>::T*>(t.grad), (long long)t.count);
  const long long s0 = (long long)(chunk - t.first_chunk) * kChunkSlots;
  const long long n = in.count();
  if (in.whole(s0) && s0 + kChunkSlots <= n && in.whole(s0 + kChunkSlots - 1)) {
    uint4 r[kSlotsPerThread];
    const uint4* p = reinterpret_cast<const uint4*>(in.row + in.first(s0)) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kSlotsPerThread; ++k) r[k] = ld_row(p + k * kThreads);
#pragma unroll
    for (int k = 0; k < kSlotsPerThread; ++k) {
      const Acc<DT> a = widen<DT>(r[k]);
      f(in, s0 + threadIdx.x + k * kThreads, a.v);
    }
  } else {
    const long long e = min(n, s0 + kChunkSlots);
    for (long long s = s0 + threadIdx.x; s < e; s += kThreads) {
      float x[N];
      in.load(s, x, 0.0f);
      f(in, s, x);
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) square_sum_kernel(const __grid_constant__ Table<CAP> tab, float* partial) {
  pdl_enter();
  __shared__ float sh[kThreads / 32];
  float acc[4] = {};
  for (unsigned int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const Tensor& t = tab.t[tensor_of(tab, c)];
    const auto add = [&](const auto&, long long, const auto& x) {
      constexpr int N = sizeof(x) / sizeof(float);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i & 3] = fmaf(x[i], x[i], acc[i & 3]);
    };
    if (t.dtype == kF32) for_chunk<kF32>(t, c, add);
    else for_chunk<kBF16>(t, c, add);
  }
  const float v = block_sum<kThreads>((acc[0] + acc[1]) + (acc[2] + acc[3]), sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// The norm from the partial sums, the same in every block.
__device__ __forceinline__ float norm_of(const float* partial, int nparts, double* sh) {
  double v = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) v += (double)partial[i];
  return (float)sqrt(block_sum<kThreads>(v, sh));
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const float* partial, int nparts, float* norm) {
  pdl_enter();
  __shared__ double sh[kThreads / 32];
  const float v = norm_of(partial, nparts, sh);
  if (threadIdx.x == 0) *norm = v;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<CAP> tab, const float* partial,
                                                         int nparts, float max_norm, float eps, float* norm) {
  pdl_enter();
  __shared__ double sh[kThreads / 32];
  const float v = norm_of(partial, nparts, sh);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  const float q = max_norm / (v + eps);
  const float coef = q > 1.0f ? 1.0f : q;  // NaN stays NaN
  for (unsigned int b = blockIdx.x; b < tab.chunks; b += gridDim.x) {
    const unsigned int c = tab.chunks - 1 - b;
    const Tensor& t = tab.t[tensor_of(tab, c)];
    if (coef == 1.0f && t.out == t.grad) continue;
    const bool same = (((uintptr_t)t.grad ^ (uintptr_t)t.out) & 15) == 0;
    const auto scale = [&](const auto& in, long long s, const auto& x) {
      constexpr int N = sizeof(x) / sizeof(float);
      constexpr int DT = N == Lanes<kF32>::N ? kF32 : kBF16;
      float y[N];
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = x[i] * coef;
      store_slot<DT>(in, static_cast<typename ElemOf<DT>::T*>(t.out), same, s, y);
    };
    if (t.dtype == kF32) for_chunk<kF32>(t, c, scale);
    else for_chunk<kBF16>(t, c, scale);
  }
}

template <int CAP>
size_t fill(const GradsCall& c, size_t i, bool outs, Table<CAP>& tab) {
  unsigned long long chunks = 0;
  tab.n = 0;
  for (; i < c.ntensors && tab.n < CAP; ++i) {
    if (c.counts[i] == 0) continue;
    const size_t es = elem_bytes(c.dtypes[i]), lead = ((uintptr_t)c.grads[i] & 15) / es;
    const unsigned long long slots = (c.counts[i] + lead + 16 / es - 1) / (16 / es);
    const unsigned long long n = (slots + kChunkSlots - 1) / kChunkSlots;
    if (chunks + n > 0xffffffffull) break;
    tab.t[tab.n++] = Tensor{c.grads[i], !outs ? nullptr : c.outs ? c.outs[i] : const_cast<void*>(c.grads[i]),
                            c.counts[i], (unsigned int)chunks, c.dtypes[i]};
    chunks += n;
  }
  tab.chunks = (unsigned int)chunks;
  return i;
}

template <int CAP>
cudaError_t run(const GradsCall& c, bool clip) {
  float* partial = static_cast<float*>(c.workspace);
  const size_t launches = std::max<size_t>(1, (c.ntensors + CAP - 1) / CAP);
  if (launches > (size_t)kMaxPartials) return cudaErrorInvalidValue;
  const unsigned most = std::max(1u, std::min<unsigned>(c.sms * kBlocksPerSm, kMaxPartials / (unsigned)launches));
  Table<CAP> tab;
  int nparts = 0;
  for (size_t i = 0; i < c.ntensors;) {
    const size_t next = fill(c, i, false, tab);
    if (tab.chunks) {
      const unsigned grid = std::min(tab.chunks, most);
      if (nparts + (int)grid > kMaxPartials) return cudaErrorInvalidValue;
      const cudaError_t e = launch_kernel(square_sum_kernel<CAP>, grid, kThreads, 0, c.stream, true, tab,
                                          partial + nparts);
      if (e != cudaSuccess) return e;
      nparts += (int)grid;
    } else if (next == i) {
      return cudaErrorInvalidValue;
    }
    i = next;
  }
  if (!clip || nparts == 0)
    return launch_kernel(norm_kernel, 1, kThreads, 0, c.stream, true, (const float*)partial, nparts, c.norm);
  for (size_t i = 0; i < c.ntensors;) {
    const size_t next = fill(c, i, true, tab);
    if (tab.chunks) {
      const cudaError_t e = launch_kernel(scale_kernel<CAP>, std::min(tab.chunks, most), kThreads, 0, c.stream, true,
                                          tab, (const float*)partial, nparts, c.max_norm, c.eps, c.norm);
      if (e != cudaSuccess) return e;
    }
    i = next;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_norm_workspace() { return kMaxPartials * sizeof(float); }

cudaError_t launch_grad_norm(const GradsCall& c) {
  return c.ntensors <= kSmallTable ? run<kSmallTable>(c, false) : run<kLargeTable>(c, false);
}

cudaError_t launch_clip_grads(const GradsCall& c) {
  return c.ntensors <= kSmallTable ? run<kSmallTable>(c, true) : run<kLargeTable>(c, true);
}

}  // namespace ar
