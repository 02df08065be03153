// ar_clip.cu -- the global norm over many gradient tensors and clipping by it
// (ar_train.h).
//
// norm = sqrt(sum g^2), out = g * min(1, max_norm / (norm + eps)).
// The tensors are cut into chunks of 32 KiB, numbered over all tensors, and every
// block takes the same number of runs of consecutive chunks, whatever the tensors'
// sizes.  Each block leaves one partial sum of squares; the clipping kernel's blocks
// each add all partials, in the same order, and scale their chunks; with many chunks
// one block adds them and blocks of half a chunk scale.  No atomics: the bits of the
// norm depend on the sizes and the device alone.
//
// Bound by HBM: the coefficient needs every element, so a gradient that does not
// stay in L2 (129 MB) is read twice and written once.  The clipping kernel takes
// the chunks from the last to the first, so that it starts with what the norm
// kernel has left in L2.
#include <algorithm>

#include "ar_logits.cuh"
#include "ar_train.h"
#include "ar_train_launch.h"

namespace ar {

namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 8;                            // 16-byte slots per thread in a chunk, all loaded before any is used
// Blocks per SM: with eight 16-byte loads on the way per thread, four are resident.
constexpr int kBlocksPerSm = 4;
constexpr int kMaxBlocks = 640;                      // of one launch
constexpr int kMaxPartials = 8192;
constexpr int kSmallTable = 64, kLargeTable = 768;   // tensors per launch
// Chunks in a run: a block that walks through consecutive chunks looks its tensor
// up once, but 608 blocks in 608 far places of 5 GB are slower than all blocks in
// one moving window (2608 against 2365 us).
constexpr unsigned int kRun = 16;

// What L2 does with a load's lines.  Up to kHintChunks (512 MB) the norm kernel asks
// L2 to keep the last kKeptChunks (40 MB; the two halves of L2 may each hold a copy)
// and to drop the rest first, and the clipping kernel, which begins with the kept
// ones, drops them as it goes: 160 MB read and written 38.5 -> 34.9 us, 480 MB 118 ->
// 112.  (In place with coefficient 1 it reads nothing.  The next kernel's first pass over
// 20 to 120 MB then takes up to 3 us longer than behind a plain sum, its second none.)  Above, nothing is gained and a hint of any kind costs 2% (9.7 GB: 2152 us
// without, 2190 with), so the kernels come without them too.
constexpr unsigned int kHintChunks = 16384, kKeptChunks = 1250;

struct Tensor {
  const void* grad;
  void* out;                  // NULL in the norm kernel
  unsigned long long count;
  unsigned int first_chunk;   // of this launch
  int dtype;
};

// In the kernel's parameters (at most 26 KiB of the 32 they may have): nothing to
// copy to the device first, and a captured call keeps its own.
template <int CAP>
struct Table {
  Tensor t[CAP];
  unsigned short start[kMaxBlocks];  // tensor of the first chunk of each block's first run
  unsigned int chunks, rounds;       // of this launch
  unsigned int kept;                 // chunks at the end that L2 is to keep for the clipping kernel (0: no hints)
  int n;
};

// The launch's chunks are cut into `rounds` equal windows, each window into one
// run of consecutive chunks for every block.
struct Run {
  unsigned int begin, end;
};
__host__ __device__ __forceinline__ Run run_of(unsigned int chunks, unsigned int rounds, unsigned int round,
                                               unsigned int block, unsigned int blocks) {
  const unsigned long long a = (unsigned long long)chunks * round / rounds;
  const unsigned long long n = (unsigned long long)chunks * (round + 1) / rounds - a;
  return Run{(unsigned int)(a + n * block / blocks), (unsigned int)(a + n * (block + 1) / blocks)};
}

// The tensor of a chunk: the last whose first chunk is not after it.
__device__ __forceinline__ int tensor_of(const unsigned int* first, int n, unsigned int chunk) {
  int lo = 0;
  for (int hi = n; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// f(tensor, chunk) for this block's chunks; with BACKWARDS they are numbered, and
// gone through, from the last.
template <bool BACKWARDS, int CAP, class F>
__device__ __forceinline__ void for_chunks(const Table<CAP>& tab, F&& f) {
  __shared__ unsigned int first[CAP];
  if (tab.rounds > 1) {  // a second run has its tensor to find
    for (int i = threadIdx.x; i < tab.n; i += kThreads) first[i] = tab.t[i].first_chunk;
    __syncthreads();
  }
  int i = tab.start[blockIdx.x];
  for (unsigned int round = 0; round < tab.rounds; ++round) {
    const Run r = run_of(tab.chunks, tab.rounds, round, blockIdx.x, gridDim.x);
    if (r.begin == r.end) continue;
    if (round) i = tensor_of(first, tab.n, BACKWARDS ? tab.chunks - 1 - r.begin : r.begin);
    for (unsigned int k = r.begin; k < r.end; ++k) {
      const unsigned int c = BACKWARDS ? tab.chunks - 1 - k : k;
      if (BACKWARDS) {
        while (tab.t[i].first_chunk > c) --i;
      } else {
        while (i + 1 < tab.n && tab.t[i + 1].first_chunk <= c) ++i;
      }
      f(tab.t[i], c);
    }
  }
}

// This thread's slots of one chunk of a tensor.  The chunks lie on 128-byte lines,
// so a tensor may begin up to 127 bytes into its first one.  All whole slots are
// loaded (zeros for the others) before any is used; a partial slot, where the
// tensor begins or ends inside it, by elements.
template <int DT, int K = kSlots>
struct Chunk {
  static constexpr int N = Lanes<DT>::N;
  using E = typename ElemOf<DT>::T;
  const E* run;               // the tensor
  long long count, s0;        // its elements; the chunk's first slot
  int lead;                   // elements of its first line before it
  int lo, lim;                // slots lo .. lim - 1 of the chunk are whole
  int ends[2];                // partial slots: the first, the last (-1: none; the same one only once)
  uint4 r[K];

  // part: which K of a chunk's kSlots slots per thread
  template <bool HINTS>
  __device__ __forceinline__ void load(const Tensor& t, unsigned int chunk, uint64_t policy, int part = 0) {
    run = static_cast<const E*>(t.grad);
    count = (long long)t.count;
    s0 = (long long)(chunk - t.first_chunk) * (kSlots * kThreads) + part * (K * kThreads);
    lead = (int)(((uintptr_t)run & 127) / sizeof(E));
    const long long full = (count + lead) / N - s0;
    lo = s0 == 0 ? (lead + N - 1) / N : 0;
    lim = (int)min((long long)(K * kThreads), full);
    ends[0] = s0 == 0 && lead % N ? lead / N : -1;
    ends[1] = (count + lead) % N && full >= lo && full < K * kThreads ? (int)full : -1;
    const uint4* src = reinterpret_cast<const uint4*>(run - lead) + s0 + threadIdx.x;
    if (lo == 0 && lim == K * kThreads) {
#pragma unroll
      for (int k = 0; k < K; ++k) r[k] = ld_hint<HINTS>(src + k * kThreads, policy);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int q = k * kThreads + (int)threadIdx.x;
        r[k] = make_uint4(0, 0, 0, 0);
        if (q >= lo && q < lim) r[k] = ld_hint<HINTS>(src + k * kThreads, policy);
      }
    }
  }
  __device__ __forceinline__ long long element(int slot) const { return (s0 + slot) * N - lead; }
  // f(first index, values) for a partial slot of this thread; zeros outside the tensor
  template <class F>
  __device__ __forceinline__ void partial_slots(F&& f) const {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (ends[e] >= 0 && ends[e] % kThreads == (int)threadIdx.x) {
        const long long j = element(ends[e]);
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = j + i >= 0 && j + i < count ? to_float(run[j + i]) : 0.0f;
        f(j, x);
      }
  }
};

// A thread's sum of squares: four accumulators of 8 or 16 squares each per chunk, then
// a compensated sum over the chunks.  (Four accumulators over all chunks add up to
// thousands of squares each, and where these are alike the roundings all go one way:
// the norm of 1.2G equal values was off by 1.4e-5.)
struct Squares {
  Carried sum;
  template <int DT, bool HINTS>
  __device__ __forceinline__ void add(const Tensor& t, unsigned int chunk, uint64_t policy) {
    float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    Chunk<DT> c;
    c.template load<HINTS>(t, chunk, policy);
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const Acc<DT> x = widen<DT>(c.r[k]);
#pragma unroll
      for (int i = 0; i < Lanes<DT>::N; i += 2) {
        const float2 v = make_float2(x.v[i], x.v[i + 1]);
        acc[i >> 1 & 1] = fma2(v, v, acc[i >> 1 & 1]);
      }
    }
    c.partial_slots([&](long long, const auto& x) {
#pragma unroll
      for (int i = 0; i < Lanes<DT>::N; ++i) acc[0].x = fmaf(x[i], x[i], acc[0].x);
    });
    sum.add((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y));
  }
};

template <int CAP, bool HINTS>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
square_sum_kernel(const __grid_constant__ Table<CAP> tab, float* partial) {
  pdl_enter();
  __shared__ float sh[kThreads / 32];
  Squares squares;
  const uint64_t keep = keep_policy(true), rest = keep_policy(false);
  for_chunks<false>(tab, [&](const Tensor& t, unsigned int c) {
    const uint64_t policy = tab.chunks - c <= tab.kept ? keep : rest;
    if (t.dtype == kF32) squares.add<kF32, HINTS>(t, c, policy);
    else squares.add<kBF16, HINTS>(t, c, policy);
  });
  const float v = block_sum<kThreads>(squares.sum.value(), sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// The norm from the partial sums, the same in every block.  In fp32: at most 32
// sums per thread, then a tree (fp64 additions and the fp64 root took 3 us of
// every block's start).
__device__ __forceinline__ float norm_of(const float* partial, int nparts, float* sh) {
  float v = 0.0f;
  for (int i = threadIdx.x; i < nparts; i += kThreads) v += partial[i];
  return sqrtf(block_sum<kThreads>(v, sh));
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const float* partial, int nparts, float* norm) {
  pdl_enter();
  __shared__ float sh[kThreads / 32];
  const float v = norm_of(partial, nparts, sh);
  if (threadIdx.x == 0) *norm = v;
}

template <int DT, bool HINTS, int K>
__device__ __forceinline__ void scale_chunk(const Tensor& t, unsigned int chunk, float coef, uint64_t policy, int part = 0) {
  constexpr int N = Lanes<DT>::N;
  using E = typename ElemOf<DT>::T;
  Chunk<DT, K> c;
  c.template load<HINTS>(t, chunk, policy, part);
  E* const out = static_cast<E*>(t.out);
  const bool same = (((uintptr_t)t.grad ^ (uintptr_t)t.out) & 15) == 0;
  const float2 f = make_float2(coef, coef);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int q = k * kThreads + (int)threadIdx.x;
    if (q >= c.lo && q < c.lim) {
      Acc<DT> y = widen<DT>(c.r[k]);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 v = mul2(make_float2(y.v[i], y.v[i + 1]), f);
        y.v[i] = v.x;
        y.v[i + 1] = v.y;
      }
      E* to = out + c.element(q);
      const uint4 v = narrow<DT>(y, 1.0f, false);
      if (same) st_stream(reinterpret_cast<uint4*>(to), v);
      else store_apart(to, v, warp_within(q, c.lo, c.lim));
    }
  }
  c.partial_slots([&](long long j, const auto& x) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (j + i >= 0 && j + i < c.count) from_float(out + j + i, x[i] * coef);
  });
}

template <int CAP, bool HINTS>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
scale_kernel(const __grid_constant__ Table<CAP> tab, const float* partial, int nparts, float max_norm, float eps,
             float* norm) {
  pdl_enter();
  __shared__ float sh[kThreads / 32];
  const float v = norm_of(partial, nparts, sh);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  const float q = max_norm / (v + eps);
  const float coef = q > 1.0f ? 1.0f : q;  // NaN stays NaN
  const uint64_t policy = keep_policy(false);
  for_chunks<true>(tab, [&](const Tensor& t, unsigned int c) {
    if (coef == 1.0f && t.out == t.grad) return;  // in place and nothing to scale
    if (t.dtype == kF32) scale_chunk<kF32, HINTS, kSlots>(t, c, coef, policy);
    else scale_chunk<kBF16, HINTS, kSlots>(t, c, coef, policy);
  });
}

// The same from kPieceChunks (46 MB) on, after a kernel that joins the partial sums:
// a block takes half a chunk and is gone, and the reads and writes of blocks that come
// and go overlap better than those of resident ones (9.7 GB: 2191 -> 2034 us; 96 MB
// 19.0 -> 17.5; 76 MB 17.0, the other way 17.6).
constexpr unsigned long long kPieceChunks = 1400;
template <int CAP, bool HINTS>
__global__ void __launch_bounds__(kThreads, 6)
scale_piece_kernel(const __grid_constant__ Table<CAP> tab, const float* norm, float max_norm, float eps) {
  pdl_enter();
  const float q = max_norm / (*norm + eps);
  const float coef = q > 1.0f ? 1.0f : q;  // NaN stays NaN
  const unsigned int c = tab.chunks - 1 - blockIdx.x / 2;
  int i = 0;
  for (int hi = tab.n; hi - i > 1;) {
    const int mid = (i + hi) >> 1;
    if (tab.t[mid].first_chunk <= c) i = mid;
    else hi = mid;
  }
  const Tensor& t = tab.t[i];
  if (coef == 1.0f && t.out == t.grad) return;  // in place and nothing to scale
  const uint64_t policy = keep_policy(false);
  const int part = 1 - (int)(blockIdx.x & 1);
  if (t.dtype == kF32) scale_chunk<kF32, HINTS, kSlots / 2>(t, c, coef, policy, part);
  else scale_chunk<kBF16, HINTS, kSlots / 2>(t, c, coef, policy, part);
}

// Tensors from i on until the table is full; returns the first that is not in it.
template <int CAP>
size_t fill(const GradsCall& c, size_t i, bool clip, Table<CAP>& tab) {
  unsigned long long chunks = 0;
  tab.n = 0;
  for (; i < c.ntensors && tab.n < CAP; ++i) {
    if (c.counts[i] == 0) continue;
    // chunks of 32 KiB from the 128-byte line that the tensor begins in
    const unsigned long long bytes = ((uintptr_t)c.grads[i] & 127) + c.counts[i] * elem_bytes(c.dtypes[i]);
    const unsigned long long n = (bytes + kSlots * kThreads * 16 - 1) / (kSlots * kThreads * 16);
    if (chunks + n > 0x3fffffffull) break;
    tab.t[tab.n++] = Tensor{c.grads[i], !clip ? nullptr : c.outs ? c.outs[i] : const_cast<void*>(c.grads[i]),
                            c.counts[i], (unsigned int)chunks, c.dtypes[i]};
    chunks += n;
  }
  tab.chunks = (unsigned int)chunks;
  tab.kept = 0;
  return i;
}

// Runs of about kRun chunks; the tensors that the blocks start with.  Returns the
// number of blocks.
template <int CAP>
unsigned plan_runs(Table<CAP>& tab, unsigned most, bool backwards) {
  const unsigned blocks = std::min(most, tab.chunks);
  tab.rounds = (unsigned)(((unsigned long long)tab.chunks + blocks * kRun - 1) / (blocks * kRun));
  int i = backwards ? tab.n - 1 : 0;
  for (unsigned b = 0; b < blocks; ++b) {
    const unsigned k = run_of(tab.chunks, tab.rounds, 0, b, blocks).begin, c = backwards ? tab.chunks - 1 - k : k;
    if (backwards) {
      while (tab.t[i].first_chunk > c) --i;
    } else {
      while (i + 1 < tab.n && tab.t[i + 1].first_chunk <= c) ++i;
    }
    tab.start[b] = (unsigned short)i;
  }
  return blocks;
}

template <int CAP>
cudaError_t run(const GradsCall& c, bool clip) {
  float* partial = static_cast<float*>(c.workspace);
  const size_t launches = std::max<size_t>(1, (c.ntensors + CAP - 1) / CAP);
  if (launches > (size_t)kMaxPartials) return cudaErrorInvalidValue;
  const unsigned most = std::max(1u, std::min<unsigned>(std::min(c.sms * kBlocksPerSm, kMaxBlocks),
                                                        kMaxPartials / (unsigned)launches));
  Table<CAP> tab;
  int nparts = 0;
  unsigned long long all_chunks = 0;
  bool pieces = false;
  for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
    for (size_t i = 0; i < c.ntensors;) {
      const size_t next = fill(c, i, pass == 1, tab);
      if (tab.chunks) {
        const unsigned grid = plan_runs(tab, most, pass == 1);
        if (pass == 0) all_chunks += tab.chunks;
        if (clip && launches == 1 && tab.chunks <= kHintChunks) tab.kept = std::min(tab.chunks, kKeptChunks);
        cudaError_t e;
        if (pass == 0) {
          if (nparts + (int)grid > kMaxPartials) return cudaErrorInvalidValue;
          e = launch_kernel(tab.kept ? square_sum_kernel<CAP, true> : square_sum_kernel<CAP, false>, grid, kThreads, 0,
                            c.stream, true, tab, partial + nparts);
          nparts += (int)grid;
        } else if (pieces) {
          e = launch_kernel(tab.kept ? scale_piece_kernel<CAP, true> : scale_piece_kernel<CAP, false>, 2 * tab.chunks,
                            kThreads, 0, c.stream, true, tab, (const float*)c.norm, c.max_norm, c.eps);
        } else {
          e = launch_kernel(tab.kept ? scale_kernel<CAP, true> : scale_kernel<CAP, false>, grid, kThreads, 0, c.stream,
                            true, tab, (const float*)partial, nparts, c.max_norm, c.eps, c.norm);
        }
        if (e != cudaSuccess) return e;
      } else if (next == i) {
        return cudaErrorInvalidValue;
      }
      i = next;
    }
    pieces = all_chunks >= kPieceChunks;
    if (pass == 0 && (!clip || pieces || nparts == 0)) {
      const cudaError_t e = launch_kernel(norm_kernel, 1, kThreads, 0, c.stream, true, (const float*)partial, nparts,
                                          c.norm);
      if (e != cudaSuccess || !clip || nparts == 0) return e;
    }
  }
  return cudaSuccess;
}

cudaError_t dispatch(const GradsCall& c, bool clip) {
  return c.ntensors <= kSmallTable ? run<kSmallTable>(c, clip) : run<kLargeTable>(c, clip);
}

}  // namespace

size_t grad_norm_workspace() { return kMaxPartials * sizeof(float); }
cudaError_t launch_grad_norm(const GradsCall& c) { return dispatch(c, false); }
cudaError_t launch_clip_grads(const GradsCall& c) { return dispatch(c, true); }

}  // namespace ar
