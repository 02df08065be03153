// ar_logits.cu -- kernels of the operators on a logits matrix (ar_train.h):
// token log-probabilities, the policy loss and the preference loss with the
// gradient of the logits.
//
// With M the largest logit of a row and S the sum of e^(x - M), the target's
// log-probability is (x_y - M) - log S and p_j = e^(x_j - M) / S.  Every kernel takes
// them in one pass: a running maximum and a sum that is rescaled when it grows, in
// fp32, joined over threads, warps, blocks and clusters.  All of them are bound by
// HBM where the matrix is large (a row is 8 to 600 KB); the policy loss keeps the row on
// the chip between the sum and the gradient, so it reads and writes the matrix once.
// Comments give times on one GB300 (152 SMs; a copy reaches 6.79 TB/s).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdlib>

#include "ar_logits.cuh"
#include "ar_train.h"
#include "ar_train_launch.h"

namespace ar {

namespace {

constexpr int kThreads = 256;
constexpr size_t kMaxPolicySums = 65536;

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

// grad[j] = c * ([j == y] - p[j]).  The target's 1 - p is -expm1(log p).
template <int DT>
__device__ __forceinline__ void row_grad(const typename ElemOf<DT>::T* row, typename ElemOf<DT>::T* grad,
                                         long long vocab, long long y, float lp, float m, float sum, float c) {
  constexpr int N = Lanes<DT>::N;
  const Slots<DT> in(row, vocab);
  const bool same = (((uintptr_t)row ^ (uintptr_t)grad) & 15) == 0;
  const float f = -c / sum;
  const long long n = in.count();
  for (long long s = threadIdx.x; s < n; s += kThreads) {
    float x[N];
    in.load(s, x, -INFINITY);
    const long long j = in.first(s);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = j + i == y ? -c * expm1f(lp) : f * exp_diff(x[i], m);
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

template <int DT>
__device__ __forceinline__ float max_of(uint4 r) {
  const Acc<DT> a = widen<DT>(r);
  float m = a.v[0];
#pragma unroll
  for (int i = 1; i < Lanes<DT>::N; ++i) m = fmaxf(m, a.v[i]);
  return m;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));  // a NaN yields to the other operand
  return r;
}

template <int DT, int K>
__device__ __forceinline__ float max_of(const uint4 (&r)[K]) {
  if constexpr (DT == kBF16) {
    uint32_t m = max_bf16x2(max_bf16x2(r[0].x, r[0].y), max_bf16x2(r[0].z, r[0].w));
#pragma unroll
    for (int k = 1; k < K; ++k)
      m = max_bf16x2(m, max_bf16x2(max_bf16x2(r[k].x, r[k].y), max_bf16x2(r[k].z, r[k].w)));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  } else {
    float m = max_of<DT>(r[0]);
#pragma unroll
    for (int k = 1; k < K; ++k) m = fmaxf(m, max_of<DT>(r[k]));
    return m;
  }
}

// e^(x - m) of a pair.  The difference is formed first (for most logits it is
// exact, and 0 at the maximum), then scaled: a multiply-add would save half an
// instruction per element, but round the largest terms, and lowest * log2(e) is
// -infinity.
__device__ __forceinline__ float2 exp_pair(float x, float y, float2 minus_m) {
  float2 z = mul2(add2(make_float2(x, y), minus_m), make_float2(kLog2e, kLog2e));
  z.x = ex2(z.x);
  z.y = ex2(z.y);
  return z;
}

__device__ __forceinline__ float2 minus(float2 a) { return make_float2(-a.x, -a.y); }

__device__ __forceinline__ uint4 no_logits(int dtype) {  // a slot of -infinity
  const uint32_t v = dtype == kBF16 ? 0xff80ff80u : 0xff800000u;
  return make_uint4(v, v, v, v);
}

// A row's slice in one block, all the same in every thread.  The row's slots are
// counted from the 128-byte line in which it begins: a warp's 512 bytes then lie on four
// lines, not on parts of five (policy losses, counted from the row's first 16 bytes: 2489 x
// 50000 bf16 99 us, now 94; 1111 x 50001 fp32 79, now 75; rows of whole lines 639, now 644).
// Slots lo .. lim - 1 of the slice lie wholly in the row; slot `head` (or none, -1) holds
// its first elements behind others, slot `tail` (or none) its last `left` elements.
template <int DT>
struct Slice {
  static constexpr int N = Lanes<DT>::N;
  const typename ElemOf<DT>::T* row;
  int lead, lo, lim, head, tail, left;
  __device__ __forceinline__ Slice(const typename ElemOf<DT>::T* r, int V, int s0, int per) : row(r) {
    lead = (int)(((uintptr_t)r & 127) / sizeof(*r));
    const int full = (V + lead) / N - s0;
    left = (V + lead) % N;
    head = s0 == 0 && lead % N ? lead / N : -1;
    lo = s0 == 0 ? (lead + N - 1) / N : 0;
    lim = min(per, full);
    tail = left && full >= lo && full < per ? full : -1;
  }
};

// -------------------------------------------------------------- one row's sum

// The lanes' pairs (m, rest), each (1 + rest) e^m, as one; in every lane.
__device__ __forceinline__ float2 warp_rest(float2 v) {
  const float M = warp_max(v.x);
  const int first = __ffs(__ballot_sync(~0u, v.x == M)) - 1;  // its 1 is the pair's, all the others are rest
  const float part = (int)(threadIdx.x & 31) == first ? v.y : (1.0f + v.y) * exp_diff(v.x, M);
  return make_float2(M, warp_sum(part));
}

// The same over a block of kThreads.  `sh` holds a pair per warp; the block must
// synchronize before it is written again.
__device__ __forceinline__ float2 block_rest(float2 v, float2* sh) {
  const int lane = threadIdx.x & 31;
  v = warp_rest(v);
  if (lane == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_rest(lane < kThreads / 32 ? sh[lane] : make_float2(-FLT_MAX, -1.0f));
}

// One thread's share of a slice, by GROUP threads: the pair (m, rest) that stands for
// (1 + rest) e^m.  One pass with a running maximum, four slots on the way while four are
// worked on.
template <int DT, int GROUP, bool HINTS>
__device__ __forceinline__ float2 row_part(const Slice<DT>& in, int V, int s0, int tid, uint64_t policy) {
  constexpr int N = Lanes<DT>::N, U = 4;
  const uint4* src = reinterpret_cast<const uint4*>(in.row - in.lead) + s0 + tid;
  const auto load = [&](int at, uint4 (&r)[U]) {
    if (at + U * GROUP <= in.lim && at >= in.lo) {
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = ld_hint<HINTS>(src + at + u * GROUP, policy);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = at + u * GROUP + tid;
        r[u] = no_logits(DT);
        if (q >= in.lo && q < in.lim) r[u] = ld_hint<HINTS>(src + at + u * GROUP, policy);
      }
    }
  };
  float m = -FLT_MAX;                              // never -infinity: differences from it have to exist
  float2 s2 = make_float2(0.0f, 0.0f), lost = s2;
  const auto grow = [&](float top) {
    const float to = fmaxf(m, top), f = exp_diff(m, to);
    s2 = mul2(s2, make_float2(f, f));
    lost = mul2(lost, make_float2(f, f));
    m = to;
  };
  uint4 r[U], next[U] = {};
  load(0, r);
  // the row's ends by elements
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int q = e == 0 ? in.head : in.tail;
    if (q >= 0 && q % GROUP == tid) {
      const int j = (s0 + q) * N - in.lead;
      float v[N], top = -INFINITY;
#pragma unroll
      for (int x = 0; x < N; ++x) v[x] = j + x >= 0 && j + x < V ? to_float(in.row[j + x]) : -INFINITY;
#pragma unroll
      for (int x = 0; x < N; ++x) top = fmaxf(top, v[x]);
      grow(top);
#pragma unroll
      for (int x = 0; x < N; ++x) s2.x += exp_diff(v[x], m);
    }
  }
  for (int at = 0; at < in.lim; at += U * GROUP) {
    if (at + U * GROUP < in.lim) load(at + U * GROUP, next);
    grow(max_of<DT>(r));
    const float2 minus_m = make_float2(-m, -m);
    float2 part[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Acc<DT> x = widen<DT>(r[u]);
      part[u] = exp_pair(x.v[0], x.v[1], minus_m);
#pragma unroll
      for (int c = 2; c < N; c += 2) part[u] = add2(part[u], exp_pair(x.v[c], x.v[c + 1], minus_m));
      r[u] = next[u];
    }
    // where the maximum is among the terms, every addition to its 1 rounds: four slots are added up first, and what
    // that addition loses, of the larger or of the smaller, is carried over to the next
    const float2 add = add2(add2(add2(part[0], part[1]), add2(part[2], part[3])), lost);
    const float2 sum = add2(s2, add), had = add2(sum, minus(add));
    lost = add2(add2(s2, minus(had)), add2(add, minus(add2(sum, minus(had)))));
    s2 = sum;
  }
  // for a near-certain token the sum is 1 and a little, and the little is its log-probability
  const bool swap = s2.y > s2.x;                   // not fmaxf: a NaN has to stay
  const float more = swap ? s2.y : s2.x, less = (swap ? s2.x : s2.y) + (lost.x + lost.y);
  return make_float2(m, (more - 1.0f) + less);
}

// ----------------------------------------------------------- log-probabilities

// Log-probability of every row's target; stats != NULL: {maximum, sum of e^(x -
// maximum)} too, and 0 into factors[t], for the preference loss.
//
// GROUP threads take a row: a warp (eight rows in a block) where there are many
// rows, else the block; with few long rows, a cluster of C blocks.
// Bound by HBM: rows vocab es bytes; 4096 x 131072 bf16 154 us, 7.0 TB/s (reads alone are
// faster than the copy); one row of 32768 2.5 us.
struct LogprobPlan {
  int C, per;  // blocks per row; slots per block
};

// Where the gradient follows and the matrix is not far larger than L2 (HINTS), the rows
// that it begins with, `keep` and later, the last kKeptBytes (the two halves of L2 may
// each hold a copy), are to stay in L2 and the others to make room for them: the whole
// loss 55.3 -> 51.7 us at 51 MB, 116.4 -> 113.6 at 240 MB, 187.5 -> 186.5 at 400 MB; nothing
// at 512 MB and 1.8 GB.
constexpr unsigned long long kKeptBytes = 40ull << 20, kHintBytes = 400ull << 20;

template <int DT, int GROUP, bool HINTS>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const Matrix<DT> a, const LogprobPlan plan, float2* stats,
                                                           float* factors, unsigned long long keep) {
  using E = typename ElemOf<DT>::T;
  pdl_enter();
  __shared__ float2 sh[kThreads / 32], mine;
  const int tid = threadIdx.x % GROUP, lane = threadIdx.x & 31;
  const unsigned long long t = GROUP == kThreads ? blockIdx.x / plan.C
                                                 : blockIdx.x * (unsigned long long)(kThreads / GROUP) +
                                                       threadIdx.x / GROUP;
  if (t >= a.rows) return;                         // whole warps; never with GROUP == kThreads
  const int rank = GROUP == kThreads ? (int)cluster_rank() : 0;
  const bool writer = rank == 0 && tid == 0;
  if (writer && stats) factors[t] = 0.0f;
  if (a.weights && a.weights[t] == 0.0f) {         // the same in all blocks of the cluster
    if (writer) a.logprobs[t] = 0.0f;
    return;
  }
  const int V = (int)a.vocab, s0 = rank * plan.per;
  const E* row = a.logits + t * a.stride;
  const Slice<DT> in(row, V, s0, plan.per);
  const long long y = writer ? load_index(a.targets, a.target_bytes, t) : 0;

  const uint64_t policy = HINTS ? keep_policy(t >= keep) : 0;
  // joined: threads, warps, blocks
  float2 v = row_part<DT, GROUP, HINTS>(in, V, s0, tid, policy);
  if constexpr (GROUP != kThreads) {
    v = warp_rest(v);
  } else {
    v = block_rest(v, sh);
    if (plan.C > 1) {
      if (threadIdx.x == 0) mine = v;
      cluster_sync();
      v = warp_rest(lane < plan.C ? ld_cluster(cluster_address((uint32_t)__cvta_generic_to_shared(&mine), lane))
                                  : make_float2(-FLT_MAX, -1.0f));
      cluster_meet();                              // nobody leaves before the others have read
    }
  }
  if (writer) {
    a.logprobs[t] = y >= 0 && y < V ? (to_float(row[y]) - v.x) - log1pf(v.y) : __int_as_float(0x7fffffff);
    if (stats) stats[t] = make_float2(v.x, 1.0f + v.y);
  }
}

// --------------------------------------------------------------- policy loss

// Rows too long to be held (above 65536 slots, 524,288 bf16 logits): a block per row,
// which it reads twice.  1000 x 1048576 bf16 1395 us, 500 x 700000 497 us, 64 x 600001 322 us:
// 0.44, 0.41 and 0.07 of one read and one write at the copy's rate (the second read is from
// HBM too, with one slot per thread on the way; few rows leave SMs idle).
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
    const int V = (int)a.vocab;
    const Slice<DT> in(row, V, 0, INT_MAX);
    const float2 v = block_rest(row_part<DT, kThreads, false>(in, V, 0, threadIdx.x, 0), sh);
    if (threadIdx.x == 0) {
      const float lp = y >= 0 && y < V ? (to_float(row[y]) - v.x) - log1pf(v.y) : __int_as_float(0x7fffffff);
      a.logprobs[t] = lp;
      sh_c[0] = policy_token(p, p.old_logprobs[t], p.advantages[t], p.ref_logprobs ? p.ref_logprobs[t] : 0.0f, w, lp,
                             sum);
      sh_c[1] = lp;
    }
    __syncthreads();  // also: the target's logit is read before an in-place gradient is written
    row_grad<DT>(row, grad, V, y, sh_c[1], v.x, 1.0f + v.y, sh_c[0]);
    __syncthreads();
  }
  if (threadIdx.x == 0) partial[blockIdx.x] = make_float4(sum.loss, sum.kl, sum.clipped, sum.weight);
}

// The same with the row kept on the chip: read once, written once.
//
// A cluster of C blocks takes `run` rows, one after the other; each block holds
// a slice of the row in registers, K slots of 16 bytes per thread.  The slice of
// the next row is on its way into shared memory (cp.async) while a row is worked
// on; a thread reads only what it copied itself, so the copies need no barrier.
// Each warp takes its maximum and its sum of exponentials, and sends the two to
// every block of the cluster (st.async, counted by an mbarrier); one warp of each
// block joins them and computes the token's loss, and one block barrier hands the
// factors to the others, which write the gradient from their registers.
//
// Bound by HBM: 2 rows vocab es bytes.  8192 x 131072 bf16: 639 us, 6.72 TB/s; 4096 x 131072
// fp32: 629 us, 6.82 TB/s; 4096 x 32768 bf16: 90 us, 5.94 TB/s.  Below that a row's own
// chain (copies, sum, exchange, loss, stores: 3.7 us) shows: 2489 x 50001 95 us, 5.2 TB/s;
// 300 x 70000 21 us, 4.1 TB/s.
struct RowPlan {
  int C;        // blocks per cluster
  int per;      // slots per block: at most THREADS * K
  int most;     // slots of a row at its worst alignment
  int run;      // rows per cluster, at most 32
  uint32_t zero;  // 0, which the compiler does not know
  int late;     // for tests: the block of every cluster that gives its first wait up (-1: none)
};

constexpr int kMaxCluster = 16;
// Polls, together about a second.  A block whose wait for the cluster's pairs runs out waits for no others and uses its
// barriers no more.  It goes on through its rows and sends its pairs, so that the other blocks end, each with one such
// wait at most.  When all have ended, it waits as long again: what was sent to it has arrived, what they stored is in
// place.  Then it makes all the cluster's rows NaN: a wrong one may be among the others.
constexpr uint32_t kWaitPolls = 1u << 16;

template <int DT, int THREADS, int K, int BLOCKS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, BLOCKS)
policy_row_kernel(const Matrix<DT> a, const PolicyParams p, const RowPlan plan, float4* partial) {
  constexpr int N = Lanes<DT>::N, W = THREADS / 32;
  constexpr bool kEachWarp = !CLUSTER && W <= 4;  // every warp computes the token's loss for itself
  // A gradient at another alignment, in a loop as the aligned one has / by elements: bf16 2489 x 50001 175 / 328 us; fp32
  // 8192 x 8000 (one block of 8 slots per thread) 95 / 99, other fp32, 1111 x 50001 105 / 89, 2000 x 60000 230 / 182,
  // 16000 x 2000 56.5 / 52, and 4096 x 30000 204 / 213, where the loop's registers cost aligned rows more (2000 x 30000
  // 80.4 / 78.2).
  constexpr bool kWords = DT == kBF16 || (!CLUSTER && THREADS == 256 && K == 8);
  using E = typename ElemOf<DT>::T;
  extern __shared__ uint4 next[];                   // [K][THREADS]: the row that is on its way
  // (maximum, rest) of every warp, by parity: a block may be one row ahead
  __shared__ float2 pairs[2][(CLUSTER ? kMaxCluster : 1) * W];
  __shared__ float4 result;
  __shared__ uint64_t bars[2];
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CLUSTER ? (int)cluster_rank() : 0, C = CLUSTER ? plan.C : 1;
  const unsigned long long cluster = blockIdx.x / C, row0 = cluster * plan.run;
  const int rows = (int)min((unsigned long long)plan.run, a.rows - row0);
  const int V = (int)a.vocab, s0 = rank * plan.per;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(next) + tid * 16;
  const uint32_t bars_at = (uint32_t)__cvta_generic_to_shared(bars);
  // this warp's pair and the barriers in the block that this lane sends to
  uint32_t pair_to = 0, bars_to = 0;
  if constexpr (CLUSTER) {
    pair_to = cluster_address((uint32_t)__cvta_generic_to_shared(&pairs[0][rank * W + warp]), min(lane, C - 1));
    bars_to = cluster_address(bars_at, min(lane, C - 1));
    if (tid == 0) {
      mbar_init(bars_at, 1);
      mbar_init(bars_at + 8, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    cluster_arrive();  // waited for before the first pair is sent
  }

  // lane i holds row i's scalars
  float w_l = 0.0f;
  if (lane < rows) w_l = a.weights ? a.weights[row0 + lane] : 1.0f;
  const uint32_t live = __ballot_sync(~0u, w_l != 0.0f);  // bit i: row i is not masked

  const E* const logits = a.logits + row0 * a.stride;
  const auto issue = [&](int i) {
    if (i < rows && (live >> i & 1)) {
      const Slice<DT> in(logits + i * a.stride, V, s0, plan.per);
      // the head slot also brings what lies before the row, but nothing from before the matrix
      const int head = in.lead / N;
      const bool before = in.head >= 0 && in.row - in.lead % N < a.logits;
      const int first = in.head >= 0 && !before ? head : in.lo;
      const char* src = reinterpret_cast<const char*>(in.row - in.lead) + (s0 + tid) * 16ll;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k * THREADS + tid < in.lim && (k > 0 || tid >= first))
          cp_async16(mine + k * THREADS * 16, src + k * THREADS * 16, 16);
      if (in.tail >= 0 && in.tail % THREADS == tid)
        cp_async16(mine + in.tail / THREADS * (THREADS * 16), src + in.tail / THREADS * (THREADS * 16),
                   in.left * (int)sizeof(E));
      if (in.head == tid) {
        if (before) {
          E* to = reinterpret_cast<E*>(&next[tid]);
          for (int x = in.lead % N; x < N && x < in.lead % N + V; ++x) to[x] = in.row[x - in.lead % N];
        } else if (in.lead % N + V < N) {  // the row begins and ends inside one slot
          cp_async16(mine, src, (in.lead % N + V) * (int)sizeof(E));
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k * THREADS + tid >= plan.per || s0 + k * THREADS + tid >= plan.most)
      st_shared16(mine + k * THREADS * 16, no_logits(DT));
  issue(0);

  int y_l = -1;
  float old_l = 0.0f, adv_l = 0.0f, ref_l = 0.0f, x_l = 0.0f;
  if (live >> lane & 1) {
    const unsigned long long t = row0 + lane;
    const long long y = load_index(a.targets, a.target_bytes, t);
    y_l = y >= 0 && y < V ? (int)y : -1;
    if (kEachWarp || warp == 0) {
      old_l = p.old_logprobs[t];
      adv_l = p.advantages[t];
      if (p.ref_logprobs) ref_l = p.ref_logprobs[t];
      x_l = y_l < 0 ? __int_as_float(0x7fffffff) : to_float(a.logits[t * a.stride + y_l]);
    }
  }
  if constexpr (CLUSTER) cluster_wait();  // every block's barriers are set up

  PolicySums sum;
  int done = 0;  // live rows; negative in warp 0 from where its wait for the cluster ran out
  for (int i = 0; i < rows; ++i) {
    if (!(live >> i & 1)) {
      E* const grad = a.grad + (row0 + i) * a.grad_stride;
      const Slots<DT> out(grad, V);
      const int n = (int)out.count();
      const float zero[N] = {};
      for (int q = rank * THREADS + tid; q < n; q += C * THREADS) store_slot<DT>(out, grad, true, q, zero);
      if (rank == 0 && tid == 0) a.logprobs[row0 + i] = 0.0f;
      issue(i + 1);
      continue;
    }
    const int b = done & 1;
    if (CLUSTER && tid == 0 && done >= 0) mbar_expect_tx(bars_at + 8 * b, C * W * 8);
    {
      const Slice<DT> in(logits + i * a.stride, V, s0, plan.per);

      cp_async_wait<0>();
      // -infinity into what the slots at the row's ends hold beside the row, and into the slots before and after
      // them, which an earlier row of another alignment may have filled
      if (s0 == 0 && tid < in.lead / N) st_shared16(mine, no_logits(DT));
      if (in.head == tid) {
        E* to = reinterpret_cast<E*>(&next[tid]);
        for (int x = 0; x < N; ++x)
          if (x < in.lead % N || x >= in.lead % N + V) from_float(to + x, -INFINITY);
      }
      if (in.tail >= 0 && in.tail % THREADS == tid) {
        E* to = reinterpret_cast<E*>(&next[in.tail / THREADS * THREADS + tid]);
        for (int x = in.left; x < N; ++x) from_float(to + x, -INFINITY);
      }
      const int end = max(0, (V + in.lead + N - 1) / N - s0);  // the slot after the row's last
      const int after = end + ((tid - end) & (THREADS - 1));   // this thread's first one from there
      if (after < min(plan.per, plan.most - s0)) st_shared16(mine + after / THREADS * (THREADS * 16), no_logits(DT));
    }

    // the slots as they are, kept until the gradient is written
    uint4 r[K];
#pragma unroll
    for (int k = 0; k < K; ++k) r[k] = ld_shared16(mine + k * THREADS * 16);
    const float m = fmaxf(warp_max(max_of<DT>(r)), -FLT_MAX);

    float2 s2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};  // short chains of roundings
    const float2 minus_m = make_float2(-m, -m);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Acc<DT> x = widen<DT>(r[k]);
      float2 part;
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const float2 z = exp_pair(x.v[c], x.v[c + 1], minus_m);
        part = c == 0 ? z : add2(part, z);
        if constexpr (DT == kF32) {  // the exponentials fit where the logits were
          if (c == 0) { r[k].x = __float_as_uint(z.x); r[k].y = __float_as_uint(z.y); }
          else { r[k].z = __float_as_uint(z.x); r[k].w = __float_as_uint(z.y); }
        }
      }
      s2[k & 1] = add2(s2[k & 1], part);
    }
    // What is added to the maximum's 1 rounds, and for a near-certain token it is all that its log-probability is made
    // of: each 1 is taken out before the others are added, and (m, rest) stands for (1 + rest) e^m from here on.
    // (Compared and swapped, not fmaxf: a NaN has to stay.)
    const float2 both = add2(s2[0], s2[1]);
    const bool swap = both.y > both.x;
    const float most = swap ? both.y : both.x, less = swap ? both.x : both.y;
    const bool one = most >= 1.0f;                 // in the maximum's lane, and perhaps in others
    const float rest = warp_sum((one ? most - 1.0f : most) + less) + (float)(__popc(__ballot_sync(~0u, one)) - 1);
    // Once all pairs are there, gradients may overwrite the row (in place): not before the targets' logits have arrived,
    // in every lane, whichever lanes send.  So the addresses of the first pairs come from a vote on them.
    uint32_t zero = 0;
    if (done == 0) zero = __ballot_sync(~0u, __float_as_uint(x_l) & plan.zero);
    if constexpr (CLUSTER) {
      if (lane < C) st_async(pair_to + b * (kMaxCluster * W * 8) + zero, make_float2(m, rest), bars_to + 8 * b);
    } else {
      if (lane == 0) pairs[b][warp + zero] = make_float2(m, rest);
    }
    issue(i + 1);

    // the token's loss and what the gradient needs of it
    float4 res = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (!CLUSTER) __syncthreads();
    if (kEachWarp || warp == 0) {
      // the row's maximum M and sum 1 + R
      if constexpr (CLUSTER)
        if (done < 0 || !mbar_wait(bars_at + 8 * b, done >> 1 & 1, kWaitPolls) || rank == plan.late) done |= INT_MIN;
      float M = -FLT_MAX, R = 0.0f;
      for (int q = lane; q < C * W; q += 32) M = fmaxf(M, pairs[b][q].x);
      M = warp_max(M);
      int ones = -1;                               // pairs of the maximum, but for one
      for (int q = lane; q - lane < C * W; q += 32) {
        const float2 v = q < C * W ? pairs[b][q] : make_float2(-FLT_MAX, -1.0f);
        R += v.x == M ? v.y : (1.0f + v.y) * exp_diff(v.x, M);
        ones += __popc(__ballot_sync(~0u, v.x == M));
      }
      R = warp_sum(R) + (float)ones;
      // log(1 + R): the logarithm of the rounded sum, and what its rounding took
      const float S = 1.0f + R, inverse = 1.0f / S;
      const float lp = (__shfl_sync(~0u, x_l, i) - M) - (logf(S) + __fdividef(R - (S - 1.0f), S));
      const float c = policy_token(p, __shfl_sync(~0u, old_l, i), __shfl_sync(~0u, adv_l, i),
                                   __shfl_sync(~0u, ref_l, i), __shfl_sync(~0u, w_l, i), lp, sum);
      res = make_float4(M, -c * inverse, -c, lp);
      if (rank == 0 && tid == 0) a.logprobs[row0 + i] = lp;
      if (!kEachWarp && lane == 0) result = res;
    }
    if constexpr (!kEachWarp) {
      __syncthreads();
      res = result;
    }
    ++done;
    // Where registers are shortest the slice is computed once more, not kept (4096 x 32768 bf16 94 -> 92 us, 2000 x
    // 30000 fp32 92 -> 85, 2000 x 26000 fp32 72.5 -> 70; with 7 slots of bf16 per thread it costs more than it frees,
    // 2489 x 50001 99 -> 105).
    int again = i;
    if constexpr (THREADS == 256 && (K == 8 || (K == 7 && DT == kF32))) asm volatile("" : "+r"(again));
    const Slice<DT> in(logits + again * a.stride, V, s0, plan.per);
    E* const grad = a.grad + (row0 + again) * a.grad_stride;
    // fp32: the exponentials, to the warp's maximum; bf16: the logits, whose exponentials are taken again (half the
    // registers, so that more rows are on the SM at a time), to the row's
    const float f = DT == kF32 ? res.y * exp_diff(m, res.x) : res.y;
    const float2 f2 = make_float2(f, f), minus_M = make_float2(-res.x, -res.x);
    if constexpr (DT == kBF16)  // unpacked again, not kept unpacked
#pragma unroll
      for (int k = 0; k < K; ++k) asm volatile("" : "+r"(r[k].x), "+r"(r[k].y), "+r"(r[k].z), "+r"(r[k].w));
    const auto values = [&](int k) {
      Acc<DT> g = widen<DT>(r[k]);
#pragma unroll
      for (int x = 0; x < N; x += 2) {
        float2 v = make_float2(g.v[x], g.v[x + 1]);
        if constexpr (DT == kBF16) v = exp_pair(v.x, v.y, minus_M);
        v = mul2(v, f2);
        g.v[x] = v.x;
        g.v[x + 1] = v.y;
      }
      return g;
    };
    const bool same = (((uintptr_t)in.row ^ (uintptr_t)grad) & 15) == 0;
    if (same) {
      char* dst = reinterpret_cast<char*>(grad - in.lead) + (s0 + tid) * 16ll;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k * THREADS + tid < in.lim && (k > 0 || tid >= in.lo))
          st_stream(reinterpret_cast<uint4*>(dst + k * THREADS * 16), narrow<DT>(values(k), 1.0f, false));
    } else if constexpr (kWords) {  // the gradient's rows start at another alignment (by words and halves: the registers
                                    // of a shuffle slowed the other rows down, 4096 x 32768 bf16 91 -> 95 us)
      E* dst = grad + ((s0 + tid) * N - in.lead);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k * THREADS + tid < in.lim && (k > 0 || tid >= in.lo))
          store_apart(dst + k * THREADS * N, narrow<DT>(values(k), 1.0f, false), false);
    }
    // by elements: slots at the row's ends, and all at another alignment but kWords
    const bool each = !kWords && !same;
    const bool first = in.head == tid, last = in.tail >= 0 && in.tail % THREADS == tid;
    if (each || first || last) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int q = k * THREADS + tid;
        if ((each && q < plan.per) || (q == in.head && first) || (q == in.tail && last)) {
          const int j = (s0 + q) * N - in.lead;
          const Acc<DT> g = values(k);
#pragma unroll
          for (int x = 0; x < N; ++x)
            if (j + x >= 0 && j + x < V) from_float(grad + j + x, g.v[x]);
        }
      }
    }
    const int y = __shfl_sync(~0u, y_l, i);
    const int yq = (y + in.lead) / N - s0;
    if (y >= 0 && yq >= 0 && yq < plan.per && yq % THREADS == tid) from_float(grad + y, res.z * expm1f(res.w));  // over its own store
  }
  if (rank == 0 && tid == 0) partial[cluster] = make_float4(sum.loss, sum.kl, sum.clipped, sum.weight);
  if constexpr (CLUSTER) {
    cluster_meet();  // no block leaves while another may still send to it
    if (done < 0) {
      const float nan = __int_as_float(0x7fffffff);
      for (uint32_t k = 0; k < kWaitPolls; ++k) __nanosleep(16000);
      for (int i = 0; i < rows; ++i)
        if (live >> i & 1) {
          E* const grad = a.grad + (row0 + i) * a.grad_stride;
#pragma unroll 1
          for (int j = lane; j < V; j += 32) from_float(grad + j, nan);
          if (lane == 0) a.logprobs[row0 + i] = nan;
        }
      if (lane == 0) partial[cluster] = make_float4(nan, nan, nan, nan);
    }
  }
}

// The blocks' sums in a fixed order.
__global__ void __launch_bounds__(kThreads) policy_sum_kernel(const float4* partial, int n, float scale, float* stats) {
  pdl_enter();
  __shared__ float sh[4][kThreads / 32];
  Carried v[4];
  for (int i = threadIdx.x; i < n; i += 4 * kThreads) {
    float4 q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      q[u] = i + u * kThreads < n ? partial[i + u * kThreads] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    v[0].add((q[0].x + q[1].x) + (q[2].x + q[3].x));
    v[1].add((q[0].y + q[1].y) + (q[2].y + q[3].y));
    v[2].add((q[0].z + q[1].z) + (q[2].z + q[3].z));
    v[3].add((q[0].w + q[1].w) + (q[2].w + q[3].w));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float r = block_sum<kThreads>(v[k].value(), sh[k]);
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
  float* factors;    // rows: d(loss)/d(lp), 0 on entry
  float* loss;
};

__device__ __forceinline__ unsigned long long offset_at(const PairParams& p, unsigned long long k) {
  const long long v = load_index(p.offsets, p.offset_bytes, k);
  return v < 0 ? 0ull : min((unsigned long long)v, p.rows);
}

// One block per pair: the two sequences' sums, the pair's loss and its rows'
// factors.
__global__ void __launch_bounds__(kThreads) pair_kernel(const PairParams p) {
  pdl_enter();
  __shared__ float sh[kThreads / 32], side;
  for (unsigned long long i = blockIdx.x; i < p.pairs; i += gridDim.x) {
    // The two sequences in one signed sum, token against token: their log-probabilities cancel before they are large
    // (two sums of some thousands each would round the difference at 1e-4).
    const unsigned long long b0 = offset_at(p, 2 * i), b1 = offset_at(p, 2 * i + 1), b2 = offset_at(p, 2 * i + 2);
    const unsigned long long n0 = b1 > b0 ? b1 - b0 : 0, n1 = b2 > b1 ? b2 - b1 : 0;
    const auto term = [&](unsigned long long t) {
      const float w = p.weights ? p.weights[t] : 1.0f;
      if (w == 0.0f) return 0.0f;
      return w * (p.ref_logprobs ? p.logprobs[t] - p.ref_logprobs[t] : p.logprobs[t]);
    };
    Carried sum;
    for (unsigned long long k = threadIdx.x; k < n0 || k < n1; k += kThreads) {
      if (k < n0) sum.add(term(b0 + k));
      if (k < n1) sum.add(-term(b1 + k));
    }
    const float v = block_sum<kThreads>(sum.value(), sh);
    if (threadIdx.x == 0) {
      const float z = p.beta * v;
      // softplus(-z) = max(-z, 0) + log1p(e^-|z|)
      const float e = expf(-fabsf(z));
      const float sp = fmaxf(-z, 0.0f) + log1pf(e);
      p.margins[i] = z;
      // (a side of weight 0 is left out: it may be infinite)
      float l = z != z ? z : 0.0f;
      if (p.ls < 1.0f) l += (1.0f - p.ls) * sp;
      if (p.ls > 0.0f) l += p.ls * (fmaxf(z, 0.0f) + log1pf(e));
      p.pair_loss[i] = l;
      // sigmoid(-z) and sigmoid(z), the smaller one without cancellation
      const float small = e / (1.0f + e), big = 1.0f / (1.0f + e);
      const float neg = z >= 0.0f ? small : big, pos = z >= 0.0f ? big : small;
      const float dz = z != z ? z : p.ls * pos - (1.0f - p.ls) * neg;
      side = p.scale * p.beta * dz;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
      const unsigned long long b = offset_at(p, 2 * i + k), e = offset_at(p, 2 * i + k + 1);
      const float f = k == 0 ? side : -side;
      for (unsigned long long t = b + threadIdx.x; t < e; t += kThreads) {
        const float w = p.weights ? p.weights[t] : 1.0f;
        if (w != 0.0f) p.factors[t] = w * f;
      }
    }
    __syncthreads();
  }
}

// The gradient of one piece of a row: kGradSlots slots per thread, all loaded
// before the first is used.  The rows go from the last to the first: what the
// statistics' pass has read last is still in L2.
// Bound by HBM: with the statistics' pass the logits are read twice, since a row's
// factor needs its whole pair's log-probabilities: 6800 x 131072 bf16 765 us for the whole
// loss, 6.99 TB/s of two reads and one write; 2400 x 50001 114 us.  2 / 4 / 8 slots: 120 / 114 /
// 115 us (2400 x 50001).
constexpr int kGradSlots = 4, kPiece = kThreads * kGradSlots;

template <int DT, bool HINTS>
__global__ void __launch_bounds__(kThreads, 6) preference_grad_kernel(const Matrix<DT> a, const PairParams p,
                                                                      const float2* stats, unsigned pieces) {
  constexpr int N = Lanes<DT>::N;
  using E = typename ElemOf<DT>::T;
  pdl_enter();
  __shared__ float sh[kThreads / 32];
  if (blockIdx.x == 0) {
    Carried sum;
    for (unsigned long long i = threadIdx.x; i < p.pairs; i += kThreads) sum.add(p.pair_loss[i]);
    const float v = block_sum<kThreads>(sum.value(), sh);
    if (threadIdx.x == 0) *p.loss = p.scale * v;
  }
  const unsigned back = blockIdx.x / pieces;
  if (back >= a.rows) return;
  const unsigned long long t = a.rows - 1 - back;
  const int V = (int)a.vocab, s0 = (int)(blockIdx.x % pieces) * kPiece, tid = threadIdx.x;
  E* grad = a.grad + t * a.grad_stride;
  const float c = p.factors[t];
  const E* row = a.logits + t * a.stride;
  if (c == 0.0f) {  // masked, of no sequence, or of a pair whose loss is flat
    const Slots<DT> out(grad, V);
    const float zero[N] = {};
#pragma unroll
    for (int k = 0; k < kGradSlots; ++k)
      if (s0 + k * kThreads + tid < out.count()) store_slot<DT>(out, grad, true, s0 + k * kThreads + tid, zero);
    return;
  }
  const Slice<DT> in(row, V, s0, kPiece);
  const uint4* src = reinterpret_cast<const uint4*>(row - in.lead) + s0 + tid;
  const uint64_t once = HINTS ? keep_policy(false) : 0;
  uint4 r[kGradSlots];
#pragma unroll
  for (int k = 0; k < kGradSlots; ++k) {
    const int q = k * kThreads + tid;
    if (q >= in.lo && q < in.lim) r[k] = ld_hint<HINTS>(src + k * kThreads, once);
  }
  const float2 st = stats[t];
  const bool same = (((uintptr_t)row ^ (uintptr_t)grad) & 15) == 0;
  const float f = -c / st.y;
  const float2 minus_m = make_float2(-st.x, -st.x), f2 = make_float2(f, f);
  E* dst = grad + ((long long)(s0 + tid) * N - in.lead);
#pragma unroll
  for (int k = 0; k < kGradSlots; ++k) {
    const int q = k * kThreads + tid;
    if (q >= in.lo && q < in.lim) {
      Acc<DT> g = widen<DT>(r[k]);
#pragma unroll
      for (int x = 0; x < N; x += 2) {
        const float2 v = mul2(exp_pair(g.v[x], g.v[x + 1], minus_m), f2);
        g.v[x] = v.x;
        g.v[x + 1] = v.y;
      }
      const uint4 v = narrow<DT>(g, 1.0f, false);
      if (same) st_stream(reinterpret_cast<uint4*>(dst + k * kThreads * N), v);
      else store_apart(dst + k * kThreads * N, v, warp_within(q, in.lo, in.lim));
    }
  }
  __syncwarp();  // the target's element follows, perhaps from another lane than its store
  // slots at the row's ends, by elements
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const int q = e == 0 ? in.head : in.tail;
    if (q < 0 || q % kThreads != tid) continue;
    const int j = (s0 + q) * N - in.lead;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = j + i >= 0 && j + i < V ? to_float(row[j + i]) : -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float g = f * exp_diff(x[i], st.x);
      if (j + i >= 0 && j + i < V) from_float(grad + j + i, g);
    }
  }
  // the target's element, over its thread's own store
  const long long y = load_index(a.targets, a.target_bytes, t);
  if (y >= 0 && y < V) {
    const int q = ((int)y + in.lead) / N - s0;
    if (q >= 0 && q < kPiece && q % kThreads == tid) from_float(grad + y, -c * expm1f(a.logprobs[t]));
  }
}

inline unsigned grid_of(unsigned long long work) {
  return (unsigned)std::max(1ull, std::min<unsigned long long>(work, kMaxLossBlocks));
}

// Slots of a matrix's row, from the line it begins in, at its worst alignment.
template <int DT>
unsigned long long row_slots(const LogitsCall& c, const void* matrix, size_t stride) {
  constexpr int N = Lanes<DT>::N;
  const size_t es = sizeof(typename ElemOf<DT>::T), at = ((uintptr_t)matrix & 127) / es;
  // the rows' places in their lines: all the same, at a distance of whole slots, or any
  const unsigned long long lead = c.rows == 1 || stride * es % 128 == 0 ? at
                                  : stride * es % 16 == 0              ? 128 / es - N + at % N
                                                                       : 128 / es - 1;
  return (c.vocab + lead + N - 1) / N;
}

// Programmatic dependent launch in clusters of C blocks (attr: room for two).
inline cudaLaunchConfig_t cluster_config(unsigned grid, unsigned threads, int smem, int C, cudaStream_t stream,
                                         cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <int DT>
bool small_for_l2(const LogitsCall& c) {
  return c.rows * row_slots<DT>(c, c.logits, c.row_stride) * 16 <= kHintBytes;
}

template <int DT>
cudaError_t run_logprobs(const LogitsCall& c, float2* stats, float* factors) {
  const unsigned long long n = row_slots<DT>(c, c.logits, c.row_stride);
  const bool hints = stats && small_for_l2<DT>(c);
  const unsigned long long kept = kKeptBytes / (n * 16), keep = c.rows > kept ? c.rows - kept : 0;
  // A warp per row where that makes 16 warps for every SM (8192 x 9000 bf16: 27 us, a block per row 41; 4096 x 32768
  // 46 and 46; but 4096 x 131072 163 and 155, 1000 x 32768 34 and 11) or a row has no more for a warp to do.  Thousands of
  // warps leave no whole rows in L2, though: where the gradient follows, long rows take a block (preference 4096 x
  // 131072: 465 us, with a warp per row 481).
  if (n <= 256 || (c.rows >= 16ull * c.sms && n <= (stats ? 2048 : 8192)))
    return launch_kernel(hints ? logprob_kernel<DT, 32, true> : logprob_kernel<DT, 32, false>,
                         (unsigned)((c.rows + 7) / 8), kThreads, 0, c.stream, true, Matrix<DT>(c),
                         LogprobPlan{1, (int)n}, stats, factors, keep);
  // a row over several blocks until there are two blocks for every SM, each with 1024 slots at least
  int C = 1;
  while (C < 8 && c.rows * C < 2ull * c.sms && n >= 2048ull * C) C *= 2;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = cluster_config((unsigned)c.rows * C, kThreads, 0, C, c.stream, attr);
  return cudaLaunchKernelEx(&cfg, hints ? logprob_kernel<DT, kThreads, true> : logprob_kernel<DT, kThreads, false>,
                            Matrix<DT>(c), LogprobPlan{C, (int)(((n + C - 1) / C + 7) / 8 * 8)}, stats, factors, keep);
}

// Rows per cluster, of 1 .. most.  A row takes a resident cluster 3.7 us by itself
// (2.0 in blocks of 128 threads: copies, sum, exchange, loss, stores); all resident
// clusters' rows take 2 wave row_bytes / 6.8 TB/s together.
// Where HBM is the longer by a fifth, the clusters' start-ups hide behind others'
// transfers and small runs end evenly: one wave's share of the rows, at most 3, or 8
// where two blocks fill an SM (us at 1 / 2 / 3 / 4 / 5 / 8 rows: 5000 x 30000 bf16 121 / 106 / 102 / 103 /
// 105 / 111, 1500 x 30000 43 / 39 / 37 / 41 / 37 / 48, 1800 x 30000 50 / 44 / 42 / 46 / 49 / 50; 8192 x 131072
// at 1 / 2 / 4 / 8 / 16: 769 / 680 / 641 / 641 / 653).
// Where the row itself is, a wave takes its rows' time and a start-up of about one
// row whether it is full or not: the least ceil(waves) (rows + 1) (300 x 70000 at 3 / 4 / 5 /
// 6: 21.4 / 26.3 / 20.7 / 24.0; 700 x 100000 at 4 / 5 / 8 / 10: 58 / 55 / 67 / 52; 2489 x 50001 at
// 2 / 3 / 4 / 6 / 8: 98 / 95 / 94 / 94 / 99).  More only to bound the number of partial sums.
inline int rows_per_cluster(unsigned long long rows, int wave, double row_bytes, int threads, bool two_blocks) {
  const double row_us = threads >= 256 ? 3.7 : 2.0, wave_us = 2.0 * wave * row_bytes / 6.8e6;
  int run = 1;
  if (wave_us > 1.2 * row_us) {
    run = (int)std::max(1ull, std::min<unsigned long long>(two_blocks ? 8 : 3, (rows + wave / 2) / wave));
  } else {
    unsigned long long least = ~0ull;
    for (int k = 1; k <= (two_blocks ? 12 : 8); ++k) {
      const unsigned long long clusters = (rows + k - 1) / k, time = (clusters + wave - 1) / wave * (k + 1);
      if (time < least) {
        least = time;
        run = k;
      }
    }
  }
  const unsigned long long bound = (rows + kMaxPolicySums - 1) / kMaxPolicySums;
  return (int)std::min(32ull, std::max((unsigned long long)run, bound));
}

// Clusters of C of this kernel's blocks that the device holds at a time; asked
// once per device (a cluster's blocks have to fit one group of SMs).  0: clusters
// of 16, which a device need not offer, do not fit.
template <int DT, int THREADS, int K, int BLOCKS, bool CLUSTER>
int resident_clusters(const cudaLaunchConfig_t& cfg, int C, int sms) {
  if (!CLUSTER) return sms * BLOCKS;
  static std::atomic<int> known[16][5];  // by device, log2 C
  int dev = -1, log2 = 0;
  while (1 << log2 < C) ++log2;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) dev = -1;
  int n = dev < 0 ? 0 : known[dev][log2].load(std::memory_order_relaxed);
  if (n > 0) return n;
  n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, policy_row_kernel<DT, THREADS, K, BLOCKS, CLUSTER>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (n <= 0) return C > 8 ? 0 : std::max(1, sms * BLOCKS / C);
  if (dev >= 0) known[dev][log2].store(n, std::memory_order_relaxed);
  return n;
}

// AR_LATE_BLOCK=<rank> (ar_train.h); read once.
inline int late_block() {
  static const int rank = [] {
    const char* s = std::getenv("AR_LATE_BLOCK");
    return s ? std::atoi(s) : -1;
  }();
  return rank;
}

template <int DT, int THREADS, int K, int BLOCKS, bool CLUSTER>
cudaError_t launch_policy_row(const LogitsCall& c, const PolicyParams& p, unsigned long long slots, int C,
                              float4* partial, unsigned* sums) {
  constexpr int smem = K * THREADS * 16;
  const auto kernel = policy_row_kernel<DT, THREADS, K, BLOCKS, CLUSTER>;
  RowPlan plan;
  plan.C = C;
  plan.per = (int)(((slots + C - 1) / C + 7) / 8 * 8);  // whole lines; still at most THREADS * K
  plan.zero = 0;
  plan.late = late_block();
  plan.most = (int)slots;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = cluster_config(C, THREADS, smem, C, c.stream, attr);
  const int wave = resident_clusters<DT, THREADS, K, BLOCKS, CLUSTER>(cfg, C, c.sms);
  if (wave == 0) return cudaErrorNotSupported;
  plan.run = rows_per_cluster(c.rows, wave, 16.0 * slots, THREADS, BLOCKS == 2);
  *sums = (unsigned)((c.rows + plan.run - 1) / plan.run);
  cfg.gridDim = *sums * C;
  return cudaLaunchKernelEx(&cfg, kernel, Matrix<DT>(c), p, plan, partial);
}

// The shape by the row's length in 16-byte slots.  Registers hold the row: a
// slice of up to 32 KiB in 256 threads leaves room for four blocks on an SM, which was
// faster than two blocks of 512 threads with three rows on the way (8192 x 131072 bf16
// 690 against 984 us) and than keeping the exponentials instead of the logits in twice
// the registers (826).  From a cluster of more than 4 such blocks on, slices of
// up to 64 KiB, two on an SM, in half the blocks (131072 bf16: 672 against 690 us; fp32:
// 666 against 687; at 65536 they are level).  Short rows take small blocks, many
// on an SM, and no cluster (8192 x 4096 bf16: 64 threads 30 us, 128 threads 40, 256 threads
// 52).
template <int DT>
cudaError_t run_policy(const LogitsCall& c, const PolicyParams& p, float* stats, float4* partial) {
  const unsigned long long n = row_slots<DT>(c, c.logits, c.row_stride);
  unsigned sums = 0;
  cudaError_t e;
#define AR_ROW(THREADS, K, BLOCKS, CLUSTER) \
  launch_policy_row<DT, THREADS, K, BLOCKS, CLUSTER>(c, p, n, C, partial, &sums)
  const auto streamed = [&] {
    sums = grid_of(c.rows);
    return launch_kernel(policy_kernel<DT>, sums, kThreads, 0, c.stream, true, Matrix<DT>(c), p, partial);
  };
  if (c.rows == 0 || n > 16 * 4096) {
    e = streamed();
  } else if (n <= 2048) {
    constexpr int C = 1;
    e = n <= 512    ? AR_ROW(64, 8, 12, false)
        : n <= 1024 ? AR_ROW(128, 8, 7, false)
        : n <= 1536 ? AR_ROW(256, 6, 4, false)
                    : AR_ROW(256, 8, 4, false);
  } else if (n <= 8192) {
    const int C = n <= 4096 ? 2 : 4;
    const unsigned long long k = (n + 256 * C - 1) / (256 * C);  // 5 .. 8
    e = k <= 5   ? AR_ROW(256, 5, 4, true)
        : k == 6 ? AR_ROW(256, 6, 4, true)
        : k == 7 ? AR_ROW(256, 7, 4, true)
                 : AR_ROW(256, 8, 4, true);
  } else {
    const int C = n <= 16384 ? 4 : n <= 32768 ? 8 : 16;
    const unsigned long long k = (n + 256 * C - 1) / (256 * C);  // 9 .. 16
    e = k <= 10   ? AR_ROW(256, 10, 2, true)
        : k <= 12 ? AR_ROW(256, 12, 2, true)
        : k <= 14 ? AR_ROW(256, 14, 2, true)
                  : AR_ROW(256, 16, 2, true);
    if (e == cudaErrorNotSupported) e = streamed();
  }
#undef AR_ROW
  if (e == cudaSuccess)
    e = launch_kernel(policy_sum_kernel, 1, kThreads, 0, c.stream, true, (const float4*)partial, (int)sums, p.scale,
                      stats);
  return e;
}

template <int DT>
cudaError_t run_preference(const LogitsCall& c, const PairParams& p, float2* stats) {
  const unsigned long long slots = std::max(row_slots<DT>(c, c.logits, c.row_stride),
                                            row_slots<DT>(c, c.grad, c.grad_stride));
  const unsigned long long pieces = std::max(1ull, (slots + kPiece - 1) / kPiece);
  if (c.rows * pieces > 0x7fffffffull) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (c.rows) e = run_logprobs<DT>(c, stats, p.factors);
  if (e == cudaSuccess && p.pairs) e = launch_kernel(pair_kernel, grid_of(p.pairs), kThreads, 0, c.stream, true, p);
  if (e == cudaSuccess)
    e = launch_kernel(small_for_l2<DT>(c) ? preference_grad_kernel<DT, true> : preference_grad_kernel<DT, false>,
                      (unsigned)std::max(1ull, c.rows * pieces), kThreads, 0, c.stream, true, Matrix<DT>(c), p,
                      (const float2*)stats, (unsigned)pieces);
  return e;
}

}  // namespace

cudaError_t launch_logprobs(const LogitsCall& c) {
  return c.dtype == kF32 ? run_logprobs<kF32>(c, nullptr, nullptr) : run_logprobs<kBF16>(c, nullptr, nullptr);
}

cudaError_t launch_policy(const LogitsCall& c, const PolicyCall& q) {
  const PolicyParams p{q.old_logprobs, q.advantages, q.ref_logprobs, q.lo, q.hi, q.kl_coef, q.scale};
  float4* partial = static_cast<float4*>(q.workspace);
  return c.dtype == kF32 ? run_policy<kF32>(c, p, q.stats, partial) : run_policy<kBF16>(c, p, q.stats, partial);
}

// one partial sum per cluster of rows (rows_per_cluster)
size_t policy_workspace(size_t rows) {
  return std::max<size_t>(1, std::max(std::min(rows, kMaxPolicySums), (rows + 31) / 32)) * sizeof(float4);
}

// workspace: the rows' statistics and factors, then the pairs' losses
size_t preference_workspace(size_t rows, size_t pairs) {
  return rows * (sizeof(float2) + sizeof(float)) + pairs * sizeof(float);
}

cudaError_t launch_preference(const LogitsCall& c, const PreferenceCall& q) {
  float2* stats = static_cast<float2*>(q.workspace);
  float* factors = reinterpret_cast<float*>(stats + c.rows);
  const PairParams p{q.offsets, q.offset_bytes, q.pairs, c.rows, c.weights, c.logprobs, q.ref_logprobs, q.beta,
                     q.label_smoothing, q.scale, q.margins, factors + c.rows, factors, q.loss};
  return c.dtype == kF32 ? run_preference<kF32>(c, p, stats) : run_preference<kBF16>(c, p, stats);
}

}  // namespace ar
