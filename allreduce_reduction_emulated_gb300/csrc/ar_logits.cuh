// ar_logits.cuh -- device-side building blocks of the operators on a logits
// matrix (ar_logits.cu): a row cut into 16-byte slots, softmax statistics and
// the losses' per-token arithmetic.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cuda_runtime.h>

#include "ar_device.cuh"

namespace ar {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x in one instruction (relative error 2^-22, results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// e^(x - m).  The difference is formed before it is scaled: x and m may be the
// type's lowest value, and lowest * log2(e) is already -infinity.
__device__ __forceinline__ float exp_diff(float x, float m) { return ex2((x - m) * kLog2e); }

// ----------------------------------------------------------------- rows

// 16-byte load of data that this block reads once or twice: not kept in L1.
// Volatile, so it stays behind the wait for the kernel before it (pdl_enter).
__device__ __forceinline__ uint4 ld_row(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// A load whose lines L2 keeps for longest (keep) or drops first; where there is no
// reason for either, ld_row.
__device__ __forceinline__ uint64_t keep_policy(bool keep) {
  uint64_t p;
  if (keep) asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
template <bool HINTS>
__device__ __forceinline__ uint4 ld_hint(const uint4* p, uint64_t policy) {
  if constexpr (!HINTS) return ld_row(p);
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p), "l"(policy));
  return r;
}

template <int DT> struct ElemOf;
template <> struct ElemOf<kF32> { using T = float; };
template <> struct ElemOf<kBF16> { using T = uint16_t; };

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return bf16_lo((uint32_t)x); }
__device__ __forceinline__ void from_float(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_float(uint16_t* p, float x) { *p = (uint16_t)(pack_bf16x2(x, 0.0f) & 0xffffu); }

// A slot's 16 bytes to an address of any other alignment, by words.  Where bf16 elements
// begin between two words, the last word takes its second half from the next lane if a whole
// warp stores consecutive slots (`warp`, the same in all lanes: an element may then be stored
// by the lane before the one that holds it), else by halves at both ends.
// Element by element, at an even / odd distance, these took (2489 x 50001 bf16) 334 / 330 us,
// now 110 / 174 (policy), 301 / 296, now 125 / 137 (preference); clipping 100M bf16 232 / 221, now
// 94 / 108.  A whole slot put together by shuffles and stored as one took 140, 148 and 111.
// fp32 (1111 x 50001): preference 125, now 103; the policy loss stores its fp32 elements one by one.
template <class E>
__device__ __forceinline__ void store_apart(E* to, uint4 v, bool warp) {
  if (sizeof(E) == 4 || ((uintptr_t)to & 2) == 0) {
    uint32_t* w = reinterpret_cast<uint32_t*>(to);
    __stcs(w, v.x); __stcs(w + 1, v.y); __stcs(w + 2, v.z); __stcs(w + 3, v.w);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(to) + 2);
    uint16_t* half = reinterpret_cast<uint16_t*>(to);
    const int lane = threadIdx.x & 31;
    const uint32_t after = warp ? __shfl_down_sync(~0u, v.x, 1) : 0u;
    __stcs(w, __funnelshift_r(v.x, v.y, 16));
    __stcs(w + 1, __funnelshift_r(v.y, v.z, 16));
    __stcs(w + 2, __funnelshift_r(v.z, v.w, 16));
    if (warp && lane < 31) __stcs(w + 3, __funnelshift_r(v.w, after, 16));
    else half[7] = (uint16_t)(v.w >> 16);
    if (!warp || lane == 0) half[0] = (uint16_t)v.x;
  }
}
// Whether the slots q of this thread's whole warp are among lo .. lim - 1.
__device__ __forceinline__ bool warp_within(int q, int lo, int lim) { return (q & ~31) >= lo && (q | 31) < lim; }

// A row (or any run of elements) as slots of 16 aligned bytes.  Its start needs
// element alignment only: slot 0 is the aligned 16 bytes that hold element 0,
// so every slot but the first and the last holds N elements of the run, and
// slot s holds elements [s * N - lead, s * N - lead + N) of it.
template <int DT>
struct Slots {
  using E = typename ElemOf<DT>::T;
  static constexpr int N = Lanes<DT>::N;
  E* row;
  long long len;     // elements
  int lead;          // elements of slot 0 that lie before the run

  __device__ __forceinline__ Slots(const E* p, long long n)
      : row(const_cast<E*>(p)), len(n), lead((int)(((uintptr_t)p & 15) / sizeof(E))) {}
  __device__ __forceinline__ long long count() const { return (len + lead + N - 1) / N; }
  __device__ __forceinline__ long long first(long long s) const { return s * N - lead; }

  // slot s widened to fp32; elements outside the run read as `fill`
  __device__ __forceinline__ void load(long long s, float (&x)[N], float fill) const {
    const long long j = first(s);
    if (j >= 0 && j + N <= len) {
      const Acc<DT> a = widen<DT>(ld_row(reinterpret_cast<const uint4*>(row + j)));
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = a.v[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = (j + i >= 0 && j + i < len) ? to_float(row[j + i]) : fill;
    }
  }
};

// Stores N elements of slot s of `in` at the same element indices of `out`
// (which may start at another alignment).
template <int DT>
__device__ __forceinline__ void store_slot(const Slots<DT>& in, typename ElemOf<DT>::T* out, bool same_align,
                                           long long s, const float (&y)[Lanes<DT>::N]) {
  constexpr int N = Lanes<DT>::N;
  const long long j = in.first(s);
  if (j >= 0 && j + N <= in.len) {
    Acc<DT> a;
#pragma unroll
    for (int i = 0; i < N; ++i) a.v[i] = y[i];
    const uint4 v = narrow<DT>(a, 1.0f, false);
    if (same_align) st_stream(reinterpret_cast<uint4*>(out + j), v);
    else store_apart(out + j, v, false);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (j + i >= 0 && j + i < in.len) from_float(out + j + i, y[i]);
  }
}

__device__ __forceinline__ long long load_index(const void* p, int bytes, size_t i) {
  return bytes == 8 ? static_cast<const long long*>(p)[i] : (long long)static_cast<const int*>(p)[i];
}

// ---------------------------------------------------- asynchronous copies

// 16 bytes to shared memory, not through L1; the first `bytes` are read from
// global memory, the rest are zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
  return r;
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of `at` (shared memory of this block) in the cluster's block `rank`.
__device__ __forceinline__ uint32_t cluster_address(uint32_t at, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
// 8 bytes into the shared memory of a block of the cluster (`at`, `bar` from
// cluster_address), counted by that block's mbarrier when they have arrived.
__device__ __forceinline__ void st_async(uint32_t at, float2 v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(at),
               "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(bar)
               : "memory");
}
__device__ __forceinline__ float2 ld_cluster(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// True once the phase of this parity has completed; false after `limit` polls
// (a poll waits in hardware itself, for about 15 us).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint32_t limit) {
  for (uint32_t i = 0; i < limit; ++i) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
  }
  return false;
}
// All threads of the cluster; what they wrote before is seen after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// All threads of the cluster are here; orders no memory accesses.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The warp's largest value; NaN yields to any number.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// ------------------------------------------------------- pairs of fp32 values

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 x, y, u, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 u, {%6, %7}; "
      "fma.rn.f32x2 z, x, y, u; mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// ------------------------------------------------------------------ block sums

// One thread's sum of many values: what an addition loses, of the larger or of the
// smaller, is carried along.  (Where the values are alike the roundings of a plain sum all
// go one way: 1500 additions 1.6e-5.)
struct Carried {
  float sum = 0.0f, lost = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float t = sum + v, b = t - sum;
    lost += (sum - (t - b)) + (v - b);
    sum = t;
  }
  __device__ __forceinline__ float value() const {
    const float v = sum + lost;
    return v == v ? v : sum;  // an infinite sum has lost infinity - infinity
  }
};

// Sum over a block of THREADS threads; valid in every thread.  `sh` holds
// THREADS / 32 values; the block must synchronize before it is written again.
template <int THREADS, class T>
__device__ __forceinline__ T block_sum(T v, T* sh) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  T r = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) r += sh[w];
  return r;
}

// ------------------------------------------------------------ per token

struct PolicyParams {
  const float* old_logprobs;
  const float* advantages;
  const float* ref_logprobs;  // NULL: no KL term
  float lo, hi;               // 1 - clip_low, 1 + clip_high
  float kl_coef, scale;
};

struct PolicySums {
  float loss = 0.0f, kl = 0.0f, clipped = 0.0f, weight = 0.0f;
};

// One token's loss into `sum`; returns its derivative by the log-probability,
// weight and scale included (scale multiplies the sums at the end).
__device__ __forceinline__ float policy_token(const PolicyParams& p, float old, float A, float ref, float w, float lp,
                                              PolicySums& sum) {
  const float r = expf(lp - old);
  const bool clip = (A > 0.0f && r > p.hi) || (A < 0.0f && r < p.lo);
  // a NaN ratio is neither clipped nor clamped away
  float term = -(clip ? (A > 0.0f ? p.hi : p.lo) * A : r * A);
  float d = clip ? 0.0f : -A * r;
  if (p.ref_logprobs) {
    const float q = ref - lp;
    const float e = expm1f(q);  // e^q - 1 without cancellation: policies start at their reference
    const float kl = e - q;
    if (p.kl_coef != 0.0f) {  // of a statistic alone nothing is added: it may be infinite
      term += p.kl_coef * kl;
      d -= p.kl_coef * e;
    }
    sum.kl += w * kl;
  }
  sum.loss += w * term;
  sum.clipped += clip ? w : 0.0f;
  sum.weight += w;
  return p.scale * w * d;
}

}  // namespace ar
