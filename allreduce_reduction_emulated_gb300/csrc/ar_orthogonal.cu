// ar_orthogonal.cu -- updates orthogonalised by Newton-Schulz products (ar_train.h), on the
// tensor-core product of ar_mma.cuh.
//
//   u = g + beta m (or m, or g);  X = u / (|u| + eps)
//   `steps` times:  A = X X^T (of a tall matrix X^T X),  B = a I + b A + c A^2,  X <- B X
//
// Two passes over the gradients (momentum and sums of squares; the scaled 16-bit copy), then one launch for all
// products of all steps and shapes.  A and B are symmetric: only their blocks on one
// side of the diagonal are computed, and stored to both.
//
// Between products X, A and B are held in fp16, not in bf16: its 11 bits keep the result of a matrix of normal values
// within 2^-9 (2-norm) of fp32 arithmetic from sides of about 16 on where bf16's 8 would be off by 2% after five steps, and the
// tensor cores are as fast.  A direction whose singular value is a small part s of the norm is known to 3e-4 / (s
// sqrt(side)), so matrices of two or three directions, or square ones, have a tail: of 4096 each, 99% (and the worst) are off
// by, bf16's 1.7e-3 included, 2 x 2 6.4e-3 (7e-2), 13 x 2 4.8e-3 (6.8e-3), 3 x 300 3.8e-3 (4.5e-3), 8 x 8 5.5e-3 (1.6e-2),
// 16 x 16 3.8e-3 (5.6e-3), 16 x 40 2.4e-3 (2.6e-3), 128 x 128 2.1e-3, 1024 x 2048 1.8e-3.  fp16's range is met by powers of two: all singular values of
// X have a bound that follows from the coefficients, so that every element's has, and each
// matrix is held times the power of two that brings the bound to 2^13.  Sums are fp32, and
// a I + b A is added in fp32 before B's one rounding.  B's diagonal is most of it, and where the singular
// values are alike (a short matrix) its roundings do not average out: what each element of it
// loses is kept in fp32, as a factor of its row.  30 x 512: 2.9e-3 of the 2-norm before the last
// rounding without, 1.4e-3 with it; 300 x 310: 1.3e-3 and 1.0e-3.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_fp16.h>

#include "ar_mma.cuh"
#include "ar_train.h"
#include "ar_train_launch.h"

namespace ar {

namespace {

using mma::Tile;

constexpr int kMaxShapes = 16, kMaxStacks = 256;  // of one group of launches
constexpr long long kMaxTiles = 1 << 24;          // and of each stage of one group
constexpr int kMaxSteps = AR_MAX_ORTHOGONAL_STEPS;
constexpr int kCoefs = 5;                          // of a matrix and step

// ------------------------------------------------------------------ momentum, norm, 16-bit copy

struct Stack {
  const void* grad;
  float* momentum;
  void* out;
  __half* x;              // of its first matrix, in the workspace
  unsigned int rows, cols, pitch, slots;  // slots: 8 columns each, per row
  unsigned int chunks;    // per matrix
  unsigned int first;     // chunk of its first matrix
  unsigned int matrix;    // number of its first matrix
  bool bf16, vectors;     // vectors: rows of the gradient are whole 16 bytes
  bool out_vectors;       // and of the result
  float scale;
};

struct PrepareParams {
  Stack stack[kMaxStacks];
  int stacks;
  float beta;
  bool nesterov;
  float eps, a, b, c, growth;
  float cap[kMaxSteps + 1];  // bounds of the singular values before each step
  int steps;
  unsigned int chunk;        // slots of a chunk
  float* partial;            // one per chunk
  float* coefs;              // kCoefs per matrix and step
  void** outs;               // one per matrix
  unsigned int* done;        // one per matrix: made 0
};

// A chunk is what one block takes: up to 2048 slots, fewer where that would leave multiprocessors idle.
constexpr int kThreads = 256;
constexpr unsigned int kMostChunk = 2048;

// Sum over the block, in a fixed order; every thread gets it.
template <int THREADS = kThreads>
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[THREADS / 32];
#pragma unroll
  for (int d = 16; d; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) s += part[i];
  return s;
}

// Eight columns of a row as fp32, 0 behind the row's end.
template <class T>
__device__ __forceinline__ void load8(const T* p, int left, bool vectors, float (&v)[8]) {
  if (vectors && left >= 8) {
    if constexpr (sizeof(T) == 2) {
      const uint4 r = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
    } else {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) v[i] = i < left ? bf16_lo(p[i]) : 0.0f;
    else v[i] = i < left ? p[i] : 0.0f;
  }
}

struct Place {
  const Stack* s;
  unsigned int matrix, chunk;  // of the stack, of the matrix
};

__device__ __forceinline__ Place place(const PrepareParams& p, unsigned int block) {
  int lo = 0;
  for (int hi = p.stacks; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (p.stack[mid].first <= block) lo = mid;
    else hi = mid;
  }
  const Stack& s = p.stack[lo];
  const unsigned int k = block - s.first;
  return Place{&s, k / s.chunks, k % s.chunks};
}

// Slots [begin, end) of one matrix, `threads` at a time: the update u of each to `use`.  With momentum, the new one
// is written where WRITE, else it is there already.
template <bool WRITE, class F>
__device__ __forceinline__ void walk(const PrepareParams& p, const Stack& s, unsigned int matrix, unsigned int begin,
                                     unsigned int end, unsigned int threads, F use) {
  const size_t base = (size_t)matrix * s.rows * s.cols;
#pragma unroll 4
  for (unsigned int slot = begin + threadIdx.x; slot < end; slot += threads) {
    const unsigned int row = slot / s.slots, col = (slot - row * s.slots) * 8;
    const int left = (int)(s.cols - col);
    const size_t e = base + (size_t)row * s.cols + col;
    float g[8];
    if (s.bf16) load8(static_cast<const uint16_t*>(s.grad) + e, left, s.vectors, g);
    else load8(static_cast<const float*>(s.grad) + e, left, s.vectors, g);
    if (s.momentum) {
      float m[8];
      load8(s.momentum + e, left, s.vectors, m);
      if (WRITE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = p.beta * m[j] + g[j];
        if (s.vectors && left >= 8) {
          float4* d = reinterpret_cast<float4*>(s.momentum + e);
          d[0] = make_float4(m[0], m[1], m[2], m[3]);
          d[1] = make_float4(m[4], m[5], m[6], m[7]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left) s.momentum[e + j] = m[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = p.nesterov ? g[j] + p.beta * m[j] : m[j];
    }
    use(row, col, left, g);
  }
}

// One chunk of one matrix.
template <bool WRITE, class F>
__device__ __forceinline__ void walk_chunk(const PrepareParams& p, const Place& at, F use) {
  const unsigned int begin = at.chunk * p.chunk, total = at.s->rows * at.s->slots;
  walk<WRITE>(p, *at.s, at.matrix, begin, min(begin + p.chunk, total), kThreads, use);
}

// Momentum, and a chunk's sum of squares.  Bound by HBM: momentum is read and written, the gradient read (2 layers of 101M
// fp32 elements: 6.6 to 6.8 TB/s).  A second pass has to follow, as the norm needs all chunks; both read 8 elements at once,
// four times before the first is used.
__global__ void __launch_bounds__(kThreads) norm_sum_kernel(const __grid_constant__ PrepareParams p) {
  pdl_enter();
  const Place at = place(p, blockIdx.x);
  float sum = 0.0f;
  walk_chunk<true>(p, at, [&](unsigned, unsigned, int, const float (&u)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += u[j] * u[j];
  });
  sum = block_sum(sum);
  if (threadIdx.x == 0) p.partial[blockIdx.x] = sum;
}

// The power of two that brings `bound` to at most 2^13 (1 for a bound of 0).
__device__ __forceinline__ float power_for(float bound) {
  if (bound == 0.0f) return 1.0f;
  const float e = floorf(13.0f - log2f(bound));
  return exp2f(fminf(fmaxf(e, -100.0f), 100.0f) + (bound - bound));  // NaN stays NaN
}

// What the epilogues multiply with.  With X = r X', A = A' / sa, B = B' / sb (primed: as held):
//   A' = sa r^2 X' X'^T;  B' = sb a I + sb b / sa A' + sb c / sa^2 A' A';  X_next' = s r / sb B' X'
__device__ __forceinline__ void coefficients(const PrepareParams& p, float norm, float scale, int step, float* to) {
  const float part = norm == 0.0f ? 0.0f : norm / (norm + p.eps);  // of the first X; below 1 where eps counts
  const auto bound = [&](int k) {
    float b = part;
    for (int i = 0; i < k; ++i) b *= p.growth;
    return fminf(p.cap[k], b) + (part - part);
  };
  const float now = bound(step), sq = now * now;
  const float r = norm == 0.0f ? 1.0f : step == 0 ? 1.0f / (norm + p.eps) / power_for(norm) : 1.0f / power_for(now);
  const float sa = power_for(sq), sb = power_for(fabsf(p.a) + fabsf(p.b) * sq + fabsf(p.c) * sq * sq);
  const float s = step + 1 == p.steps ? scale : power_for(bound(step + 1));
  to[0] = sa * r * r;
  to[1] = sb / sa * p.b;
  to[2] = sb / sa * p.c / sa;
  to[3] = sb * p.a;
  to[4] = s * r / sb;
}

// The norm from its parts (every block for itself, in one order), the factors of all steps, and u times a power of two
// in fp16.  Bound by HBM, but for what the kernel before has left in L2; of one matrix of very many chunks by their
// sums, which every block reads: 8192 x 28672 (14336 chunks) fp32 takes 217 us, 6.5 TB/s, 65536 x 16384 (65536) 1500 to 2100,
// 4.3 to 3.1 TB/s.
__global__ void __launch_bounds__(kThreads) halve_kernel(const __grid_constant__ PrepareParams p) {
  pdl_enter();
  // from the last chunk to the first: it begins with what the kernel before has left in L2
  const unsigned int block = gridDim.x - 1 - blockIdx.x;
  const Place at = place(p, block);
  const Stack& s = *at.s;
  const float* partial = p.partial + (block - at.chunk);
  float sum = 0.0f;
  for (unsigned int i = threadIdx.x; i < s.chunks; i += kThreads) sum += partial[i];
  const float norm = sqrtf(block_sum(sum));
  const unsigned int matrix = s.matrix + at.matrix;
  if (at.chunk == 0) {
    if (threadIdx.x < p.steps)
      coefficients(p, norm, s.scale, threadIdx.x, p.coefs + ((size_t)matrix * p.steps + threadIdx.x) * kCoefs);
    if (threadIdx.x == 0) p.done[matrix] = 0;
    if (threadIdx.x == 0) p.outs[matrix] = static_cast<uint16_t*>(s.out) + (size_t)at.matrix * s.rows * s.cols;
  }
  const float power = power_for(norm);
  __half* x = s.x + (size_t)at.matrix * s.rows * s.pitch;
  walk_chunk<false>(p, at, [&](unsigned row, unsigned col, int, const float (&u)[8]) {
    __half2 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(u[2 * j] * power, u[2 * j + 1] * power);
    *reinterpret_cast<uint4*>(x + (size_t)row * s.pitch + col) = *reinterpret_cast<const uint4*>(h);
  });
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What B's diagonal loses when it is rounded: the factor of B's rows (or, as B is symmetric, columns) in the last
// product's epilogue that makes up for it.  It goes with the whole row, so it may only be a rounding's, 1 +- 2^-11: under
// coefficients whose polynomial has a root the element can come below fp16's normal values, where a step is a larger part of
// it than the row's other elements can bear, and what it loses is at most 2^-25 beside a bound of 2^12 or more.
__device__ __forceinline__ float rounding_rest(float exact, float rounded) {
  return fabsf(rounded) < 0x1p-14f ? 1.0f : __fdividef(exact, rounded);  // (NaN stays)
}

// ------------------------------------------------------------------ small matrices, whole in one block

// Up to 128 by 512 a matrix stays in one block's shared memory through all steps, and so do A and B: what
// a step costs is the matrix instructions' way and three turns through the registers (about 3 us), where the
// tiles of the launch below go through L2 and wait for one another (10 us).
//
// X lies as boxes of 128 rows (the short side) by 64 columns, 128-byte swizzle.  The first product reads
// it with the columns as k, the third with the rows as k: the tensor cores take the same bytes both ways.
// A and B are symmetric boxes of 128 x 64 each, two behind one another.
constexpr int kSmallSide = 128, kSmallLong = 512, kSmallThreads = 512;
constexpr int kBox = kSmallSide * 128;  // bytes
constexpr int kSquareBytes = 2 * kBox;

struct SmallShared {
  uint64_t done;
  uint32_t tmem, late;
  float coefs[kMaxSteps * kCoefs], rest[kSmallSide];
};

constexpr int small_bytes(int boxes) { return 1024 + 2 * kSquareBytes + boxes * kBox + (int)sizeof(SmallShared); }

// Address of 16 bytes: row, 8 columns from `col` on.
__device__ __forceinline__ uint32_t swizzled(uint32_t base, int row, int col) {
  return base + (col >> 6) * kBox + row * 128 + (((col >> 3 & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ void put16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Eight columns of x old + y sum, rounded to fp16 (or bf16).
__device__ __forceinline__ uint4 combine8(float x, uint4 old, float y, const float* v, bool bf16) {
  const uint32_t o[4] = {old.x, old.y, old.z, old.w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
    const float lo = x * b.x + y * v[2 * i], hi = x * b.y + y * v[2 * i + 1];
    w[i] = bf16 ? pack_bf16x2(lo, hi) : half2_bits(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int COLUMNS>  // of tensor memory: at least 128, at least the long side
__global__ void __launch_bounds__(kSmallThreads, COLUMNS == 128 ? 2 : 1) small_kernel(const __grid_constant__ PrepareParams p) {
  extern __shared__ uint8_t raw[];
  const uint32_t base = (mma::saddr(raw) + 1023) & ~1023u;
  const uint32_t sa = base, sb = base + kSquareBytes, sx = base + 2 * kSquareBytes;
  constexpr int kBoxes = COLUMNS / 64;
  auto& s = *reinterpret_cast<SmallShared*>(raw + (sx + kBoxes * kBox - mma::saddr(raw)));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mma::bar_init(mma::saddr(&s.done), 1);
    s.late = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_enter();
  if (warp == 0) mma::tmem_alloc<1>(mma::saddr(&s.tmem), COLUMNS);
  const Place at = place(p, blockIdx.x);  // a chunk is a whole matrix here
  const Stack& k = *at.s;
  const unsigned int matrix = at.matrix;
  const bool wide = k.rows <= k.cols;
  const int side = wide ? k.rows : k.cols, length = wide ? k.cols : k.rows;
  const int boxes = (length + 63) / 64;
  const unsigned int total = k.rows * k.slots;

  float sum = 0.0f;
  walk<true>(p, k, matrix, 0, total, kSmallThreads, [&](unsigned, unsigned, int, const float (&u)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += u[j] * u[j];
  });
  const float norm = sqrtf(block_sum<kSmallThreads>(sum));
  if (threadIdx.x < p.steps) coefficients(p, norm, k.scale, threadIdx.x, s.coefs + threadIdx.x * kCoefs);
  const float power = power_for(norm);
  // zeros behind the matrix' sides
  for (int v = threadIdx.x; v < boxes * (kBox / 16); v += kSmallThreads) put16(sx + v * 16, make_uint4(0, 0, 0, 0));
  __syncthreads();
  walk<false>(p, k, matrix, 0, total, kSmallThreads, [&](unsigned row, unsigned col, int left, const float (&u)[8]) {
    __half h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __float2half_rn(u[j] * power);
    if (wide) {  // u is 0 behind the row's end
      put16(swizzled(sx, row, col), *reinterpret_cast<const uint4*>(h));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left)
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(swizzled(sx, col + j, row) + (row & 7) * 2),
                       "h"(__half_as_ushort(h[j]))
                       : "memory");
    }
  });
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  mma::fence_before();
  __syncthreads();
  mma::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s.tmem);
  volatile uint32_t* late = &s.late;
  uint32_t phase = 0;
  const int row = (warp & 3) * 32 + lane, group = warp >> 2;   // of four groups of columns
  const uint32_t mine = tmem + ((uint32_t)(warp & 3) * 32 << 16);
  const bool one = mma::elect();
  bool ok = true;
  const auto wait = [&] {  // for the matrix instructions
    ok = mma::warp_wait(mma::saddr(&s.done), phase, late) && ok;
    phase ^= 1;
    mma::fence_after();
  };
  const auto hand_over = [&] {  // what the threads have stored, to the matrix instructions
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    mma::fence_before();
    __syncthreads();
    mma::fence_after();
  };
  const auto sums = [&](int col, float (&v)[32]) {
    if (ok) {
      mma::tmem_rows(mine + col, v);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __int_as_float(0x7fc00000);
    }
  };
  const uint32_t square = mma::instruction<1>(false, true, true, kSmallSide);
  for (int step = 0; step < p.steps; ++step) {
    const float* f = s.coefs + step * kCoefs;
    const bool last = step + 1 == p.steps;
    if (warp == 0 && one) {
      for (int b = 0; b < boxes; ++b)
        for (int i = 0; i < 4; ++i) {
          const uint64_t d = mma::operand_desc(sx + b * kBox, true) + i * mma::depth_step(true);
          mma::mma_f16<1>(tmem, d, d, square, b + i > 0);
        }
      mma::mma_commit<1>(mma::saddr(&s.done));
    }
    __syncwarp();
    wait();
    float v[32];
    uint4 a[4];
    sums(group * 32, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = combine8(0.0f, make_uint4(0, 0, 0, 0), f[0], v + 8 * i, false);
      put16(swizzled(sa, row, group * 32 + 8 * i), a[i]);
    }
    hand_over();
    if (warp == 0 && one) {
      for (int b = 0; b < 2; ++b)
        for (int i = 0; i < 4; ++i) {
          const uint64_t d = mma::operand_desc(sa + b * kBox, true) + i * mma::depth_step(true);
          mma::mma_f16<1>(tmem, d, d, square, b + i > 0);
        }
      mma::mma_commit<1>(mma::saddr(&s.done));
    }
    __syncwarp();
    wait();
    sums(group * 32, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = f[2] * v[i] + (group * 32 + i == row ? f[3] : 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) put16(swizzled(sb, row, group * 32 + 8 * i), combine8(f[1], a[i], 1.0f, v + 8 * i, false));
    if ((warp & 3) == group) {  // lane l has row and column l of a block on the diagonal
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) sum = i == lane ? v[i] : sum;
      const auto at = [&](uint32_t base) {
        uint16_t h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(swizzled(base, row, row) + (row & 7) * 2) : "memory");
        return __half2float(__ushort_as_half(h));
      };
      s.rest[row] = rounding_rest(f[1] * at(sa) + sum, at(sb));
    }
    hand_over();
    if (warp == 0 && one) {
      // X with its columns contiguous: the next 64 of them are a box away
      for (int n = 0; n < boxes * 64; n += 256) {
        const int columns = min(256, boxes * 64 - n);
        const uint32_t idesc = mma::instruction<1>(false, true, false, columns);
        for (int i = 0; i < kSmallSide / 16; ++i) {
          const uint64_t l = mma::operand_desc(sb + (i >> 2) * kBox, true) + (i & 3) * mma::depth_step(true);
          const uint64_t r = mma::operand_desc(sx + (n >> 6) * kBox, false, kBox) + i * mma::depth_step(false);
          mma::mma_f16<1>(tmem + n, l, r, idesc, i > 0);
        }
      }
      mma::mma_commit<1>(mma::saddr(&s.done));
    }
    __syncwarp();
    wait();
    for (int col = group * 32; col < boxes * 64; col += 128) {
      sums(col, v);
      uint16_t* out = static_cast<uint16_t*>(k.out) + (size_t)matrix * k.rows * k.cols;
      if (wide) out += (size_t)row * length + col;
      else out += (size_t)col * side + row;
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = swizzled(sx, row, col + 8 * i);
        const uint4 r = combine8(0.0f, make_uint4(0, 0, 0, 0), f[4] * s.rest[row], v + 8 * i, last);
        if (!last) put16(x, r);
        else if (wide && k.out_vectors && row < side && col + 8 * i + 8 <= length) *reinterpret_cast<uint4*>(out + 8 * i) = r;
        w[4 * i] = r.x, w[4 * i + 1] = r.y, w[4 * i + 2] = r.z, w[4 * i + 3] = r.w;
      }
      if (last && row < side && !(wide && k.out_vectors)) {
        const size_t stride = wide ? 1 : side;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i < length) out[i * stride] = (uint16_t)(w[i / 2] >> (i % 2 * 16));
      }
    }
    hand_over();
  }
  if (__syncthreads_or(*late != 0)) {  // what the matrix instructions still do takes microseconds; 10 ms are theirs
    for (int i = 0; i < 10000; ++i) __nanosleep(1000);
    __syncthreads();
  }
  if (warp == 0) mma::tmem_free<1>(tmem, COLUMNS);
}

// ------------------------------------------------------------------ the products

enum Stage : int { kGram, kSquare, kApply };

// The matrices of one shape in the product kernel.  A stage's result has nj rows of ni.
struct Shape {
  CUtensorMap gram[2][2], apply[2], a[2], b;   // of X in either place, as either operand; of A, as either; of B
  mma::Kind gram_kind, apply_kind;
  int rows, cols, side;
  int x_pitch, a_pitch;          // multiples of 64; what lies behind a row's end counts nowhere
  int count, matrix;             // matrices, and the number of the first
  int first[3], tiles[3];        // of each stage: first tile in it, tiles of a matrix
  __half *x[2], *to_a, *to_b;
  float* rest;                   // of B's diagonal, a_pitch apart
  bool vectors;                  // the results' rows are whole 16 bytes
};

struct StepsParams {
  Shape shape[kMaxShapes];
  int shapes, steps;
  int stage_tiles[3], width;     // columns of a tile
  const float* coefs;            // kCoefs per matrix and step
  void* const* outs;             // where the results of the last step go
  unsigned int* done;            // per matrix: blocks that have stored their part of a tile
};

// All tiles of all steps in one launch: those of the first product of all matrices, of the second, of the
// third, then the next step's.  A tile waits until all tiles of its matrix before it are stored, which
// with several matrices they mostly are: nobody waits for the last tile of a launch, and a step of a small
// matrix costs three times the way through the chip, not three launches (256 x 256, five steps: 144 us
// so, 98 in one launch, 74 with tiles of half the width).  16 x 1024 x 2048: 590 us, of which 93 are the passes over the
// gradients; a further step takes 84 us for 133 GFLOP executed, 1.58 PFLOP/s.  2 layers of 101M elements: 2590 to 2730 us,
// passes 316, a step 462 us for 721 GFLOP, 1.56 PFLOP/s.  Bound by the matrix instructions under the power cap (cuBLAS's
// sustained rate is 1.72) and, at 1024 x 2048, by epilogues of 5 us beside products of 6.5 us a tile.  Not so far: a short
// side's A is one tile or two whose sum runs over the whole long side (16 of 64 x 8192: 260 us, 48 a step), and many of a
// middle size are bound by the epilogues of their short sums (300 of 200 x 300: 465 us, 200 of 256 x 256 211).
template <int CG>
struct Steps {
  static constexpr bool kBf16 = false, kOrdered = true;
  static constexpr int kStages = 6, kBytesB = 2 * mma::kBoxBytes, kAreas = 1, kArea = 2048, kRun = 0;
  static constexpr int kSide = 128 * CG;
  static constexpr unsigned int kFailed = 1u << 31;  // in a matrix' count: a block that had tiles of it has given up
  using Params = StepsParams;
  struct Local {};
  static __device__ __forceinline__ void begin(const Params&, Local&) {}
  static __device__ __forceinline__ bool tile(const Params& p, const Local&, int t, Tile& w) {
    const int per_step = p.stage_tiles[0] + p.stage_tiles[1] + p.stage_tiles[2];
    const int step = t / per_step;
    if (step >= p.steps) return false;
    t -= step * per_step;
    int stage = 0;
    while (t >= p.stage_tiles[stage]) t -= p.stage_tiles[stage++];
    int q = 0;
    while (q + 1 < p.shapes && p.shape[q + 1].first[stage] <= t) ++q;
    const Shape& s = p.shape[q];
    const int z = (t - s.first[stage]) / s.tiles[stage];
    int j = (t - s.first[stage]) - z * s.tiles[stage], i;
    const bool wide = s.rows <= s.cols;
    int nj = s.side;
    if (stage == kApply) {
      // the shorter side first: what is on the GPU at once covers all of it, and X is read once
      const int fi = (s.cols + kSide - 1) / kSide, fj = (s.rows + p.width - 1) / p.width;
      i = wide ? j / fj : j % fi;
      j = wide ? j % fj : j / fi;
      nj = s.rows;
      // lanes are the columns of X: D[i, j] = sum_k X[k, i] B[j, k] of a wide one, sum_k B[i, k] X[j, k] of a tall one
      w.a = wide ? &s.apply[step & 1] : &s.b;
      w.b = wide ? &s.b : &s.apply[step & 1];
      w.a_kind = wide ? s.apply_kind : mma::kDepthRows;
      w.b_kind = wide ? mma::kDepthRows : s.apply_kind;
    } else if (p.width == kSide) {  // on and above the diagonal: column j of blocks has j + 1 of them
      int c = (int)((sqrtf(8.0f * j + 1.0f) - 1.0f) * 0.5f);
      while ((c + 1) * (c + 2) / 2 <= j) ++c;
      while (c * (c + 1) / 2 > j) --c;
      i = j - c * (c + 1) / 2;
      j = c;
    } else {  // columns 2 c and 2 c + 1 of half blocks have c + 1 each
      int c = (int)((sqrtf(4.0f * j + 1.0f) - 1.0f) * 0.5f);
      while ((c + 1) * (c + 2) <= j) ++c;
      while (c * (c + 1) > j) --c;
      const int rest = j - c * (c + 1);
      i = rest % (c + 1);
      j = 2 * c + rest / (c + 1);
    }
    if (stage != kApply) {
      w.a = stage == kGram ? &s.gram[step & 1][0] : &s.a[0];
      w.b = stage == kGram ? &s.gram[step & 1][1] : &s.a[1];
      w.a_kind = w.b_kind = stage == kGram ? s.gram_kind : mma::kDepthRows;
    }
    w.a_row = i * kSide;
    w.b_row = j * p.width;
    w.a_z = w.b_z = z;
    w.k = 0;
    w.blocks = ((stage == kGram ? max(s.rows, s.cols) : s.side) + mma::kDepth - 1) / mma::kDepth;
    w.last = mma::kDepth;
    const int unit = (w.b_kind == mma::kDepthRows ? 16 : 64) * CG;
    w.columns = min(p.width, (nj - w.b_row + unit - 1) / unit * unit);
    w.b_bytes = p.width / CG * 128;
    w.shape = q;
    w.stage = stage;
    w.step = step;
    return true;
  }

  // The tiles of this matrix before this stage, each in CG parts.
  static __device__ __forceinline__ bool wait(const Params& p, const Tile& w, volatile uint32_t* late) {
    const Shape& s = p.shape[w.shape];
    unsigned int before = (s.tiles[0] + s.tiles[1] + s.tiles[2]) * w.step;
    for (int i = 0; i < w.stage; ++i) before += s.tiles[i];
    before *= CG;
    if (before == 0) return true;
    const unsigned int* at = p.done + s.matrix + w.a_z;
    bool ok = false;
    const uint64_t begin = mma::nanoseconds();
    for (uint32_t n = 1;; ++n) {
      unsigned int v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
      ok = v >= before && !(v & kFailed);
      if (ok || *late || (v & kFailed) || (n % 256 == 0 && mma::nanoseconds() - begin > mma::kLimit)) break;
    }
    if (!ok) *late = 1;
    return __all_sync(~0u, ok);
  }
  static __device__ __forceinline__ void done(const Params& p, const Tile& w, bool ok) {
    unsigned int* at = p.done + p.shape[w.shape].matrix + w.a_z;
    __threadfence();
    if (ok) atomicAdd(at, 1u);
    else atomicOr(at, kFailed);
  }
  // Whether the tile is of the results, not of what goes between the products.
  static __device__ __forceinline__ bool result(const Params& p, const Tile& w) {
    return w.stage == kApply && w.step + 1 == p.steps;
  }

  // Of the sum (0) and, of the second product, of A (1) in the epilogue.
  static __device__ __forceinline__ float factor(const Params& p, const Tile& w, int which) {
    const float* f = p.coefs + ((long long)(p.shape[w.shape].matrix + w.a_z) * p.steps + w.step) * kCoefs;
    if (which == 0) return __ldcg(f + 2 * w.stage);
    return w.stage == kSquare ? __ldcg(f + 1) : 0.0f;
  }

  struct Epilogue {
    float x, y, diagonal;        // of A, of the sum; what is added where row and column are the same
    int row, column;             // of the warp's first lane, of the tile
    const __half* old;           // A, of the tile's first column, the warp's first lane; NULL: none
    uint16_t *to, *mirror;       // likewise; a block above the diagonal is stored a second time, lanes as rows
    long long stride, stride_in; // of the results' columns; of A's, and of the mirrored rows
    int lanes, columns, pads, pad_columns;  // of the sides, and with what lies behind a row's end
    bool last, vectors, on_diagonal, tall;
    uint32_t staging;
    float* rest;                 // of the second product: where to keep the diagonal's; of the third: its columns'
    float rows[4];               // of the third: of a lane's rows
    uint4 next[4];               // of the next chunk, loaded ahead: A, or the columns' factors

    __device__ __forceinline__ Epilogue(const Params& p, const Local&, const Tile& w, int row, int c,
                                        mma::Staging& area, const float* factors)
        : x(factors[1]), y(factors[0]), diagonal(0.0f), row(row), column(w.b_row), staging(area.base) {
      const Shape& s = p.shape[w.shape];
      const int z = w.a_z, matrix = s.matrix + z;
      const int ni = w.stage == kApply ? s.cols : s.side, nj = w.stage == kApply ? s.rows : s.side;
      const int pitch = w.stage == kApply ? s.x_pitch : s.a_pitch;
      const long long at = (long long)z * nj * pitch, here = at + (long long)w.b_row * pitch + row;
      last = w.stage == kApply && w.step + 1 == p.steps;
      vectors = true;
      on_diagonal = false;
      stride = stride_in = pitch;
      old = nullptr;
      mirror = nullptr;
      rest = nullptr;
      tall = w.stage == kApply && s.rows > s.cols;
      if (w.stage == kApply) {
        const float* factors = s.rest + (long long)z * s.a_pitch;
        if (!tall) {
          rest = const_cast<float*>(factors);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = row + (threadIdx.x & 31) / 4 + 8 * i;
            rows[i] = at < ni ? __ldcg(factors + at) : 1.0f;
          }
        }
        to = reinterpret_cast<uint16_t*>(s.x[(w.step + 1) & 1]) + here;
        if (last) {
          stride = ni;
          to = static_cast<uint16_t*>(p.outs[matrix]) + (long long)w.b_row * ni + row;
          vectors = s.vectors;
        }
      } else {
        uint16_t* result = reinterpret_cast<uint16_t*>(w.stage == kGram ? s.to_a : s.to_b);
        to = result + here;
        if (w.b_row >= w.a_row + kSide) mirror = result + at + (long long)row * pitch + w.b_row;
        if (w.stage == kSquare) {
          old = s.to_a + here;
          rest = s.rest + (long long)z * s.a_pitch;
          on_diagonal = !mirror;
          if (on_diagonal) diagonal = __ldcg(p.coefs + ((long long)matrix * p.steps + w.step) * kCoefs + 3);
        }
      }
      lanes = ni - row;
      pads = pitch - row;
      columns = min(w.columns, nj - w.b_row);
      pad_columns = pitch - w.b_row;
      load_next(c);
    }

    __device__ __forceinline__ void load_next(int c) {
      if (!old) {
        if (!rest) return;
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // whole pairs: `rest` is as long as a padded row
          const int at = c + 8 * q + 2 * (threadIdx.x & 3);
          const float2 f = at < columns ? __ldcg(reinterpret_cast<const float2*>(rest + column + at)) : make_float2(1.0f, 1.0f);
          next[q].x = __float_as_uint(f.x);
          next[q].y = __float_as_uint(f.y);
        }
        return;
      }
      const int lane = threadIdx.x & 31, part = lane & 3, column = c + (lane >> 2);
      const __half* from = old + column * stride_in + part * 8;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        next[q] = make_uint4(0, 0, 0, 0);
        if (column + 8 * q < columns && part * 8 < pads)
          next[q] = __ldcg(reinterpret_cast<const uint4*>(from + q * (8 * stride_in)));
      }
    }

    __device__ __forceinline__ void chunk(uint32_t at, int c, mma::Source source, bool) {
      const int lane = threadIdx.x & 31;
      uint32_t o[16] = {};
      if (old) {
        // A's columns into the staging memory, and out again as fragments
        const int part = lane & 3;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                           mma::staged(staging, 8 * q + (lane >> 2), part)),
                       "r"(next[q].x), "r"(next[q].y), "r"(next[q].z), "r"(next[q].w)
                       : "memory");
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(o[2 * q]), "=r"(o[2 * q + 1]), "=r"(o[8 + 2 * q]), "=r"(o[8 + 2 * q + 1])
                       : "r"(mma::staged(staging, 8 * q + (lane & 7), lane >> 3))
                       : "memory");
        __syncwarp();
      } else if (rest) {
#pragma unroll
        for (int q = 0; q < 4; ++q) o[2 * q] = next[q].x, o[2 * q + 1] = next[q].y;
      }
      load_next(c + mma::kChunkStep);
      float v[32];
      if (source == mma::kSums) {
        mma::tmem_fragments(at, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = source == mma::kZeros ? 0.0f : __int_as_float(0x7fc00000);
      }
      uint32_t w[16];
      // A 32 x 32 block lies on the diagonal or off it.  On it a lane's rows lane / 4 + 8 k meet the columns 8 k +
      // 2 (lane % 4) and the next: four elements of every fourth lane are the diagonal's.
      const bool mine = on_diagonal && row == column + c && lane >> 3 == (lane & 3), upper = lane >> 2 & 1;
      if (old) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
          float lo = y * v[2 * i] + x * b.x, hi = y * v[2 * i + 1] + x * b.y;
          const int k = (i & 1) + 2 * (i >> 3);
          if ((i >> 1 & 3) == k && mine) {
            if (upper) hi += diagonal;
            else lo += diagonal;
            if ((lane >> 2) + 8 * k < lanes)
              rest[row + (lane >> 2) + 8 * k] =
                  rounding_rest(upper ? hi : lo, __half2float(__float2half_rn(upper ? hi : lo)));
          }
          w[i] = half2_bits(lo, hi);
        }
      } else {
        // the columns' factors, or the lane's rows'
        float f[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = rest ? y * __uint_as_float(o[q]) : y;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int q = i >> 1 & 3;
          float lo = f[2 * q] * v[2 * i], hi = f[2 * q + 1] * v[2 * i + 1];
          if (tall) lo *= rows[(i & 1) + 2 * (i >> 3)], hi *= rows[(i & 1) + 2 * (i >> 3)];
          w[i] = last ? pack_bf16x2(lo, hi) : half2_bits(lo, hi);
        }
      }
      mma::stage_columns(staging, w);
      __syncwarp();
      mma::put_columns(staging, to + c * stride, stride, last ? lanes : pads, columns - c, vectors);
      __syncwarp();
      if (mirror) {
        // as rows: the four matrices of rows 8 h and on are its columns 0, 8, 16 and 24
#pragma unroll
        for (int h = 0; h < 4; ++h)
          asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                           mma::staged(staging, 8 * h + (lane & 7), lane >> 3)),
                       "r"(w[8 * (h / 2) + h % 2]), "r"(w[8 * (h / 2) + 2 + h % 2]), "r"(w[8 * (h / 2) + 4 + h % 2]),
                       "r"(w[8 * (h / 2) + 6 + h % 2])
                       : "memory");
        __syncwarp();
        mma::put_columns(staging, mirror + c, stride_in, pad_columns - c, lanes, true);
        __syncwarp();
      }
    }
  };
};

// How the products are cut: blocks alone or in pairs, columns of a tile.
struct Cut {
  int pair, width;
};
// A tile's slice and its epilogue, in us: the loads of 16 KiB of A and 8 or 16 of B a block bound a slice but of the
// whole pair's tile, which the matrix instructions do.  Updates measured with each cut, us: 256 x 256 104, 83, 89, 75;
// 1024 x 1024 170, 134, 137, 119; 4 x 1024 x 2048 214, 196, 206, 282; 16 of them 468, 609, 624, 1054.  Not always the
// best: 2048 x 8192 527, 544, 595, 989 (takes the second), and many short sums take longer than estimated, as kEnd is less than
// half of their epilogue (300 x 200 x 300: 447, 571, 422, 594, estimated 240 for the third).
constexpr Cut kCuts[4] = {{2, 256}, {2, 128}, {1, 128}, {1, 64}};
constexpr double kSlice[4] = {0.30, 0.17, 0.18, 0.14}, kEnd[4] = {1.5, 0.8, 0.8, 0.4};
constexpr double kTurn = 3.0;  // of a stage, from its last tile's sums to the next stage's first

long long stage_tiles(int stage, long long rows, long long cols, const Cut& cut) {
  const auto over = [](long long n, long long d) { return (n + d - 1) / d; };
  const long long side = 128 * cut.pair;
  if (stage == kApply) return over(cols, side) * over(rows, cut.width);
  const long long fj = over(std::min(rows, cols), cut.width), q = fj / 2;
  return cut.width == side ? fj * (fj + 1) / 2 : q * (q + 1) + (fj & 1 ? q + 1 : 0);
}

// Time of a step of `n` shapes: a stage takes its tiles' time over all multiprocessors, but at least a tile's.
struct Sizes {
  long long rows, cols, count;
};
double step_time(const Sizes* sizes, int n, int cut, int sms) {
  double time = 0.0;
  for (int stage = 0; stage < 3; ++stage) {
    double work = 0.0, longest = 0.0;
    for (int q = 0; q < n; ++q) {
      const Sizes& s = sizes[q];
      const long long depth = stage == kGram ? std::max(s.rows, s.cols) : std::min(s.rows, s.cols);
      const double tile = kSlice[cut] * ((depth + 63) / 64) + kEnd[cut];
      work += tile * (double)(stage_tiles(stage, s.rows, s.cols, kCuts[cut]) * s.count);
      longest = std::max(longest, tile);
    }
    time += std::max(work / std::max(1, sms / kCuts[cut].pair), longest) + kTurn;
  }
  return time;
}
int best_cut(const Sizes* sizes, int n, int sms) {
  int best = 0;
  for (int i = 1; i < 4; ++i)
    if (step_time(sizes, n, i, sms) < step_time(sizes, n, best, sms)) best = i;
  return best;
}

// ------------------------------------------------------------------ one group of stacks

// Tensor-memory columns of the kernel that takes matrices of this shape whole; 0: they go in tiles.
int whole_columns(size_t rows, size_t cols) {
  const size_t side = std::min(rows, cols), length = std::max(rows, cols);
  return side > kSmallSide || length > kSmallLong ? 0 : length <= 128 ? 128 : length <= 256 ? 256 : 512;
}

// The small matrices go whole where that is faster.  Alone they nearly always do; beside others, whose tiles
// leave room for theirs, it is the time of a launch more.  Times in us, measured,
// whole and in the best tiles: 128 x 128 27 and 58, 400 of them 60 and 105, 128 x 512 50 and 70, 1000 of 16 x 16 95 and 191.
bool take_whole(const OrthogonalCall& c) {
  double alone = 0.0;
  Sizes rest[kMaxShapes], all[kMaxShapes];
  int nr = 0, na = 0;
  double whole[3] = {}, longest[3] = {};
  for (size_t i = 0; i < c.nstacks; ++i) {
    if (!c.counts[i] || !c.rows[i] || !c.cols[i]) continue;
    const Sizes s = {(long long)c.rows[i], (long long)c.cols[i], (long long)c.counts[i]};
    const auto put = [&](Sizes* to, int& n) {  // shapes beyond kMaxShapes count as the last
      for (int q = 0; q < n; ++q)
        if ((to[q].rows == s.rows && to[q].cols == s.cols) || q == kMaxShapes - 1) {
          to[q].count += s.count;
          return;
        }
      to[n++] = s;
    };
    put(all, na);
    const int columns = whole_columns(c.rows[i], c.cols[i]);
    if (!columns) {
      put(rest, nr);
      continue;
    }
    const int k = columns == 512 ? 2 : columns == 256 ? 1 : 0;
    const double length = (double)std::max(c.rows[i], c.cols[i]);
    whole[k] += (double)c.counts[i];
    longest[k] = std::max(longest[k], 6.0 + 0.035 * length + c.steps * (2.2 + 0.008 * length));
  }
  for (int k = 0; k < 3; ++k) alone += longest[k] * std::ceil(whole[k] / (c.sms * (k == 0 ? 2 : 1)));
  const double start = 10.0;
  const auto tiles = [&](const Sizes* s, int n) {
    return n ? start + c.steps * step_time(s, n, best_cut(s, n, c.sms), c.sms) : 0.0;
  };
  return alone + tiles(rest, nr) <= tiles(all, na);
}

// The matrices of one shape, and where they lie in the workspace.
struct Class {
  size_t rows, cols, count;
  unsigned int matrix;           // number of the first
  __half *x[2], *a, *b;
  float* rest;
  bool vectors;
};

size_t up(size_t n, size_t unit) { return (n + unit - 1) / unit * unit; }

// Stacks [first, end) of the call with at most kMaxShapes shapes; their workspace, laid out from `base`.
struct Group {
  size_t end;
  int classes;
  Class cls[kMaxShapes];
  short of[kMaxStacks];          // class of each stack, -1: empty, or taken whole
  size_t matrices, chunks, bytes;
  unsigned int chunk;            // slots
  float *partial, *coefs;
  void** outs;
  unsigned int* done;
};

size_t slots_of(size_t rows, size_t cols) { return rows * (up(cols, 8) / 8); }
// Slots of a chunk for so many in all: about 1200 blocks, whole rounds of a block's threads.
unsigned int chunk_for(size_t slots) {
  return (unsigned int)std::min<size_t>(kMostChunk, std::max<size_t>(kThreads, slots / 1200 / kThreads * kThreads));
}

// The tiles of a matrix in the stage that has most, cut as finely as any cut does.
long long most_tiles(size_t rows, size_t cols) {
  long long most = 0;
  for (int stage = 0; stage < 3; ++stage)
    most = std::max(most, stage_tiles(stage, (long long)rows, (long long)cols, kCuts[3]));
  return most;
}

// `whole`: without the small matrices.  A group ends where its tiles would be too many, but has one stack at least.
void gather(const OrthogonalCall& c, size_t first, bool whole, uint8_t* base, Group& g) {
  g.classes = 0;
  g.matrices = g.chunks = 0;
  size_t slots = 0;
  long long tiles = 0;
  size_t i = first;
  for (; i < c.nstacks && i - first < kMaxStacks; ++i) {
    short k = -1;
    if (c.counts[i] && c.rows[i] && c.cols[i] && !(whole && whole_columns(c.rows[i], c.cols[i]))) {
      const long long more = most_tiles(c.rows[i], c.cols[i]) * (long long)c.counts[i];
      if (tiles && tiles + more > kMaxTiles) break;
      tiles += more;
      for (k = 0; k < g.classes && !(g.cls[k].rows == c.rows[i] && g.cls[k].cols == c.cols[i]); ++k) {}
      if (k == g.classes) {
        if (g.classes == kMaxShapes) break;
        g.cls[g.classes++] = Class{c.rows[i], c.cols[i], 0, 0, {}, nullptr, nullptr, nullptr, true};
      }
      g.cls[k].count += c.counts[i];
      g.cls[k].vectors &= c.cols[i] % 8 == 0 && (c.outs == nullptr || ((uintptr_t)c.outs[i] & 15) == 0);
      g.matrices += c.counts[i];
      slots += c.counts[i] * slots_of(c.rows[i], c.cols[i]);
    }
    g.of[i - first] = k;
  }
  g.end = i;
  g.chunk = chunk_for(slots);
  for (i = first; i < g.end; ++i)
    if (g.of[i - first] >= 0) g.chunks += c.counts[i] * ((slots_of(c.rows[i], c.cols[i]) + g.chunk - 1) / g.chunk);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    uint8_t* p = base + at;
    at += up(bytes, 256);
    return p;
  };
  size_t matrix = 0;
  for (int k = 0; k < g.classes; ++k) {
    Class& l = g.cls[k];
    const size_t side = std::min(l.rows, l.cols), x = l.rows * up(l.cols, 64) * 2, a = side * up(side, 64) * 2;
    for (int j = 0; j < 2; ++j) l.x[j] = reinterpret_cast<__half*>(take(l.count * x));
    l.a = reinterpret_cast<__half*>(take(l.count * a));
    l.b = reinterpret_cast<__half*>(take(l.count * a));
    l.rest = reinterpret_cast<float*>(take(l.count * up(side, 64) * 4));
    l.matrix = (unsigned int)matrix;
    matrix += l.count;
  }
  g.partial = reinterpret_cast<float*>(take(g.chunks * 4));
  g.coefs = reinterpret_cast<float*>(take(g.matrices * c.steps * kCoefs * 4));
  g.outs = reinterpret_cast<void**>(take(g.matrices * 8));
  g.done = reinterpret_cast<unsigned int*>(take(g.matrices * 4));
  g.bytes = at;
}

// Bounds of the singular values before each step, from 1 on, and how far a step can multiply a small one.
// False where they grow out of any range.
bool bounds(const OrthogonalCall& c, float* cap, float* growth) {
  const double a = c.a, b = c.b, q = c.c;
  double most = 1.0, grow = 1e-30;
  for (int k = 0; k <= c.steps; ++k) {
    cap[k] = (float)most;
    if (!(cap[k] < 1e6f)) return false;
    // over [0, most], of f(s) = a + b s^2 + c s^4 and of s f(s): at the end, and where a derivative is 0
    double next = 1e-30;
    const auto at = [&](double t) {  // t = s^2
      if (!(t >= 0.0 && t <= most * most)) return;
      const double f = std::fabs(a + t * (b + t * q));
      next = std::max(next, std::sqrt(t) * f);
      grow = std::max(grow, f);
    };
    at(0.0);
    at(most * most);
    if (q != 0.0) at(-b / (2.0 * q));
    const double root = 9.0 * b * b - 20.0 * a * q;
    if (q != 0.0 && root >= 0.0) {
      at((-3.0 * b + std::sqrt(root)) / (10.0 * q));
      at((-3.0 * b - std::sqrt(root)) / (10.0 * q));
    } else if (q == 0.0 && b != 0.0) {
      at(-a / (3.0 * b));
    }
    most = 1.01 * next;
  }
  *growth = (float)(1.01 * grow);
  return *growth < 1e12f;
}

// What the kernels that read gradients have in common; no stacks yet.
void start(const OrthogonalCall& c, const float* cap, float growth, PrepareParams& p) {
  p.stacks = 0;
  p.beta = c.beta, p.nesterov = c.nesterov, p.eps = c.eps;
  p.a = c.a, p.b = c.b, p.c = c.c, p.growth = growth, p.steps = c.steps;
  std::memcpy(p.cap, cap, sizeof p.cap);
  p.chunk = 0;
  p.partial = p.coefs = nullptr, p.outs = nullptr, p.done = nullptr;
}

Stack& add(const OrthogonalCall& c, size_t i, size_t chunk, size_t chunks, PrepareParams& p) {
  float* m = c.momentum ? c.momentum[i] : nullptr;
  Stack& s = p.stack[p.stacks++];
  s.grad = c.grads[i], s.momentum = m, s.out = c.outs[i], s.x = nullptr;
  s.rows = (unsigned)c.rows[i], s.cols = (unsigned)c.cols[i], s.pitch = (unsigned)up(c.cols[i], 64);
  s.slots = (unsigned)(up(c.cols[i], 8) / 8);
  s.chunks = (unsigned)chunks, s.first = (unsigned)chunk, s.matrix = 0;
  s.bf16 = c.dtypes[i] == AR_BFLOAT16;
  s.vectors = c.cols[i] % 8 == 0 && ((uintptr_t)c.grads[i] & 15) == 0 && ((uintptr_t)m & 15) == 0;
  s.out_vectors = c.cols[i] % 8 == 0 && ((uintptr_t)c.outs[i] & 15) == 0;
  s.scale = c.scales ? c.scales[i] : 1.0f;
  return s;
}

// The stacks of small matrices, kMaxStacks at a time.
template <int COLUMNS>
cudaError_t run_whole(const OrthogonalCall& c, const float* cap, float growth) {
  constexpr int bytes = small_bytes(COLUMNS / 64);
  PrepareParams p;
  start(c, cap, growth, p);
  size_t matrices = 0;
  const auto launch = [&]() -> cudaError_t {
    if (p.stacks == 0) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(small_kernel<COLUMNS>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
      e = launch_kernel(small_kernel<COLUMNS>, dim3((unsigned)matrices), dim3(kSmallThreads), bytes, c.stream, true, p);
    p.stacks = 0;
    matrices = 0;
    return e;
  };
  for (size_t i = 0; i < c.nstacks; ++i) {
    if (!c.counts[i] || !c.rows[i] || !c.cols[i] || whole_columns(c.rows[i], c.cols[i]) != COLUMNS) continue;
    add(c, i, matrices, 1, p);
    matrices += c.counts[i];
    if (p.stacks == kMaxStacks) {
      const cudaError_t e = launch();
      if (e != cudaSuccess) return e;
    }
  }
  return launch();
}

cudaError_t run(const OrthogonalCall& c, const Group& g, size_t first, const float* cap, float growth) {
  PrepareParams p;
  start(c, cap, growth, p);
  p.chunk = g.chunk;
  p.partial = g.partial, p.coefs = g.coefs, p.outs = g.outs, p.done = g.done;
  size_t used[kMaxShapes] = {}, chunk = 0;
  for (size_t i = first; i < g.end; ++i) {
    const short k = g.of[i - first];
    if (k < 0) continue;
    const Class& l = g.cls[k];
    Stack& s = add(c, i, chunk, (slots_of(l.rows, l.cols) + g.chunk - 1) / g.chunk, p);
    s.x = l.x[0] + used[k] * l.rows * s.pitch;
    s.matrix = l.matrix + (unsigned)used[k];
    used[k] += c.counts[i];
    chunk += c.counts[i] * s.chunks;
  }
  if (p.stacks == 0) return cudaSuccess;
  cudaError_t e = launch_kernel(norm_sum_kernel, dim3((unsigned)chunk), dim3(kThreads), 0, c.stream, true, p);
  if (e == cudaSuccess) e = launch_kernel(halve_kernel, dim3((unsigned)chunk), dim3(kThreads), 0, c.stream, true, p);
  StepsParams q;
  Sizes sizes[kMaxShapes];
  for (int k = 0; k < g.classes; ++k)
    sizes[k] = Sizes{(long long)g.cls[k].rows, (long long)g.cls[k].cols, (long long)g.cls[k].count};
  const Cut cut = kCuts[best_cut(sizes, g.classes, c.sms)];
  const uint32_t half = (uint32_t)(cut.width / cut.pair);  // j of a block
  long long total[3] = {};
  for (int k = 0; e == cudaSuccess && k < g.classes; ++k) {
    const Class& l = g.cls[k];
    Shape& s = q.shape[k];
    const bool wide = l.rows <= l.cols;
    const size_t side = std::min(l.rows, l.cols), px = up(l.cols, 64), pa = up(side, 64);
    s.rows = (int)l.rows, s.cols = (int)l.cols, s.side = (int)side;
    s.x_pitch = (int)px, s.a_pitch = (int)pa;
    s.count = (int)l.count, s.matrix = (int)l.matrix;
    s.to_a = l.a, s.to_b = l.b, s.rest = l.rest;
    s.vectors = l.vectors;
    mma::Kind depth;
    const auto map = [&](CUtensorMap* to, mma::Kind* kind, const __half* at, size_t rows, size_t cols, size_t pitch,
                         bool depth, uint32_t box) {
      // as i or j the padded row is read: what lies behind its end becomes lanes or columns that nothing uses
      if (e == cudaSuccess)
        e = mma::make_map(to, kind, false, at, depth ? cols : pitch, rows, l.count, pitch, rows * pitch, depth, box);
    };
    for (int j = 0; j < 2; ++j) {
      s.x[j] = l.x[j];
      map(&s.gram[j][0], &s.gram_kind, l.x[j], l.rows, l.cols, px, wide, 128);
      map(&s.gram[j][1], &s.gram_kind, l.x[j], l.rows, l.cols, px, wide, half);
      map(&s.apply[j], &s.apply_kind, l.x[j], l.rows, l.cols, px, !wide, wide ? 128 : half);
    }
    map(&s.a[0], &depth, l.a, side, side, pa, true, 128);
    map(&s.a[1], &depth, l.a, side, side, pa, true, half);
    map(&s.b, &depth, l.b, side, side, pa, true, wide ? half : 128);
    for (int stage = 0; stage < 3; ++stage) {
      const long long one = stage_tiles(stage, sizes[k].rows, sizes[k].cols, cut);
      if (total[stage] + one * sizes[k].count > kMaxTiles) return cudaErrorInvalidValue;  // (one stack of 275 GB or more)
      s.first[stage] = (int)total[stage];
      s.tiles[stage] = (int)one;
      total[stage] += one * sizes[k].count;
    }
  }
  for (int stage = 0; stage < 3; ++stage) q.stage_tiles[stage] = (int)total[stage];
  q.width = cut.width;
  q.shapes = g.classes, q.steps = c.steps;
  q.coefs = g.coefs, q.outs = g.outs, q.done = g.done;
  if (e != cudaSuccess) return e;
  const long long most = std::max(total[0], std::max(total[1], total[2]));
  return cut.pair == 2 ? mma::launch_product<2, Steps<2>>(q, most, c.sms, c.stream, true)
                       : mma::launch_product<1, Steps<1>>(q, most, c.sms, c.stream, true);
}

}  // namespace

size_t orthogonal_workspace(const OrthogonalCall& c) {
  // the groups depend on whether the small matrices are taken whole, and that on the device
  size_t most = 0;
  Group g;
  for (const bool whole : {false, true})
    for (size_t i = 0; i < c.nstacks; i = g.end) {
      gather(c, i, whole, nullptr, g);
      most = std::max(most, g.bytes);
    }
  return most;
}

bool orthogonal_bounded(const OrthogonalCall& c) {
  float cap[kMaxSteps + 1], growth;
  return bounds(c, cap, &growth);
}

cudaError_t launch_orthogonal(const OrthogonalCall& c) {
  float cap[kMaxSteps + 1] = {}, growth;
  if (!bounds(c, cap, &growth)) return cudaErrorInvalidValue;
  const bool whole = take_whole(c);
  cudaError_t e = cudaSuccess;
  if (whole) {
    e = run_whole<512>(c, cap, growth);
    if (e == cudaSuccess) e = run_whole<256>(c, cap, growth);
    if (e == cudaSuccess) e = run_whole<128>(c, cap, growth);
    if (e != cudaSuccess) return e;
  }
  Group g;
  for (size_t i = 0; i < c.nstacks; i = g.end) {
    gather(c, i, whole, static_cast<uint8_t*>(c.workspace), g);
    if (g.chunks > 1u << 30 || g.matrices > 1u << 20) return cudaErrorInvalidValue;
    e = run(c, g, i, cap, growth);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ar
