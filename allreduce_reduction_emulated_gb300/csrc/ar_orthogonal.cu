// ar_orthogonal.cu -- updates orthogonalised by Newton-Schulz products (ar_train.h), on the
// tensor-core product of ar_mma.cuh.
//
//   u = g + beta m (or m, or g);  X = u / (|u| + eps)
//   `steps` times:  A = X X^T (of a tall matrix X^T X),  B = b A + c A^2,  X <- a X + B X
//
// Two passes over the gradients (momentum and sums of squares; the scaled 16-bit copy), then one launch for all
// products of all steps and shapes.  A and B are symmetric: only their blocks on one
// side of the diagonal are computed, and stored to both.
//
// Between products X, A and B are held in fp16, not in bf16: its 11 bits keep the result within
// 2^-9 (2-norm) of fp32 arithmetic where bf16's 8 would be off by 2% after five steps, and the
// tensor cores are as fast.  fp16's range is met by powers of two: all singular values of
// X have a bound that follows from the coefficients, so that every element's has, and each
// matrix is held times the power of two that brings the bound to 2^13.  Sums are fp32, and
// b A and a X are added in fp32 from the 16-bit values before the one rounding.
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
  float* partial;            // one per chunk
  float* coefs;              // kCoefs per matrix and step
  void** outs;               // one per matrix
  unsigned int* done;        // one per matrix: made 0
};

constexpr int kThreads = 256, kSlotsPerThread = 8;
constexpr unsigned int kChunk = kThreads * kSlotsPerThread;  // slots

// Sum over the block, in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int d = 16; d; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
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

__device__ __forceinline__ Place place(const PrepareParams& p) {
  int lo = 0;
  for (int hi = p.stacks; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (p.stack[mid].first <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  const Stack& s = p.stack[lo];
  const unsigned int k = blockIdx.x - s.first;
  return Place{&s, k / s.chunks, k % s.chunks};
}

// One chunk of one matrix: the update u of every slot to `use`.  With MOMENTUM, the new momentum is
// written where WRITE, else it is there already.
template <bool WRITE, class F>
__device__ __forceinline__ void walk(const PrepareParams& p, const Place& at, F use) {
  const Stack& s = *at.s;
  const size_t base = (size_t)at.matrix * s.rows * s.cols;
  const unsigned int total = s.rows * s.slots;
#pragma unroll 2
  for (int i = 0; i < kSlotsPerThread; ++i) {
    const unsigned int slot = at.chunk * kChunk + i * kThreads + threadIdx.x;
    if (slot >= total) break;
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

__global__ void __launch_bounds__(kThreads) norm_sum_kernel(const __grid_constant__ PrepareParams p) {
  pdl_enter();
  const Place at = place(p);
  float sum = 0.0f;
  walk<true>(p, at, [&](unsigned, unsigned, int, const float (&u)[8]) {
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
//   A' = sa r^2 X' X'^T;  B' = sb b / sa A' + sb c / sa^2 A' A';  X_next' = s a r X' + s r / sb B' X'
__device__ __forceinline__ void coefficients(const PrepareParams& p, float norm, float scale, int step, float* to) {
  const float part = norm == 0.0f ? 0.0f : norm / (norm + p.eps);  // of the first X; below 1 where eps counts
  const auto bound = [&](int k) {
    float b = part;
    for (int i = 0; i < k; ++i) b *= p.growth;
    return fminf(p.cap[k], b) + (part - part);
  };
  const float now = bound(step), sq = now * now;
  const float r = norm == 0.0f ? 1.0f : step == 0 ? 1.0f / (norm + p.eps) / power_for(norm) : 1.0f / power_for(now);
  const float sa = power_for(sq), sb = power_for(fabsf(p.b) * sq + fabsf(p.c) * sq * sq);
  const float s = step + 1 == p.steps ? scale : power_for(bound(step + 1));
  to[0] = sa * r * r;
  to[1] = sb / sa * p.b;
  to[2] = sb / sa * p.c / sa;
  to[3] = s * r * p.a;
  to[4] = s * r / sb;
}

__global__ void __launch_bounds__(kThreads) halve_kernel(const __grid_constant__ PrepareParams p) {
  pdl_enter();
  const Place at = place(p);
  const Stack& s = *at.s;
  const float* partial = p.partial + (blockIdx.x - at.chunk);
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
  walk<false>(p, at, [&](unsigned row, unsigned col, int, const float (&u)[8]) {
    __half2 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(u[2 * j] * power, u[2 * j + 1] * power);
    *reinterpret_cast<uint4*>(x + (size_t)row * s.pitch + col) = *reinterpret_cast<const uint4*>(h);
  });
}

// ------------------------------------------------------------------ the products

enum Stage : int { kGram, kSquare, kApply };

// The matrices of one shape in the product kernel.  A stage's result has nj rows of ni.
struct Shape {
  CUtensorMap gram[2], apply[2], a, b;   // of X in either place for either product; of A; of B
  mma::Kind gram_kind, apply_kind;
  int rows, cols, side;
  int x_pitch, a_pitch;          // multiples of 64; what is stored behind a row's end is read by nothing
  int count, matrix;             // matrices, and the number of the first
  int first[3], tiles[3];        // of each stage: first tile in it, tiles of a matrix
  __half *x[2], *to_a, *to_b;
  bool vectors;                  // the results' rows are whole 16 bytes
};

struct StepsParams {
  Shape shape[kMaxShapes];
  int shapes, steps;
  int stage_tiles[3];
  const float* coefs;            // kCoefs per matrix and step
  void* const* outs;             // where the results of the last step go
  unsigned int* done;            // per matrix: blocks that have stored their part of a tile
};

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// All tiles of all steps in one launch: those of the first product of all matrices, of the second, of the
// third, then the next step's.  A tile waits until all tiles of its matrix before it are stored, which
// with several matrices they mostly are: nobody waits for the last tile of a launch, and a step of a small
// matrix costs three times the way through the chip, not three launches (8.4 us each).
template <int CG>
struct Steps {
  static constexpr bool kBf16 = false, kOrdered = true;
  static constexpr int kSide = 128 * CG;
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
      const int fi = (s.cols + kSide - 1) / kSide, fj = (s.rows + kSide - 1) / kSide;
      i = wide ? j / fj : j % fi;
      j = wide ? j % fj : j / fi;
      nj = s.rows;
      // lanes are the columns of X: D[i, j] = sum_k X[k, i] B[j, k] of a wide one, sum_k B[i, k] X[j, k] of a tall one
      w.a = wide ? &s.apply[step & 1] : &s.b;
      w.b = wide ? &s.b : &s.apply[step & 1];
      w.a_kind = wide ? s.apply_kind : mma::kDepthRows;
      w.b_kind = wide ? mma::kDepthRows : s.apply_kind;
    } else {  // on and above the diagonal: block column j has j + 1 of them
      int c = (int)((sqrtf(8.0f * j + 1.0f) - 1.0f) * 0.5f);
      while ((c + 1) * (c + 2) / 2 <= j) ++c;
      while (c * (c + 1) / 2 > j) --c;
      i = j - c * (c + 1) / 2;
      j = c;
      w.a = w.b = stage == kGram ? &s.gram[step & 1] : &s.a;
      w.a_kind = w.b_kind = stage == kGram ? s.gram_kind : mma::kDepthRows;
    }
    w.a_row = i * kSide;
    w.b_row = j * kSide;
    w.a_z = w.b_z = z;
    w.k = 0;
    w.blocks = ((stage == kGram ? max(s.rows, s.cols) : s.side) + mma::kDepth - 1) / mma::kDepth;
    w.last = mma::kDepth;
    const int unit = (w.b_kind == mma::kDepthRows ? 16 : 64) * CG;
    w.columns = min(kSide, (nj - w.b_row + unit - 1) / unit * unit);
    w.b_bytes = 2 * mma::kBoxBytes;
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
    for (uint32_t n = 0; n < 16 * mma::kPolls; ++n) {  // about 0.7 us each
      unsigned int v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
      ok = v >= before;
      if (ok || *late) break;
    }
    if (!ok) *late = 1;
    // what was stored there is read by TMA too
    asm volatile("fence.proxy.async.global;" ::: "memory");
    return __all_sync(~0u, ok);
  }
  static __device__ __forceinline__ void done(const Params& p, const Tile& w) {
    __threadfence();
    atomicAdd(p.done + p.shape[w.shape].matrix + w.a_z, 1u);
  }

  struct Epilogue {
    float x, y;                  // of the old value, of the sum
    const __half* old;           // of the tile's first column, the warp's first lane; NULL: none
    uint16_t *to, *mirror;
    long long stride, stride_in;   // of the results' columns; of the old values' and the mirrored rows
    int lanes, columns, pads, pad_columns;  // of the sides, and with what lies behind a row's end
    bool last, vectors;
    uint32_t staging;
    uint4 next[4];               // the old values of the next chunk, loaded ahead

    __device__ __forceinline__ Epilogue(const Params& p, const Local&, const Tile& w, int row, int c, uint32_t staging)
        : staging(staging) {
      const Shape& s = p.shape[w.shape];
      const int z = w.a_z, matrix = s.matrix + z;
      const float* f = p.coefs + ((long long)matrix * p.steps + w.step) * kCoefs;
      const int ni = w.stage == kApply ? s.cols : s.side, nj = w.stage == kApply ? s.rows : s.side;
      const int pitch = w.stage == kApply ? s.x_pitch : s.a_pitch;
      const long long at = (long long)z * nj * pitch, here = at + (long long)w.b_row * pitch + row;
      last = w.stage == kApply && w.step + 1 == p.steps;
      vectors = true;
      stride = stride_in = pitch;
      mirror = nullptr;
      if (w.stage == kGram) {
        x = 0.0f, y = f[0];
        old = nullptr;
        to = reinterpret_cast<uint16_t*>(s.to_a) + here;
      } else if (w.stage == kSquare) {
        x = f[1], y = f[2];
        old = s.to_a + here;
        to = reinterpret_cast<uint16_t*>(s.to_b) + here;
      } else {
        x = f[3], y = f[4];
        old = s.x[w.step & 1] + here;
        to = reinterpret_cast<uint16_t*>(s.x[(w.step + 1) & 1]) + here;
        if (last) {
          stride = ni;
          to = static_cast<uint16_t*>(p.outs[matrix]) + (long long)w.b_row * ni + row;
          vectors = s.vectors;
        }
      }
      // a block off the diagonal is stored a second time, lanes as rows
      if (w.stage != kApply && w.a_row != w.b_row)
        mirror = reinterpret_cast<uint16_t*>(w.stage == kGram ? s.to_a : s.to_b) + at + (long long)row * pitch + w.b_row;
      lanes = ni - row;
      pads = pitch - row;
      columns = min(w.columns, nj - w.b_row);
      pad_columns = pitch - w.b_row;
      load_next(c);
    }

    __device__ __forceinline__ void load_next(int c) {
      if (!old) return;
      const int lane = threadIdx.x & 31, part = lane & 3, column = c + (lane >> 2);
      const __half* from = old + column * stride_in + part * 8;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        next[q] = make_uint4(0, 0, 0, 0);
        if (column + 8 * q < columns && part * 8 < pads)
          next[q] = __ldcg(reinterpret_cast<const uint4*>(from + q * (8 * stride_in)));
      }
    }

    __device__ __forceinline__ void chunk(uint32_t at, int c, mma::Source source) {
      const int lane = threadIdx.x & 31;
      uint32_t o[16] = {};
      if (old) {
        // the old values' columns into the staging memory, and out again as fragments
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
        load_next(c + mma::kChunkStep);
      }
      float v[32];
      if (source == mma::kSums) {
        mma::tmem_fragments(at, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = source == mma::kZeros ? 0.0f : __int_as_float(0x7fc00000);
      }
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
        float lo = y * v[2 * i], hi = y * v[2 * i + 1];
        if (old) lo += x * b.x, hi += x * b.y;
        w[i] = last ? pack_bf16x2(lo, hi) : half2_bits(lo, hi);
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

// Tiles of all shapes at this side of a tile, and an estimate of the time in units of a 64-deep slice of a
// pair's tile: a stage takes at least one tile's way, and 5 slices' time go into its epilogue.
double count_tiles(StepsParams& p, int side, int workers, double slice) {
  double time = 0.0;
  for (int stage = 0; stage < 3; ++stage) {
    long long total = 0;
    double work = 0.0, longest = 0.0;
    for (int q = 0; q < p.shapes; ++q) {
      Shape& s = p.shape[q];
      const auto blocks = [&](long long n) { return (n + side - 1) / side; };
      const long long fs = blocks(s.side);
      const long long one = stage == kApply ? blocks(s.rows) * blocks(s.cols) : fs * (fs + 1) / 2;
      s.tiles[stage] = (int)one;
      s.first[stage] = (int)std::min<long long>(total, 1 << 30);
      total += one * s.count;
      const double tile = slice * ((stage == kGram ? std::max(s.rows, s.cols) : s.side) / 64.0) + 5.0;
      work += tile * one * s.count;
      longest = std::max(longest, tile);
    }
    p.stage_tiles[stage] = (int)std::min<long long>(total, 1 << 30);
    time += std::max(work / workers, longest);
  }
  return time;
}

cudaError_t launch_steps(StepsParams& p, int sms, cudaStream_t stream) {
  // Pairs of blocks (256 x 256) or blocks alone: 128 x 128, a quarter, whose slices take 0.75 as long.
  const int pairs = std::max(1, sms / 2);
  const double pair = count_tiles(p, 256, pairs, 1.0), alone = count_tiles(p, 128, sms, 0.75);
  const bool in_pairs = pair <= alone;
  if (in_pairs) count_tiles(p, 256, pairs, 1.0);
  long long tiles = 0;
  int most = 0;
  for (int stage = 0; stage < 3; ++stage) {
    tiles += p.stage_tiles[stage];
    most = std::max(most, p.stage_tiles[stage]);
  }
  if (tiles * p.steps > 1 << 30) return cudaErrorInvalidValue;
  return in_pairs ? mma::launch_product<2, Steps<2>>(p, most, sms, stream, true)
                  : mma::launch_product<1, Steps<1>>(p, most, sms, stream, true);
}

// ------------------------------------------------------------------ one group of stacks

// The matrices of one shape, and where they lie in the workspace.
struct Class {
  size_t rows, cols, count;
  unsigned int matrix;           // number of the first
  __half *x[2], *a, *b;
  bool vectors;
};

size_t up(size_t n, size_t unit) { return (n + unit - 1) / unit * unit; }

// Stacks [first, end) of the call with at most kMaxShapes shapes; their workspace, laid out from `base`.
struct Group {
  size_t end;
  int classes;
  Class cls[kMaxShapes];
  short of[kMaxStacks];          // class of each stack, -1: empty
  size_t matrices, chunks, bytes;
  float *partial, *coefs;
  void** outs;
  unsigned int* done;
};

size_t chunks_of(size_t rows, size_t cols) { return (rows * up(cols, 8) / 8 + kChunk - 1) / kChunk; }

void gather(const OrthogonalCall& c, size_t first, uint8_t* base, Group& g) {
  g.classes = 0;
  g.matrices = g.chunks = 0;
  size_t i = first;
  for (; i < c.nstacks && i - first < kMaxStacks; ++i) {
    short k = -1;
    if (c.counts[i] && c.rows[i] && c.cols[i]) {
      for (k = 0; k < g.classes && !(g.cls[k].rows == c.rows[i] && g.cls[k].cols == c.cols[i]); ++k) {}
      if (k == g.classes) {
        if (g.classes == kMaxShapes) break;
        g.cls[g.classes++] = Class{c.rows[i], c.cols[i], 0, 0, {}, nullptr, nullptr, true};
      }
      g.cls[k].count += c.counts[i];
      g.cls[k].vectors &= c.cols[i] % 8 == 0 && (c.outs == nullptr || ((uintptr_t)c.outs[i] & 15) == 0);
      g.matrices += c.counts[i];
      g.chunks += c.counts[i] * chunks_of(c.rows[i], c.cols[i]);
    }
    g.of[i - first] = k;
  }
  g.end = i;
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

cudaError_t run(const OrthogonalCall& c, const Group& g, size_t first, const float* cap, float growth) {
  PrepareParams p;
  p.stacks = 0;
  p.beta = c.beta, p.nesterov = c.nesterov, p.eps = c.eps;
  p.a = c.a, p.b = c.b, p.c = c.c, p.growth = growth, p.steps = c.steps;
  std::memcpy(p.cap, cap, sizeof p.cap);
  p.partial = g.partial, p.coefs = g.coefs, p.outs = g.outs, p.done = g.done;
  size_t used[kMaxShapes] = {}, chunk = 0;
  for (size_t i = first; i < g.end; ++i) {
    const short k = g.of[i - first];
    if (k < 0) continue;
    const Class& l = g.cls[k];
    const size_t pitch = up(l.cols, 64);
    const bool bf16 = c.dtypes[i] == AR_BFLOAT16;
    float* m = c.momentum ? c.momentum[i] : nullptr;
    Stack& s = p.stack[p.stacks++];
    s.grad = c.grads[i], s.momentum = m, s.out = c.outs[i];
    s.x = l.x[0] + used[k] * l.rows * pitch;
    s.rows = (unsigned)l.rows, s.cols = (unsigned)l.cols, s.pitch = (unsigned)pitch;
    s.slots = (unsigned)(up(l.cols, 8) / 8);
    s.chunks = (unsigned)chunks_of(l.rows, l.cols);
    s.first = (unsigned)chunk;
    s.matrix = l.matrix + (unsigned)used[k];
    s.bf16 = bf16;
    s.vectors = l.cols % 8 == 0 && ((uintptr_t)c.grads[i] & 15) == 0 && ((uintptr_t)m & 15) == 0;
    s.scale = c.scales ? c.scales[i] : 1.0f;
    used[k] += c.counts[i];
    chunk += c.counts[i] * s.chunks;
  }
  if (p.stacks == 0) return cudaSuccess;
  cudaError_t e = launch_kernel(norm_sum_kernel, dim3((unsigned)chunk), dim3(kThreads), 0, c.stream, true, p);
  if (e == cudaSuccess) e = launch_kernel(halve_kernel, dim3((unsigned)chunk), dim3(kThreads), 0, c.stream, true, p);
  StepsParams q;
  for (int k = 0; e == cudaSuccess && k < g.classes; ++k) {
    const Class& l = g.cls[k];
    Shape& s = q.shape[k];
    const bool wide = l.rows <= l.cols;
    const size_t side = std::min(l.rows, l.cols), px = up(l.cols, 64), pa = up(side, 64);
    s.rows = (int)l.rows, s.cols = (int)l.cols, s.side = (int)side;
    s.x_pitch = (int)px, s.a_pitch = (int)pa;
    s.count = (int)l.count, s.matrix = (int)l.matrix;
    s.to_a = l.a, s.to_b = l.b;
    s.vectors = l.vectors;
    mma::Kind depth;
    const auto map = [&](CUtensorMap* to, mma::Kind* kind, const __half* at, size_t rows, size_t cols, size_t pitch,
                         bool depth) {
      // as i or j the padded row is read: what lies behind its end becomes lanes or columns that nothing uses
      if (e == cudaSuccess)
        e = mma::make_map(to, kind, false, at, depth ? cols : pitch, rows, l.count, pitch, rows * pitch, depth, 128);
    };
    for (int j = 0; j < 2; ++j) {
      s.x[j] = l.x[j];
      map(&s.gram[j], &s.gram_kind, l.x[j], l.rows, l.cols, px, wide);
      map(&s.apply[j], &s.apply_kind, l.x[j], l.rows, l.cols, px, !wide);
    }
    map(&s.a, &depth, l.a, side, side, pa, true);
    map(&s.b, &depth, l.b, side, side, pa, true);
  }
  q.shapes = g.classes, q.steps = c.steps;
  q.coefs = g.coefs, q.outs = g.outs, q.done = g.done;
  return e == cudaSuccess ? launch_steps(q, c.sms, c.stream) : e;
}

}  // namespace

size_t orthogonal_workspace(const OrthogonalCall& c) {
  size_t most = 0;
  Group g;
  for (size_t i = 0; i < c.nstacks; i = g.end) {
    gather(c, i, nullptr, g);
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
  Group g;
  for (size_t i = 0; i < c.nstacks; i = g.end) {
    gather(c, i, static_cast<uint8_t*>(c.workspace), g);
    if (g.chunks > 1u << 30 || g.matrices > 1u << 20) return cudaErrorInvalidValue;
    const cudaError_t e = run(c, g, i, cap, growth);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ar
