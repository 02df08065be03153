// ar_experts.cu -- products of rows sorted by expert with their expert's weights, and
// the gradient of the weights (ar_train.h), on the tensor-core product of ar_mma.cuh.
//
//   y[t, f] = sum_k W_e[f, k] x[t, k]      rows t of expert e
//   dW_e[j, i] = sum_t b[t, j] a[t, i]     a, b: x and dy
//
// In both the 128 lanes of an accumulator are the side that is contiguous in the
// output, so that a warp stores whole 64-byte (fp32: 128-byte) runs; and in the first the
// rows of an expert are the columns, of which the matrix instructions take any multiple
// of 16: an expert's ragged rest costs what its rows cost, not a whole tile.
//
// The offsets are read on the device, by every block: nothing waits for the host.
#include <algorithm>
#include <cmath>

#include "ar_mma.cuh"
#include "ar_train.h"
#include "ar_train_launch.h"

namespace ar {

namespace mma {

namespace {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  return encode;
}

}  // namespace

cudaError_t make_map(CUtensorMap* map, Kind* kind, bool bf16, const void* base, uint64_t nx, uint64_t ny, uint64_t nz,
                     uint64_t y_stride, uint64_t z_stride, bool depth, uint32_t box_rows) {
  const Encode encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  *kind = depth ? kDepthRows : nx % 64 == 0 ? kWideRows : kNarrowRows;
  // A side of length one has no stride of its own; the map wants one that is whole all the same.
  const cuuint64_t y = ny > 1 ? y_stride * 2 : (nx * 2 + 15) / 16 * 16;
  const cuuint64_t z = nz > 1 ? z_stride * 2 : y;
  const bool wide = *kind == kWideRows;
  const cuuint64_t dims[4] = {wide ? 64 : nx, ny, wide ? nx / 64 : nz, wide ? nz : 1};
  const cuuint64_t strides[3] = {y, wide ? 128 : z, z};
  const cuuint32_t box[4] = {64, depth ? box_rows : 64, wide ? box_rows / 64 : 1, 1}, step[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_store_map(CUtensorMap* map, const void* base, uint64_t nx, uint64_t ny, uint64_t nz, uint64_t y_stride,
                           uint64_t z_stride) {
  const Encode encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t y = ny > 1 ? y_stride * 2 : (nx * 2 + 15) / 16 * 16;
  const cuuint64_t dims[3] = {nx, ny, nz}, strides[2] = {y, nz > 1 ? z_stride * 2 : y};
  const cuuint32_t box[3] = {32, 32, 1}, step[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace mma

namespace {

using mma::Tile;

// Row ranges of the experts, and what every block works out of them.
struct Offsets {
  const void* at;
  int bytes, experts;
  long long rows;
  __device__ __forceinline__ int get(int i) const {
    const long long v = bytes == 8 ? static_cast<const long long*>(at)[i] : (long long)static_cast<const int*>(at)[i];
    return (int)(v < 0 ? 0 : v > rows ? rows : v);
  }
};

// start[e]: first row of expert e, the largest offset so far (so that the ranges never
// overlap, whatever the offsets hold); first[e]: tiles before it.
struct Ranges {
  int start[kMaxExperts + 1];
  int first[kMaxExperts + 3];
};

// One warp; `count(rows)` is an expert's number of tiles.
template <class Count>
__device__ __forceinline__ void lay_out(const Offsets& o, Ranges& r, Count count) {
  const int lane = threadIdx.x & 31;
  int most = 0, tiles = 0;
  for (int base = 0; base <= o.experts; base += 32) {
    const int e = base + lane;
    int a = e <= o.experts ? o.get(e) : 0;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(~0u, a, d);
      if (lane >= d) a = max(a, v);
    }
    a = max(a, most);
    // tiles of the expert before this offset
    int before = __shfl_up_sync(~0u, a, 1);
    if (lane == 0) before = most;
    int n = e >= 1 && e <= o.experts ? count(a - before) : 0;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(~0u, n, d);
      if (lane >= d) n += v;
    }
    if (e <= o.experts) {
      r.start[e] = a;
      r.first[e] = tiles + n;
    }
    most = __shfl_sync(~0u, a, 31);
    tiles += __shfl_sync(~0u, n, 31);
  }
}

// Last e in [0, n) with first[e] <= t.
__device__ __forceinline__ int find(const int* first, int n, int t) {
  int lo = 0;
  for (int hi = n; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) { return (uint16_t)pack_bf16x2(v, 0.0f); }

// Stores a warp's chunks of 32 lanes by 32 columns: column c of a tile is `stride` elements behind column
// c - 1, a lane next to its neighbour.
struct Store {
  void* to;             // of the tile's first column, the warp's first lane
  long long stride;
  int lanes, columns;   // that are stored: of the warp (may be negative), of the tile
  bool fp32, add, vectors;
  const CUtensorMap* map;   // at whole 16 bytes: of the results, in boxes of 32 x 32
  int x, y, z;              // in it
  mma::Staging& staging;

  // A lane's 32 columns as they are: a warp stores whole 128-byte runs of fp32.  `add`: to what is there.
  __device__ __forceinline__ void put(int c, const float (&v)[32], bool add) const {
    const int lane = threadIdx.x & 31;
    if (lane >= lanes) return;
    if (fp32) {
      float* y = static_cast<float*>(to) + lane + c * stride;
      if (add) {
        // One thread's, one behind the other: the order is fixed.  Nothing is waited for (as loads, additions and stores
        // 16384 rows of 8 experts, dW of 2048 x 2048: 139 us, now 120).  Subnormal values become 0, sums and what was
        // there (join_kernel's additions keep them).
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < columns)
            asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(y + i * stride), "f"(v[i]) : "memory");
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < columns) y[i * stride] = v[i];
      }
    } else {
      uint16_t* y = static_cast<uint16_t*>(to) + lane + c * stride;
#pragma unroll
      for (int h = 0; h < 32; h += 8) {
        float old[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) old[i] = add && c + h + i < columns ? bf16_lo(y[(h + i) * stride]) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + h + i < columns) y[(h + i) * stride] = bf16_bits(add ? old[i] + v[h + i] : v[h + i]);
        asm volatile("" ::: "memory");
      }
    }
  }
  // `more`: a later run of a tile, added to the ones before.
  __device__ __forceinline__ void chunk(uint32_t at, int c, mma::Source source, bool more) const {
    float v[32];
    if (fp32 || add || source != mma::kSums) {
      if (source == mma::kSums) {
        mma::tmem_rows(at, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = source == mma::kZeros ? 0.0f : __int_as_float(0x7fc00000);
      }
      put(c, v, add || more);
      return;
    }
    // bf16: 8 x 8 matrices are transposed on their way through shared memory, 64 bytes a column
    mma::tmem_fragments(at, v);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    const uint32_t area = staging.next();
    mma::stage_columns(area, w);
    if (vectors && c + 32 <= columns) {  // whole chunks by TMA; the map ends where a row of results does
      staging.store(area, map, x, y + c, z, lanes > 0);
    } else {
      __syncwarp();
      mma::put_columns(area, static_cast<uint16_t*>(to) + c * stride, stride, lanes, columns - c, vectors);
      staging.release();
    }
  }
};

// Of a tile's slices those of one of `parts` parts.
__device__ __forceinline__ void cut(Tile& w, int part, int parts) {
  const int begin = (int)((long long)w.blocks * part / parts), end = (int)((long long)w.blocks * (part + 1) / parts);
  if (end < w.blocks) w.last = mma::kDepth;
  w.k += begin * mma::kDepth;
  w.blocks = end - begin;
}

struct ForwardParams {
  CUtensorMap weights, x, x_few, y_map;  // x_few: boxes of 32 rows
  mma::Kind w_kind;
  Offsets offsets;
  int out, in;             // W_e: out x in
  void* y;
  long long y_stride;
  bool vectors, zero_rest;
  int splits;              // parts of the sums, fp32, each with results of its own
  long long split_stride;
};

// The experts' weights are read once for every 128 CG rows of theirs, x once for every 128 CG outputs, both
// mostly from L2: what is on the GPU at once are neighbours.  4096 rows of 8 uneven experts, 2048 -> 8192: 104 us (1.3
// PFLOP/s; what is left of the last wave costs the rest), 16384 rows of 64, 2048 -> 1024: 75 us (4.9 TB/s).
// An expert's rows are cut into tiles of one width, rather than whole ones and a rest: the last wave is as wide as the
// first.
//
// FP32: of the results.  The tensor cores cut what an addition to the accumulators loses: over 1000 k a sum
// is off by 1e-6 of itself, over 16000 by 2e-5.  So 960 k are the longest run that they add up; a later run is
// added, rounded, to what the runs before have stored.  A bf16 result's own rounding is larger than all that.  4096 rows of
// 8 experts, 2048 -> 8192: fp32 117 us, bf16 89; 1024 -> 8192 68 and 51; 960 -> 8192, one run, 57 and 49.
template <int CG, bool FP32>
struct Forward {
  static constexpr bool kBf16 = true, kOrdered = false;
  static constexpr int kStages = FP32 ? 6 : 5, kBytesB = 2 * mma::kBoxBytes;
  static constexpr int kAreas = FP32 ? 0 : 2, kArea = 2048, kRun = FP32 ? 15 : 0;
  static constexpr int kWide = 128 * CG, kUnit = 16 * CG;  // most columns of a tile, and what they are a multiple of
  using Params = ForwardParams;
  struct Local {
    Ranges r;
  };
  static __device__ __forceinline__ void begin(const Params& p, Local& l) {
    if ((threadIdx.x >> 5) != 3) return;
    const int f = (p.out + kRowsOfTile - 1) / kRowsOfTile;
    const auto tiles = [&](int rows) { return (rows + kWide - 1) / kWide * f; };
    lay_out(p.offsets, l.r, tiles);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      const int E = p.offsets.experts, n = l.r.first[E];
      // the rows of no expert: in front, behind
      const int front = p.zero_rest ? tiles(l.r.start[0]) : 0;
      const int behind = p.zero_rest ? tiles((int)p.offsets.rows - l.r.start[E]) : 0;
      l.r.first[E + 1] = n + front;
      l.r.first[E + 2] = n + front + behind;
    }
  }
  static constexpr int kRowsOfTile = mma::kRows * CG;
  static __device__ __forceinline__ bool tile(const Params& p, const Local& l, int t, Tile& w) {
    const int E = p.offsets.experts, total = l.r.first[E + 2];
    int part = 0;
    if constexpr (FP32) {
      if (p.splits > 1 && t >= total) {
        if (total == 0) return false;
        part = t / total;
        if (part >= p.splits) return false;
        t -= part * total;
      }
      w.shape = part;
    }
    if (t >= total) return false;
    const int e = find(l.r.first, E + 2, t), j = t - l.r.first[e];
    const int begin = e < E ? l.r.start[e] : e == E ? 0 : l.r.start[E];
    const int end = e < E ? l.r.start[e + 1] : e == E ? l.r.start[0] : (int)p.offsets.rows;
    const int n = (end - begin + kWide - 1) / kWide;
    const int width = ((end - begin + n - 1) / n + kUnit - 1) / kUnit * kUnit;
    w.a = &p.weights;
    w.a_row = j / n * kRowsOfTile;
    w.b_row = begin + j % n * width;
    w.a_z = e;
    w.b_z = 0;
    w.k = 0;
    w.blocks = e < E ? (p.in + mma::kDepth - 1) / mma::kDepth : 0;
    w.last = mma::kDepth;
    if constexpr (FP32)
      if (p.splits > 1) cut(w, part, p.splits);
    // the tiles before may have taken all rows (rounding up to whole units)
    const int left = end - w.b_row;
    w.columns = left < width ? max(kUnit, (left + kUnit - 1) / kUnit * kUnit) : width;
    w.a_kind = p.w_kind;
    w.b_kind = mma::kDepthRows;
    const bool few = w.columns <= 32 * CG;
    w.b = few ? &p.x_few : &p.x;
    w.b_bytes = few ? mma::kBoxBytes / 2 : 2 * mma::kBoxBytes;
    w.end = end;
    return true;
  }
  struct Epilogue : Store {
    __device__ __forceinline__ Epilogue(const Params& p, const Local&, const Tile& w, int row, int, mma::Staging& staging,
                                        const float*)
        : Store{static_cast<uint8_t*>(p.y) + (w.b_row * p.y_stride + row) * (FP32 ? 4 : 2) +
                    (FP32 ? w.shape * p.split_stride * 4 : 0), p.y_stride, p.out - row,
                min(w.columns, w.end - w.b_row), FP32, false, p.vectors, &p.y_map, row, w.b_row, 0, staging} {}
  };
};

struct GradientParams {
  CUtensorMap a, b, dw_map;  // rows by ni, rows by nj; dW
  mma::Kind a_kind, b_kind;
  Offsets offsets;
  int ni, nj;
  void* dw;                // dW_e[j, i] at e * e_stride + j * j_stride + i
  long long e_stride, j_stride;
  bool add, vectors;
  int splits;              // as above
  long long split_stride;
};

// Sums over an expert's rows, which are k here: of both operands the outer side, so a slice is whole rows of
// boxes and the last one's rest is cleared in shared memory (warp 3; by the loading warp 64 rows of 8 experts, 2048 ->
// 2048, took 47 us, now 38).  Bound by the matrix instructions where experts have many rows (dx and dW of 16384 rows of
// 16 experts, 2048 -> 8192: 767 us, 1.43 PFLOP/s), by storing dW where they have few (4096 rows of 8, 8192 -> 2048, fp32:
// 155 us for 537 MB and 137 GFLOP).
template <int CG, bool FP32>
struct WeightGradient {
  static constexpr bool kBf16 = true, kOrdered = false;
  static constexpr int kStages = FP32 ? 6 : 5, kBytesB = 2 * mma::kBoxBytes;
  static constexpr int kAreas = FP32 ? 0 : 2, kArea = 2048, kRun = FP32 ? 15 : 0;
  static constexpr int kWide = 128 * CG, kUnit = 64 * CG, kRowsOfTile = mma::kRows * CG;
  using Params = GradientParams;
  struct Local {
    Ranges r;
  };
  static __device__ __forceinline__ void begin(const Params& p, Local& l) {
    if ((threadIdx.x >> 5) == 3) lay_out(p.offsets, l.r, [](int) { return 0; });
  }
  static __device__ __forceinline__ bool tile(const Params& p, const Local& l, int t, Tile& w) {
    const int fi = (p.ni + kRowsOfTile - 1) / kRowsOfTile, fj = (p.nj + kWide - 1) / kWide;
    int part = 0;
    if constexpr (FP32) {
      const long long total = (long long)fi * fj * p.offsets.experts;
      if (p.splits > 1 && t >= total) {
        part = (int)(t / total);
        if (part >= p.splits) return false;
        t -= (int)(part * total);
      }
      w.shape = part;
    }
    const int e = t / (fi * fj), rest = t % (fi * fj);
    if (e >= p.offsets.experts) return false;
    const int begin = l.r.start[e], n = l.r.start[e + 1] - begin;
    w.a = &p.a;
    w.b = &p.b;
    w.a_row = rest % fi * kRowsOfTile;
    w.b_row = rest / fi * kWide;
    w.a_z = w.b_z = 0;
    w.k = begin;
    w.blocks = (n + mma::kDepth - 1) / mma::kDepth;
    w.last = n - (w.blocks - 1) * mma::kDepth;
    if constexpr (FP32)
      if (p.splits > 1) cut(w, part, p.splits);
    w.columns = min(kWide, (p.nj - w.b_row + kUnit - 1) / kUnit * kUnit);
    w.a_kind = p.a_kind;
    w.b_kind = p.b_kind;
    w.b_bytes = p.b_kind == mma::kNarrowRows && w.columns <= 64 * CG ? mma::kBoxBytes : 2 * mma::kBoxBytes;
    w.end = e;
    return true;
  }
  struct Epilogue : Store {
    __device__ __forceinline__ Epilogue(const Params& p, const Local&, const Tile& w, int row, int, mma::Staging& staging,
                                        const float*)
        : Store{static_cast<uint8_t*>(p.dw) + (w.end * p.e_stride + w.b_row * p.j_stride + row) * (FP32 ? 4 : 2) +
                    (FP32 ? w.shape * p.split_stride * 4 : 0),
                p.j_stride, p.add && w.blocks == 0 ? 0 : p.ni - row, min(w.columns, p.nj - w.b_row), FP32, p.add,
                p.vectors, &p.dw_map, row, w.b_row, w.end, staging} {}
  };
};

// ------------------------------------------------------------------ operands that TMA cannot read

// nz x ny rows of nx bf16 each, at any alignment and strides, into rows of whole slots of eight elements one behind the
// other; of the weights only experts that may have rows.  Bound by HBM, a pass over the operand more: 57 matrices of
// 240 x 5549 are laid out and multiplied with 2000 rows in 91 us (by single elements and 64-bit divisions 99), with 30
// rows, which half of the experts have, in 58 (85).  A slot takes two aligned loads, the second of which is the next
// thread's first, and is shifted in registers.  More slots of a thread at once are slower (16336 x 163: 14 us of
// the call, one 12.6).
struct PackParams {
  const uint16_t* from;
  uint16_t* to;
  unsigned int nx, ny, slots;   // slots: of a row
  long long total;              // slots in all
  long long y_stride, z_stride;
  Offsets offsets;              // experts 0: not the weights
};
constexpr int kPackThreads = 256;

template <class I>  // of slots: 32 bits where they fit
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const __grid_constant__ PackParams p) {
  __shared__ uint32_t has_rows[(kMaxExperts + 31) / 32];
  pdl_enter();
  const bool some = p.offsets.experts > 0;
  if (some) {
    for (int e = threadIdx.x; e - (int)(threadIdx.x & 31) < p.offsets.experts; e += kPackThreads) {
      const bool has = e < p.offsets.experts && p.offsets.get(e + 1) > p.offsets.get(e);
      const uint32_t bits = __ballot_sync(~0u, has);
      if ((threadIdx.x & 31) == 0) has_rows[e >> 5] = bits;
    }
    __syncthreads();
  }
  const I total = (I)p.total, step = (I)gridDim.x * kPackThreads;
  for (I v = (I)blockIdx.x * kPackThreads + threadIdx.x; v < total; v += step) {
    const I row = v / p.slots;
    const unsigned int x = (unsigned int)(v - row * p.slots) * 8, z = (unsigned int)(row / p.ny);
    if (some && !(has_rows[z >> 5] >> (z & 31) & 1)) continue;
    const uint16_t* from = p.from + z * p.z_stride + (long long)(row - (I)z * p.ny) * p.y_stride + x;
    const int left = (int)(p.nx - x);                      // of the row
    const int before = (int)((uintptr_t)from & 15) >> 1;   // elements in front of the slot in its first 16 bytes
    const uint4* aligned = reinterpret_cast<const uint4*>(from - before);
    const uint4 lo = __ldg(aligned);
    uint4 hi = make_uint4(0, 0, 0, 0);
    if (before && before + left > 8) hi = __ldg(aligned + 1);  // (it has elements of the row)
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < 6; ++j) w[j] = before & 4 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = before & 2 ? w[j + 1] : w[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before & 1) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
      if (left < 8) w[j] = 2 * j >= left ? 0 : 2 * j + 1 >= left ? w[j] & 0xffff : w[j];  // zeros behind the row's end
    }
    reinterpret_cast<uint4*>(p.to)[v] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------ sums in parts

// Few tiles of long sums leave multiprocessors idle: their slices are split into parts, each a tile of its own with
// fp32 results in the workspace, and this adds them up, in their order.  Bound by a launch, the parts are in L2 mostly.
// 5 rows of 4 experts, 8192 -> 1024: 31.8 us whole, 14.4 in parts; dx and dW of 16336 rows of 2 experts, 163 -> 264: 63.5,
// 28.3; dx and dW of 1355 rows of 19, 93 -> 7512: 78, 50; dW of 100000 rows, 1024 x 1024: 382, by blocks alone 233, by pairs
// 170 to 190.
struct JoinParams {
  const float* parts;
  long long split_stride;
  int splits;
  unsigned int count, cols, per;   // values, of a row, rows of a matrix
  void* to;
  long long z_stride, y_stride;
  bool fp32, add, zero_rest;
  Offsets offsets;                 // experts 0: all rows are somebody's
};

__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ int most;
  pdl_enter();
  int begin = 0, end = 0;
  if (p.offsets.experts) {
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    int last = 0;
    for (int i = threadIdx.x; i <= p.offsets.experts; i += 256) last = max(last, p.offsets.get(i));
    atomicMax(&most, last);
    __syncthreads();
    begin = p.offsets.get(0), end = most;
  }
  for (unsigned int i = blockIdx.x * 256 + threadIdx.x; i < p.count; i += gridDim.x * 256) {
    const unsigned int row = i / p.cols, z = row / p.per;
    const long long at = z * p.z_stride + (row - z * p.per) * p.y_stride + (i - row * p.cols);
    float sum = 0.0f;
    if (!p.offsets.experts || ((int)row >= begin && (int)row < end)) {
#pragma unroll 4
      for (int s = 0; s < p.splits; ++s) sum += __ldcg(p.parts + s * p.split_stride + i);
    } else if (!p.zero_rest) {
      continue;
    }
    if (p.fp32) {
      float* y = static_cast<float*>(p.to) + at;
      *y = p.add ? *y + sum : sum;
    } else {
      uint16_t* y = static_cast<uint16_t*>(p.to) + at;
      *y = bf16_bits(p.add ? bf16_lo(*y) + sum : sum);
    }
  }
}

cudaError_t join(const JoinParams& p, int sms, cudaStream_t stream) {
  const unsigned int blocks = std::min<unsigned int>((p.count + 255) / 256, (unsigned int)sms * 8);
  return launch_kernel(join_kernel, dim3(blocks), dim3(256), 0, stream, true, p);
}

constexpr size_t whole(size_t n) { return (n + 7) / 8 * 8; }

// TMA wants addresses and strides of whole 16 bytes (strides that nothing follows do not count).
bool direct(const ExpertMatrix& m) {
  return ((uintptr_t)m.at & 15) == 0 && (m.ny <= 1 || m.y_stride % 8 == 0) && (m.nz <= 1 || m.z_stride % 8 == 0);
}

// The map of an operand; where it cannot be read as it is, of a copy in the workspace.
cudaError_t operand(ExpertMatrix m, bool depth, uint8_t*& workspace, const Offsets& offsets, int sms,
                    cudaStream_t stream, CUtensorMap* map, mma::Kind* kind, CUtensorMap* few = nullptr) {
  if (!m.nx || !m.ny || !m.nz) return cudaSuccess;  // no tile reads it
  if (!direct(m)) {
    const size_t pitch = whole(m.nx), rows = m.ny * m.nz;
    uint16_t* to = reinterpret_cast<uint16_t*>(workspace);
    workspace += expert_matrix_workspace(m);
    PackParams p = {static_cast<const uint16_t*>(m.at), to, (unsigned)m.nx, (unsigned)m.ny, (unsigned)(pitch / 8),
                    (long long)(rows * (pitch / 8)), (long long)m.y_stride, (long long)m.z_stride, offsets};
    if (m.nz != (size_t)offsets.experts) p.offsets.experts = 0;
    const long long blocks = std::min<long long>((p.total + kPackThreads - 1) / kPackThreads, sms * 8);
    const bool few = p.total + blocks * kPackThreads < 1ll << 32;
    const cudaError_t e = launch_kernel(few ? pack_kernel<unsigned int> : pack_kernel<unsigned long long>,
                                        dim3((unsigned)blocks), dim3(kPackThreads), 0, stream, true, p);
    if (e != cudaSuccess) return e;
    m = ExpertMatrix{to, m.nx, m.ny, m.nz, pitch, m.ny * pitch};
  }
  const cudaError_t e = mma::make_map(map, kind, true, m.at, m.nx, m.ny, m.nz, m.y_stride, m.z_stride, depth, 128);
  if (e != cudaSuccess || !few) return e;
  return mma::make_map(few, kind, true, m.at, m.nx, m.ny, m.nz, m.y_stride, m.z_stride, depth, 32);
}

// Whether rows of results can be stored 16 bytes at a time.
bool vectors(const void* at, size_t stride, size_t matrix_stride = 0) {
  return ((uintptr_t)at & 15) == 0 && stride % 8 == 0 && matrix_stride % 8 == 0;
}

// splits > 1: the sums in so many parts, joined from the workspace behind the operands'.
template <int CG, bool FP32>
cudaError_t forward(const ExpertsCall& c, int splits = 1) {
  using Policy = Forward<CG, FP32>;
  ForwardParams p = {};
  p.offsets = Offsets{c.offsets, c.offset_bytes, (int)c.experts, (long long)c.rows};
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  mma::Kind kind;
  cudaError_t e = operand(c.w, c.w_in_contiguous, ws, p.offsets, c.sms, c.stream, &p.weights, &p.w_kind);
  if (e == cudaSuccess) e = operand(c.x, true, ws, p.offsets, c.sms, c.stream, &p.x, &kind, &p.x_few);
  p.vectors = !FP32 && vectors(c.y, c.y_stride);
  if (e == cudaSuccess && p.vectors)
    e = mma::make_store_map(&p.y_map, c.y, c.out, c.rows, 1, c.y_stride, 0);
  if (e != cudaSuccess) return e;
  p.out = (int)c.out;
  p.in = (int)c.in;
  p.y = c.y;
  p.y_stride = (long long)c.y_stride;
  p.zero_rest = c.zero_rest;
  const long long f = ((long long)c.out + Policy::kRowsOfTile - 1) / Policy::kRowsOfTile;
  const long long groups = (long long)std::min<size_t>(c.experts, c.rows) + 2 + (long long)(c.rows / Policy::kWide);
  p.splits = splits;
  if (splits > 1) {
    p.y = ws, p.y_stride = p.out, p.zero_rest = false;
    p.split_stride = (long long)c.rows * p.out;
  }
  e = mma::launch_product<CG, Policy>(p, f * groups * splits, c.sms, c.stream);
  if (e != cudaSuccess || splits == 1) return e;
  return join(JoinParams{static_cast<const float*>(p.y), p.split_stride, splits, (unsigned)p.split_stride, (unsigned)p.out,
                         (unsigned)c.rows, c.y, 0, (long long)c.y_stride, c.dtype == AR_FLOAT32, false, c.zero_rest,
                         p.offsets}, c.sms, c.stream);
}

template <int CG, bool FP32>
cudaError_t weight_gradient(const ExpertsCall& c, int splits = 1) {
  using Policy = WeightGradient<CG, FP32>;
  GradientParams p = {};
  p.offsets = Offsets{c.offsets, c.offset_bytes, (int)c.experts, (long long)c.rows};
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  // the contiguous side of dW is the lanes'
  const bool lanes_in = c.w_in_contiguous;
  cudaError_t e = operand(lanes_in ? c.x : c.dy, false, ws, p.offsets, c.sms, c.stream, &p.a, &p.a_kind);
  if (e == cudaSuccess)
    e = operand(lanes_in ? c.dy : c.x, false, ws, p.offsets, c.sms, c.stream, &p.b, &p.b_kind);
  p.ni = (int)(lanes_in ? c.in : c.out);
  p.nj = (int)(lanes_in ? c.out : c.in);
  p.dw = c.y;
  p.e_stride = (long long)c.w.z_stride;
  p.j_stride = (long long)c.w.y_stride;
  p.add = c.accumulate;
  p.vectors = !FP32 && vectors(c.y, c.w.y_stride, c.w.z_stride);
  if (e == cudaSuccess && p.vectors)
    e = mma::make_store_map(&p.dw_map, c.y, p.ni, p.nj, c.experts, c.w.y_stride, c.w.z_stride);
  if (e != cudaSuccess) return e;
  const auto over = [](long long n, long long d) { return (n + d - 1) / d; };
  const long long tiles = over(p.ni, Policy::kRowsOfTile) * over(p.nj, Policy::kWide) * (long long)c.experts;
  p.splits = splits;
  if (splits > 1) {
    p.dw = ws, p.add = false;
    p.j_stride = p.ni, p.e_stride = (long long)p.nj * p.ni;
    p.split_stride = p.e_stride * (long long)c.experts;
  }
  e = mma::launch_product<CG, Policy>(p, tiles * splits, c.sms, c.stream);
  if (e != cudaSuccess || splits == 1) return e;
  return join(JoinParams{static_cast<const float*>(p.dw), p.split_stride, splits, (unsigned)p.split_stride, (unsigned)p.ni,
                         (unsigned)p.nj, c.y, (long long)c.w.z_stride, (long long)c.w.y_stride, c.dtype == AR_FLOAT32,
                         c.accumulate, false, Offsets{}}, c.sms, c.stream);
}

}  // namespace

size_t expert_matrix_workspace(const ExpertMatrix& m) {
  return direct(m) ? 0 : (whole(m.nx) * m.ny * m.nz * 2 + 127) / 128 * 128;
}

// What the choice between pairs, blocks alone and sums in parts goes by.  The offsets are on the device: as if all experts
// had the same number of rows.
struct Work {
  double in_pairs, alone, slices, values;   // tiles, 64-deep slices of a tile, results
};
static Work product_work(const ExpertsCall& c) {
  const double some = (double)std::min(c.experts, c.rows);   // 0: no tiles
  const auto tiles = [&](double side) { return some ? std::ceil(c.out / side) * some * std::ceil(c.rows / some / side) : 0; };
  return Work{tiles(256), tiles(128), std::ceil(c.in / 64.0), (double)c.rows * (double)c.out};
}
static Work gradient_work(const ExpertsCall& c) {
  const auto tiles = [&](double side) { return std::ceil(c.out / side) * std::ceil(c.in / side) * (double)c.experts; };
  return Work{tiles(256), tiles(128), std::ceil((double)c.rows / std::max<size_t>(1, c.experts) / 64.0),
              (double)c.experts * (double)c.out * (double)c.in};
}
// Pairs of blocks or blocks alone, and into how many parts the sums are split: where the tiles take less time so, with a
// launch that adds the parts up (about 3 us, and what it reads and writes, from L2 mostly).  Without a workspace for
// the parts, whole sums.
struct Plan {
  bool pairs;
  int splits;
  size_t bytes;
};
static Plan whole_sums(const Work& w, int sms) {
  return Plan{mma::better_in_pairs(w.in_pairs, w.alone, w.slices, sms), 1, 0};
}
static Plan plan(const Work& w, int sms) {
  const auto time = [&](bool pairs, int n) {
    const double tiles = (pairs ? w.in_pairs : w.alone) * n, at_once = pairs ? sms / 2 : sms;
    return std::ceil(tiles / at_once) * ((pairs ? 0.27 : 0.20) * std::ceil(w.slices / n) + (pairs ? 3.0 : 2.0)) +
           (n > 1 ? 3.0 + w.values * 4 * (2 * n + 1) / 4e6 : 0.0);
  };
  Plan best = whole_sums(w, sms);
  // (Without tiles nobody would write the parts that the join adds up.)
  if (w.values > 1 << 26 || w.alone == 0 || sms < 2) return best;
  double least = 0.9 * time(best.pairs, 1);
  for (const bool pairs : {false, true})
    for (int n = 2; n <= 16 && (pairs ? w.in_pairs : w.alone) <= (pairs ? sms / 2 : sms); ++n)
      if (time(pairs, n) < least) least = time(pairs, n), best = Plan{pairs, n, (size_t)w.values * 4 * n};
  return best;
}

size_t expert_parts_workspace(const ExpertsCall& c, bool of_weights) {
  return plan(of_weights ? gradient_work(c) : product_work(c), c.sms).bytes;
}

cudaError_t launch_expert_product(const ExpertsCall& c) {
  const Work w = product_work(c);
  Plan to = plan(w, c.sms);
  if (to.bytes > c.spare) to = whole_sums(w, c.sms);
  if (c.dtype == AR_FLOAT32 || to.splits > 1) return to.pairs ? forward<2, true>(c, to.splits) : forward<1, true>(c, to.splits);
  return to.pairs ? forward<2, false>(c) : forward<1, false>(c);
}

cudaError_t launch_expert_weight_gradient(const ExpertsCall& c) {
  const Work w = gradient_work(c);
  Plan to = plan(w, c.sms);
  if (to.bytes > c.spare) to = whole_sums(w, c.sms);
  if (c.dtype == AR_FLOAT32 || to.splits > 1)
    return to.pairs ? weight_gradient<2, true>(c, to.splits) : weight_gradient<1, true>(c, to.splits);
  return to.pairs ? weight_gradient<2, false>(c) : weight_gradient<1, false>(c);
}

}  // namespace ar
