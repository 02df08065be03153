// ar_mma.cuh -- the tensor-core product that the expert products (ar_experts.cu) and
// the orthogonalisation (ar_orthogonal.cu) are made of: one persistent kernel whose
// tiles, operands and epilogue come from a policy class.
//
//   D[i, j] = sum_k A[i, k] B[j, k]      A, B 16-bit (bf16 or fp16), D fp32 in tensor memory
//
// i runs over 128 lanes per block (256 per pair of blocks), j over up to 128 columns
// per block of a pair (256 per pair; alone 128).  Either operand may lie with k or
// with i / j next to each other in memory: the tensor cores read both.
//
// Roles of a block's 12 warps: warp 2 works out the tiles, warp 0 issues the TMA loads of a
// tile's 64-deep slices into a ring of shared-memory stages, warp 1 issues the matrix
// instructions (of a pair only the even block's), warps 4 to 11 read finished accumulators and
// hand them to the policy's epilogue, in chunks of 32 columns; warp 3 clears what does not belong to a
// last slice, or tells of stored tiles where others wait for them.  There are two accumulators, so that
// one tile's epilogue overlaps the next tile's products.
//
// What bounds it: with 256 columns or so the matrix instructions (a pair's slice takes them 0.27 us at full clocks, 0.37
// in loops long enough for the power cap, which is cuBLAS's sustained rate; 4096 rows of 8
// even experts, 2048 -> 8192: 85 us in a captured graph, 1.6 PFLOP/s), with few columns the loads (16 rows of 8 experts: 47 us, 5.7 TB/s of
// weights).  Five or six stages keep 160 to 192 KB a block on their way; one thread issues all loads without a
// branch, as a slice's instructions in a whole warp took longer (0.36 us) than its products.
//
// Every wait is bounded (two seconds).  A block that gives up tells its other warps;
// what they have not computed by then becomes NaN in the output, copies and matrix
// instructions on their way are let finish, tensor memory is freed and the block ends.
#pragma once

#include <atomic>
#include <cstdint>
#include <cstdlib>

#include <cuda.h>
#include <cuda_runtime.h>

#include "ar_device.cuh"

namespace ar {
namespace mma {

constexpr int kRows = 128;                 // i per block
constexpr int kDepth = 64;                 // k per stage: 128 bytes, one swizzled row
constexpr int kBoxBytes = 64 * kDepth * 2; // 64 x 64 elements, 128-byte rows
constexpr int kAhead = 8;                  // tiles worked out ahead
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
constexpr uint64_t kLimit = 2000000000;    // ns that anything may be waited for
constexpr int kChunkStep = 32 * (kEpilogueWarps / 4);  // from one chunk of a warp to its next

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint32_t b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
}
// Of a barrier anywhere in the cluster.
__device__ __forceinline__ void bar_arrive_cluster(uint32_t b) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(b) : "memory");
}
// Relaxed: for what is no longer in use, not for what was written.  Releasing at the cluster's scope waits for
// the warp's stores on their way to memory, 2 us of every tile.
__device__ __forceinline__ void bar_free_cluster(uint32_t b) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(b) : "memory");
}
// Relaxed: what it announces is counted by the barrier itself.  With release semantics, and waits that acquire
// at the cluster's scope, every slice took 0.3 us more (4864 x 2048 x 8192: 235 us against 107).
__device__ __forceinline__ void bar_expect_cluster(uint32_t b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(b), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t b, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(done)
               : "r"(b), "r"(parity)
               : "memory");
  return done != 0;
}
__device__ __forceinline__ uint64_t nanoseconds() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// False where the phase did not end in time, or another warp of the block has given up.
__device__ __forceinline__ bool bar_wait(uint32_t b, uint32_t parity, volatile uint32_t* late) {
  if (bar_try(b, parity)) return true;
  const uint64_t begin = nanoseconds();
  for (uint32_t n = 1;; ++n) {
    if (bar_try(b, parity)) return true;
    if (*late) return false;
    if (n % 256 == 0 && nanoseconds() - begin > kLimit) {
      *late = 1;
      return false;
    }
  }
}
// The same for a whole warp: all its lanes get one answer.
__device__ __forceinline__ bool warp_wait(uint32_t b, uint32_t parity, volatile uint32_t* late) {
  return __all_sync(~0u, bar_wait(b, parity, late));
}
__device__ __forceinline__ uint32_t of_rank(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
  return one != 0;
}

// A box of `map` at (x, y, z, u) into shared memory; its bytes count on `bar`, which for
// a pair may be the other block's.
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t to, const CUtensorMap* map, int x, int y, int z, int u, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
        : "memory");
}

// 32 x 32 values from shared memory to (x, y, z) of `map`; what lies outside the map is not stored.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t from, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(from)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t to, uint32_t columns) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (CG == 2)
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// An arrival on `bar` (of a pair: on both blocks') once all matrix instructions issued so far are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32 columns of a warp's 32 lanes; a thread gets its lane's.
__device__ __forceinline__ void tmem_rows(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(at));
  tmem_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The same 32 x 32 values as the fragments of 8 x 8 matrices that stmatrix takes: v[16 h + 4 q + i] is
// row 16 h + lane / 4 + 8 (i / 2), column 8 q + 2 (lane % 4) + i % 2.
__device__ __forceinline__ void tmem_fragments(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(at));
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(at + (16u << 16)));
  tmem_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Four 8 x 8 matrices of 16-bit values, columns as rows: lane l gives the address of column l % 8 of matrix l / 8.
__device__ __forceinline__ void store_transposed(uint32_t to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// ------------------------------------------------------------------ a warp's 32 x 32 results

// In a warp's staging memory 32 columns of 32 16-bit rows lie 64 bytes each; their 16-byte parts are
// exchanged by (column / 2) % 4, so that neither side has bank conflicts.
__device__ __forceinline__ uint32_t staged(uint32_t staging, int column, int part) {
  return staging + column * 64 + ((part ^ (column >> 1 & 3)) << 4);
}
// The fragments of tmem_fragments, packed in pairs of columns: w[8 h + 2 q + i].
__device__ __forceinline__ void stage_columns(uint32_t staging, const uint32_t (&w)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    store_transposed(staged(staging, 8 * q + (lane & 7), lane >> 3), w[2 * q], w[2 * q + 1], w[8 + 2 * q],
                     w[8 + 2 * q + 1]);
}
// An epilogue warp's two staging areas in turn.  Every use ends in a commit, of stores or of nothing, so
// that "all but the last" are those from the area that comes next.
struct Staging {
  uint32_t base, bytes;          // of the first, of each
  uint32_t used = 0;
  __device__ __forceinline__ Staging(uint32_t base, uint32_t bytes) : base(base), bytes(bytes) {}
  __device__ __forceinline__ uint32_t next() {
    if ((threadIdx.x & 31) == 0) bulk_wait_read<1>();
    __syncwarp();
    return base + (used++ & 1) * bytes;
  }
  // What the warp has staged at `from` to (x, y, z) of map, where that is inside.
  __device__ __forceinline__ void store(uint32_t from, const CUtensorMap* map, int x, int y, int z, bool inside) const {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      if (inside) tma_store(map, from, x, y, z);
      bulk_commit();
    }
  }
  __device__ __forceinline__ void release() const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bulk_commit();
  }
};

// The staged columns to memory, `stride` elements apart; `rows` of each, `columns` of them.
__device__ __forceinline__ void put_columns(uint32_t staging, uint16_t* to, long long stride, int rows, int columns,
                                            bool vectors) {
  const int lane = threadIdx.x & 31, part = lane & 3;
  if (!vectors) {
    // a column at a time, a lane an element: 64 bytes in one store instruction (as 8 elements a lane, a sector each:
    // 700 x 700 x 700 18.0 us, now 12.1; dW of 7 x 1431 x 1001 67, now 28)
    columns = min(columns, 32);
#pragma unroll 8
    for (int c = 0; c < columns; ++c) {
      uint16_t v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(staged(staging, c, lane >> 3) + (lane & 7) * 2));
      if (lane < rows) to[c * stride + lane] = v;
    }
    return;
  }
  uint4 o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(o[q].x), "=r"(o[q].y), "=r"(o[q].z), "=r"(o[q].w)
                 : "r"(staged(staging, 8 * q + (lane >> 2), part)));
  uint16_t* d = to + (lane >> 2) * stride + part * 8;
  if (rows >= 32 && columns >= 32) {  // of the whole warp: no branches between the stores
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(d + q * (8 * stride)) = o[q];
    return;
  }
  for (int q = 0; q < 4; ++q, d += 8 * stride) {
    if (8 * q + (lane >> 2) >= columns) break;
    const uint4 v = q == 0 ? o[0] : q == 1 ? o[1] : q == 2 ? o[2] : o[3];
    if (part * 8 + 8 <= rows) {
      *reinterpret_cast<uint4*>(d) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (part * 8 + i < rows) d[i] = (uint16_t)(w[i / 2] >> (i % 2 * 16));
    }
  }
}

// ------------------------------------------------------------------ descriptors

// Of an operand in shared memory, 128-byte swizzle, as its 64 x 64 boxes lie there
// one behind the other: groups of eight 128-byte rows are 1024 bytes apart; where i
// (or j) is contiguous, the next 64 of it are a box (8192 bytes, or `box`) away.
__device__ __forceinline__ uint64_t operand_desc(uint32_t at, bool depth_contiguous, int box = kBoxBytes) {
  const uint64_t lead = depth_contiguous ? 1 : box >> 4;
  return (uint64_t)((at & 0x3ffff) >> 4) | lead << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Sixteen further in k, in the descriptor's units of 16 bytes.
__device__ __forceinline__ uint32_t depth_step(bool depth_contiguous) { return depth_contiguous ? 2 : 128; }

// fp32 accumulators of 16-bit operands; columns: of both blocks of a pair.
template <int CG>
__device__ __forceinline__ uint32_t instruction(bool bf16, bool a_depth, bool b_depth, int columns) {
  const uint32_t type = bf16 ? 1 : 0;
  return 1u << 4 | type << 7 | type << 10 | (a_depth ? 0u : 1u) << 15 | (b_depth ? 0u : 1u) << 16 |
         (uint32_t)(columns >> 3) << 17 | (uint32_t)(CG * kRows >> 4) << 24;
}

// ------------------------------------------------------------------ the kernel

// How an operand lies in memory, which says what its map and its boxes are like.
enum Kind : int {
  kDepthRows,   // k contiguous: a box is 64 k of up to 128 rows
  kWideRows,    // i (or j) contiguous, a multiple of 64 of them: a box is one or two times 64 i of 64 k
  kNarrowRows,  // i contiguous, any number of them: 64 i of 64 k, two loads
};

// One tile of one product.
struct Tile {
  const CUtensorMap *a, *b;
  Kind a_kind, b_kind;
  int a_row, b_row;        // first i of the pair, first j
  int a_z, b_z;            // which matrix of the map
  int k, blocks;           // first k, number of 64-deep slices (0: the sum is 0)
  int last;                // k of the last slice that count (64: all)
  int columns;             // j of the tile, a multiple of 16 * CG (kWideRows: 64 * CG), at most 128 * CG
  int b_bytes;             // of B's box(es) per block and slice
  int end, shape, stage, step;  // the policy's own
};

// What a chunk of a tile's epilogue is made of.
enum Source : int { kZeros, kSums, kLate };

template <int kStages, int kStageBytes, int kStaging>
struct Shared {
  alignas(1024) uint8_t stage[kStages][kStageBytes];
  alignas(1024) uint8_t staging[kEpilogueWarps][kStaging ? kStaging : 16];
  alignas(8) uint64_t full[kStages], empty[kStages], tail[kStages], ready[2], drained[2], done;
  // Tiles that have been worked out, with their epilogue's factors (columns 0: there are no more).
  uint64_t filled[kAhead], taken[kAhead], stored[kAhead];
  Tile tiles[kAhead];
  float factors[kAhead][2];
  uint32_t tmem, late;
};

template <class Policy>
using SharedOf = Shared<Policy::kStages, 2 * kBoxBytes + Policy::kBytesB, Policy::kAreas * Policy::kArea>;

// Where the next slice of an operand is, and how far the one behind it.
struct Boxes {
  const CUtensorMap* map;
  int x, y, z, u, dx, dy;
  bool two;                // a second box, 64 rows further
  __device__ __forceinline__ Boxes(const CUtensorMap* map, Kind kind, int row, int k, int matrix, int bytes)
      : map(map), two(kind == kNarrowRows && bytes > kBoxBytes) {
    x = kind == kDepthRows ? k : kind == kWideRows ? 0 : row;
    y = kind == kDepthRows ? row : k;
    z = kind == kWideRows ? row >> 6 : matrix;
    u = kind == kWideRows ? matrix : 0;
    dx = kind == kDepthRows ? kDepth : 0;
    dy = kDepth - dx;
  }
  template <int CG>
  __device__ __forceinline__ void load(uint32_t to, uint32_t bar) {
    tma_load<CG>(to, map, x, y, z, u, bar);
    if (two) tma_load<CG>(to + kBoxBytes, map, x + 64, y, z, u, bar);
    x += dx;
    y += dy;
  }
};

// Into how many runs, of at most kRun slices, a tile's sums are cut, and the slices of one: all alike, so that an
// epilogue has as many behind it as the next.  (So many slices a run make exactly so many runs: fewer would take r (r - 1) >=
// blocks > most (r - 1), so r > most, and then a run has `most`.)
__device__ __forceinline__ int runs_of(int blocks, int most) { return max(1, (blocks + most - 1) / most); }
__device__ __forceinline__ int run_length(int blocks, int most) {
  const int runs = runs_of(blocks, most);
  return (blocks + runs - 1) / runs;
}

template <int CG, class Policy>
constexpr int shared_bytes() {
  return (int)sizeof(SharedOf<Policy>) + (int)sizeof(typename Policy::Local) + 1024;
}

template <int CG, class Policy>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ typename Policy::Params p, int late_block) {
  extern __shared__ uint8_t raw[];
  constexpr int kStages = Policy::kStages, kStageBytes = 2 * kBoxBytes + Policy::kBytesB;
  auto& s = *reinterpret_cast<SharedOf<Policy>*>(raw + ((1024 - (saddr(raw) & 1023)) & 1023));
  auto& local = *reinterpret_cast<typename Policy::Local*>(&s + 1);
  constexpr uint32_t kColumns = 2 * 128 * CG;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int first = blockIdx.x / CG, pairs = gridDim.x / CG;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(saddr(&s.full[i]), CG);
      bar_init(saddr(&s.empty[i]), 1);
      bar_init(saddr(&s.tail[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(saddr(&s.ready[i]), 1);
      bar_init(saddr(&s.drained[i]), CG * kEpilogueWarps);
    }
    bar_init(saddr(&s.done), 1);
    for (int i = 0; i < kAhead; ++i) {
      bar_init(saddr(&s.filled[i]), 1);
      bar_init(saddr(&s.taken[i]), kEpilogueWarps + 2 + (rank == 0 ? 1 : 0));
      bar_init(saddr(&s.stored[i]), kEpilogueWarps);
    }
    s.late = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_enter();
  // Tensor memory is taken behind the wait for the kernel before: a kernel that holds
  // it has all it waits for.
  if (warp == 2) tmem_alloc<CG>(saddr(&s.tmem), kColumns);
  Policy::begin(p, local);
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s.tmem);
  volatile uint32_t* late = &s.late;

  if (warp == 2) {
    // Works the tiles out for all others, and waits for what they depend on, up to kAhead tiles early: in the loading
    // warp this took 2 us of every tile.
    for (uint32_t t = 0;; ++t) {
      Tile w;
      const bool more = Policy::tile(p, local, first + (int)t * pairs, w);
      const uint32_t place = t % kAhead;
      if (!warp_wait(saddr(&s.taken[place]), (t / kAhead & 1) ^ 1, late)) break;
      if constexpr (Policy::kOrdered) {
        if (more && !Policy::wait(p, w, late)) break;
        // what other blocks have stored is read by TMA from here on (in the loading warp the fence holds the loads up)
        asm volatile("fence.proxy.async.global;" ::: "memory");
        if (more && lane < 2) s.factors[place][lane] = Policy::factor(p, w, lane);
      }
      if (!more) w.columns = 0;
      if (lane == 0) s.tiles[place] = w;
      __syncwarp();
      if (lane == 0) bar_arrive(saddr(&s.filled[place]));
      if (!more) break;
    }
  } else if (warp == 0) {
    const bool gives_up = (int)blockIdx.x == late_block;
    if (gives_up) *late = 1;
    const bool one = elect();
    const uint32_t empty = saddr(&s.empty[0]), stages = saddr(s.stage[0]);
    const uint32_t full = CG == 2 ? of_rank(saddr(&s.full[0]), 0) : saddr(&s.full[0]);
    uint32_t slot = 0, phase = 0;
    // (Whether a warp goes on is decided by votes alone: its lanes may read `late` at different times.)
    for (uint32_t t = 0; !gives_up; ++t) {
      const uint32_t place = t % kAhead;
      if (!warp_wait(saddr(&s.filled[place]), t / kAhead & 1, late)) break;
      const Tile w = s.tiles[place];
      __syncwarp();
      if (lane == 0) bar_arrive(saddr(&s.taken[place]));
      if (w.columns == 0) break;
      const uint32_t bytes = 2 * kBoxBytes + w.b_bytes;
      Boxes a(w.a, w.a_kind, w.a_row + (int)rank * kRows, w.k, w.a_z, 2 * kBoxBytes);
      Boxes b(w.b, w.b_kind, w.b_row + (int)rank * (w.columns / CG), w.k, w.b_z, w.b_bytes);
      bool ok = true;
      if (one) {  // one thread issues them all
        for (int i = 0; i < w.blocks; ++i) {
          ok = bar_wait(empty + 8 * slot, phase ^ 1, late);
          if (!ok) break;
          const bool tail = w.last < kDepth && i == w.blocks - 1;  // warp 3 passes it on
          const uint32_t bar = tail ? saddr(&s.tail[slot]) : full + 8 * slot;
          if (CG == 2 && !tail) bar_expect_cluster(bar, bytes);
          else bar_expect(bar, bytes);
          const uint32_t at = stages + slot * kStageBytes;
          a.load<CG>(at, bar);
          b.load<CG>(at + 2 * kBoxBytes, bar);
          if (++slot == kStages) slot = 0, phase ^= 1;
        }
      }
      __syncwarp();
      if (!__all_sync(~0u, ok)) break;
      if (!one) {  // the others keep count
        const uint32_t n = slot + w.blocks;
        phase ^= n / kStages & 1;
        slot = n % kStages;
      }
    }
  } else if (warp == 1 && rank == 0) {
    const bool one = elect();  // one thread issues them all: a commit counts its own thread's
    uint32_t slot = 0, phase = 0, n = 0;
    for (uint32_t t = 0;; ++t) {
      const uint32_t place = t % kAhead;
      if (!warp_wait(saddr(&s.filled[place]), t / kAhead & 1, late)) break;
      const Tile w = s.tiles[place];
      __syncwarp();
      if (lane == 0) bar_arrive(saddr(&s.taken[place]));
      if (w.columns == 0) break;
      if (w.blocks == 0) continue;
      const uint32_t idesc = instruction<CG>(Policy::kBf16, w.a_kind == kDepthRows, w.b_kind == kDepthRows, w.columns);
      const uint32_t a_step = depth_step(w.a_kind == kDepthRows), b_step = depth_step(w.b_kind == kDepthRows);
      bool ok = true;
      for (int begin = 0; ok && begin < w.blocks;) {
        int end = w.blocks;
        if constexpr (Policy::kRun > 0) end = min(begin + run_length(w.blocks, Policy::kRun), end);
        const uint32_t buffer = n & 1, d = tmem + buffer * (kColumns / 2);
        ok = warp_wait(saddr(&s.drained[buffer]), ((n >> 1) & 1) ^ 1, late);
        ++n;
        fence_after();
        for (int i = begin; ok && i < end; ++i) {
          ok = warp_wait(saddr(&s.full[slot]), phase, late);
          if (!ok) break;
          // zeros that the other block's threads have stored
          if (CG == 2 && w.last < kDepth && i == w.blocks - 1) asm volatile("fence.acq_rel.cluster;" ::: "memory");
          fence_after();
          if (one) {
            const uint32_t at = saddr(s.stage[slot]);
            const uint64_t a = operand_desc(at, w.a_kind == kDepthRows),
                           b = operand_desc(at + 2 * kBoxBytes, w.b_kind == kDepthRows);
            if (i < w.blocks - 1 || w.last == kDepth) {
#pragma unroll
              for (int k = 0; k < kDepth / 16; ++k)
                mma_f16<CG>(d, a + k * a_step, b + k * b_step, idesc, i > begin || k > 0);
            } else {
              for (int k = 0; k < (w.last + 15) / 16; ++k)
                mma_f16<CG>(d, a + k * a_step, b + k * b_step, idesc, i > begin || k > 0);
            }
            mma_commit<CG>(saddr(&s.empty[slot]));
            if (i == end - 1) mma_commit<CG>(saddr(&s.ready[buffer]));
          }
          __syncwarp();
          if (++slot == kStages) slot = 0, phase ^= 1;
        }
        begin = end;
      }
      if (!ok) break;
    }
    if (__any_sync(~0u, *late)) {  // let what was issued finish
      if (one) mma_commit<CG>(saddr(&s.done));
      __syncwarp();
      for (const uint64_t begin = nanoseconds(); !bar_try(saddr(&s.done), 0) && nanoseconds() - begin < kLimit;) {}
    }
  } else if (warp >= 4) {
    const int e = warp - 4;
    uint32_t n = 0;
    bool ok = true;
    Staging staging(saddr(s.staging[e]), Policy::kArea);
    for (uint32_t t = 0;; ++t) {
      const uint32_t place = t % kAhead;
      Tile w;
      float factors[2] = {0.0f, 0.0f};
      ok = ok && warp_wait(saddr(&s.filled[place]), t / kAhead & 1, late);
      if (ok) {
        w = s.tiles[place];
        if constexpr (Policy::kOrdered) factors[0] = s.factors[place][0], factors[1] = s.factors[place][1];
        __syncwarp();
        if (lane == 0) bar_arrive(saddr(&s.taken[place]));
        if (w.columns == 0) break;
      } else {
        // The block has given up: from here on its tiles' results are NaN.  (The ring is not asked again: a barrier
        // that nothing arrives on any more lets every other round through.)
        if (!Policy::tile(p, local, first + (int)t * pairs, w)) break;
        if constexpr (Policy::kOrdered)
          if (!Policy::result(p, w)) continue;
      }
      const int row = w.a_row + (int)rank * kRows + (e & 3) * 32, first_column = (e >> 2) * 32;
      // The accumulators of one run are ready: `use` reads them, then they are handed back.
      const auto run = [&](auto use) {
        const uint32_t buffer = n & 1, at = tmem + buffer * (kColumns / 2) + ((uint32_t)(e & 3) * 32 << 16);
        if (w.blocks) {
          ok = ok && warp_wait(saddr(&s.ready[buffer]), (n >> 1) & 1, late);
          fence_after();
        }
        use(at);
        if (w.blocks) {
          ++n;
          fence_before();
          __syncwarp();
          if (lane == 0 && ok) {
            if constexpr (CG == 2) bar_free_cluster(of_rank(saddr(&s.drained[buffer]), 0));
            else bar_arrive(saddr(&s.drained[buffer]));
          }
        }
      };
      typename Policy::Epilogue out(p, local, w, row, first_column, staging, factors);
      int runs = 1;
      if constexpr (Policy::kRun > 0) runs = runs_of(w.blocks, Policy::kRun);
      for (int r = 0; r < runs; ++r)
        run([&](uint32_t at) {
          for (int c = first_column; c < w.columns; c += kChunkStep)
            out.chunk(at + c, c, !w.blocks ? kZeros : ok ? kSums : kLate, r > 0);
        });
      if constexpr (Policy::kOrdered) {  // warp 3 says so once all warps have stored their parts
        __syncwarp();
        if (lane == 0) bar_arrive(saddr(&s.stored[place]));
      }
    }
    if (lane == 0) bulk_wait();
  } else if (warp == 3) {
    if constexpr (!Policy::kOrdered) {
      // The last slice of an expert's rows: those of the next expert, or of none, come along, and both operands'
      // become 0 (the other operand's could be infinite).  k is a box's outer side there: whole 128-byte rows.
      const uint32_t full = CG == 2 ? of_rank(saddr(&s.full[0]), 0) : saddr(&s.full[0]);
      uint32_t slices = 0, phases = 0;
      for (uint32_t t = 0;; ++t) {
        const uint32_t place = t % kAhead;
        if (!warp_wait(saddr(&s.filled[place]), t / kAhead & 1, late)) break;
        const Tile w = s.tiles[place];
        __syncwarp();
        if (lane == 0) bar_arrive(saddr(&s.taken[place]));
        if (w.columns == 0) break;
        slices += w.blocks;
        if (w.blocks == 0 || w.last == kDepth) continue;
        const uint32_t slot = (slices - 1) % kStages;
        if (!warp_wait(saddr(&s.tail[slot]), phases >> slot & 1, late)) break;
        phases ^= 1u << slot;
        // up to whole sixteens, the rest is not multiplied
        const int end = (w.last + 15) & ~15, boxes = (2 * kBoxBytes + w.b_bytes) / kBoxBytes;
        for (int box = 0; box < boxes; ++box)
          for (int row = w.last + (lane >> 3); row < end; row += 4)
            *reinterpret_cast<uint4*>(s.stage[slot] + box * kBoxBytes + row * 128 + (lane & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) bar_arrive_cluster(full + 8 * slot);
          else bar_arrive(full + 8 * slot);
        }
      }
    }
    if constexpr (Policy::kOrdered) {
      bool ok = true;
      for (uint32_t t = 0;; ++t) {
        const uint32_t place = t % kAhead;
        Tile w;
        ok = ok && warp_wait(saddr(&s.filled[place]), t / kAhead & 1, late);
        if (ok) {
          w = s.tiles[place];
          __syncwarp();
          if (lane == 0) bar_arrive(saddr(&s.taken[place]));
          if (w.columns == 0) break;
          ok = warp_wait(saddr(&s.stored[place]), t / kAhead & 1, late);
        } else if (!Policy::tile(p, local, first + (int)t * pairs, w)) {
          break;
        }
        // the fence covers what the epilogue's warps stored before they arrived; who waits for a tile of a
        // block that has given up gives up too
        if (lane == 0) Policy::done(p, w, ok);
      }
    }
  }
  __syncwarp();
  if (*late) {
    // Copies on their way into this block's memory take microseconds; 10 ms are theirs.
    for (int i = 0; i < 10000; ++i) __nanosleep(1000);
  }
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 2) {
    fence_after();
    tmem_free<CG>(tmem, kColumns);
  }
}

// ------------------------------------------------------------------ host

// The map of `nz` matrices of `ny` rows of `nx` contiguous 16-bit elements; 128-byte swizzle, zeros outside.
// Strides in elements; addresses and strides are whole 16 bytes.  depth: nx is k; else nx is i (or j).  A box has
// `box` i (64 or 128; of kNarrowRows always 64).  Returns how it is to be loaded.
cudaError_t make_map(CUtensorMap* map, Kind* kind, bool bf16, const void* base, uint64_t nx, uint64_t ny, uint64_t nz,
                     uint64_t y_stride, uint64_t z_stride, bool depth, uint32_t box);

// The same for bf16 results stored in boxes of 32 x 32, 64-byte swizzle, as staged() lays them out.
cudaError_t make_store_map(CUtensorMap* map, const void* base, uint64_t nx, uint64_t ny, uint64_t nz, uint64_t y_stride,
                           uint64_t z_stride);

// Whether `in_pairs` tiles of pairs of blocks (256 x 256) take less time than `alone` tiles of blocks (128 x
// 128, a quarter of the work): both in whole waves over the multiprocessors, a slice at 0.27 us (the matrix
// instructions at full clocks) against 0.20 (its loads), and what a tile takes besides.  Measured, us, in pairs and alone: 4096 rows of 8
// experts, 2048 -> 8192, 85 and 125; 16384 of 64, 2048 -> 1024, 69 and 75; 700 x 700 x 700 26 and 17; 5 rows of 4, 512
// -> 1024, 6.7 and 5.9.
inline bool better_in_pairs(double in_pairs, double alone, double slices, int sms) {
  const double pairs = sms / 2 > 0 ? sms / 2 : 1;
  const auto whole = [](double n) { return (double)(long long)(n + 0.999999); };
  return whole(in_pairs / pairs) * (0.27 * slices + 3.0) <= whole(alone / sms) * (0.20 * slices + 2.0);
}

// AR_LATE_BLOCK=<number> in the environment: a block that gives up at once, for tests; -1: none.
inline int late_block() {
  static const int block = [] {
    const char* s = std::getenv("AR_LATE_BLOCK");
    return s ? std::atoi(s) : -1;
  }();
  return block;
}

// `together`: the blocks wait for one another, so all of them have to be on the GPU at once.
template <int CG, class Policy>
cudaError_t launch_product(const typename Policy::Params& p, long long tiles, int sms, cudaStream_t stream,
                           bool together = false) {
  constexpr int bytes = shared_bytes<CG, Policy>();
  static_assert(bytes <= 227 * 1024, "shared memory of a block");
  const cudaError_t e =
      cudaFuncSetAttribute(product_kernel<CG, Policy>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  if (together) {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  long long most = sms / CG;
  if (together) {  // as many as fit at once, asked once per device
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
      cfg.gridDim = dim3((unsigned)(most * CG));
      const cudaError_t q = cudaOccupancyMaxActiveClusters(&n, product_kernel<CG, Policy>, &cfg);
      if (q != cudaSuccess) return q;
      if (n <= 0) return cudaErrorCooperativeLaunchTooLarge;
      known[dev].store(n, std::memory_order_relaxed);
    }
    if (n < most) most = n;
  }
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * CG));
  return cudaLaunchKernelEx(&cfg, product_kernel<CG, Policy>, p, late_block());
}

}  // namespace mma
}  // namespace ar
