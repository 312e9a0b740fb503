// tc_gemm.cuh -- matrix products on the tensor cores of sm_103a: operands staged
// in shared memory by TMA, tcgen05.mma over a pair of CTAs, sums in TMEM.
//
// A pair of CTAs (a cluster of two) computes a 256 x 256 tile of sum_k A(i, k)
// B(j, k): each CTA stages 128 rows of A and 128 of B, the leader issues the
// products for both (cta_group::2), and each CTA holds the sums of its own 128
// rows: 256 of its 512 TMEM columns, so that the epilogue of one tile overlaps
// the products of the next.  A 128 x 256 tile by one CTA would stage 48 KB for the
// products that a CTA of the pair does with 32 KB: 96 bytes a clock per SM from L2
// against 64.
// Warps: 0-7 epilogue (TMEM lanes 32 (w % 4) on, columns 128 (w / 4) on), 8 producer,
// 9 products.  With four epilogue warps a tile's epilogue takes longer than the products
// of a tile of k up to about 1024.
// Operands of bf16, sums of fp32.
#pragma once

#include <cuda.h>

#include "rows.cuh"

namespace sv {

constexpr int kTcTile = 256;                 // tile rows and columns of a pair
constexpr int kTcHalf = 128;                 // of one CTA
constexpr int kTcK = 64;                     // k per stage: 128 bytes of bf16, one swizzle row
constexpr int kTcStages = 6;
constexpr int kTcOperand = kTcHalf * kTcK * 2;           // 16 KB
constexpr int kTcStage = 2 * kTcOperand;
constexpr int kTcEpilogue = 8;                           // warps
constexpr int kTcThreads = kTcEpilogue * 32 + 64;
constexpr int kTcProducer = kTcEpilogue, kTcIssuer = kTcEpilogue + 1;
constexpr uint32_t kTcColumns = 512;

// Places for the halves' values: a warp that is a tile ahead of its other half writes to
// one of its own, and its products wait for that half two tiles later at the latest.
constexpr int kTcTurns = 4;

struct TcShared {
  uint64_t full[kTcStages], empty[kTcStages], done[2], drained[2];
  uint64_t half[kTcTurns][kTcEpilogue / 2];
  uint32_t tmem;
  int failed;
};
constexpr int kTcBox = 32 * 128;                        // 32 rows of 64 bf16 on their way to memory
constexpr int kTcStaging = kTcEpilogue * kTcBox;
constexpr size_t kTcSmem = kTcStages * (size_t)kTcStage + kTcStaging + 1024 + sizeof(TcShared);
static_assert(kTcSmem <= 232448, "shared memory of a CTA");

// One box of a 2-D tensor map into this CTA's shared memory, counted on a
// barrier of either CTA of the pair.  x is a multiple of 8 elements (16 bytes).
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle, 64 bf16 wide rows.
//   k inner:  rows of 64 k; 8 rows a swizzle atom (1 KB apart); 16 k are 32 bytes.
//   k outer:  64 k rows of 64 i (8 KB); 8 k an atom (1 KB apart), the next 64 i
//             8 KB on; 16 k are 2 KB.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, bool k_inner) {
  const uint64_t lead = k_inner ? 1 : 8192 >> 4;
  return (uint64_t)((addr & 0x3FFFF) >> 4) | lead << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// kind::f16 instruction: fp32 sums, bf16 operands, M = N = 256
__device__ __forceinline__ uint32_t tc_idesc(bool a_k_inner, bool b_k_inner) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (a_k_inner ? 0u : 1u << 15) | (b_k_inner ? 0u : 1u << 16) |
         (kTcTile >> 3) << 17 | (kTcTile >> 4) << 24;
}
__device__ __forceinline__ void tc_mma(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// the barrier at this offset in both CTAs, once the products issued so far are done
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's 32 lanes: v[c] is column col + c of the thread's row
__device__ __forceinline__ void tc_load32(float (&v)[32], uint32_t addr) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(r[c]);
}

// 16 columns, added to x
__device__ __forceinline__ void tc_add16(float* x, uint32_t addr) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int c = 0; c < 16; ++c) x[c] += __uint_as_float(r[c]);
}

// An epilogue warp's stores: 32 rows of 64 bf16 at a time, thread = row, through
// shared memory (swizzled: no bank conflicts, and whole lines to L2; 16-byte stores
// by rows halve the write rate).  The map has boxes of 64 columns x 32 rows; what
// lies outside the matrix is left out.  x is a multiple of 8.
struct TcStore {
  uint32_t box;
  __device__ __forceinline__ void put(const CUtensorMap* map, int x, int y, const uint4 (&v)[8]) {
    const int lane = threadIdx.x & 31;
    const uint32_t row = box + lane * 128;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");       // the last one has left
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (uint32_t)((c ^ (lane & 7)) << 4)), "r"(v[c].x),
                   "r"(v[c].y), "r"(v[c].z), "r"(v[c].w)
                   : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                   "r"(y), "r"(box)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  __device__ __forceinline__ void finish() const {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
};

// One operand of a tile: rows i0 .. i0 + 255 (the CTA's half from i0 + 128 rank)
// over k0 .. of a matrix whose map has k inner (box 64 x 128) or i inner (box 64 x 64).
struct TcOperand {
  const CUtensorMap* map;
  bool k_inner;
  int i0, k0;
};
__device__ __forceinline__ void tc_stage(uint32_t dst, const TcOperand& o, uint32_t rank, int k, uint32_t bar) {
  const int i = o.i0 + (int)rank * kTcHalf;
  if (o.k_inner) {
    tma_box(dst, o.map, o.k0 + k, i, bar);
  } else {
    tma_box(dst, o.map, i, o.k0 + k, bar);
    tma_box(dst + kTcOperand / 2, o.map, i + 64, o.k0 + k, bar);
  }
}

// The persistent kernel.  Work::index(l, pair, pairs) is a pair's l-th tile, -1 after
// its last; Work::tile(t) gives a tile's operands and the number of stages of k
// (0: no product); Work::epilogue(t, e) is called by the epilogue threads.
// With CHUNK > 0 a tile's sum is taken in parts of CHUNK stages, each from 0 in a TMEM
// buffer of its turn, and the parts are added in registers, rounded to nearest: the
// tensor cores cut their sums off at every addition, and a part is smaller and has
// fewer of them.  The epilogue gets the sums, epilogue(t, e, x), of half rows for which
// Work::counts(t, e) holds; every tile has a product.
struct TcTile {
  TcOperand a, b;
  int steps;
};
// An epilogue thread's half row of a tile: the tile row, its first column of 128, the
// TMEM address of that, and whether there is a product (else the sums are 0).
struct TcHalfRow {
  int row, col;
  uint32_t tmem;
  bool any;
  float2* halves;                            // of this tile, by row % 128 (in the staging: either is used)
  uint64_t* ready;                           // and the barrier that counts this quarter's 32 of them
  uint32_t turn, joined;                     // tile mod kTcTurns; joins so far mod 2, a bit for each turn
  Waits waits;
  TcStore store;
  // The second half's value to the thread of the first half, which gets it (after a
  // wait that ran out, any value); at most once a tile, by both halves of a quarter.
  __device__ __forceinline__ float2 join(float2 v) {
    const int at = row & (kTcHalf - 1);
    if (col != 0) {
      halves[at] = v;
      mbar_arrive(ready);
      return v;
    }
    bounded_wait(ready, joined >> turn & 1, waits);
    joined ^= 1u << turn;
    return halves[at];
  }
};
// `make` gives the work, once the kernel before has ended.
template <int CHUNK, class Make>
__device__ __forceinline__ void tc_run(Make&& make, long long wait_limit, int* error) {
  extern __shared__ unsigned char tc_smem[];
  const uint32_t base = (smem_u32(tc_smem) + 1023) & ~1023u;
  TcShared& S = *reinterpret_cast<TcShared*>(tc_smem + (base - smem_u32(tc_smem)) + kTcStages * (size_t)kTcStage + kTcStaging);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const Waits waits{&S.failed, wait_limit};

  if (threadIdx.x == 0) {
    S.failed = 0;
    for (int i = 0; i < kTcStages; ++i) { mbar_init(&S.full[i], 1); mbar_init(&S.empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&S.done[i], 1); mbar_init(&S.drained[i], 2 * kTcEpilogue); }
    for (int i = 0; i < kTcTurns * kTcEpilogue / 2; ++i) mbar_init(&S.half[i % kTcTurns][i / kTcTurns], 32);
    fence_mbar_init();
  }
  __syncthreads();
  cluster_sync();                            // both CTAs' barriers are ready
  if (warp == kTcIssuer) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)),
                 "r"(kTcColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                            // both halves of the tensor memory are allocated
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  griddep_launch();
  griddep_wait();
  const auto work = make();

  if (warp == kTcProducer) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int l = 0, t; ok && (t = work.index(l, pair, pairs)) >= 0; ++l) {
        const TcTile tile = work.tile(t);
        for (int k = 0; k < tile.steps; ++k, ++it) {
          const int st = it % kTcStages;
          if (!(ok = bounded_wait(&S.empty[st], ((it / kTcStages) & 1) ^ 1, waits))) break;
          const uint32_t bar = map_rank(smem_u32(&S.full[st]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&S.full[st], 2 * kTcStage);   // both CTAs' halves
          const uint32_t at = base + st * kTcStage;
          tc_stage(at, tile.a, rank, k * kTcK, bar);
          tc_stage(at + kTcOperand, tile.b, rank, k * kTcK, bar);
        }
      }
    }
  } else if (warp == kTcIssuer) {
    if (rank == 0 && lane == 0) {
      int it = 0, n = 0;
      bool ok = true;
      for (int l = 0, t; ok && (t = work.index(l, pair, pairs)) >= 0; ++l) {
        const TcTile tile = work.tile(t);
        if (tile.steps == 0) continue;
        const uint32_t idesc = tc_idesc(tile.a.k_inner, tile.b.k_inner);
        const uint32_t sa = tile.a.k_inner ? 32 >> 4 : 2048 >> 4, sb = tile.b.k_inner ? 32 >> 4 : 2048 >> 4;
        int first = 0;
        do {
          const int buf = n & 1, end = CHUNK > 0 && first + CHUNK < tile.steps ? first + CHUNK : tile.steps;
          if (!(ok = bounded_wait(&S.drained[buf], ((n >> 1) & 1) ^ 1, waits))) break;
          tc_fence_after();
          const uint32_t d = tmem + buf * kTcTile;
          for (int k = first; k < end; ++k, ++it) {
            const int st = it % kTcStages;
            if (!(ok = bounded_wait(&S.full[st], (it / kTcStages) & 1, waits))) break;
            tc_fence_after();
            const uint64_t da = tc_desc(base + st * kTcStage, tile.a.k_inner);
            const uint64_t db = tc_desc(base + st * kTcStage + kTcOperand, tile.b.k_inner);
#pragma unroll
            for (int q = 0; q < kTcK / 16; ++q)
              tc_mma(d, da + (uint64_t)(q * sa), db + (uint64_t)(q * sb), idesc, k > first || q > 0);
            tc_commit(&S.empty[st]);
          }
          if (ok) tc_commit(&S.done[buf]);
          ++n;
          first = end;
        } while (CHUNK > 0 && ok && first < tile.steps);
      }
    }
  } else {
    int n = 0;
    TcHalfRow e;
    e.row = (int)rank * kTcHalf + (warp & 3) * 32 + lane;
    e.col = (warp >> 2) * kTcHalf;
    e.joined = 0;
    e.waits = waits;
    e.store.box = base + kTcStages * kTcStage + (uint32_t)warp * kTcBox;
    float2* const halves =
        reinterpret_cast<float2*>(tc_smem + (base - smem_u32(tc_smem)) + kTcStages * (size_t)kTcStage);
    for (int l = 0, t; (t = work.index(l, pair, pairs)) >= 0; ++l) {
      const int steps = work.tile(t).steps;
      const int turn = l % kTcTurns;
      e.halves = halves + turn * kTcHalf;
      e.ready = &S.half[turn][warp & 3];
      e.turn = (uint32_t)turn;
      if constexpr (CHUNK > 0) {
        float x[kTcHalf];
        const bool counts = work.counts(t, e);
        bool ok = true;
        int buf = 0;
#pragma unroll
        for (int c = 0; c < kTcHalf; ++c) x[c] = 0.f;
        for (int k = 0; k < steps; k += CHUNK, ++n) {
          buf = n & 1;
          ok = __all_sync(0xffffffffu, bounded_wait(&S.done[buf], (n >> 1) & 1, waits));
          if (!ok) break;
          tc_fence_after();
          if (counts) {
            const uint32_t at = tmem + buf * kTcTile + e.col + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll
            for (int c = 0; c < kTcHalf; c += 16) tc_add16(x + c, at + c);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&S.drained[buf]), 0));
        }
        if (!ok) break;
        if (counts) work.epilogue(t, e, x);
        continue;
      }
      const int buf = n & 1;
      if (steps > 0) {
        const bool ok = bounded_wait(&S.done[buf], (n >> 1) & 1, waits);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
      }
      e.tmem = tmem + buf * kTcTile + e.col + ((uint32_t)((warp & 3) * 32) << 16);
      e.any = steps > 0;
      if constexpr (CHUNK == 0) work.epilogue(t, e);
      if (steps > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&S.drained[buf]), 0));
        ++n;
      }
    }
    e.store.finish();
  }
  __syncwarp();
  if (any_failed(waits)) {    // copies or products may still be in flight
    drain_after_failure();
    if (lane == 0) *error = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();                            // neither CTA leaves while the other signals it
  tc_fence_after();
  if (warp == kTcIssuer)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcColumns) : "memory");
}

}  // namespace sv
