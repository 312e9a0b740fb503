// w4_linear.cu -- products with 4-bit weights on the tensor cores of sm_103a.
//
// logits[r, v] = sum over groups g of s[v, g] sum_{k in g} (q[v, k] - z[v, g]) h[r, k].
//
// The inner sums are products of bf16 with small whole numbers, which bf16 holds exactly:
// tcgen05.mma takes them, the weights as the operand A of 128 vocabulary rows in tensor
// memory and the hidden states as the operand B in shared memory, and starts a sum for each
// group.  Its fp32 sum is read back and added, times the group's scale, to registers.  No
// weight is rounded, and a sum of the tensor cores, which cut off at every addition, is at
// most 128 long.
//
// A CTA (one an SM) takes tiles of 128 vocabulary rows x NT rows of hidden states (16 to 128, the
// least that holds them: 35 us for one row and 36 for 16 against 151936 x 2048 weights in groups of
// 128, 39 for 32, 45 for 64, 69 for 128, 247 to 263 for 512).  The k of a tile goes by stages of 256 (16 KB of
// weights), cut into slots of whole groups: a slot has its own columns of tensor memory for A and
// for the sums of its groups, and two barriers, "ready" (unpacked, and the sums of its last use
// taken) and "done" (products finished): one wait and one commit of the issuing warp a slot.
// Roles, in warps:
//   teams of four  weights from shared memory to bf16 in tensor memory, thread = vocabulary row;
//                  the teams take slots in turn;
//   four or eight  groups' sums to registers, and out;
//   one each       copies of weights, copies of hidden states;
//   one or two     products, in turn.
// Where there are few tiles and much k, a cluster of CTAs splits the k of a tile, and the parts
// are joined through distributed shared memory in the order of their ranks.
//
// What bounds it: for few rows launch and first copies, and unpacking (2.75 instructions a pair of
// weights) with the hand-overs between the roles; the weights alone stream through the ring in 28 us
// (5.8 TB/s).  For many rows the way from a slot's products to its sums and on to the next products
// in its columns of tensor memory, which hold two slots: a slot of 128 k takes 1000 clocks, 512 of
// them products.  With barriers of their own for A, hidden
// states and sums at every 128 k one row took 54 us; with products issued by a single lane of a
// diverged warp 132.  mma.sync with the weights straight in registers took 108 us for up to 8 rows
// (its m16n8k16 goes out every 20 clocks of a scheduler, and needs the scales of 16 rows a warp).
#include "serve.cuh"
#include "tc_gemm.cuh"

namespace sv {
namespace {

constexpr int kRows = 128;                   // vocabulary rows of a tile
constexpr int kStageK = 256;                 // k of a stage of weights
constexpr int kWeightStage = kRows * kStageK / 2;        // 16 KB
constexpr int kMaxSplit = 4, kSplitStages = 16;          // of a tile's k, from so many stages on

template <int NT, int GROUP>
struct Shape {
  // a slot: whole groups, as many k as leave tensor memory for two slots (the sums of a group of a slot
  // take NT columns, the weights of 2 k one)
  static constexpr int cost(int k) { return k / 2 + k / GROUP * NT; }
  static constexpr int SlotK = 2 * cost(256) <= (int)kTcColumns ? 256 : GROUP >= 128 || 2 * cost(128) <= (int)kTcColumns ? 128
                               : GROUP >= 64 || 2 * cost(64) <= (int)kTcColumns ? 64 : 32;
  static constexpr int GS = SlotK / GROUP, Subs = kStageK / SlotK, ACols = SlotK / 2, DCols = GS * NT;
  static constexpr int Fit = (int)kTcColumns / (ACols + DCols), Slots = NT == 128 || Fit < 3 ? 2 : 3;
  static constexpr int DColumn = Slots * ACols;                  // where the sums begin
  static constexpr int Chunks = SlotK / 32;                      // of 16 bytes of a row
  // warps: teams of four unpack, and take slots in turn, as the issuers do
  static constexpr int Teams = NT == 128 ? 1 : Slots == 3 ? 3 : 2, UnpackWarps = 4 * Teams, Issuers = Slots == 3 ? 1 : 2;
  static constexpr int Columns = NT == 128 ? 64 : NT < 32 ? NT : 32, SumWarps = 4 * NT / Columns;       // columns of a thread
  static constexpr int Threads = (UnpackWarps + SumWarps + 2 + Issuers) * 32;
  // Whoever takes every n-th slot, stage or copy of a ring has a ring of a multiple of n: it waits
  // for every phase of the barriers that it waits for, and so never takes one for another.
  static constexpr int WS = NT > 16 ? 6 : Teams == 3 ? 9 : 8;     // stages of weights
  static constexpr int XK = NT == 128 ? 128 : 256, XS = NT <= 32 ? 6 : 4;   // of hidden states
  static constexpr int XSlot = NT * XK * 2, XBox = NT * 128;     // bytes
  static constexpr int Ring = WS * kWeightStage + XS * XSlot;
};
template <class Z>
struct W4Shared {
  uint64_t w_full[Z::WS], w_empty[Z::WS], x_full[Z::XS], x_empty[Z::XS], ready[Z::Slots], done[Z::Slots];
  uint32_t tmem;
  int failed;
};
template <class Z>
constexpr size_t linear_smem() { return Z::Ring + 1024 + sizeof(W4Shared<Z>); }

__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
                   "r"(dst), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
               : "memory");
}
// Whether a phase of a barrier is over.
__device__ __forceinline__ uint32_t over(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok;
}
// bounded_wait of a barrier that only this CTA arrives on, all lanes of a warp alike; `seen` is
// what over() said before (a test takes about 130 clocks from issue to use)
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const Waits& waits, uint32_t seen = 0) {
  if (__all_sync(0xffffffffu, seen)) return true;
  uint32_t ok;
  long long t0 = 0;
  for (;;) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(waits.limit < kSleepNs ? (uint32_t)waits.limit : kSleepNs)
        : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    const long long t = clock64();
    if (t0 == 0) t0 = t;
    if (__any_sync(0xffffffffu, *waits.failed || t - t0 > waits.limit)) {
      *waits.failed = 1;
      return false;
    }
  }
}
// The same without sleep.  Hardware sleeps for microseconds whatever shorter time it is asked for, so
// wait_for never gives up on what comes sooner, however low the limit.
__device__ __forceinline__ bool poll_for(uint64_t* bar, uint32_t parity, const Waits& waits) {
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, over(bar, parity))) {
    if (__any_sync(0xffffffffu, *waits.failed || clock64() - t0 > waits.limit)) {
      *waits.failed = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
// A in tensor memory, B in shared memory
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
               : "memory");
}
__device__ __forceinline__ void commit_to(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void store32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
      "r"(addr)
      : "memory");
}
__device__ __forceinline__ void store16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void load16(float (&v)[16], uint32_t addr) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(r[c]);
}
// once loads have been issued: what they give may be used after wait_loads and keep
__device__ __forceinline__ void wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void keep(float (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 16; ++c) asm volatile("" : "+f"(v[c]));
}
__device__ __forceinline__ uint4 shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// A scale on its way, and as a number once it is needed.  Both stay where they are written: a
// conversion that the compiler moves up to its load makes every turn wait for memory (500 clocks).
__device__ __forceinline__ uint32_t scale_bits(const __nv_bfloat16* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// 2, 4 or 8 scales, two in each even place (a single one has no pairs)
template <int N>
__device__ __forceinline__ void scale_pairs(uint32_t (&to)[N], const __nv_bfloat16* p) {
  if constexpr (N == 2) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(to[0]) : "l"(p));
  else if constexpr (N == 4) asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(to[0]), "=r"(to[2]) : "l"(p));
  else if constexpr (N == 8)
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(to[0]), "=r"(to[2]), "=r"(to[4]), "=r"(to[6]) : "l"(p));
}
__device__ __forceinline__ float scale_of_bits(uint32_t v) {
  float f;
  asm volatile("shl.b32 %0, %1, 16;" : "=f"(f) : "r"(v));
  return f;
}
// Zero points on their way: one, or 1, 2, 4 or 8 as bytes.
__device__ __forceinline__ void zero_byte(uint32_t& to, const uint8_t* p) { asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(to) : "l"(p)); }
template <int N>
__device__ __forceinline__ void zero_bytes(uint32_t* to, const uint8_t* p) {
  if constexpr (N == 1) zero_byte(to[0], p);
  else if constexpr (N == 2) asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(to[0]) : "l"(p));
  else if constexpr (N == 4) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(to[0]) : "l"(p));
  else asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(to[0]), "=r"(to[1]) : "l"(p));
}
// less_of(byte i of z): the byte, 0x43, the byte, 0x43
__device__ __forceinline__ uint32_t less_of_byte(uint32_t z, int i) { return __byte_perm(z, 0x43u, 0x4040u | (uint32_t)i * 0x0101u); }
// a += s x, two at once: each rounded once, as by fmaf
__device__ __forceinline__ void add_two(float* a, float s, const float* x) {
  asm("{\n .reg .b64 a, x, s;\n mov.b64 a, {%0, %1};\n mov.b64 x, {%3, %4};\n mov.b64 s, {%2, %2};\n"
      " fma.rn.f32x2 a, x, s, a;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(a[0]), "+f"(a[1])
      : "f"(s), "f"(x[0]), "f"(x[1]));
}
// acc[c] += s * column c of a group's sums
template <int N>
__device__ __forceinline__ void add_unit(float (&acc)[N], uint32_t from, float s) {
#pragma unroll
  for (int c = 0; c < N; c += 16) {          // (32 at once left too few registers: 64 rows, groups of 32: 113 us, here 100)
    float x[16];
    load16(x, from + c);
    wait_loads();
    keep(x);
#pragma unroll
    for (int i = 0; i < 16; i += 2) add_two(acc + c + i, s, x + i);
  }
}
// asks `count` elements from p + at on into L2
template <class T>
__device__ __forceinline__ void ahead(const T* p, size_t at, int count) {
  for (int i = 0; i < count; i += 128 / (int)sizeof(T))
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p + at + i));
}

struct W4Maps {
  CUtensorMap weight, hidden;
};

// What a CTA does: its tiles, and of each the stages [first, first + stages) of 256 k.
template <int NT>
struct Plan {
  static constexpr bool One = NT < 128;      // tile of rows (a call with more rows has tiles of 128)
  int items, step, row_tiles, first, stages;
  __device__ __forceinline__ int row0(int item) const { return One ? 0 : item % row_tiles * NT; }
  __device__ __forceinline__ int col0(int item) const { return (One ? item : item / row_tiles) * kRows; }
};

template <int NT, int GROUP, bool ZERO>
__global__ void __launch_bounds__(Shape<NT, GROUP>::Threads, 1)
linear_kernel(const __grid_constant__ W4Params P, const __grid_constant__ W4Maps M, int split) {
  using Z = Shape<NT, GROUP>;
  extern __shared__ unsigned char w4_smem[];
  const uint32_t base = (smem_u32(w4_smem) + 1023) & ~1023u;
  unsigned char* const ring = w4_smem + (base - smem_u32(w4_smem));
  W4Shared<Z>& S = *reinterpret_cast<W4Shared<Z>*>(ring + Z::Ring);
  const uint32_t w_ring = base, x_ring = base + Z::WS * kWeightStage;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kWeightCopies = Z::UnpackWarps + Z::SumWarps, kHiddenCopies = kWeightCopies + 1, kProducts = kWeightCopies + 2;
  const Waits waits{&S.failed, P.wait_limit};

  Plan<NT> plan;
  plan.row_tiles = (P.n + NT - 1) / NT;
  plan.items = plan.row_tiles * ((P.V + kRows - 1) / kRows);
  const int rank = blockIdx.x % split, item0 = blockIdx.x / split;
  plan.step = gridDim.x / split;
  {
    const int stages = (P.H + kStageK - 1) / kStageK;
    plan.first = rank * stages / split;
    plan.stages = (rank + 1) * stages / split - plan.first;
  }

  if (threadIdx.x == 0) {
    S.failed = 0;
    for (int i = 0; i < Z::WS; ++i) { mbar_init(&S.w_full[i], 1); mbar_init(&S.w_empty[i], 4 * Z::Subs); }
    for (int i = 0; i < Z::XS; ++i) { mbar_init(&S.x_full[i], 1); mbar_init(&S.x_empty[i], Z::XK / Z::SlotK); }
    for (int i = 0; i < Z::Slots; ++i) { mbar_init(&S.ready[i], 4 + Z::SumWarps); mbar_init(&S.done[i], 1); }
    fence_mbar_init();
  }
  if (warp == kProducts) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)), "r"(kTcColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;

  const int tiles = item0 < plan.items ? (plan.items - 1 - item0) / plan.step + 1 : 0;
  bool ok = true;
  if (warp < Z::UnpackWarps) {
    const int quarter = warp & 3, team = warp >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    // the team's next slot: `sub` of a stage, and where it goes
    RingAt w, a;
    int sub = team, stage = 0, item = item0;
    const auto whole = [&] {                 // sub back into a stage
#pragma unroll
      for (int i = 0; i < (Z::Teams + Z::Subs - 1) / Z::Subs; ++i) {
        if (sub >= Z::Subs) {
          sub -= Z::Subs;
          ++stage;
          w.next(Z::WS);
        }
      }
    };
    whole();
    a.skip(team, Z::Slots);
    uint4 v[Z::Chunks];
    // chunk c of a row's eight lies at c ^ (row % 8) times 16 bytes
    const uint32_t mine = w_ring + row * 128 + ((row & 7) << 4);
    const auto weights = [&] {
      const uint32_t at = (mine + w.stage * kWeightStage) ^ (sub * (Z::Chunks * 16));
#pragma unroll
      for (int c = 0; c < Z::Chunks; ++c) v[c] = shared16(at ^ (c * 16));
    };
    // zero points of the next slot's groups: all at once, GS bytes in zero[0] and zero[1], where those are
    // aligned, or one by one
    constexpr int kZeros = ZERO ? (Z::GS < 2 ? 2 : Z::GS) : 1;
    uint32_t zero[kZeros];
    const bool packed = ZERO && P.groups % Z::GS == 0 && reinterpret_cast<uintptr_t>(P.zero) % Z::GS == 0;
    const uint8_t* zeros_of = nullptr;
    const auto seek = [&] {                  // the tile of the next slot
      while (stage >= plan.stages) {
        stage -= plan.stages;
        item += plan.step;
      }
      zeros_of = P.zero + (size_t)min(plan.col0(item) + row, P.V - 1) * P.groups;
      ahead(P.zero, (size_t)min(plan.col0(item + plan.step) + row, P.V - 1) * P.groups, P.groups);
    };
    const auto zeros = [&] {
      if constexpr (ZERO) {
        const int g = (plan.first + stage) * (kStageK / GROUP) + sub * Z::GS;
        if (packed) {
          zero_bytes<Z::GS>(zero, zeros_of + min(g, P.groups - Z::GS));
        } else {
#pragma unroll
          for (int i = 0; i < Z::GS; ++i) zero_byte(zero[i], zeros_of + min(g + i, P.groups - 1));
        }
      }
    };
    const auto less = [&](int c) {           // of chunk c
      if constexpr (!ZERO) {
        return less_of(8);
      } else {
        const int i = c * 32 / GROUP;
        return packed ? less_of_byte(zero[i / 4], i % 4) : less_of(zero[i]);
      }
    };
    long long left = ((long long)tiles * plan.stages * Z::Subs - team + Z::Teams - 1) / Z::Teams;       // the team's slots
    if (left > 0) {
      if constexpr (ZERO) {
        seek();
        zeros();
      }
      ok = wait_for(&S.w_full[w.stage], w.phase, waits);
      weights();
    }
    while (ok && left > 0) {
      uint64_t* const emptied = &S.w_empty[w.stage];
      const uint32_t a_seen = over(&S.done[a.stage], a.phase ^ 1);
      const uint32_t to = lanes + a.stage * Z::ACols;
      // two chunks at a time; where there are registers, four before the slot's last use is waited for
      constexpr int kAtOnce = Z::Chunks < 2 ? 1 : 2, kFirst = Z::Chunks >= 4 && Z::Threads <= 512 ? 2 : 1;
      uint32_t r[kFirst][16 * kAtOnce];
      const auto unpack = [&](int c, uint32_t (&to)[16 * kAtOnce]) {
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const uint32_t l = less(c + u);
          unpack8(to + 16 * u, v[c + u].x, l);
          unpack8(to + 16 * u + 4, v[c + u].y, l);
          unpack8(to + 16 * u + 8, v[c + u].z, l);
          unpack8(to + 16 * u + 12, v[c + u].w, l);
        }
      };
#pragma unroll
      for (int i = 0; i < kFirst; ++i) unpack(i * kAtOnce, r[i]);
      if (!(ok = wait_for(&S.done[a.stage], a.phase ^ 1, waits, a_seen))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < Z::Chunks; c += kAtOnce) {
        const int i = c / kAtOnce;
        if (i >= kFirst) unpack(c, r[i % kFirst]);
        if constexpr (kAtOnce == 1) store16(to, r[0]);
        else store32(to + 16 * c, r[i % kFirst]);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.ready[a.stage]);
        // only here: the loads of a slot are sure to be done once what they gave has been
        // stored (an arrival before the stores has let the next copy into the stage under them)
        mbar_arrive(emptied);
      }
      sub += Z::Teams;
      whole();
      if (--left > 0) {
        if constexpr (ZERO) {
          if (stage >= plan.stages) seek();
          zeros();
        }
        if (!(ok = wait_for(&S.w_full[w.stage], w.phase, waits))) break;
        weights();
      }
      a.skip(Z::Teams, Z::Slots);
    }
  } else if (warp < kWeightCopies) {
    float acc[Z::Columns];
    const int quarter = warp & 3, part = (warp - Z::UnpackWarps) >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + Z::DColumn + part * Z::Columns;
    if (lane < Z::Slots) mbar_arrive(&S.ready[lane]);            // nothing to take of the first use
    RingAt d;
    uint32_t seen = 0;
    const int g0 = plan.first * (kStageK / GROUP), g1 = (plan.first + plan.stages) * (kStageK / GROUP);
    constexpr int kAhead = Z::GS <= 2 && NT < 128 ? 2 : 1;   // slots whose scales are on their way
    // Scales are asked for in the order of use, over the ends of tiles: a slot's at once, where its
    // groups' 2 GS bytes are aligned (then as pairs in the even places), or one by one.
    const bool pairs = Z::GS > 1 && P.groups % Z::GS == 0 && reinterpret_cast<uintptr_t>(P.scale) % (2 * Z::GS) == 0;
    const bool even = P.V % 2 == 0 && reinterpret_cast<uintptr_t>(P.out) % 4 == 0;
    uint32_t next[kAhead][Z::GS];
    int ask_item = item0, ask = g0;
    const __nv_bfloat16* scale = nullptr;
    const auto seek = [&] {
      scale = P.scale + (size_t)min(plan.col0(ask_item) + row, P.V - 1) * P.groups;
      ahead(P.scale, (size_t)min(plan.col0(ask_item + plan.step) + row, P.V - 1) * P.groups, P.groups);
    };
    const auto fetch = [&](uint32_t (&to)[Z::GS]) {
      if (pairs) {
        scale_pairs(to, scale + min(ask, P.groups - Z::GS));
      } else {
#pragma unroll
        for (int i = 0; i < Z::GS; ++i) to[i] = scale_bits(scale + min(ask + i, P.groups - 1));
      }
      if ((ask += Z::GS) >= g1) {
        ask = g0;
        ask_item += plan.step;
        seek();
      }
    };
    seek();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(next[u]);
    for (int item = item0; item < plan.items; item += plan.step) {
      const int v = plan.col0(item) + row;
#pragma unroll
      for (int c = 0; c < Z::Columns; ++c) acc[c] = 0.f;
      for (int g = g0; ok && g < g1; g += Z::GS) {
        float s[Z::GS];
#pragma unroll
        for (int i = 0; i < Z::GS; ++i)
          s[i] = pairs && (i & 1) ? scale_of_bits(next[0][i & ~1] >> 16) : scale_of_bits(next[0][i]);
#pragma unroll
        for (int u = 1; u < kAhead; ++u)
#pragma unroll
          for (int i = 0; i < Z::GS; ++i) next[u - 1][i] = next[u][i];
        fetch(next[kAhead - 1]);
        if (!(ok = wait_for(&S.done[d.stage], d.phase, waits, seen))) break;
        tc_fence_after();
        const uint32_t from = lanes + d.stage * Z::DCols;
#pragma unroll
        for (int i = 0; i < Z::GS; i += Z::Columns == 16 && Z::GS > 1 ? 2 : 1) {
          if (g + i >= P.groups) break;      // behind the row's end
          if constexpr (Z::Columns == 16 && Z::GS > 1) {
            float x[2][16];
            load16(x[0], from + i * NT);
            load16(x[1], from + (i + 1) * NT);
            wait_loads();
            keep(x[0]);
            keep(x[1]);
#pragma unroll
            for (int c = 0; c < 16; c += 2) add_two(acc + c, s[i], x[0] + c);
            if (g + i + 1 < P.groups) {
#pragma unroll
              for (int c = 0; c < 16; c += 2) add_two(acc + c, s[i + 1], x[1] + c);
            }
          } else {
            add_unit<Z::Columns>(acc, from + i * NT, s[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.ready[d.stage]);
        d.next(Z::Slots);
        seen = over(&S.done[d.stage], d.phase);
      }
      if (!ok) {
#pragma unroll
        for (int c = 0; c < Z::Columns; ++c) acc[c] = NAN;
      }
      if (split == 1) {
        const int r0 = plan.row0(item) + part * Z::Columns, rows = P.n - r0;
        const size_t o = (size_t)r0 * P.V + v;
        if (P.dtype == SPEC_BF16 && even) {
          // two lanes exchange columns: each stores two neighbours of a row at once
          __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(P.out) + o + (lane & 1 ? (ptrdiff_t)P.V - 1 : 0);
#pragma unroll
          for (int c = 0; c < Z::Columns; c += 2, to += 2 * (size_t)P.V) {
            if (NT == 16 && c >= rows) break;
            const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? acc[c] : acc[c + 1], 1);
            const __nv_bfloat162 two = lane & 1 ? __floats2bfloat162_rn(other, acc[c + 1]) : __floats2bfloat162_rn(acc[c], other);
            if (c + (lane & 1) < rows && v < P.V) *reinterpret_cast<__nv_bfloat162*>(to) = two;
          }
        } else if (v < P.V) {
          if (P.dtype == SPEC_BF16) {
            __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(P.out) + o;
#pragma unroll
            for (int c = 0; c < Z::Columns; ++c, to += P.V)
              if (c < rows) *to = __float2bfloat16_rn(acc[c]);
          } else {
            float* to = reinterpret_cast<float*>(P.out) + o;
#pragma unroll
            for (int c = 0; c < Z::Columns; ++c, to += P.V)
              if (c < rows) *to = acc[c];
          }
        }
      }
    }
    if (split > 1) {
      // With its last sums taken a warp knows that every product and so every copy is done: the ring is
      // free.  Otherwise copies may be in flight, and NaN stands for the sums.
      if (!ok) drain_after_failure();
      float* const parts = reinterpret_cast<float*>(ring);         // [NT][128]
#pragma unroll
      for (int c = 0; c < Z::Columns; ++c) parts[(part * Z::Columns + c) * kRows + row] = acc[c];
    }
  } else if (warp == kWeightCopies) {
    RingAt w;
    for (int item = item0; ok && item < plan.items; item += plan.step) {
      for (int j = 0; j < plan.stages; ++j) {
        if (!(ok = wait_for(&S.w_empty[w.stage], w.phase ^ 1, waits))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&S.w_full[w.stage], kWeightStage);
          copy_box(w_ring + w.stage * kWeightStage, &M.weight, (plan.first + j) * (kStageK / 2), plan.col0(item), &S.w_full[w.stage]);
        }
        w.next(Z::WS);
      }
    }
  } else if (warp == kHiddenCopies) {
    RingAt x;
    const uint32_t box_bytes = min(P.n, NT) * 128;
    for (int item = item0; ok && item < plan.items; item += plan.step) {
      for (int k = plan.first * kStageK; k < (plan.first + plan.stages) * kStageK; k += Z::XK) {
        if (!(ok = wait_for(&S.x_empty[x.stage], x.phase ^ 1, waits))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&S.x_full[x.stage], box_bytes * (Z::XK / 64));
#pragma unroll
          for (int c = 0; c < Z::XK / 64; ++c)
            copy_box(x_ring + x.stage * Z::XSlot + c * Z::XBox, &M.hidden, k + 64 * c, plan.row0(item), &S.x_full[x.stage]);
        }
        // a limit shorter than a sleep holds for each of these copies (polled for in every wait: 1 to 4 % of a call)
        if (waits.limit < kSleepNs && !(ok = poll_for(&S.x_full[x.stage], x.phase, waits))) break;
        x.next(Z::XS);
      }
    }
  } else {
    constexpr uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(NT >> 3) << 17 | (uint32_t)(kRows >> 4) << 24;
    constexpr int kSteps = GROUP / 16;       // 16 k each, 4 to a box
    // an issuer's slots: every Issuers-th of the CTA's, the copies of hidden states likewise
    constexpr int kPer = Z::XK / Z::SlotK;                       // slots to a copy
    const int mine = warp - kProducts;
    RingAt x, a;
    a.skip(mine, Z::Slots);
    x.skip(mine / kPer, Z::XS);
    int sub = mine % kPer;
    uint32_t a_seen = 0, x_seen = 0;
    for (long long slot = mine, slots = (long long)tiles * plan.stages * Z::Subs; slot < slots; slot += Z::Issuers) {
      if (!(ok = wait_for(&S.x_full[x.stage], x.phase, waits, x_seen) && wait_for(&S.ready[a.stage], a.phase, waits, a_seen))) break;
      tc_fence_after();
      const uint32_t at = tmem + a.stage * Z::ACols, to = tmem + Z::DColumn + a.stage * Z::DCols;
      const uint64_t desc = tc_desc(x_ring + x.stage * Z::XSlot + sub * Z::SlotK / 64 * Z::XBox + sub * Z::SlotK % 64 * 2, true);
      if (elect_one()) {
#pragma unroll
        for (int q = 0; q < Z::GS * kSteps; ++q)
          product(to + q / kSteps * NT, at + q * 8, desc + (uint64_t)((q >> 2) * (Z::XBox >> 4) + (q & 3) * 2), idesc, q % kSteps > 0);
        commit_to(&S.done[a.stage]);
        commit_to(&S.x_empty[x.stage]);
      }
      __syncwarp();
      a.skip(Z::Issuers, Z::Slots);
      a_seen = over(&S.ready[a.stage], a.phase);
      sub += Z::Issuers;
      x.skip(sub / kPer, Z::XS);
      sub %= kPer;
      x_seen = over(&S.x_full[x.stage], x.phase);
    }
  }
  __syncwarp();
  const bool failed = any_failed(waits);
  if (failed) drain_after_failure();         // copies or products may still be in flight
  __syncwarp();

  if (split > 1) {
    const bool sums = warp >= Z::UnpackWarps && warp < kWeightCopies;
    const int row = (warp & 3) * 32 + lane, part = (warp - Z::UnpackWarps) >> 2;
    cluster_sync();
    if (sums) {
      const int v = plan.col0(item0) + row, r0 = plan.row0(item0);
      for (int c = rank + part * split; c < NT && r0 + c < P.n; c += split * (Z::SumWarps / 4)) {
        float sum = 0.f;
        for (int k = 0; k < split; ++k) {
          float x;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(map_rank(base + (uint32_t)(c * kRows + row) * 4, k)) : "memory");
          sum += x;
        }
        if (v < P.V) {
          const size_t o = (size_t)(r0 + c) * P.V + v;
          if (P.dtype == SPEC_BF16) reinterpret_cast<__nv_bfloat16*>(P.out)[o] = __float2bfloat16_rn(sum);
          else reinterpret_cast<float*>(P.out)[o] = sum;
        }
      }
    }
    cluster_sync();                          // a part is read until here
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kProducts)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcColumns) : "memory");
}

// rows of `width` elements of `size` bytes, boxes of 128 bytes x `box` rows
bool encode(CUtensorMap* map, CUtensorMapDataType type, int size, const void* p, uint64_t width, uint64_t height, uint32_t box) {
  const cuuint64_t dims[2] = {width, height}, strides[1] = {width * size};
  const cuuint32_t boxes[2] = {(cuuint32_t)(128 / size), box}, ones[2] = {1, 1};
  return encoder()(map, type, 2, const_cast<void*>(p), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, int GROUP>
cudaError_t launch(const W4Params& P, int nsm, cudaStream_t s) {
  W4Maps M;
  if (!encode(&M.weight, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, P.packed, P.H / 2, P.V, kRows) ||
      // boxes of no more rows than there are: 36.4 us for one row, 39 with a box of 16 that TMA fills
      // up with zeros.  What the other rows of a tile hold reaches columns of the sums that nothing takes.
      !encode(&M.hidden, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, P.hidden, P.H, P.n, P.n < NT ? P.n : NT))
    return cudaErrorInvalidValue;
  const long long items = ((P.n + NT - 1ll) / NT) * ((P.V + kRows - 1ll) / kRows);
  const int stages = (P.H + kStageK - 1) / kStageK;
  // V = 2048, 8 rows: 12.3 us in one part and 8.2 in four for 16 stages, 18.5 and 10.3 for 32; 8.2 either way
  // for 8 (64 rows: 10.3 and 11.9), where the joining costs what it saves
  int split = 1;
  while (split < kMaxSplit && stages >= kSplitStages && 2 * split * items <= nsm) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(split > 1 ? items * split : items < nsm ? items : nsm));
  cfg.blockDim = dim3(Shape<NT, GROUP>::Threads);
  cfg.dynamicSmemBytes = linear_smem<Shape<NT, GROUP>>();
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)split, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return P.zero ? cudaLaunchKernelEx(&cfg, linear_kernel<NT, GROUP, true>, P, M, split)
                : cudaLaunchKernelEx(&cfg, linear_kernel<NT, GROUP, false>, P, M, split);
}
template <int NT>
cudaError_t of_group(const W4Params& P, int nsm, cudaStream_t s) {
  return P.group == 128 ? launch<NT, 128>(P, nsm, s) : P.group == 64 ? launch<NT, 64>(P, nsm, s) : launch<NT, 32>(P, nsm, s);
}
template <int NT, int GROUP>
cudaError_t allow() {
  using Z = Shape<NT, GROUP>;
  static_assert(linear_smem<Z>() <= 232448, "shared memory of a CTA");
  static_assert(Z::Slots % Z::Teams == 0 && Z::Slots % Z::Issuers == 0 && Z::WS * Z::Subs % Z::Teams == 0 &&
                (Z::XK >= Z::Issuers * Z::SlotK || Z::XS % Z::Issuers == 0), "phases");
  static_assert(Z::Slots >= Z::Teams && Z::DColumn + Z::Slots * Z::DCols <= (int)kTcColumns, "tensor memory");
  static_assert(Z::Ring >= NT * kRows * 4, "parts of a split tile");
  const int smem = (int)linear_smem<Z>();
  const cudaError_t e = cudaFuncSetAttribute(linear_kernel<NT, GROUP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(linear_kernel<NT, GROUP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}
template <int NT>
cudaError_t allow_all() {
  cudaError_t e = allow<NT, 32>();
  if (e == cudaSuccess) e = allow<NT, 64>();
  if (e == cudaSuccess) e = allow<NT, 128>();
  return e;
}

}  // namespace

cudaError_t configure_w4() {
  cudaError_t e = find_encoder();
  if (e != cudaSuccess) return e;
  e = allow_all<16>();
  if (e == cudaSuccess) e = allow_all<32>();
  if (e == cudaSuccess) e = allow_all<64>();
  if (e == cudaSuccess) e = allow_all<128>();
  return e;
}

cudaError_t launch_w4_linear(const W4Params& P, int nsm, cudaStream_t s) {
  if (P.n <= 16) return of_group<16>(P, nsm, s);
  if (P.n <= 32) return of_group<32>(P, nsm, s);
  if (P.n <= 64) return of_group<64>(P, nsm, s);
  return of_group<128>(P, nsm, s);
}

}  // namespace sv
