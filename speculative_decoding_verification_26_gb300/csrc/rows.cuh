// rows.cuh -- one logit row read by a CTA: the split into a scalar head, a body
// of 16-byte vectors and a scalar tail; clusters and bounded waits.
#pragma once

#include "common.cuh"

namespace sv {

// Logits of a row of dtype DT; PER of them fill a 16-byte vector.
template <int DT>
struct RowType;
template <>
struct RowType<SPEC_BF16> {
  static constexpr int ES = 2, PER = 8;
};
template <>
struct RowType<SPEC_F32> {
  static constexpr int ES = 4, PER = 4;
};

// One logit by a plain load (a row that the same kernel also writes).
template <int DT>
__device__ __forceinline__ float row_logit(const unsigned char* row, int e) {
  if constexpr (DT == SPEC_BF16)
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(row)[e]) << 16);
  else
    return reinterpret_cast<const float*>(row)[e];
}

// log2(e) / T = c + lo: c the fp32 quotient, lo what it leaves (an fma gives the
// exact remainder of the division), together good to about 2^-46.  Weights
// 2^{(x - m) c} take c alone, which scales an exponent by 1 + 2^-24 at most (and
// x - m first: m c of a row of the type's lowest value would overflow); lo enters
// where a logarithm is put back into units of the logits.
struct Scale {
  float c, lo;
};
constexpr float kLog2eHi = 1.4426950216293335f, kLog2eLo = 1.9259629911266175e-8f;
__device__ __forceinline__ Scale scale_split(float T) {
  Scale s;
  s.c = __fdiv_rn(kLog2eHi, T);
  s.lo = __fdiv_rn(__fmaf_rn(-s.c, T, kLog2eHi) + kLog2eLo, T);
  return s;
}

// Elements [0, head) and [tail0, V) are read one by one, the nvec vectors
// between them start on 16-byte boundaries.  Both ends hold fewer than PER
// elements.
struct RowSpan {
  int head, nvec, tail0;
};
template <int DT>
__device__ __forceinline__ RowSpan row_span(const unsigned char* row, int V) {
  constexpr int ES = RowType<DT>::ES, PER = RowType<DT>::PER;
  const int mis = (int)(reinterpret_cast<uintptr_t>(row) & 15u);
  RowSpan s;
  s.head = mis == 0 ? 0 : (16 - mis) / ES;
  if (s.head > V) s.head = V;
  s.nvec = (V - s.head) / PER;
  s.tail0 = s.head + s.nvec * PER;
  return s;
}

// A 16-byte vector as pairs of logits.
template <int DT>
__device__ __forceinline__ float2 vec_pair(const uint4& w, int k) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (DT == SPEC_BF16) return make_float2(bf16_lo(u[k]), bf16_hi(u[k]));
  else return make_float2(__uint_as_float(u[2 * k]), __uint_as_float(u[2 * k + 1]));
}
__device__ __forceinline__ uint32_t max_bf2(uint32_t a, uint32_t b) {  // a number before a NaN
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// The largest logit of a vector, NaNs left out.
template <int DT>
__device__ __forceinline__ float vec_max(const uint4& w) {
  if constexpr (DT == SPEC_BF16) {
    const uint32_t m = max_bf2(max_bf2(w.x, w.y), max_bf2(w.z, w.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  } else {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
}

// The largest logit of several vectors, NaNs left out.
template <int DT, int N>
__device__ __forceinline__ float vecs_max(const uint4 (&w)[N]) {
  if constexpr (DT == SPEC_BF16) {
    uint32_t m[N];
#pragma unroll
    for (int u = 0; u < N; ++u) m[u] = max_bf2(max_bf2(w[u].x, w[u].y), max_bf2(w[u].z, w[u].w));
#pragma unroll
    for (int u = 1; u < N; ++u) m[0] = max_bf2(m[0], m[u]);
    return fmaxf(bf16_lo(m[0]), bf16_hi(m[0]));
  } else {
    float m = vec_max<DT>(w[0]);
#pragma unroll
    for (int u = 1; u < N; ++u) m = fmaxf(m, vec_max<DT>(w[u]));
    return m;
  }
}

template <int DT>
__device__ __forceinline__ uint4 minus_infinity() {
  const uint32_t v = DT == SPEC_BF16 ? 0xFF80FF80u : 0xFF800000u;
  return make_uint4(v, v, v, v);
}
// Marks (bit u PER + k) of the logits of vectors that are at least `least` (of a
// bf16 row: a bf16 value).
template <int DT, int N>
__device__ __forceinline__ uint32_t mark_from(const uint4 (&w)[N], float least) {
  uint32_t mark = 0;
  const __nv_bfloat162 bar = __float2bfloat162_rn(least);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const uint32_t word[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == SPEC_BF16) {
        __nv_bfloat162 x;
        memcpy(&x, &word[i], 4);
        const uint32_t ge = __hge2_mask(x, bar);             // 0xFFFF per half
        mark |= ((ge & 1u) | (ge >> 31 << 1)) << (8 * u + 2 * i);
      } else {
        if (__uint_as_float(word[i]) >= least) mark |= 1u << (4 * u + i);
      }
    }
  }
  return mark;
}
// Vectors whose marked logits (bit u PER + k) become -inf.
template <int DT, int N>
__device__ __forceinline__ void drop_marked(uint4 (&w)[N], uint32_t mark) {
#pragma unroll
  for (int u = 0; u < N; ++u) {
    uint32_t* word[4] = {&w[u].x, &w[u].y, &w[u].z, &w[u].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == SPEC_BF16) {
        const uint32_t two = mark >> (8 * u + 2 * i) & 3u, cover = (two & 1u) * 0xFFFFu | (two >> 1) * 0xFFFF0000u;
        *word[i] = (*word[i] & ~cover) | (0xFF80FF80u & cover);
      } else {
        if (mark >> (4 * u + i) & 1u) *word[i] = 0xFF800000u;
      }
    }
  }
}

// A CTA's share of a row that a cluster of CS CTAs reads: vectors [lo, hi), and
// both ends' single elements by the first.
struct RowShare {
  int lo, hi;
  bool ends;
};
template <int CS>
__device__ __forceinline__ RowShare row_share(const RowSpan& sp, int rank) {
  if constexpr (CS == 1) return {0, sp.nvec, true};
  const int per = (sp.nvec + CS - 1) / CS, lo = rank * per;
  return {lo < sp.nvec ? lo : sp.nvec, lo + per < sp.nvec ? lo + per : sp.nvec, rank == 0};
}

// CTAs per row: the largest cluster that keeps every CTA resident at once, two per
// SM, and leaves each at least 16 KB of the row (two vectors a thread).
inline int row_cluster(int n, int V, int es, int nsm) {
  for (int cs = 8; cs > 1; cs /= 2)
    if ((long long)n * cs <= 2 * nsm && (long long)V * es >= cs * 16384ll) return cs;
  return 1;
}

inline int log2_of(int cs) { return cs == 8 ? 3 : cs == 4 ? 2 : cs == 2 ? 1 : 0; }

// Clusters of `cs` CTAs of a kernel that the current device holds at once: fewer
// than its SMs allow, where the SMs of a GPC do not divide by cs.  A persistent
// grid of more would leave whole clusters for a second wave.
template <class K>
inline cudaError_t resident_clusters(K kernel, int cs, int threads, size_t smem, int* out) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1024 * cs);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)cs, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(out, kernel, &cfg);
  if (e == cudaSuccess && *out < 1) *out = 1;
  return e;
}

constexpr float kLn2 = 0.693147180559945f;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A place in a ring of stages: the stage, and the phase of its barriers.
struct RingAt {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) { stage = 0; phase ^= 1; }
  }
};

// ---------------------------------------------------------------------------
// clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster; writes before it, to shared memory too, are seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// the same shared address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// 16 bytes to the same shared address of CTA `rank` of the cluster, counted there
// on a barrier: no fence on this side, the barrier's phase orders them for the reader.
__device__ __forceinline__ void send16(const void* at, const uint64_t* bar, uint32_t rank, uint32_t a, uint32_t b,
                                       uint32_t c, uint32_t d) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(
                   map_rank(smem_u32(at), rank)),
               "r"(map_rank(smem_u32(bar), rank)), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// 8 bytes to a shared address of the cluster, counted on a barrier of the same CTA.
__device__ __forceinline__ void send8(uint32_t addr, uint32_t bar, unsigned long long v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %2, [%1];" ::"r"(addr), "r"(bar),
               "l"(v)
               : "memory");
}

// A wait for a phase of a barrier gives up after `limit` cycles (by default about 2 s,
// which no healthy call comes near), or once another role of the CTA has (*failed).
// The thread sleeps in hardware in between (a polling warp takes issue slots from the
// others).  A CTA with a failed wait lets kDrainCycles (~1 ms) pass before it ends, for
// the copies still in flight.
struct Waits {
  volatile int* failed;
  long long limit;
};
constexpr long long kDrainCycles = 2000000ll;
constexpr uint32_t kSleepNs = 100000;
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, const Waits& waits) {
  uint32_t ok;
  long long t0 = 0;
  for (;;) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(waits.limit < kSleepNs ? (uint32_t)waits.limit : kSleepNs)
        : "memory");
    if (ok) return true;
    const long long t = clock64();
    if (t0 == 0) t0 = t;
    if (*waits.failed || t - t0 > waits.limit) {
      *waits.failed = 1;
      return false;
    }
  }
}
// whether a wait of this CTA ran out, the same for the warp
__device__ __forceinline__ bool any_failed(const Waits& waits) { return __any_sync(0xffffffffu, *waits.failed); }
__device__ __forceinline__ void drain_after_failure() {
  const long long t0 = clock64();
  while (clock64() - t0 < kDrainCycles) {}
}

}  // namespace sv
