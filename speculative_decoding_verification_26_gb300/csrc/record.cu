// record.cu -- the record of a teacher row: its K largest logits and the log
// mass of the rest.
//
// Per row x[V] at temperature T: the K largest logits, by value, ties to the
// lowest index, and tail = ln sum_{v not among them} e^{x_v / T}.  The tail is
// summed over the rest itself: as a difference of two full sums it would cancel
// where the K logits carry nearly all of the mass.
//
// What bounds it: the row is read once from HBM.  Two passes: a row's own CTA
// streams it twice (the second time from L2); where rows are few, a cluster of CS
// CTAs shares one, and the shares stay in shared memory between the passes.  Persistent CTAs, two per SM, of four roles:
//   producer  streams the shares into a ring of stages (bulk copies);
//   consumers pass A: 256 running maxima, one per thread over its own part of the
//             share (1024 where a share has to yield more than 64); pass B: candidates (logits above the bound, and
//             those equal to it) to shared memory, the weights of all others
//             summed: they are in the tail for certain;
//   picker    (one warp) takes a lower bound of the row's K-th largest logit from
//             the maxima: the K-th largest of a share's maxima is one, since K
//             parts each hold a logit that large, and so is the least, over the
//             shares, of each one's ceil(K / CS)-th largest; the greater of the
//             two leaves little more than K candidates.  Gathers the candidates
//             of the cluster in the row's leader (CTAs take turns);
//   rankers   (four warps) give each candidate its place, the number of candidates
//             before it, while the others are at the next row; they write the
//             record and add the candidates past K to the tail.
// Keys hold value and index, so no two are equal and the order in which candidates
// were found does not matter.  Where more than kTies logits equal the
// bound (a mask of finite values), the first of them are found by a scan in index
// order; where more than kAbove lie above it, the K-th largest is searched by
// counting over the row.
#include <cuda_runtime.h>

#include <cstdint>

#include "rows.cuh"

namespace sv {
namespace {

constexpr int kRecWarps = 8;                               // consumers
constexpr int kRecConsumers = kRecWarps * 32;
constexpr int kRankWarps = 4, kRankThreads = kRankWarps * 32;
constexpr int kRecThreads = kRecConsumers + 64 + kRankThreads;       // picker, rankers, producer
constexpr int kRecPer = 4;                                 // vectors of a stage per thread
constexpr int kRecStageVecs = kRecPer * kRecConsumers;
constexpr int kRecStage = 16 * kRecStageVecs;
constexpr int kRecMaxStages = 5;
constexpr int kMaxima = 4 * kRecConsumers;
constexpr int kAbove = 768, kTies = 256, kList = kAbove + kTies;
constexpr float kLn2 = 0.693147180559945f;

// order of a float as an unsigned integer, -0 and +0 alike
__device__ __forceinline__ uint32_t order_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // order_key(-inf)
// a candidate: larger comes first
__device__ __forceinline__ unsigned long long candidate(float x, int e) {
  return (unsigned long long)order_key(x) << 32 | (uint32_t)~e;
}

struct RecJob {
  int row, above, ties;                      // row -1: no more
  float below, m, T;
  uint32_t bound;
  bool counted;                              // above, ties and bound are the K-th largest key's
};
struct RecShared {
  uint64_t full[kRecMaxStages], empty[kRecMaxStages];
  // by row parity: the maxima are in; the bound is in; the candidates are in; every
  // CTA's bound, and candidate count, is in
  uint64_t maxed[2], bounded[2], found[2], bounds_in[2], counts_in[2];
  uint64_t listed[2], ranked[2];             // by job parity
  unsigned long long list[2][kList + 2];     // above from 0, ties from kAbove (in a leader's list: behind the others)
  float maxima[kMaxima];
  float part[kRecWarps], rank_part[kRankWarps];
  int part_above[kRecWarps], part_ties[kRecWarps];
  uint4 bounds[2][8], counts[2][8];          // of each CTA of the cluster
  RecJob job[2];
  int above, ties;                           // this share's candidates listed
  float m, c, least;                         // row maximum, scale, value of the bound
  int error, into;                           // whether the row is refused; which list the consumers fill
  int todo;                                  // of the rankers
  int failed;
};
enum { kRank = 0, kRecount = 1, kStop = 2 };

// The ring's place: stage and phase.
struct RecRing {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) { stage = 0; phase ^= 1; }
  }
};

// Four running maxima of a thread; NaN when one was seen.
template <int DT>
struct Maxima;
template <>
struct Maxima<SPEC_BF16> {                   // both halves of two words
  uint32_t m[2] = {0xFF80FF80u, 0xFF80FF80u};
  __device__ __forceinline__ void add(int u, const uint4& w) {
    m[u & 1] = max_nan_bf2(m[u & 1], max_nan_bf2(max_nan_bf2(w.x, w.y), max_nan_bf2(w.z, w.w)));
  }
  __device__ __forceinline__ float get(int i) const { return i & 1 ? bf16_hi(m[i >> 1]) : bf16_lo(m[i >> 1]); }
};
template <>
struct Maxima<SPEC_F32> {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  __device__ __forceinline__ void add(int u, const uint4& w) {
    m[u] = max_nan(m[u], max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                                 max_nan(__uint_as_float(w.z), __uint_as_float(w.w))));
  }
  __device__ __forceinline__ float get(int i) const { return m[i]; }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A bound of a share's want-th largest logit from N of its maxima per lane: a key
// that `want` or more of them reach, at most an eighth more where there is one.
// Keys of bf16 logits are told apart by their upper halves.  A bound of
// kKeyNegInf + 1 takes every finite logit (-inf is never recorded).
template <int DT, int N>
__device__ __forceinline__ uint32_t bound_of(const uint32_t (&key)[N], int want) {
  constexpr int shift = DT == SPEC_BF16 ? 16 : 0;
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) { lo = min(lo, key[j]); hi = max(hi, key[j]); }
  lo = __reduce_min_sync(0xffffffffu, lo) >> shift;
  hi = __reduce_max_sync(0xffffffffu, hi) >> shift;
  const uint32_t least = (kKeyNegInf >> shift) + 1;
  if (lo < least) {
    lo = least;
    int n = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) n += (key[j] >> shift) >= lo;
    if ((int)__reduce_add_sync(0xffffffffu, (unsigned)n) < want) hi = lo;
  }
  while (lo < hi) {                          // lo is reached by `want` or more, hi + 1 by fewer
    // four keys between at a time; two counts to a word (at most 1024 each)
    const uint32_t gap = hi - lo, p1 = lo + gap / 5 + 1, p2 = max(p1, lo + gap / 5 * 2 + 1),
                   p3 = max(p2, lo + gap / 5 * 3 + 1), p4 = max(p3, lo + gap / 5 * 4 + 1);
    unsigned low = 0, high = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t k = key[j] >> shift;
      low += (k >= p1 ? 1u : 0u) + (k >= p2 ? 65536u : 0u);
      high += (k >= p3 ? 1u : 0u) + (k >= p4 ? 65536u : 0u);
    }
    low = __reduce_add_sync(0xffffffffu, low);
    high = __reduce_add_sync(0xffffffffu, high);
    const int n1 = (int)(low & 0xFFFFu), n2 = (int)(low >> 16), n3 = (int)(high & 0xFFFFu), n4 = (int)(high >> 16);
    int n;
    if (n4 >= want) { lo = p4; n = n4; }
    else if (n3 >= want) { lo = p3; hi = p4 - 1; n = n3; }
    else if (n2 >= want) { lo = p2; hi = p3 - 1; n = n2; }
    else if (n1 >= want) { lo = p1; hi = p2 - 1; n = n1; }
    else { hi = p1 - 1; n = 1 << 30; }
    if (n <= want + want / 8) break;
  }
  return shift == 0 ? lo : lo << 16 | (lo & 0x8000u ? 0u : 0xFFFFu);
}
// Both bounds of a share (for K, and for its part of K) and its maximum, NaN first.
template <int DT, int N>
__device__ __forceinline__ float bounds_of(const float* maxima, int K, int part, uint32_t& whole, uint32_t& share) {
  uint32_t key[N];
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float x = maxima[(threadIdx.x & 31) + 32 * j];
    m = max_nan(m, x);
    key[j] = order_key(x);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
  whole = share = kKeyNegInf + 1;
  if (isfinite(m)) {
    if (K <= 32 * N) whole = bound_of<DT>(key, K);
    share = part == K ? whole : bound_of<DT>(key, part);
  }
  return m;
}

// Calls f(e, x) for every logit of a row, by one warp.
template <int DT, class F>
__device__ __forceinline__ void warp_row(const unsigned char* row, int V, F&& f) {
  constexpr int PER = RowType<DT>::PER;
  const RowSpan sp = row_span<DT>(row, V);
  const uint4* vec = reinterpret_cast<const uint4*>(row + (size_t)sp.head * RowType<DT>::ES);
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int j = lane; j < sp.nvec; j += 32) {
    const uint4 w = vec[j];
#pragma unroll
    for (int k = 0; k < PER / 2; ++k) {
      const float2 x = vec_pair<DT>(w, k);
      f(sp.head + j * PER + 2 * k, x.x);
      f(sp.head + j * PER + 2 * k + 1, x.y);
    }
  }
  const int ends = sp.head + (V - sp.tail0);
  if (lane < ends) {
    const int e = lane < sp.head ? lane : sp.tail0 + (lane - sp.head);
    f(e, row_logit<DT>(row, e));
  }
}

__device__ __forceinline__ void rank_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kRankThreads) : "memory"); }

// The K-th largest key of a row by counting, for a row with more candidates above
// the bound than are listed; one warp.  Lists what lies above it (less than K).
template <int DT>
__device__ __noinline__ void recount(const RecordParams& P, RecJob& job, unsigned long long* list) {
  const int K = P.K, V = P.V, lane = threadIdx.x & 31;
  const unsigned char* row = P.logits + (size_t)job.row * V * RowType<DT>::ES;
  const float c = scale_split(job.T).c, ref = ref_of(job.m, c);
  auto count = [&](auto&& pred) {
    int n = 0;
    warp_row<DT>(row, V, [&](int, float x) { n += pred(order_key(x)); });
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
  };
  uint32_t lo = job.bound + 1, hi = order_key(job.m);
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    if (count([&](uint32_t k) { return k >= mid; }) >= K) lo = mid;
    else hi = mid - 1;
  }
  const int ties = count([&](uint32_t k) { return k == lo; });
  float s = 0.f;
  int at = 0;
  for (int e0 = 0; e0 < V; e0 += 32) {
    const int e = e0 + lane;
    const float x = e < V ? row_logit<DT>(row, e) : -INFINITY;
    const uint32_t k = order_key(x);
    const bool above = e < V && k > lo;
    const unsigned vote = __ballot_sync(0xffffffffu, above);
    if (above) list[at + __popc(vote & ((1u << lane) - 1))] = candidate(x, e);
    at += __popc(vote);
    if (e < V && k < lo) s += ex2(fmaf(x, c, -ref));
  }
  s = warp_sum(s);
  __syncwarp();
  if (lane == 0) { job.above = at; job.ties = ties; job.below = s; job.bound = lo; job.counted = true; }
  __syncwarp();
}

// The rankers' work on one row.
template <int DT>
__device__ __forceinline__ void rank_row(const RecordParams& P, RecShared& S, RecJob& shared, unsigned long long* list) {
  const int K = P.K, V = P.V, t = (int)threadIdx.x - kRecConsumers - 32, lane = t & 31, warp = t >> 5;
  if (S.todo == kRecount) {
    if (warp == 0) recount<DT>(P, shared, list);
    rank_sync();
  }
  const RecJob job = shared;
  const int r = job.row;
  const unsigned char* row = P.logits + (size_t)r * V * RowType<DT>::ES;
  float* top = P.top_logits + (size_t)r * K;
  int32_t* ti = P.top_index + (size_t)r * K;
  const Scale sc = scale_split(job.T);
  const float ref = ref_of(job.m, sc.c);
  auto weight = [&](float x) { return ex2(fmaf(x, sc.c, -ref)); };
  const bool listed_ties = !job.counted && job.ties <= kTies;
  const int above = job.above, n = above + (listed_ties ? job.ties : 0);
  if (t == 0) list[n] = 0;                   // the keys are read by twos
  rank_sync();
  constexpr int kEach = kList / kRankThreads;
  int place[kEach];
  unsigned long long mine[kEach];
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    if (q * kRankThreads >= n) break;
    const int i = t + q * kRankThreads;
    mine[q] = i < n ? list[i] : 0;
    int before = 0;
    const ulonglong2* pair = reinterpret_cast<const ulonglong2*>(list);
#pragma unroll 4
    for (int j = 0; j < (n + 1) / 2; ++j) {
      const ulonglong2 p = pair[j];
      before += (p.x > mine[q]) + (p.y > mine[q]);
    }
    place[q] = before;
  }
  rank_sync();                               // the list is read: it takes the weights past K, by place
  float* left = reinterpret_cast<float*>(list);
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    if (q * kRankThreads >= n) break;
    if (t + q * kRankThreads >= n) continue;
    const float x = key_value((uint32_t)(mine[q] >> 32));
    const int e = (int)~(uint32_t)mine[q];
    if (place[q] < K) {
      top[place[q]] = x == 0.f ? row_logit<DT>(row, e) : x;  // the key has lost a zero's sign
      ti[place[q]] = e;
    } else {
      left[place[q] - K] = weight(x);
    }
  }
  float extra = 0.f;
  if (n > K) {
    rank_sync();
    for (int i = t; i < n - K; i += kRankThreads) extra += left[i];
    extra = warp_sum(extra);
    if (lane == 0) S.rank_part[warp] = extra;
    rank_sync();
    extra = 0.f;
    for (int w = 0; w < kRankWarps; ++w) extra += S.rank_part[w];
  }
  if (listed_ties) {
    for (int i = n + t; i < K; i += kRankThreads) { top[i] = -INFINITY; ti[i] = -1; }    // fewer finite logits than K
  } else if (warp == 0) {
    // ties in index order up to K; the others are in the tail
    int at = above;
    for (int e0 = 0; at < K && e0 < V; e0 += 128) {
      float x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int e = e0 + 32 * q + lane;
        x[q] = e < V ? row_logit<DT>(row, e) : -INFINITY;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool tie = order_key(x[q]) == job.bound;
        const unsigned vote = __ballot_sync(0xffffffffu, tie);
        const int to = at + __popc(vote & ((1u << lane) - 1));
        if (tie && to < K) { top[to] = x[q]; ti[to] = e0 + 32 * q + lane; }
        at += __popc(vote);
      }
    }
    extra += (float)(job.ties - (K > above ? K - above : 0)) * weight(key_value(job.bound));
  }
  if (t == 0) {
    // the weights are 2^{x c - ref}: ref and the scale's remainder put the exponent back
    const float tail = job.below + extra, nan = __int_as_float(0x7fc00000);
    const bool failed = *(volatile int*)&S.failed != 0;
    P.tail_lse[r] = failed ? nan : tail > 0.f ? kLn2 * (ref + (log2f(tail) + job.m * sc.lo)) : -INFINITY;
    if (P.status) P.status[r] = failed ? SPEC_ST_TIMEOUT : SPEC_ST_OK;
  }
  rank_sync();                               // before the list is filled again
}

template <int DT, int CS>
__global__ void __launch_bounds__(kRecThreads, 2) record_kernel(const __grid_constant__ RecordParams P,
                                                                const int stages, const bool keep) {
  constexpr int PER = RowType<DT>::PER, ES = RowType<DT>::ES;
  extern __shared__ __align__(128) unsigned char s_ring[];
  RecShared& S = *reinterpret_cast<RecShared*>(s_ring + (size_t)stages * kRecStage);
  const int V = P.V, K = P.K, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CS == 1 ? 0 : (int)cluster_rank();
  const int first = blockIdx.x / CS, step = gridDim.x / CS;
  volatile int* failed = &S.failed;

  if (tid == 0) {
    S.failed = 0;
    S.above = S.ties = 0;
    for (int i = 0; i < stages; ++i) { mbar_init(&S.full[i], 1); mbar_init(&S.empty[i], kRecWarps); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.maxed[i], kRecWarps);
      mbar_init(&S.bounded[i], 1);
      mbar_init(&S.found[i], kRecWarps);
      mbar_init(&S.bounds_in[i], 1);
      mbar_init(&S.counts_in[i], 1);
      mbar_init(&S.listed[i], 1);
      mbar_init(&S.ranked[i], kRankWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if constexpr (CS > 1) cluster_sync();

  const int part = (K + CS - 1) / CS;        // a share's part of the record
  const bool few = part <= 64;               // one maximum per thread is enough

  if (warp == kRecWarps + 1 + kRankWarps) {  // producer
    if (lane == 0) {
      RecRing at;
      for (int r = first; r < P.n; r += step) {
        const unsigned char* row = P.logits + (size_t)r * V * ES;
        const RowSpan sp = row_span<DT>(row, V);
        const RowShare sh = row_share<CS>(sp, rank);
        const unsigned char* body = row + (size_t)sp.head * ES;
        bool ok = true;
        for (int pass = 0; pass < (keep ? 1 : 2) && ok; ++pass)
          for (int j = sh.lo; j < sh.hi; j += kRecStageVecs) {
            const uint32_t bytes = 16u * (uint32_t)(sh.hi - j < kRecStageVecs ? sh.hi - j : kRecStageVecs);
            if (!(ok = bounded_wait(&S.empty[at.stage], at.phase ^ 1, failed))) break;
            mbar_arrive_expect_tx(&S.full[at.stage], bytes);
            bulk_load(s_ring + (size_t)at.stage * kRecStage, body + 16ll * j, bytes, &S.full[at.stage]);
            at.next(stages);
          }
        if (!ok) break;
      }
    }
  } else if (warp > kRecWarps) {             // rankers
    for (int j = 0;; ++j) {
      bounded_wait(&S.listed[j & 1], (j >> 1) & 1, failed);
      if (warp == kRecWarps + 1 && lane == 0)                // one decision for all four warps
        S.todo = *failed || S.job[j & 1].row < 0 ? kStop : S.job[j & 1].above > kAbove ? kRecount : kRank;
      rank_sync();
      if (S.todo == kStop) break;
      rank_row<DT>(P, S, S.job[j & 1], S.list[CS == 1 ? j & 1 : 1]);
      if (lane == 0) mbar_arrive(&S.ranked[j & 1]);
    }
  } else if (warp == kRecWarps) {            // picker
    int i = 0, live = 0;                     // rows, and rows not refused
    float T = first < P.n && P.temperature ? P.temperature[first] : 1.f;
    for (int r = first; r < P.n; r += step, ++i) {
      const int b = i & 1;
      const uint32_t turn = (i >> 1) & 1;
      const float given = T;
      if (P.temperature && r + step < P.n) T = P.temperature[r + step];
      bounded_wait(&S.maxed[b], turn, failed);
      __syncwarp();
      uint32_t bound, share;
      float m = few ? bounds_of<DT, kRecConsumers / 32>(S.maxima, K, part, bound, share)
                    : bounds_of<DT, kMaxima / 32>(S.maxima, K, part, bound, share);
      if constexpr (CS > 1) {
        if (lane == 0) mbar_arrive_expect_tx(&S.bounds_in[b], 16 * CS);
        __syncwarp();
        if (lane < CS) send16(&S.bounds[b][rank], &S.bounds_in[b], lane, __float_as_uint(m), bound, share, 0u);
        bounded_wait(&S.bounds_in[b], turn, failed);
        __syncwarp();
        uint32_t least = 0xFFFFFFFFu;
#pragma unroll
        for (int q = 0; q < CS; ++q) {
          const uint4 v = S.bounds[b][q];
          m = max_nan(m, __uint_as_float(v.x));
          bound = max(bound, v.y);
          least = min(least, v.z);
        }
        bound = max(bound, least);
      }
      if (bound == order_key(0.f) - 1) ++bound;              // no logit has that key, and its value compares as 0's
      int st = 0;
      if (!temperature_ok(given)) st |= SPEC_ST_BAD_TEMPERATURE;
      if (!isfinite(m)) st |= SPEC_ST_NONFINITE;             // NaN, +inf, or nothing finite
      const float Tr = st ? 1.f : given;
      const int leader = live % CS, job = live / CS;         // the same in every CTA of the cluster
      // the list that the consumers are about to fill is free again
      if (CS == 1 && st == 0 && job >= 2) bounded_wait(&S.ranked[job & 1], ((job - 2) >> 1) & 1, failed);
      __syncwarp();
      if (lane == 0) {
        S.m = m;
        S.c = scale_split(Tr).c;
        S.least = key_value(bound);
        S.error = st;
        S.into = CS == 1 ? job & 1 : 0;
        mbar_arrive(&S.bounded[b]);
      }
      if (st != 0) {
        if (rank == 0) {
          for (int k = lane; k < K; k += 32) {
            P.top_logits[(size_t)r * K + k] = __int_as_float(0x7fc00000);
            P.top_index[(size_t)r * K + k] = -1;
          }
          if (lane == 0) {
            P.tail_lse[r] = __int_as_float(0x7fc00000);
            if (P.status) P.status[r] = st;
          }
        }
        bounded_wait(&S.found[b], turn, failed);
        __syncwarp();
        continue;
      }
      bounded_wait(&S.found[b], turn, failed);
      __syncwarp();
      int above = 0, ties = 0;
      float below = 0.f;
      for (int w = 0; w < kRecWarps; ++w) { below += S.part[w]; above += S.part_above[w]; ties += S.part_ties[w]; }
      __syncwarp();
      if (lane == 0) S.above = S.ties = 0;
      ++live;
      if constexpr (CS == 1) {
        if (lane == 0) {
          S.job[job & 1] = {r, above, ties, below, m, Tr, bound, false};
        }
        // ties behind the others
        const int n = ties <= kTies ? ties : 0;
        unsigned long long* list = S.list[job & 1];
        if (above < kAbove)
          for (int t0 = 0; t0 < n; t0 += 32) {
            const unsigned long long v = t0 + lane < n ? list[kAbove + t0 + lane] : 0;
            __syncwarp();
            if (t0 + lane < n) list[above + t0 + lane] = v;
            __syncwarp();
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.listed[job & 1]);
      } else {
        // the leader's list is free again
        if (rank == leader && job >= 1) bounded_wait(&S.ranked[(job - 1) & 1], ((job - 1) >> 1) & 1, failed);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&S.counts_in[b], 16 * CS);
        __syncwarp();
        if (lane < CS)
          send16(&S.counts[b][rank], &S.counts_in[b], lane, (uint32_t)above, (uint32_t)ties, __float_as_uint(below), 0u);
        bounded_wait(&S.counts_in[b], turn, failed);
        __syncwarp();
        int total = 0, all_ties = 0, at = 0, tie_at = 0;
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < CS; ++q) {
          const uint4 v = S.counts[b][q];
          if (q == rank) { at = total; tie_at = all_ties; }
          total += (int)v.x;
          all_ties += (int)v.y;
          sum += __uint_as_float(v.z);
        }
        const bool send = total <= kAbove, send_ties = send && all_ties <= kTies;
        const int mine = send ? above : 0, my_ties = send_ties ? ties : 0;
        uint64_t* bar = &S.listed[job & 1];
        if (rank == leader) {
          if (lane == 0) {
            S.job[job & 1] = {r, total, all_ties, sum, m, Tr, bound, false};
            mbar_arrive_expect_tx(bar, 8u * (uint32_t)((send ? total : 0) + (send_ties ? all_ties : 0)));
          }
          __syncwarp();
        }
        const unsigned long long* from = S.list[0];
        const uint32_t to = map_rank(smem_u32(S.list[1]), leader), done = map_rank(smem_u32(bar), leader);
        for (int k = lane; k < mine; k += 32) send8(to + 8 * (at + k), done, from[k]);
        for (int k = lane; k < my_ties; k += 32) send8(to + 8 * (total + tie_at + k), done, from[kAbove + k]);
        __syncwarp();
      }
    }
    // no more rows
    int mine = 0;                            // jobs of this CTA's ranker
    if (CS == 1) mine = live;
    else mine = live / CS + (rank < live % CS);
    if (mine >= 2) bounded_wait(&S.ranked[mine & 1], ((mine - 2) >> 1) & 1, failed);
    __syncwarp();
    if (lane == 0) {
      S.job[mine & 1].row = -1;
      mbar_arrive(&S.listed[mine & 1]);
    }
  } else {                                   // consumers
    RecRing at;
    int i = 0;
    for (int r = first; r < P.n; r += step, ++i) {
      const int b = i & 1;
      const uint32_t turn = (i >> 1) & 1;
      const unsigned char* row = P.logits + (size_t)r * V * ES;
      const RowSpan sp = row_span<DT>(row, V);
      const RowShare sh = row_share<CS>(sp, rank);
      const int ends = sh.ends ? sp.head + (V - sp.tail0) : 0;
      const int end_e = tid < sp.head ? tid : sp.tail0 + (tid - sp.head);
      const float end_x = tid < ends ? row_logit<DT>(row, end_e) : -INFINITY;
      const RecRing row_at = at;
      // pass A
      Maxima<DT> mx;
      for (int j = sh.lo; j < sh.hi; j += kRecStageVecs) {
        bounded_wait(&S.full[at.stage], at.phase, failed);
        const uint4* vec = reinterpret_cast<const uint4*>(s_ring + (size_t)at.stage * kRecStage) + tid;
        const int left = sh.hi - j - tid;
        if (left > (kRecPer - 1) * kRecConsumers) {
          uint4 w[kRecPer];
#pragma unroll
          for (int u = 0; u < kRecPer; ++u) w[u] = vec[u * kRecConsumers];
#pragma unroll
          for (int u = 0; u < kRecPer; ++u) mx.add(u, w[u]);
        } else {
#pragma unroll
          for (int u = 0; u < kRecPer; ++u)
            if (u * kRecConsumers < left) mx.add(u, vec[u * kRecConsumers]);
        }
        if (!keep) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.empty[at.stage]);
        }
        at.next(stages);
      }
      if (few) {
        S.maxima[tid] = max_nan(max_nan(max_nan(mx.get(0), mx.get(1)), max_nan(mx.get(2), mx.get(3))), end_x);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) S.maxima[tid + q * kRecConsumers] = q == 0 ? max_nan(mx.get(q), end_x) : mx.get(q);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.maxed[b]);

      // pass B
      bounded_wait(&S.bounded[b], turn, failed);
      const bool error = S.error != 0;
      const float c = S.c, ref = ref_of(S.m, c), least = S.least;
      unsigned long long* list = S.list[S.into];
      const float2 C2 = make_float2(c, c), R2 = make_float2(-ref, -ref);
      float sum = 0.f;
      // One logit of each lane with `has`, by the whole warp: listed while there is room,
      // and counted.  A row of one value does not queue at the counter.
      int above = 0, ties = 0;
      auto take = [&](bool has, int e, float x) {
        const bool tie = !(x > least);
        const unsigned up = __ballot_sync(0xffffffffu, has && !tie), eq = __ballot_sync(0xffffffffu, has && tie);
        if (up != 0) {
          int slot = lane == 0 ? atomicAdd(&S.above, __popc(up)) : 0;
          slot = __shfl_sync(0xffffffffu, slot, 0) + __popc(up & ((1u << lane) - 1));
          if (has && !tie && slot < kAbove) list[slot] = candidate(x, e);
          above += __popc(up);
        }
        if (eq != 0) {
          int slot = kTies;
          if (lane == 0 && *(volatile int*)&S.ties < kTies) slot = atomicAdd(&S.ties, __popc(eq));
          slot = __shfl_sync(0xffffffffu, slot, 0) + __popc(eq & ((1u << lane) - 1));
          if (has && tie && slot < kTies) list[kAbove + slot] = candidate(x, e);
          ties += __popc(eq);
        }
      };
      // the candidates among a vector of each lane (j: its place in the row) are taken
      // and become -inf, so that the sums are straight code
      auto pick = [&](uint4& v, int j) {
        if (!__any_sync(0xffffffffu, vec_max<DT>(v) >= least)) return;
        uint4 w[1] = {v};
        uint32_t mark = mark_from<DT>(w, least);
        drop_marked<DT>(w, mark);
        const uint4 old = v;
        v = w[0];
        while (__any_sync(0xffffffffu, mark != 0)) {
          const int k = mark ? __ffs((int)mark) - 1 : 0;
          const uint32_t word = k < PER / 2 ? (k < PER / 4 ? old.x : old.y) : (k < PER * 3 / 4 ? old.z : old.w);
          const float x = DT == SPEC_BF16 ? (k & 1 ? bf16_hi(word) : bf16_lo(word)) : __uint_as_float(word);
          take(mark != 0, sp.head + j * PER + k, x);
          mark &= mark - 1;
        }
      };
      RecRing from = keep ? row_at : at;
      for (int j = sh.lo; j < sh.hi; j += kRecStageVecs) {
        if (!keep) bounded_wait(&S.full[from.stage], from.phase, failed);
        const uint4* vec = reinterpret_cast<const uint4*>(s_ring + (size_t)from.stage * kRecStage) + tid;
        const int left = error ? -32 : sh.hi - j - tid;
        if (left > (kRecPer - 1) * kRecConsumers + 31 - lane) {     // for all lanes of the warp
          uint4 w[kRecPer];
#pragma unroll
          for (int u = 0; u < kRecPer; ++u) w[u] = vec[u * kRecConsumers];
          if (__any_sync(0xffffffffu, vecs_max<DT>(w) >= least)) {
#pragma unroll
            for (int u = 0; u < kRecPer; ++u) pick(w[u], j + tid + u * kRecConsumers);
          }
          float2 t[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int u = 0; u < kRecPer; ++u)
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
              const float2 a = __ffma2_rn(vec_pair<DT>(w[u], k), C2, R2);
              t[k & 1] = __fadd2_rn(t[k & 1], make_float2(ex2(a.x), ex2(a.y)));
            }
          t[0] = __fadd2_rn(t[0], t[1]);
          sum += t[0].x + t[0].y;
        } else {
#pragma unroll 1
          for (int u = 0; u < kRecPer && u * kRecConsumers < left + lane; ++u) {
            const bool has = u * kRecConsumers < left;
            uint4 w = has ? vec[u * kRecConsumers] : minus_infinity<DT>();
            pick(w, j + tid + u * kRecConsumers);
            float2 t = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
              const float2 a = __ffma2_rn(vec_pair<DT>(w, k), C2, R2);
              t = __fadd2_rn(t, make_float2(ex2(a.x), ex2(a.y)));
            }
            sum += t.x + t.y;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.empty[from.stage]);
        from.next(stages);
      }
      if (!keep) at = from;
      if (!error && warp == 0) {             // at most 14 single elements
        const bool has = lane < ends && end_x >= least;
        take(has, end_e, end_x);
        if (lane < ends && !has) sum += ex2(fmaf(end_x, c, -ref));
      }
      sum = warp_sum(sum);
      if (lane == 0) { S.part[warp] = sum; S.part_above[warp] = above; S.part_ties[warp] = ties; }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.found[b]);
    }
  }
  __syncwarp();
  if (__any_sync(0xffffffffu, *failed)) drain_after_failure();
  __syncwarp();
  if constexpr (CS > 1) cluster_sync();      // no CTA leaves while another sends to it
}

struct RecShape {
  int cs, stages;
  bool keep;
};
// Dynamic shared memory: two CTAs per SM (228 KB, 1 KB of it reserved for each).
constexpr int kRecSmem = kRecMaxStages * kRecStage + (int)sizeof(RecShared);
static_assert(kRecSmem <= 112 * 1024, "two CTAs per SM");

// One CTA per row where the rows fill the GPU, and pass B reads the row again from
// L2 (304 rows in flight are 92 MB); more CTAs where the rows are few, and their
// shares stay in the rings.  (512 x 151936 bf16: 65 us with one CTA per row, 70, 75
// and 112 with two, four and eight, whose exchanges between the passes cost more
// than the second read.)
RecShape shape_of(int n, int V, int es, int nsm) {
  RecShape s{};
  s.cs = row_cluster(n, V, es, nsm);
  const long long vecs = ((long long)V * es / 16 + s.cs - 1) / s.cs, share = (vecs + kRecStageVecs - 1) / kRecStageVecs;
  s.keep = share <= kRecMaxStages;
  s.stages = s.keep && share < kRecMaxStages ? (int)share + 1 : kRecMaxStages;
  return s;
}

int g_clusters[kMaxDevices][2][4];           // resident at once, by device, dtype and log2 CS

template <int DT, int CS>
cudaError_t launch_as(const RecordParams& P, const RecShape& shape, int dev, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int most = g_clusters[dev][DT == SPEC_BF16][log2_of(CS)];
  cfg.gridDim = dim3((P.n < most ? P.n : most) * CS);
  cfg.blockDim = dim3(kRecThreads);
  cfg.dynamicSmemBytes = (size_t)shape.stages * kRecStage + sizeof(RecShared);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {CS, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, record_kernel<DT, CS>, P, shape.stages, shape.keep);
}

template <int DT>
cudaError_t launch_of(const RecordParams& P, int dev, int nsm, cudaStream_t s) {
  const RecShape shape = shape_of(P.n, P.V, RowType<DT>::ES, nsm);
  if (shape.cs == 8) return launch_as<DT, 8>(P, shape, dev, s);
  if (shape.cs == 4) return launch_as<DT, 4>(P, shape, dev, s);
  if (shape.cs == 2) return launch_as<DT, 2>(P, shape, dev, s);
  return launch_as<DT, 1>(P, shape, dev, s);
}

template <int DT, int CS>
cudaError_t configure_one(int dev) {
  const cudaError_t e = cudaFuncSetAttribute(record_kernel<DT, CS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRecSmem);
  if (e != cudaSuccess) return e;
  return resident_clusters(record_kernel<DT, CS>, CS, kRecThreads, kRecSmem, &g_clusters[dev][DT == SPEC_BF16][log2_of(CS)]);
}
template <int DT>
cudaError_t configure_as(int dev) {
  cudaError_t e = configure_one<DT, 1>(dev);
  if (e == cudaSuccess) e = configure_one<DT, 2>(dev);
  if (e == cudaSuccess) e = configure_one<DT, 4>(dev);
  if (e == cudaSuccess) e = configure_one<DT, 8>(dev);
  return e;
}

}  // namespace

cudaError_t launch_record(const RecordParams& P, int dev, int nsm, cudaStream_t s) {
  return P.dtype == SPEC_BF16 ? launch_of<SPEC_BF16>(P, dev, nsm, s) : launch_of<SPEC_F32>(P, dev, nsm, s);
}

cudaError_t configure_record(int dev) {
  const cudaError_t e = configure_as<SPEC_BF16>(dev);
  return e == cudaSuccess ? configure_as<SPEC_F32>(dev) : e;
}

}  // namespace sv
