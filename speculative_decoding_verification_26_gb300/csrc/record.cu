// record.cu -- the record of a teacher row: its K largest logits and the log
// mass of the rest.
//
// Per row x[V] at temperature T: the K largest logits, by value, ties to the
// lowest index, and tail = ln sum_{v not among them} e^{x_v / T}.  The tail is
// summed over the rest itself: as a difference of two full sums it would cancel
// where the K logits carry nearly all of the mass.
//
// What bounds it: the row is read once.  A row's logits are summed before it is
// known which of them are recorded: a consumer thread keeps the maximum and the sum
// of weights of each group of its logits (32 per stage, some stages to a group).
// When the row has been read, a lower bound of its K-th largest logit follows from
// the maxima; a group whose maximum is below it is in the tail as a whole, and the
// logits of the few others (little more than K groups) are read again.
// Persistent CTAs, two per SM, of four roles; where rows are few, a cluster of CS
// CTAs shares one:
//   producer  streams the shares into a ring of stages (bulk copies);
//   consumers the groups' maxima and sums, row after row;
//   picker    (one warp) the bound: the K-th largest of a share's 256 thread maxima
//             is one (1024 part maxima where a share has to yield more than 64),
//             since K parts each hold a logit that large, and so is the least, over
//             the shares, of each one's ceil(K / CS)-th largest; the greater of the
//             two leaves little more than K candidates;
//   finishers (four warps) sum the groups below the bound, take the others apart,
//             gather the cluster's candidates in the row's leader (CTAs take turns),
//             and give each candidate its place, the number of candidates before
//             it; candidates past K join the tail.
// Keys hold value and index, so no two are equal and the order in which candidates
// were found does not matter.  Where more than kTies logits equal the bound (a mask
// of finite values), the first of them are found by a scan in index order; where
// more than kAbove lie above it, the K-th largest is searched by counting, by one
// warp: rows whose large logits sit in few threads' vectors (0.4 s at 2^24 logits), and
// records of nearly 256 from rows of one stage, whose 256 thread maxima bound little
// (K = 256: 512 x 8192 bf16 326 us, 37 us at 16384; K = 200: 39 us).
// Measured at 512 x 151936 bf16, K = 64: reading each row twice (maxima, then
// weights with the candidates taken on the way) took 64 us with one CTA per row and
// 70 to 112 with clusters that keep their shares; taking candidates in the stream
// cost a third of that.
#include <cuda_runtime.h>

#include <cstdint>

#include "rows.cuh"

namespace sv {
namespace {

constexpr int kRecWarps = 8;                               // consumers
constexpr int kRecConsumers = kRecWarps * 32;
constexpr int kFinWarps = 4, kFinThreads = kFinWarps * 32;
constexpr int kRecThreads = kRecConsumers + 64 + kFinThreads;        // picker, finishers, producer
constexpr int kRecPer = 4;                                 // vectors of a stage per thread
constexpr int kRecStageVecs = kRecPer * kRecConsumers;
constexpr int kRecStage = 16 * kRecStageVecs;
constexpr int kRecStages = 3;
constexpr int kMaxGroups = 10;                             // of a thread and row
constexpr int kMaxima = 4 * kRecConsumers;
constexpr int kAbove = 768, kTies = 256, kList = kAbove + kTies;
static_assert(kMaxGroups * kRecConsumers * 2 <= kList * 8, "a list holds the numbers of all groups");
static_assert(kMaxGroups * kRecConsumers <= 32 * kFinThreads, "a finisher's marks");

// order of a float as an unsigned integer, -0 and +0 alike
__device__ __forceinline__ uint32_t order_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // order_key(-inf)
// order_key of the type's lowest value: a bound that takes every finite logit
template <int DT>
constexpr uint32_t kKeyLowest = DT == SPEC_BF16 ? 0x0080FFFFu : 0x00800000u;
// a candidate: larger comes first
__device__ __forceinline__ unsigned long long candidate(float x, int e) {
  return (unsigned long long)order_key(x) << 32 | (uint32_t)~e;
}

struct RecRow {                              // what the picker found of a row
  float m, T;
  uint32_t bound;
  int st;
};
struct RecShared {
  uint64_t full[kRecStages], empty[kRecStages];
  // by row parity: the groups are in; the bound is in; the groups have been read;
  // every CTA's bound, and candidate count, is in; the leader's candidates are in
  uint64_t summed[2], bounded[2], freed[2], bounds_in[2], counts_in[2], listed[2];
  uint4 bounds[2][8], counts[2][8];          // of each CTA of the cluster
  unsigned long long list[2][kList + 2];     // of this share (above from 0, ties from kAbove), and a leader's
  float group_max[2][kMaxGroups * kRecConsumers], group_sum[2][kMaxGroups * kRecConsumers];
  float maxima[kMaxima];
  RecRow row[2];
  float part[kFinWarps];
  int part_above[kFinWarps], part_ties[kFinWarps];
  int above, ties;                           // this share's candidates listed
  struct {
    int above, ties;
    float below;
    uint32_t bound;
  } counted;                                 // by recount
  int stop[3];                               // the finishers' decision after each wait
  int failed;
};

// A bound of a share's want-th largest logit from N of its maxima per lane: one of
// them that `want` or more reach, at most an eighth more where there is one.  Keys are
// told apart by their upper 16 bits for bf16 logits and 20 for fp32; the bound is the
// least of those found, whole: a value that many logits share (a mask) is met exactly.
// -inf is never recorded: a bound is at least kKeyLowest.
template <int DT, int N>
__device__ __forceinline__ uint32_t bound_of(const uint32_t (&key)[N], int want) {
  constexpr int shift = DT == SPEC_BF16 ? 16 : 12;
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
    if ((int)__reduce_add_sync(0xffffffffu, (unsigned)n) < want) return kKeyLowest<DT>;
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
  uint32_t exact = 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (key[j] >> shift >= lo) exact = min(exact, key[j]);
  return __reduce_min_sync(0xffffffffu, exact);
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
  whole = share = kKeyLowest<DT>;
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

__device__ __forceinline__ void fin_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kFinThreads) : "memory"); }

// The K-th largest key of a row by counting, for a row with more candidates above
// the bound than are listed; one warp.  Lists what lies above it (less than K).
template <int DT>
__device__ __noinline__ void recount(const RecordParams& P, RecShared& S, int r, const RecRow& info,
                                     unsigned long long* list) {
  const int K = P.K, V = P.V, lane = threadIdx.x & 31;
  const unsigned char* row = P.logits + (size_t)r * V * RowType<DT>::ES;
  const float c = scale_split(info.T).c, m = info.m;
  auto count = [&](auto&& pred) {
    int n = 0;
    warp_row<DT>(row, V, [&](int, float x) { n += pred(order_key(x)); });
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
  };
  uint32_t lo = info.bound + 1, hi = order_key(info.m);
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    if (count([&](uint32_t k) { return k >= mid; }) >= K) lo = mid;
    else hi = mid - 1;
  }
  const int ties = count([&](uint32_t k) { return k == lo; });
  // a lane sums V / 32 weights one after another: what each addition rounds off is carried along
  float s = 0.f, off = 0.f;
  int at = 0;
  for (int e0 = 0; e0 < V; e0 += 32) {
    const int e = e0 + lane;
    const float x = e < V ? row_logit<DT>(row, e) : -INFINITY;
    const uint32_t k = order_key(x);
    const bool above = e < V && k > lo;
    const unsigned vote = __ballot_sync(0xffffffffu, above);
    const int to = at + __popc(vote & ((1u << lane) - 1));
    if (above && to < kAbove) list[to] = candidate(x, e);
    at += __popc(vote);
    if (e < V && k < lo) {
      const float w = ex2((x - m) * c) - off, to_s = s + w;
      off = (to_s - s) - w;
      s = to_s;
    }
  }
  s = warp_sum(s);
  __syncwarp();
  if (lane == 0) { S.counted.above = at; S.counted.ties = ties; S.counted.below = s; S.counted.bound = lo; }
  __syncwarp();
}

// A run of keys in order, largest first, by one warp: a key's place is the number of
// keys before it.  E of them a lane at a time.
template <int E>
__device__ __forceinline__ void order_run(const unsigned long long* from, int len, unsigned long long* to) {
  const int lane = threadIdx.x & 31;
  const ulonglong2* pair = reinterpret_cast<const ulonglong2*>(from);
  for (int k0 = lane; k0 - lane < len; k0 += 32 * E) {
    unsigned long long mine[E];
    int place[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      mine[j] = k0 + 32 * j < len ? from[k0 + 32 * j] : ~0ull;
      place[j] = 0;
    }
#pragma unroll 2
    for (int p = 0; p < (len + 1) / 2; ++p) {
      const ulonglong2 two = pair[p];
#pragma unroll
      for (int j = 0; j < E; ++j) place[j] += (two.x > mine[j]) + (two.y > mine[j]);
    }
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (k0 + 32 * j < len) to[place[j]] = mine[j];
  }
}

// The record from the candidates: `above` of them above the bound, `ties` equal to
// it and listed behind the others where there are at most kTies.
template <int DT>
__device__ __forceinline__ void rank_row(const RecordParams& P, RecShared& S, int r, const RecRow& info, int above,
                                         int ties, float below, unsigned long long* list,
                                         unsigned long long* spare) {
  const int K = P.K, V = P.V, t = (int)threadIdx.x - kRecConsumers - 32, lane = t & 31, warp = t >> 5;
  uint32_t bound = info.bound;
  bool listed_ties = ties <= kTies;
  if (above > kAbove) {                      // the same in every finisher
    if (warp == 0) recount<DT>(P, S, r, info, list);
    fin_sync();
    above = S.counted.above;
    ties = S.counted.ties;
    below = S.counted.below;
    bound = S.counted.bound;
    listed_ties = false;
  }
  const unsigned char* row = P.logits + (size_t)r * V * RowType<DT>::ES;
  float* top = P.top_logits + (size_t)r * K;
  int32_t* ti = P.top_index + (size_t)r * K;
  const float c = scale_split(info.T).c;
  auto weight = [&](float x) { return ex2((x - info.m) * c); };
  const int n = above + (listed_ties ? ties : 0);
  auto record = [&](int place, unsigned long long key) {
    const float x = key_value((uint32_t)(key >> 32));
    const int e = (int)~(uint32_t)key;
    top[place] = x == 0.f ? row_logit<DT>(row, e) : x;       // the key has lost a zero's sign
    ti[place] = e;
  };
  // A candidate's place: each warp orders a quarter by counting, then each candidate
  // looks up how many of the other quarters come before it.  (305 candidates: 7000 to 9000
  // clocks with the outputs; sorting all of them in one go took 14000 to 17000.)
  const int run = ((n + kFinWarps - 1) / kFinWarps + 1) & ~1;
  if (t == 0) list[n] = 0;                   // the keys are read by twos
  fin_sync();
  auto length = [&](int w) { return n - w * run < 0 ? 0 : n - w * run < run ? n - w * run : run; };
  if (run <= 32) order_run<1>(list + warp * run, length(warp), spare + warp * run);
  else if (run <= 64) order_run<2>(list + warp * run, length(warp), spare + warp * run);
  else order_run<3>(list + warp * run, length(warp), spare + warp * run);
  fin_sync();                                // the list is read: it takes the weights past K, by place
  float* past = reinterpret_cast<float*>(list);
  const int first_step = 1 << (31 - __clz(run | 1));       // no run: only ties, none of them listed
  const unsigned long long* other[kFinWarps - 1];
  int others[kFinWarps - 1];
#pragma unroll
  for (int q = 0; q < kFinWarps - 1; ++q) {
    const int w = (warp + 1 + q) % kFinWarps;
    other[q] = spare + w * run - 1;
    others[q] = length(w);
  }
  for (int i = lane; i < length(warp); i += 32) {
    const unsigned long long mine = spare[warp * run + i];
    int at[kFinWarps - 1] = {};
    for (int step = first_step; step > 0; step >>= 1)
#pragma unroll
      for (int q = 0; q < kFinWarps - 1; ++q) {
        const int to = at[q] + step;
        if (to <= others[q] && other[q][to] > mine) at[q] = to;
      }
    int place = i;
#pragma unroll
    for (int q = 0; q < kFinWarps - 1; ++q) place += at[q];
    if (place < K) record(place, mine);
    else past[place - K] = weight(key_value((uint32_t)(mine >> 32)));
  }
  float extra = 0.f;                         // weights past K, in the order of their places
  if (n > K) {
    fin_sync();
    for (int i = t; i < n - K; i += kFinThreads) extra += past[i];
    extra = warp_sum(extra);
    if (lane == 0) S.part[warp] = extra;
    fin_sync();
    extra = 0.f;
    for (int w = 0; w < kFinWarps; ++w) extra += S.part[w];
  }
  if (listed_ties) {
    for (int i = n + t; i < K; i += kFinThreads) { top[i] = -INFINITY; ti[i] = -1; }     // fewer finite logits than K
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
        const bool tie = order_key(x[q]) == bound;
        const unsigned vote = __ballot_sync(0xffffffffu, tie);
        const int to = at + __popc(vote & ((1u << lane) - 1));
        if (tie && to < K) { top[to] = x[q]; ti[to] = e0 + 32 * q + lane; }
        at += __popc(vote);
      }
    }
    extra += (float)(ties - (K > above ? K - above : 0)) * weight(key_value(bound));
  }
  if (t == 0) {
    // the weights are beside the row's maximum
    const float tail = below + extra;
    P.tail_lse[r] = tail > 0.f ? __fdiv_rn(info.m, info.T) + kLn2 * log2f(tail) : -INFINITY;
    if (P.status) P.status[r] = SPEC_ST_OK;
  }
}

template <int DT, int CS>
__global__ void __launch_bounds__(kRecThreads, 2) record_kernel(const __grid_constant__ RecordParams P,
                                                                const int group) {
  constexpr int PER = RowType<DT>::PER, ES = RowType<DT>::ES;
  extern __shared__ __align__(128) unsigned char s_ring[];
  RecShared& S = *reinterpret_cast<RecShared*>(s_ring + (size_t)kRecStages * kRecStage);
  const int V = P.V, K = P.K, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CS == 1 ? 0 : (int)cluster_rank();
  const int first = blockIdx.x / CS, step = gridDim.x / CS;
  const Waits waits{&S.failed, P.wait_limit};

  if (tid == 0) {
    S.failed = 0;
    for (int i = 0; i < kRecStages; ++i) { mbar_init(&S.full[i], 1); mbar_init(&S.empty[i], kRecWarps); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.summed[i], kRecWarps);
      mbar_init(&S.bounded[i], 1);
      mbar_init(&S.freed[i], 1);
      mbar_init(&S.bounds_in[i], 1);
      mbar_init(&S.counts_in[i], 1);
      mbar_init(&S.listed[i], 1);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if constexpr (CS > 1) cluster_sync();

  const int part = (K + CS - 1) / CS;        // a share's part of the record
  const bool few = part <= 64;               // one maximum per thread is enough
  int left = P.n;                            // a finisher's first row after a failed wait

  if (warp == kRecWarps + 1 + kFinWarps) {   // producer
    if (lane == 0) {
      RingAt at;
      bool ok = true;
      for (int r = first; r < P.n && ok; r += step) {
        const unsigned char* row = P.logits + (size_t)r * V * ES;
        const RowSpan sp = row_span<DT>(row, V);
        const RowShare sh = row_share<CS>(sp, rank);
        const unsigned char* body = row + (size_t)sp.head * ES;
        for (int j = sh.lo; j < sh.hi; j += kRecStageVecs) {
          const uint32_t bytes = 16u * (uint32_t)(sh.hi - j < kRecStageVecs ? sh.hi - j : kRecStageVecs);
          ok = bounded_wait(&S.empty[at.stage], at.phase ^ 1, waits) && !*waits.failed;      // after it, stages are given up unread
          if (!ok) break;
          mbar_arrive_expect_tx(&S.full[at.stage], bytes);
          bulk_load(s_ring + (size_t)at.stage * kRecStage, body + 16ll * j, bytes, &S.full[at.stage]);
          at.next(kRecStages);
        }
      }
    }
  } else if (warp > kRecWarps) {             // finishers
    const int t = tid - kRecConsumers - 32, fw = t >> 5;
    int i = 0, live = 0, r = first;          // rows, and rows not refused (the same in every CTA of the cluster)
    for (; r < P.n; r += step, ++i) {
      const int b = i & 1;
      const uint32_t turn = (i >> 1) & 1;
      bounded_wait(&S.bounded[b], turn, waits);
      if (t == 0) {
        S.above = S.ties = 0;
        S.stop[0] = *waits.failed;
      }
      fin_sync();
      if (S.stop[0]) break;                     // the same for all: nothing of this row is known
      const RecRow info = S.row[b];
      const unsigned char* row = P.logits + (size_t)r * V * ES;
      const RowSpan sp = row_span<DT>(row, V);
      const RowShare sh = row_share<CS>(sp, rank);
      if (info.st != 0) {
        if (rank == 0) {
          const float nan = __int_as_float(0x7fc00000);
          for (int k = t; k < K; k += kFinThreads) { P.top_logits[(size_t)r * K + k] = nan; P.top_index[(size_t)r * K + k] = -1; }
          if (t == 0) {
            P.tail_lse[r] = nan;
            if (P.status) P.status[r] = info.st;
          }
        }
        fin_sync();                          // S.row[b] is read by all: it may take the row after next
        if (t == 0) mbar_arrive(&S.freed[b]);
        continue;
      }
      const float c = scale_split(info.T).c, top = info.m, least = key_value(info.bound);
      // the groups: whole into the tail, or marked
      float sum = 0.f;
      uint32_t marked = 0;
      const int stages = (sh.hi - sh.lo + kRecStageVecs - 1) / kRecStageVecs;
      const int groups = (stages + group - 1) / group * kRecConsumers;
#pragma unroll 4
      for (int g = t, bit = 0; g < groups; g += kFinThreads, ++bit) {
        const float gm = S.group_max[b][g], gs = S.group_sum[b][g];
        if (gm >= least) marked |= 1u << bit;
        else sum += gs * ex2((gm - top) * c);  // 0 where the group holds -inf alone
      }
      fin_sync();
      if (t == 0) mbar_arrive(&S.freed[b]);
      // The marked groups, logit by logit.
      unsigned long long* list = S.list[0];
      int above = 0, ties = 0;
      auto take = [&](int e, float x) {      // counted, and listed while there is room
        const bool tie = !(x > least);
        above += !tie;
        ties += tie;
        int* counter = tie ? &S.ties : &S.above;
        const int room = tie ? kTies : kAbove;
        if (*(volatile int*)counter >= room) return;         // a row of one value does not queue here
        const int slot = atomicAdd(counter, 1);
        if (slot < room) list[(tie ? kAbove : 0) + slot] = candidate(x, e);
      };
      // their numbers in order (in the leader's list, which fills up after the counts are
      // exchanged), so that every thread has its vectors, four at a time, in a fixed order
      uint16_t* numbers = reinterpret_cast<uint16_t*>(S.list[1]);
      int before = __popc(marked);
#pragma unroll
      for (int off = 1; off < 32; off *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += v;
      }
      if (lane == 31) S.part_ties[fw] = before;
      fin_sync();
      int nm = 0;
      before -= __popc(marked);
      for (int w = 0; w < kFinWarps; ++w) {
        if (w < fw) before += S.part_ties[w];
        nm += S.part_ties[w];
      }
      for (; marked != 0; marked &= marked - 1) numbers[before++] = (uint16_t)(t + (__ffs((int)marked) - 1) * kFinThreads);
      fin_sync();
      const uint4* vec = reinterpret_cast<const uint4*>(row + (size_t)sp.head * ES);
      const int per = kRecPer * group;       // vectors of a group: kRecConsumers apart
      auto place_of = [&](unsigned v) {      // of the v-th vector of the marked groups: its place in the row, or past it
        const unsigned q = v / (unsigned)per;
        if ((int)q >= nm) return sh.hi;
        const int g = numbers[q];
        return sh.lo + g / kRecConsumers * group * kRecStageVecs + g % kRecConsumers + (int)(v - q * per) * kRecConsumers;
      };
#pragma unroll 1
      for (int v0 = t; v0 < nm * per; v0 += 4 * kFinThreads) {               // below 2^26: V < 2^28
        uint4 w[4];
        int at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          at[u] = place_of((unsigned)(v0 + u * kFinThreads));
          w[u] = at[u] < sh.hi ? vec[at[u]] : minus_infinity<DT>();
        }
#pragma unroll 1
        for (int u = 0; u < 4 && v0 + u * kFinThreads < nm * per; ++u) {
          const uint4 old = u == 0 ? w[0] : u == 1 ? w[1] : u == 2 ? w[2] : w[3];
          const int j = u == 0 ? at[0] : u == 1 ? at[1] : u == 2 ? at[2] : at[3];
          uint4 one[1] = {old};
          uint32_t mark = 0;
          if (vec_max<DT>(old) >= least) {
            mark = mark_from<DT>(one, least);
            drop_marked<DT>(one, mark);
          }
#pragma unroll
          for (int k = 0; k < PER / 2; ++k) {
            const float2 x = vec_pair<DT>(one[0], k);
            sum += ex2((x.x - top) * c) + ex2((x.y - top) * c);
          }
          for (; mark != 0; mark &= mark - 1) {
            const int k = __ffs((int)mark) - 1;
            const uint32_t word = k < PER / 2 ? (k < PER / 4 ? old.x : old.y) : (k < PER * 3 / 4 ? old.z : old.w);
            take(sp.head + j * PER + k,
                 DT == SPEC_BF16 ? (k & 1 ? bf16_hi(word) : bf16_lo(word)) : __uint_as_float(word));
          }
        }
      }
      const int ends = sh.ends ? sp.head + (V - sp.tail0) : 0;               // single elements
      if (t < ends) {
        const int e = t < sp.head ? t : sp.tail0 + (t - sp.head);
        const float x = row_logit<DT>(row, e);
        if (x >= least) take(e, x);
        else sum += ex2((x - top) * c);
      }
      __syncwarp();
      sum = warp_sum(sum);
      above = (int)__reduce_add_sync(0xffffffffu, (unsigned)above);
      ties = (int)__reduce_add_sync(0xffffffffu, (unsigned)ties);
      if (lane == 0) { S.part[fw] = sum; S.part_above[fw] = above; S.part_ties[fw] = ties; }
      fin_sync();
      above = ties = 0;
      sum = 0.f;
      for (int w = 0; w < kFinWarps; ++w) { sum += S.part[w]; above += S.part_above[w]; ties += S.part_ties[w]; }
      fin_sync();                            // S.part is used again below
      if constexpr (CS == 1) {
        if (above < kAbove && ties <= kTies) {               // ties behind the others
          unsigned long long v[kTies / kFinThreads];
#pragma unroll
          for (int q = 0; q < kTies / kFinThreads; ++q) v[q] = list[kAbove + t + q * kFinThreads];
          fin_sync();
#pragma unroll
          for (int q = 0; q < kTies / kFinThreads; ++q)
            if (t + q * kFinThreads < ties) list[above + t + q * kFinThreads] = v[q];
          fin_sync();
        }
        rank_row<DT>(P, S, r, info, above, ties, sum, list, S.list[1]);
      } else {
        const int lb = live & 1, leader = live % CS;
        const uint32_t lturn = (live >> 1) & 1;
        if (t == 0) mbar_arrive_expect_tx(&S.counts_in[lb], 16 * CS);
        fin_sync();
        if (t < CS) send16(&S.counts[lb][rank], &S.counts_in[lb], t, (uint32_t)above, (uint32_t)ties, __float_as_uint(sum), 0u);
        bounded_wait(&S.counts_in[lb], lturn, waits);
        if (t == 0) S.stop[1] = *waits.failed;
        fin_sync();
        if (S.stop[1]) break;
        int total = 0, all_ties = 0, at = 0, tie_at = 0;
        float below = 0.f;
#pragma unroll
        for (int q = 0; q < CS; ++q) {
          const uint4 v = S.counts[lb][q];
          if (q == rank) { at = total; tie_at = all_ties; }
          total += (int)v.x;
          all_ties += (int)v.y;
          below += __uint_as_float(v.z);
        }
        const bool send = total <= kAbove, send_ties = send && all_ties <= kTies;
        // a leader's candidates, on a barrier of their own turn: its leads are CS rows apart
        const int lead = live / CS;
        uint64_t* bar = &S.listed[lead & 1];
        if (rank == leader && t == 0)
          mbar_arrive_expect_tx(bar, 8u * (uint32_t)((send ? total : 0) + (send_ties ? all_ties : 0)));
        const uint32_t to = map_rank(smem_u32(S.list[1]), leader), done = map_rank(smem_u32(bar), leader);
        if (send)
          for (int k = t; k < above; k += kFinThreads) send8(to + 8 * (at + k), done, list[k]);
        if (send_ties)
          for (int k = t; k < ties; k += kFinThreads) send8(to + 8 * (total + tie_at + k), done, list[kAbove + k]);
        if (rank == leader) {
          bounded_wait(bar, (lead >> 1) & 1, waits);
          if (t == 0) S.stop[2] = *waits.failed;
          fin_sync();
          if (S.stop[2]) break;
          rank_row<DT>(P, S, r, info, total, all_ties, below, S.list[1], S.list[0]);
        }
        ++live;
      }
      fin_sync();                            // the lists are free
    }
    left = r;
  } else if (warp == kRecWarps) {            // picker
    int i = 0;
    float T = first < P.n && P.temperature ? P.temperature[first] : 1.f;
    for (int r = first; r < P.n; r += step, ++i) {
      if (any_failed(waits)) break;
      const int b = i & 1;
      const uint32_t turn = (i >> 1) & 1;
      const float given = T;
      if (P.temperature && r + step < P.n) T = P.temperature[r + step];
      bounded_wait(&S.summed[b], turn, waits);
      __syncwarp();
      uint32_t bound, share;
      float m = few ? bounds_of<DT, kRecConsumers / 32>(S.maxima, K, part, bound, share)
                    : bounds_of<DT, kMaxima / 32>(S.maxima, K, part, bound, share);
      if constexpr (CS > 1) {
        if (lane == 0) mbar_arrive_expect_tx(&S.bounds_in[b], 16 * CS);
        __syncwarp();
        if (lane < CS) send16(&S.bounds[b][rank], &S.bounds_in[b], lane, __float_as_uint(m), bound, share, 0u);
        bounded_wait(&S.bounds_in[b], turn, waits);
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
      int st = 0;
      if (!temperature_ok(given)) st |= SPEC_ST_BAD_TEMPERATURE;
      if (!isfinite(m)) st |= SPEC_ST_NONFINITE;             // NaN, +inf, or nothing finite
      if (lane == 0) {
        S.row[b] = {m, st ? 1.f : given, bound, st};
        mbar_arrive(&S.bounded[b]);
      }
      __syncwarp();
    }
  } else {                                   // consumers
    RingAt at;
    int i = 0;
    float T = first < P.n && P.temperature ? P.temperature[first] : 1.f;      // a row ahead: a load takes 2 us here
    for (int r = first; r < P.n; r += step, ++i) {
      if (any_failed(waits)) break;
      const int b = i & 1;
      const unsigned char* row = P.logits + (size_t)r * V * ES;
      const RowSpan sp = row_span<DT>(row, V);
      const RowShare sh = row_share<CS>(sp, rank);
      const float given = T;
      if (P.temperature && r + step < P.n) T = P.temperature[r + step];
      const int ends = sh.ends ? sp.head + (V - sp.tail0) : 0;
      const float end_x = tid < ends ? row_logit<DT>(row, tid < sp.head ? tid : sp.tail0 + (tid - sp.head)) : -INFINITY;
      const float c = scale_split(temperature_ok(given) ? given : 1.f).c;
      const float2 C2 = make_float2(c, c);
      if (i >= 2) bounded_wait(&S.freed[b], ((i - 2) >> 1) & 1, waits);     // the groups of the row before last
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      float m = -INFINITY, s = 0.f, bad = 0.f;
      int left_of_group = group, g = 0;
      for (int j = sh.lo; j < sh.hi; j += kRecStageVecs) {
        bounded_wait(&S.full[at.stage], at.phase, waits);
        const uint4* vec = reinterpret_cast<const uint4*>(s_ring + (size_t)at.stage * kRecStage) + tid;
        const int left = sh.hi - j - tid;
        uint4 w[kRecPer];
        if (left > (kRecPer - 1) * kRecConsumers) {
#pragma unroll
          for (int u = 0; u < kRecPer; ++u) w[u] = vec[u * kRecConsumers];
        } else {
#pragma unroll
          for (int u = 0; u < kRecPer; ++u) w[u] = u * kRecConsumers < left ? vec[u * kRecConsumers] : minus_infinity<DT>();
        }
        const float top = vecs_max<DT>(w);
        if (top > m) {
          s = m == -INFINITY ? s : s * ex2((m - top) * c);
          m = top;
        }
        const float nm = m == -INFINITY ? 0.f : -m;          // all -inf so far: weights of 0
        const float2 M2 = make_float2(nm, nm);
        float2 t[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int u = 0; u < kRecPer; ++u)
#pragma unroll
          for (int k = 0; k < PER / 2; ++k) {
            const float2 a = __fmul2_rn(__fadd2_rn(vec_pair<DT>(w[u], k), M2), C2);
            t[k & 1] = __fadd2_rn(t[k & 1], make_float2(ex2(a.x), ex2(a.y)));
          }
        t[0] = __fadd2_rn(t[0], t[1]);
        s += t[0].x + t[0].y;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.empty[at.stage]);
        at.next(kRecStages);
        if (--left_of_group == 0 || j + kRecStageVecs >= sh.hi) {
          S.group_max[b][g * kRecConsumers + tid] = m;
          S.group_sum[b][g * kRecConsumers + tid] = s;
          bad += s;                          // NaN once any sum is: a NaN or +inf logit
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if ((g & 3) == q) mx[q] = fmaxf(mx[q], m);
          ++g;
          left_of_group = group;
          m = -INFINITY;
          s = 0.f;
        }
      }
      if (bad != bad) mx[0] = bad;
      mx[0] = max_nan(mx[0], end_x);
      if (i >= 1) bounded_wait(&S.bounded[b ^ 1], ((i - 1) >> 1) & 1, waits);             // the last row's maxima are read
      if (few) {
        S.maxima[tid] = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3]));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) S.maxima[tid + q * kRecConsumers] = mx[q];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.summed[b]);
    }
  }
  __syncwarp();
  const bool failed = any_failed(waits);
  if (failed) drain_after_failure();
  __syncwarp();
  if constexpr (CS > 1) cluster_sync();      // no CTA leaves while another sends to it
  if (!failed) return;
  for (int r = left; r < P.n; r += step) {   // over what another CTA of the cluster wrote
    const float nan = __int_as_float(0x7fc00000);
    const int t = tid - kRecConsumers - 32;
    for (int k = t; k < K; k += kFinThreads) { P.top_logits[(size_t)r * K + k] = nan; P.top_index[(size_t)r * K + k] = -1; }
    if (t == 0) {
      P.tail_lse[r] = nan;
      if (P.status) P.status[r] = SPEC_ST_TIMEOUT;
    }
  }
}

// Dynamic shared memory: two CTAs per SM (228 KB, 1 KB of it reserved for each).
constexpr int kRecSmem = kRecStages * kRecStage + (int)sizeof(RecShared);
static_assert(kRecSmem <= 112 * 1024, "two CTAs per SM");

int g_clusters[kMaxDevices][2][4];           // resident at once, by device, dtype and log2 CS

template <int DT, int CS>
cudaError_t launch_as(const RecordParams& P, int dev, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int most = g_clusters[dev][DT == SPEC_BF16][log2_of(CS)];
  cfg.gridDim = dim3((P.n < most ? P.n : most) * CS);
  cfg.blockDim = dim3(kRecThreads);
  cfg.dynamicSmemBytes = kRecSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {CS, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // stages to a group, so that a thread has at most kMaxGroups of them
  const long long vecs = ((long long)P.V * RowType<DT>::ES / 16 + CS - 1) / CS;
  const long long stages = (vecs + kRecStageVecs - 1) / kRecStageVecs;
  const int group = stages <= kMaxGroups ? 1 : (int)((stages + kMaxGroups - 1) / kMaxGroups);
  return cudaLaunchKernelEx(&cfg, record_kernel<DT, CS>, P, group);
}

// Two CTAs share a row of 256 KB or more even where the rows fill the GPU: the work
// after the stream is shared, and the last round of rows is shorter (K = 64: 512 x
// 151936 bf16 43.4 us, 46.5 with one, 57 with four; 600 x 128256 fp32 65 and 72; K = 256:
// 600 x 128256 fp32 100 and 116; but 2048 x 32000 bf16, rows of 64 KB: 89 us, 52 with
// one).
template <int DT>
cudaError_t launch_of(const RecordParams& P, int dev, int nsm, cudaStream_t s) {
  int cs = row_cluster(P.n, P.V, RowType<DT>::ES, nsm);
  if (cs == 1 && (long long)P.V * RowType<DT>::ES >= 256 * 1024) cs = 2;
  if (cs == 8) return launch_as<DT, 8>(P, dev, s);
  if (cs == 4) return launch_as<DT, 4>(P, dev, s);
  if (cs == 2) return launch_as<DT, 2>(P, dev, s);
  return launch_as<DT, 1>(P, dev, s);
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
