// distill.cu -- the loss of a student's logit rows against a teacher's records,
// with its gradient by the logits.
//
// Row i: the record holds K teacher logits x_k with their tokens and tail =
// ln sum e^{x_v / T} over the teacher's other tokens.  On the K tokens and one
// bucket r for all others,
//   p_k = e^{x_k / T} / Z,  p_r = e^{tail} / Z  (they sum to 1 by Z),
//   q = softmax(z / T),     q_r = the sum of q over the tokens not recorded;
//   KL = sum_b p_b ln(p_b / q_b),  TV = 1/2 sum_b |p_b - q_b|,  CE = -ln q_y,
//   loss = w (kl KL + tv TV + ce CE)
// (forward KL, TV and CE with position weights: the DLite page's distillation
// losses).  With s_b = sign(q_b - p_b) and S = 1/2 sum_b s_b q_b the gradient is
//   w/T [ q_v (kl + ce + tv (s_b(v)/2 - S)) - kl p_v - ce [v = y] ]  v recorded,
//   w/T [ q_v (kl + ce + tv (s_r/2 - S) - kl p_r / q_r) - ce [v = y] ]  else.
// For a token outside the record it is e^{(z_v - m) / T}, m the largest logit outside,
// times one factor of the row.
// The sum over the tokens not recorded leaves the others out by a bit map: q_r as
// 1 - sum q_k would cancel.
//
// What bounds it: the row is read once and its gradient written once.  A row is
// shared by a cluster of CS CTAs, each with a share that stays in shared memory
// between the two passes over it (a second read would come from HBM again: the
// rows in flight and the gradients do not fit L2 together).  Persistent CTAs, two per
// SM, of three roles, so that the copies never wait for the arithmetic between rows:
//   producer  streams the shares of this row and the next into a ring of
//             stages (bulk copies);
//   consumers pass 1: running maximum and sum of the unmarked logits; pass 2: the
//             gradient of every token as if outside the record;
//   recorder  (one warp) loads the next row's record, marks its tokens and sums
//             the teacher while the consumers work; merges the partial sums of
//             the CTA and, by messages through distributed shared memory, of the
//             cluster; computes losses, factors and the gradient of the K tokens
//             and the label, which the consumers store over theirs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rows.cuh"

namespace sv {
namespace {

constexpr int kDisWarps = 8;                               // consumers
constexpr int kDisConsumers = kDisWarps * 32;
constexpr int kDisThreads = kDisConsumers + 64;            // recorder, producer
constexpr int kDisPer = 4;                                 // vectors of a stage per thread
constexpr int kDisStageVecs = kDisPer * kDisConsumers;
constexpr int kDisStage = 16 * kDisStageVecs;
constexpr int kDisMaxStages = 6;

struct DisShared {
  uint64_t full[kDisMaxStages], empty[kDisMaxStages];
  // by row parity: the record is marked; the partial sums are in; the factors are
  // in; the recorded tokens' gradients are in; the gradient pass is done; every
  // CTA's message is in
  uint64_t marked[2], summed[2], factors[2], fixed[2], written[2], message[2];
  float part_m[2][kDisWarps], part_s[2][kDisWarps];
  uint4 msg[2][8];                           // maximum and sum outside the record, status, of each CTA of the cluster
  float c[2], top[2], factor[2];
  int skip[2], zero[2];
  uint32_t ends[2];                          // marks of the single elements: head from bit 0, tail from bit 8
  int fix_idx[SPEC_MAX_TOPK + 1];            // the recorded tokens and the label: token, or -1, and gradient
  float fix_g[SPEC_MAX_TOPK + 1];
  int raw_idx[SPEC_MAX_TOPK];
  float raw_x[SPEC_MAX_TOPK];
  int failed;
};

template <int DT>
__device__ __forceinline__ void store_logit(unsigned char* row, int e, float v) {
  if constexpr (DT == SPEC_BF16) reinterpret_cast<__nv_bfloat16*>(row)[e] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(row)[e] = v;
}

// Weights are 2^{(x - m) c}, m a maximum: m c apart would overflow for rows masked with
// the type's lowest value.  A sum of weights moved from one maximum to another:
__device__ __forceinline__ float moved(float sum, float from, float to, float c) {
  return from == -INFINITY ? sum : sum * ex2((from - to) * c);
}

// A token's mark, o elements into the share: a unit of kDisPer * PER bits per stage
// and consumer thread, PER for each vector that the thread reads of it.
template <int BITS>
struct MarkUnit;
template <>
struct MarkUnit<32> { using type = uint32_t; };
template <>
struct MarkUnit<16> { using type = uint16_t; };
template <>
struct MarkUnit<8> { using type = uint8_t; };
template <int PER>
__device__ __forceinline__ void mark_of(int o, int& word, int& bit) {
  const int vec = o / PER, in = vec % kDisStageVecs;
  const int at = (vec / kDisStageVecs * kDisConsumers + in % kDisConsumers) * (kDisPer * PER) +
                 in / kDisConsumers * PER + o % PER;
  word = at >> 5;
  bit = at & 31;
}

// A logit as loaded, and its value: a load is not waited for until the latter.
template <int DT>
__device__ __forceinline__ uint32_t raw_logit(const unsigned char* row, int e) {
  if constexpr (DT == SPEC_BF16) return reinterpret_cast<const unsigned short*>(row)[e];
  else return reinterpret_cast<const uint32_t*>(row)[e];
}
template <int DT>
__device__ __forceinline__ float raw_value(uint32_t raw) {
  return __uint_as_float(DT == SPEC_BF16 ? raw << 16 : raw);
}
template <int DT>
constexpr uint32_t kRawNegInf = DT == SPEC_BF16 ? 0xFF80u : 0xFF800000u;

// A row's own words as loaded.  Its record's entries lane, lane + 32, ... come to
// S.raw_idx and S.raw_x by asynchronous copies: registers would be spilled, and a
// spill waits for the load.
struct RawRow {
  float w, T, tail;
  int y;
};
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// A record worked up: teacher's share of each bucket, student weights relative to
// the record's own largest student logit, sums.
template <int NJ>
struct Record {
  int idx[NJ];                               // -1: none
  float p[NJ], f[NJ];                        // teacher's share, student's 2^{(z - zmax) c}
  uint32_t z[NJ], zy;                        // student's logits there and at the label, as loaded
  float w, T, zmax, F, A, in, pr, lpr;       // A = sum p (log2 p - (z - zmax) c), F = sum f, in = sum p
  int y, st;
  bool skip, recorded;
};

template <int DT, int CS, int NJ>
__global__ void __launch_bounds__(kDisThreads, 2) distill_kernel(const __grid_constant__ DistillParams P,
                                                                 const int stages, const int map_words,
                                                                 const bool keep) {
  constexpr int PER = RowType<DT>::PER, ES = RowType<DT>::ES;
  extern __shared__ __align__(128) unsigned char s_ring[];           // stages, then two mark maps
  __shared__ DisShared S;
  uint32_t* maps = reinterpret_cast<uint32_t*>(s_ring + (size_t)stages * kDisStage);
  const int V = P.V, K = P.K, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CS == 1 ? 0 : (int)cluster_rank();
  const int first = blockIdx.x / CS, step = gridDim.x / CS;
  const Waits waits{&S.failed, P.wait_limit};

  for (int i = tid; i < 2 * map_words; i += kDisThreads) maps[i] = 0;
  if (tid == 0) {
    S.failed = 0;
    S.ends[0] = S.ends[1] = 0;
    for (int i = 0; i < stages; ++i) { mbar_init(&S.full[i], 1); mbar_init(&S.empty[i], kDisWarps); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.marked[i], 1);
      mbar_init(&S.summed[i], kDisWarps);
      mbar_init(&S.factors[i], 1);
      mbar_init(&S.fixed[i], 1);
      mbar_init(&S.written[i], kDisWarps);
      mbar_init(&S.message[i], 1);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if constexpr (CS > 1) cluster_sync();

  if (warp == kDisWarps + 1) {               // producer
    if (lane == 0) {
      RingAt at;
      const int passes = P.grad && !keep ? 2 : 1;
      float next = first < P.n && P.row_weight ? P.row_weight[first] : 1.f; // a row ahead: a load takes 2 us here
      for (int r = first; r < P.n; r += step) {
        const float w = next;
        if (P.row_weight && r + step < P.n) next = P.row_weight[r + step];
        if (w == 0.f) continue;
        const unsigned char* row = P.logits + (size_t)r * V * ES;
        const RowSpan sp = row_span<DT>(row, V);
        const RowShare sh = row_share<CS>(sp, rank);
        const unsigned char* body = row + (size_t)sp.head * ES;
        for (int pass = 0; pass < passes; ++pass)
          for (int j = sh.lo; j < sh.hi; j += kDisStageVecs) {
            const uint32_t bytes = 16u * (uint32_t)(sh.hi - j < kDisStageVecs ? sh.hi - j : kDisStageVecs);
            // after a failed wait, stages are given up unread
            if (!bounded_wait(&S.empty[at.stage], at.phase ^ 1, waits) || *waits.failed) { r = P.n; pass = passes; break; }
            mbar_arrive_expect_tx(&S.full[at.stage], bytes);
            bulk_load(s_ring + (size_t)at.stage * kDisStage, body + 16ll * j, bytes, &S.full[at.stage]);
            at.next(stages);
          }
        if (r == P.n) break;
      }
    }
  } else if (warp == kDisWarps) {            // recorder
    auto fetch = [&](RawRow& W, int r) {
      W.w = P.row_weight ? P.row_weight[r] : 1.f;
      W.T = P.temperature ? P.temperature[r] : 1.f;
      W.tail = P.tail_lse ? P.tail_lse[r] : -INFINITY;
      W.y = P.label ? P.label[r] : -1;
      for (int k = lane; k < K; k += 32) {
        copy4(&S.raw_idx[k], P.top_index + (size_t)r * K + k);
        copy4(&S.raw_x[k], P.top_logits + (size_t)r * K + k);
      }
    };
    // marks the row's recorded tokens of this CTA's share and asks for the student's
    // logits there; the consumers may begin
    auto mark = [&](Record<NJ>& R, const RawRow& W, int r, int b) {
      R.w = W.w;
      R.skip = W.w == 0.f;                   // a padded row: its logits are not read
      R.st = 0;
      if (R.skip) {
        // the next row's copies go to the same words, and copies are not ordered among themselves
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0) { S.skip[b] = 1; mbar_arrive(&S.marked[b]); }
        return;
      }
      const unsigned char* row = P.logits + (size_t)r * V * ES;
      const RowSpan sp = row_span<DT>(row, V);
      const RowShare sh = row_share<CS>(sp, rank);
      R.T = temperature_ok(W.T) ? W.T : 1.f;
      R.y = W.y;
      if (!temperature_ok(W.T)) R.st |= SPEC_ST_BAD_TEMPERATURE;
      if (R.y < -1 || R.y >= V) { R.st |= SPEC_ST_BAD_TOKEN; R.y = -1; }
      R.recorded = false;
      asm volatile("cp.async.wait_all;" ::: "memory");       // a lane reads what it copied
      uint32_t* map = maps + b * map_words;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int k = lane + 32 * j;
        int e = k < K ? S.raw_idx[k] : -1;
        if (e < -1 || e >= V) { R.st |= SPEC_ST_BAD_TOKEN; e = -1; }
        R.idx[j] = e;
        R.p[j] = k < K ? S.raw_x[k] : -INFINITY;
        R.recorded |= e >= 0 && e == R.y;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = R.idx[j], o = e - sp.head;
        if (e < 0) continue;
        uint32_t old = 0;
        if (o < 0 || e >= sp.tail0) {
          const int bit = o < 0 ? e : 8 + e - sp.tail0;
          if (sh.ends) old = atomicOr(&S.ends[b], 1u << bit) >> bit;
        } else if (o >= sh.lo * PER && o < sh.hi * PER) {
          int word, bit;
          mark_of<PER>(o - sh.lo * PER, word, bit);
          old = atomicOr(&map[word], 1u << bit) >> bit;
        }
        if (old & 1) R.st |= SPEC_ST_BAD_TOKEN;              // recorded twice: the CTA that has it tells the others
      }
      if (lane == 0) { S.skip[b] = 0; S.c[b] = scale_split(R.T).c; }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.marked[b]);
      // after the arrival, whose release would wait for them
#pragma unroll
      for (int j = 0; j < NJ; ++j) R.z[j] = R.idx[j] >= 0 ? raw_logit<DT>(row, R.idx[j]) : kRawNegInf<DT>;
      R.zy = R.y >= 0 ? raw_logit<DT>(row, R.y) : 0u;
      R.lpr = W.tail;
    };
    // all that does not wait for the student's sums
    auto work_up = [&](Record<NJ>& R) {
      if (R.skip) return;
      const Scale sc = scale_split(R.T);
      const float tail = R.lpr;
      float z[NJ], xmax = -INFINITY, zmax = -INFINITY;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        z[j] = raw_value<DT>(R.z[j]);
        R.p[j] = R.idx[j] >= 0 ? R.p[j] : -INFINITY;
        if (R.p[j] != R.p[j] || R.p[j] == INFINITY || z[j] != z[j] || z[j] == INFINITY) R.st |= SPEC_ST_NONFINITE;
        xmax = fmaxf(xmax, R.p[j]);
        zmax = fmaxf(zmax, z[j]);
      }
      if (tail != tail || tail == INFINITY) R.st |= SPEC_ST_NONFINITE;
      // The label's logit is waited for here, with the others: once this CTA has sent its
      // sums, another may write its gradient over it.
      const float zy = raw_value<DT>(R.zy);
      if (zy != zy || zy == INFINITY) R.st |= SPEC_ST_NONFINITE;
      // The teacher's buckets in base 2, relative to its largest logit x0: a_k =
      // (x_k - x0) c, and tail log2(e) - x0 (c + lo) with the products' roundings
      // put back (x0 c alone is off by 2^-24 |x0 c|, which the K logits share and
      // the tail does not).
      xmax = warp_max(xmax);
      R.zmax = warp_max(zmax);
      const float x0 = xmax == -INFINITY ? 0.f : xmax, x0c = fmaxf(__fmul_rn(x0, sc.c), -3.4028235e38f);
      const float lt = tail == -INFINITY ? -INFINITY
                                           : (fmaf(tail, kLog2eHi, -x0c) - fmaf(x0, sc.c, -x0c)) +
                                                 (tail * kLog2eLo - x0 * sc.lo);
      const float top = fmaxf(xmax == -INFINITY ? -INFINITY : 0.f, lt);
      if (!(top > -INFINITY && top < INFINITY)) R.st |= SPEC_ST_NONFINITE;   // a record without any mass
      float a[NJ], Z = 0.f, F = 0.f, A = 0.f;
      const float z0 = R.zmax == -INFINITY ? 0.f : R.zmax;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        a[j] = R.p[j] == -INFINITY ? -INFINITY : (R.p[j] - x0) * sc.c - top;
        R.p[j] = ex2(a[j]);
        R.f[j] = ex2((z[j] - z0) * sc.c);
        Z += R.p[j];
        F += R.f[j];
      }
      const float er = lt == -INFINITY ? 0.f : ex2(lt - top);
      Z = warp_sum(Z) + er;
      R.F = warp_sum(F);
      const float rZ = 1.f / Z, l2Z = log2f(Z);
      float in = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        R.p[j] *= rZ;
        in += R.p[j];
        if (R.p[j] > 0.f) A += R.p[j] * ((a[j] - l2Z) - (z[j] - z0) * sc.c);   // +inf where z is -inf
      }
      R.A = warp_sum(A);
      R.in = warp_sum(in);                   // 1 - pr would cancel beside a lift of thousands
      R.pr = er * rZ;
      R.lpr = lt - top - l2Z;
      R.st = (int)__reduce_or_sync(0xffffffffu, (unsigned)R.st);
      R.recorded = __any_sync(0xffffffffu, R.recorded);
    };
    RawRow W;
    Record<NJ> R, N;
    if (first < P.n) {
      fetch(W, first);
      mark(N, W, first, 0);
      if (first + step < P.n) fetch(W, first + step);
      work_up(N);
    }
    int i = 0, live = 0;
    for (int r = first; r < P.n; r += step, ++i) {
      if (any_failed(waits)) break;
      const int b = i & 1;
      const bool more = r + step < P.n;
      R = N;
      // the next row's marks and loads go out while the consumers are in pass 1
      if (more) mark(N, W, r + step, b ^ 1);
      if (r + step < P.n - step) fetch(W, r + 2 * step);
      bounded_wait(&S.summed[b], (i >> 1) & 1, waits);
      __syncwarp();
      const unsigned char* row = P.logits + (size_t)r * V * ES;
      const RowSpan sp = row_span<DT>(row, V);
      const RowShare sh = row_share<CS>(sp, rank);
      const float nan = __int_as_float(0x7fc00000);
      float loss = 0.f, kl = 0.f, tv = 0.f, ce = 0.f;
      int st = 0;
      if (!R.skip) {
        const float c = S.c[b];
        float m = lane < kDisWarps ? S.part_m[b][lane] : -INFINITY;
        float s = lane < kDisWarps ? S.part_s[b][lane] : 0.f;
        // The tokens outside the record: their sum stays beside their own maximum, where it is
        // 1 or more (beside the row's, weights below 2^-126 are 0, and so would q_rest be).
        float mr = warp_max(m), sum_r = warp_sum(moved(s, m, mr, c));
        st = R.st;
        if constexpr (CS > 1) {
          const int mb = live & 1;
          if (lane == 0) mbar_arrive_expect_tx(&S.message[mb], 16 * CS);
          __syncwarp();
          if (lane < CS)                     // this CTA's sums to each CTA of the cluster
            send16(&S.msg[mb][rank], &S.message[mb], lane, __float_as_uint(mr), __float_as_uint(sum_r), (uint32_t)st, 0u);
          bounded_wait(&S.message[mb], (live >> 1) & 1, waits);
          __syncwarp();
          uint4 msg[CS];
#pragma unroll
          for (int q = 0; q < CS; ++q) {
            msg[q] = S.msg[mb][q];
            mr = fmaxf(mr, __uint_as_float(msg[q].x));
            st |= (int)msg[q].z;
          }
          sum_r = 0.f;
#pragma unroll
          for (int q = 0; q < CS; ++q) sum_r += moved(__uint_as_float(msg[q].y), __uint_as_float(msg[q].x), mr, c);
        }
        ++live;
        const float mall = fmaxf(R.zmax, mr), lift_r = mr == -INFINITY ? 0.f : (mr - mall) * c;
        const float up_r = ex2(lift_r), rest = sum_r * up_r;
        // weights are beside mall from here on: the record's own move there by `up`
        const float zy = raw_value<DT>(R.zy), lift = R.zmax == -INFINITY ? 0.f : (R.zmax - mall) * c, up = ex2(lift);
        const float sum = fmaf(R.F, up, rest);
        if (!isfinite(mall) || !isfinite(sum)) st |= SPEC_ST_NONFINITE;
        const float rS = 1.f / sum, l2S = log2f(sum), qr = rest * rS;
        const float sr = qr > R.pr ? 0.5f : qr < R.pr ? -0.5f : 0.f;
        const float kappa = up * rS;         // q_k = f_k kappa
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          if (R.idx[j] < 0) continue;
          const float q = R.f[j] * kappa;
          tv += fabsf(R.p[j] - q);
          sq += q > R.p[j] ? 0.5f * q : q < R.p[j] ? -0.5f * q : 0.f;
        }
        tv = warp_sum(tv);
        const float mean = warp_sum(sq) + sr * qr;
        const float lce = R.y >= 0 ? P.ce : 0.f, wT = R.w / R.T, base = P.kl + lce - P.tv * mean;
        // A token of the rest has q_v = e_v up_r rS and the share e_v / sum_r of the teacher's,
        // e_v = 2^{(z_v - mr) c} <= 1: one factor of e_v, no larger than its terms (pr / rest
        // would pass 2^128 long before the gradient does).  sum_r = 0: no token of the rest has
        // weight, its factor does not matter.
        const float factor = ((base + P.tv * sr) * (up_r * rS) - (sum_r > 0.f ? P.kl * R.pr / sum_r : 0.f)) * wT;
        const float e0 = mr == -INFINITY ? 0.f : mr;
        if (P.grad && lane == 0) {
          S.top[b] = e0;
          S.factor[b] = factor;
          S.zero[b] = st != 0;
          mbar_arrive(&S.factors[b]);
        }
        // log2 q_k = (z_k - zmax) c + lift - l2S, and the p_k sum to `in`;
        // log2 q_r = log2 sum_r + lift_r - l2S
        kl = R.in > 0.f ? R.A - R.in * (lift - l2S) : R.A;
        if (R.pr > 0.f) kl += R.pr * (R.lpr - (log2f(sum_r) + lift_r - l2S));
        kl *= kLn2;
        tv = 0.5f * (tv + fabsf(R.pr - qr));
        ce = R.y >= 0 ? (l2S - (zy - mall) * c) * kLn2 : 0.f;
        if (P.kl != 0.f) loss += P.kl * kl;
        if (P.tv != 0.f) loss += P.tv * tv;
        if (P.ce != 0.f) loss += P.ce * ce;
        loss *= R.w;
        if (P.grad) {
          // the consumers store these after their pass
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int k = lane + 32 * j;
            if (k >= K) continue;
            const float q = R.f[j] * kappa, sk = q > R.p[j] ? 0.5f : q < R.p[j] ? -0.5f : 0.f;
            S.fix_idx[k] = R.idx[j];
            S.fix_g[k] = wT * (q * (base + P.tv * sk) - P.kl * R.p[j] - (R.idx[j] == R.y ? lce : 0.f));
          }
          if (lane == 0) {                   // the label, where it is not recorded
            S.fix_idx[K] = R.recorded ? -1 : R.y;
            S.fix_g[K] = ex2((zy - e0) * c) * factor - wT * lce;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.fixed[b]);
        }
        // the map is clean for the row after next
        uint32_t* map = maps + b * map_words;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int o = R.idx[j] - sp.head;
          if (R.idx[j] >= 0 && o >= sh.lo * PER && o < sh.hi * PER) {
            int word, bit;
            mark_of<PER>(o - sh.lo * PER, word, bit);
            map[word] = 0;
          }
        }
        if (lane == 0) S.ends[b] = 0;
      } else if (P.grad && lane == 0) {
        S.zero[b] = 1;
        mbar_arrive(&S.factors[b]);
        mbar_arrive(&S.fixed[b]);
      }
      if (rank == 0 && lane == 0) {
        P.loss[r] = st ? nan : loss;
        if (P.parts) {
          P.parts[3 * (size_t)r] = st ? nan : kl;
          P.parts[3 * (size_t)r + 1] = st ? nan : tv;
          P.parts[3 * (size_t)r + 2] = st ? nan : ce;
        }
        if (P.status) P.status[r] = st;
      }
      __syncwarp();
      if (more) work_up(N);
    }
  } else {                                   // consumers
    RingAt at;
    int i = 0;
    for (int r = first; r < P.n; r += step, ++i) {
      if (any_failed(waits)) break;
      const int b = i & 1;
      const uint32_t turn = (i >> 1) & 1;
      const unsigned char* row = P.logits + (size_t)r * V * ES;
      unsigned char* grow = P.grad ? P.grad + (size_t)r * V * ES : nullptr;
      const RowSpan sp = row_span<DT>(row, V);
      const RowShare sh = row_share<CS>(sp, rank);
      const int ends = sh.ends ? sp.head + (V - sp.tail0) : 0;
      const int end_e = tid < sp.head ? tid : sp.tail0 + (tid - sp.head);
      bounded_wait(&S.marked[b], turn, waits);
      const int skip = S.skip[b];
      const float c = S.c[b];
      const RingAt row_at = at;
      float end_x = -INFINITY;
      if (!skip) {
        if (tid < ends) end_x = row_logit<DT>(row, end_e);
        // pass 1: running maximum and sum of the tokens not recorded
        float m = -INFINITY, s = 0.f;
        float nm = 0.f;                      // -m; 0 while all are -inf: weights of 0
        const auto* map = reinterpret_cast<const typename MarkUnit<kDisPer * PER>::type*>(maps + b * map_words);
        const float2 C2 = make_float2(c, c);
        auto raise = [&](float x) {
          s = moved(s, m, x, c);
          m = x;
          nm = -x;
        };
        for (int j = sh.lo, word = tid; j < sh.hi; j += kDisStageVecs, word += kDisConsumers) {
          bounded_wait(&S.full[at.stage], at.phase, waits);
          unsigned char* mine = s_ring + (size_t)at.stage * kDisStage + 16 * tid;
          const uint4* vec = reinterpret_cast<const uint4*>(mine);
          const int left = sh.hi - j - tid;
          // The marked logits become -inf in this thread's own vectors, so that the sums
          // below are straight code; the next copy into the stage comes after these
          // stores by the proxy fence.  (Masking the loaded registers costs more:
          // 91 us against 82 for 2048 x 128256.)
          uint32_t mark = map[word];
          if (mark != 0) {
            do {
              const int bit = __ffs((int)mark) - 1;
              mark &= mark - 1;
              store_logit<DT>(mine + (size_t)(bit / PER) * (16 * kDisConsumers), bit % PER, -INFINITY);
            } while (mark != 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          if (left > (kDisPer - 1) * kDisConsumers) {
            uint4 w[kDisPer];
#pragma unroll
            for (int u = 0; u < kDisPer; ++u) w[u] = vec[u * kDisConsumers];
            const float top = vecs_max<DT>(w);
            if (top > m) raise(top);
            const float2 M2 = make_float2(nm, nm);
            float2 t[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int u = 0; u < kDisPer; ++u)
#pragma unroll
              for (int k = 0; k < PER / 2; ++k) {
                const float2 a = __fmul2_rn(__fadd2_rn(vec_pair<DT>(w[u], k), M2), C2);
                t[k & 1] = __fadd2_rn(t[k & 1], make_float2(ex2(a.x), ex2(a.y)));
              }
            t[0] = __fadd2_rn(t[0], t[1]);
            s += t[0].x + t[0].y;
          } else {
#pragma unroll 1
            for (int u = 0; u < kDisPer && u * kDisConsumers < left; ++u) {
              const uint4 w = vec[u * kDisConsumers];
              const float top = vec_max<DT>(w);
              if (top > m) raise(top);
              const float2 M2 = make_float2(nm, nm);
              float2 t = make_float2(0.f, 0.f);
#pragma unroll
              for (int k = 0; k < PER / 2; ++k) {
                const float2 a = __fmul2_rn(__fadd2_rn(vec_pair<DT>(w, k), M2), C2);
                t = __fadd2_rn(t, make_float2(ex2(a.x), ex2(a.y)));
              }
              s += t.x + t.y;
            }
          }
          if (!(P.grad && keep)) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.empty[at.stage]);
          }
          at.next(stages);
        }
        if (tid < ends && !(S.ends[b] >> (tid < sp.head ? tid : 8 + tid - sp.head) & 1)) {
          if (end_x > m) raise(end_x);
          s += ex2((end_x + nm) * c);
        }
        const float top = warp_max(m);
        s = warp_sum(moved(s, m, top, c));
        if (lane == 0) { S.part_m[b][warp] = top; S.part_s[b][warp] = s; }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.summed[b]);
      if (!P.grad) continue;

      // pass 2: every token's gradient as if outside the record
      bounded_wait(&S.factors[b], turn, waits);
      const float top = S.top[b], factor = S.factor[b];
      const bool zero = S.zero[b] != 0;
      // vectors of the gradient row start where those of the logit row do, or it is written element by element
      const bool gvec = ((reinterpret_cast<uintptr_t>(grow) ^ reinterpret_cast<uintptr_t>(row)) & 15u) == 0;
      const float2 C2 = make_float2(c, c), M2 = make_float2(-top, -top), F2 = make_float2(factor, factor);
      uint4* gv = reinterpret_cast<uint4*>(grow + (size_t)sp.head * ES);
      RingAt from = keep ? row_at : at;
      auto gradient = [&](const uint4& w) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < PER / 2; ++k) {
          const float2 a = __fmul2_rn(__fadd2_rn(vec_pair<DT>(w, k), M2), C2);
          const float2 g = __fmul2_rn(make_float2(ex2(a.x), ex2(a.y)), F2);
          if constexpr (DT == SPEC_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(g.x, g.y);
            memcpy(&o[k], &h, 4);
          } else {
            o[2 * k] = __float_as_uint(g.x);
            o[2 * k + 1] = __float_as_uint(g.y);
          }
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
      };
      for (int j = sh.lo; j < sh.hi; j += kDisStageVecs) {
        if (!skip && !keep) bounded_wait(&S.full[from.stage], from.phase, waits);
        const uint4* vec = reinterpret_cast<const uint4*>(s_ring + (size_t)from.stage * kDisStage) + tid;
        const int left = sh.hi - j - tid;
        if (left > (kDisPer - 1) * kDisConsumers && gvec && !zero) {
          uint4 w[kDisPer];
#pragma unroll
          for (int u = 0; u < kDisPer; ++u) w[u] = vec[u * kDisConsumers];
#pragma unroll
          for (int u = 0; u < kDisPer; ++u) __stcs(gv + j + tid + u * kDisConsumers, gradient(w[u]));
        } else {
#pragma unroll 1
          for (int u = 0; u < kDisPer && u * kDisConsumers < left; ++u) {
            const uint4 g = zero ? make_uint4(0, 0, 0, 0) : gradient(vec[u * kDisConsumers]);
            const int v = j + tid + u * kDisConsumers;
            if (gvec) {
              __stcs(gv + v, g);
              continue;
            }
            const int e = sp.head + v * PER;
            const uint32_t o[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
            for (int k = 0; k < PER; ++k) {
              if constexpr (DT == SPEC_BF16)
                reinterpret_cast<uint16_t*>(grow)[e + k] = (uint16_t)(k & 1 ? o[k / 2] >> 16 : o[k / 2]);
              else
                reinterpret_cast<uint32_t*>(grow)[e + k] = o[k];
            }
          }
        }
        if (!skip) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.empty[from.stage]);
          from.next(stages);
        }
      }
      if (tid < ends) store_logit<DT>(grow, end_e, zero ? 0.f : ex2((end_x - top) * c) * factor);
      // over them, once every consumer's stores are out, one warp stores the recorded
      // tokens' and the label's (warps take turns; the others go on)
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.written[b]);
      if (warp == i % kDisWarps) {
        bounded_wait(&S.written[b], turn, waits);
        bounded_wait(&S.fixed[b], turn, waits);
        if (!zero)
          for (int k = lane; k <= K; k += 32) {
            const int e = S.fix_idx[k], o = e - sp.head;
            if (e >= 0 && e < V && (o < 0 || e >= sp.tail0 ? sh.ends : o >= sh.lo * PER && o < sh.hi * PER))
              store_logit<DT>(grow, e, S.fix_g[k]);
          }
      }
      if (!keep) at = from;
    }
  }
  __syncwarp();
  if (any_failed(waits)) drain_after_failure();
  __syncthreads();
  if constexpr (CS > 1) cluster_sync();      // no CTA leaves while another sends to it
  if (S.failed == 0 || warp != kDisWarps) return;
  // which of its rows the failed wait reached is not told apart
  for (long long r = first + (long long)lane * step; r < P.n; r += 32ll * step) {
    const float nan = __int_as_float(0x7fc00000);
    P.loss[r] = nan;
    if (P.parts)
      for (int k = 0; k < 3; ++k) P.parts[3 * r + k] = nan;
    if (P.status) P.status[r] = SPEC_ST_TIMEOUT;
  }
}

struct DisShape {
  int cs, stages, map_words;
  bool keep;
};

// Dynamic shared memory: two CTAs per SM (228 KB, 1 KB of it reserved for each).
constexpr int kDisSmem = 112 * 1024 - (int)sizeof(DisShared);

// Shares of a row: as many CTAs as leave each a bit map of 20 KB, and with the
// gradient a share that stays in the ring; more where the rows are few.
DisShape shape_of(int n, int V, int es, int nsm, bool grad) {
  DisShape s{};
  const int fill = row_cluster(n, V, es, nsm);
  for (s.cs = 1;; s.cs *= 2) {
    const int vecs = (V * es / 16 + s.cs - 1) / s.cs;
    s.map_words = (vecs + kDisStageVecs - 1) / kDisStageVecs * kDisStageVecs * (16 / es) / 32;
    const int most = (kDisSmem - 8 * s.map_words) / kDisStage, share = (vecs + kDisStageVecs - 1) / kDisStageVecs;
    s.keep = grad && share <= most;
    // no more than is used: what the ring does not take is L1, and the gathers and the
    // gradient's stores go through it (fp32 501 x 100003: 108 us with 6 stages, 98 with 5)
    const int want = s.keep ? share + 1 : 5;
    s.stages = want < most ? want : most;
    const bool fits = s.map_words <= 5120 && (!grad || s.keep);
    if (s.cs == 8 || (fits && s.cs >= fill)) return s;
  }
}

int g_clusters[kMaxDevices][4][2][4];           // resident at once, by device, record size, dtype and log2 CS

template <int DT, int CS, int NJ>
cudaError_t launch_as(const DistillParams& P, const DisShape& shape, int dev, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int most = g_clusters[dev][log2_of(NJ)][DT == SPEC_BF16][log2_of(CS)];
  cfg.gridDim = dim3((P.n < most ? P.n : most) * CS);
  cfg.blockDim = dim3(kDisThreads);
  cfg.dynamicSmemBytes = (size_t)shape.stages * kDisStage + 8 * shape.map_words;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {CS, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, distill_kernel<DT, CS, NJ>, P, shape.stages, shape.map_words, shape.keep);
}

template <int DT, int NJ>
cudaError_t launch_of(const DistillParams& P, int dev, int nsm, cudaStream_t s) {
  const DisShape shape = shape_of(P.n, P.V, RowType<DT>::ES, nsm, P.grad != nullptr);
  if (shape.cs == 8) return launch_as<DT, 8, NJ>(P, shape, dev, s);
  if (shape.cs == 4) return launch_as<DT, 4, NJ>(P, shape, dev, s);
  if (shape.cs == 2) return launch_as<DT, 2, NJ>(P, shape, dev, s);
  return launch_as<DT, 1, NJ>(P, shape, dev, s);
}

template <int DT, int CS, int NJ>
cudaError_t configure_one(int dev) {
  const auto kernel = distill_kernel<DT, CS, NJ>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDisSmem);
  if (e != cudaSuccess) return e;
  return resident_clusters(kernel, CS, kDisThreads, kDisSmem, &g_clusters[dev][log2_of(NJ)][DT == SPEC_BF16][log2_of(CS)]);
}
template <int DT, int NJ>
cudaError_t configure_as(int dev) {
  cudaError_t e = configure_one<DT, 1, NJ>(dev);
  if (e == cudaSuccess) e = configure_one<DT, 2, NJ>(dev);
  if (e == cudaSuccess) e = configure_one<DT, 4, NJ>(dev);
  if (e == cudaSuccess) e = configure_one<DT, 8, NJ>(dev);
  return e;
}

// Entries per recorder lane: records of up to 64, 128 and 256.  With 8 entries the
// recorder spills 72 to 208 bytes a thread, a few words of a row's record at a time.
template <int DT>
cudaError_t launch_entries(const DistillParams& P, int dev, int nsm, cudaStream_t s) {
  if (P.K <= 64) return launch_of<DT, 2>(P, dev, nsm, s);
  if (P.K <= 128) return launch_of<DT, 4>(P, dev, nsm, s);
  return launch_of<DT, 8>(P, dev, nsm, s);
}
template <int DT>
cudaError_t configure_entries(int dev) {
  cudaError_t e = configure_as<DT, 2>(dev);
  if (e == cudaSuccess) e = configure_as<DT, 4>(dev);
  if (e == cudaSuccess) e = configure_as<DT, 8>(dev);
  return e;
}

}  // namespace

cudaError_t launch_distill(const DistillParams& P, int dev, int nsm, cudaStream_t s) {
  return P.dtype == SPEC_BF16 ? launch_entries<SPEC_BF16>(P, dev, nsm, s) : launch_entries<SPEC_F32>(P, dev, nsm, s);
}

cudaError_t configure_distill(int dev) {
  const cudaError_t e = configure_entries<SPEC_BF16>(dev);
  return e == cudaSuccess ? configure_entries<SPEC_F32>(dev) : e;
}

}  // namespace sv
