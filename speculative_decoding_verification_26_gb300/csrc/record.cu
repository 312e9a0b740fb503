// record.cu -- the record of a teacher row: its K largest logits and the log
// mass of the rest.
//
// Per row x[V] at temperature T: the K largest logits, by value, ties to the
// lowest index, and tail = ln sum_{v not among them} e^{x_v / T}.  The tail is
// summed over the rest itself: as a difference of two full sums it would cancel
// where the K logits carry nearly all of the mass.
//
// One CTA per row.  Pass A keeps each thread's own maximum.  The K-th largest
// of those is a lower bound of the K-th largest logit, since K threads each
// hold a logit that large; for random rows the logits at or above it are little
// more than K.  Pass B copies those candidates to shared memory and sums the
// weights of all others, which are in the tail for certain.  Each candidate's
// place is the number of candidates before it (value descending, index
// ascending: no two compare equal), so the order in which they were copied does
// not matter; candidates past K join the tail in that order.
// Where more than kCap logits reach the bound (many equal values), the K-th
// largest key is found bit by bit by counting over the row, and ties are taken
// in index order.
#include <cuda_runtime.h>

#include <cstdint>

#include "rows.cuh"

namespace sv {
namespace {

constexpr int kRecThreads = 512;
constexpr int kRecWarps = kRecThreads / 32;
constexpr int kRecCap = 2048;

// order of a float as an unsigned integer, -0 and +0 alike
__device__ __forceinline__ uint32_t order_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // order_key(-inf)

template <int DT>
__global__ void __launch_bounds__(kRecThreads, 2) record_kernel(const __grid_constant__ RecordParams P) {
  constexpr int PER = RowType<DT>::PER, ES = RowType<DT>::ES;
  __shared__ float s_f[kRecWarps];
  __shared__ int s_i[kRecWarps];
  __shared__ int s_n;
  __shared__ float s_val[kRecCap];
  __shared__ int s_idx[kRecCap];
  __shared__ float s_left[kRecCap];        // weights of the candidates past K, by place
  const int V = P.V, K = P.K, tid = threadIdx.x;
  for (int r = blockIdx.x; r < P.n; r += gridDim.x) {
    const unsigned char* row = P.logits + (size_t)r * V * ES;
    const float T = P.temperature ? P.temperature[r] : 1.f;
    const RowSpan sp = row_span<DT>(row, V);
    float* top = P.top_logits + (size_t)r * K;
    int32_t* ti = P.top_index + (size_t)r * K;

    // pass A: this thread's maximum, and whether a NaN was seen
    float mx = -INFINITY;
    bool nan = false;
    for_row<DT, kRecThreads, 4>(row, sp, V,
        [&](int, const float (&x)[PER]) {
#pragma unroll
          for (int k = 0; k < PER; ++k) { mx = fmaxf(mx, x[k]); nan |= x[k] != x[k]; }
        },
        [&](int, float x) { mx = fmaxf(mx, x); nan |= x != x; });
    const int any_nan = __syncthreads_or(nan);
    const float m = cta_max<kRecWarps>(mx, s_f);
    int st = 0;
    if (!temperature_ok(T)) st |= SPEC_ST_BAD_TEMPERATURE;
    if (any_nan || !isfinite(m)) st |= SPEC_ST_NONFINITE;
    if (tid == 0) {
      s_n = 0;
      if (P.status) P.status[r] = st;
    }
    if (st != 0) {
      for (int k = tid; k < K; k += kRecThreads) { top[k] = __int_as_float(0x7fc00000); ti[k] = -1; }
      if (tid == 0) P.tail_lse[r] = __int_as_float(0x7fc00000);
      __syncthreads();
      continue;
    }
    // the K-th largest thread maximum: the largest key that K of them reach
    uint32_t bound = 0;
    const uint32_t mykey = order_key(mx);
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t t = bound | (1u << bit);
      if (__syncthreads_count(mykey >= t) >= K) bound = t;
    }
    if (bound <= kKeyNegInf) bound = kKeyNegInf + 1;     // -inf is never recorded

    // pass B: candidates, and the weights of the others
    const Scale sc = scale_split(T);
    const float c = sc.c, ref = ref_of(m, c);
    float below = 0.f;
    auto take = [&](int e, float x) {
      if (order_key(x) >= bound) {
        const int at = atomicAdd(&s_n, 1);
        if (at < kRecCap) { s_val[at] = x; s_idx[at] = e; }
      } else {
        below += ex2(fmaf(x, c, -ref));
      }
    };
    for_row<DT, kRecThreads, 4>(row, sp, V,
        [&](int j, const float (&x)[PER]) {
#pragma unroll
          for (int k = 0; k < PER; ++k) take(sp.head + j * PER + k, x[k]);
        },
        take);
    __syncthreads();
    int C = s_n;
    float extra = 0.f;                   // tail weights beside `below`
    if (C > kRecCap) {
      // many equal values: the K-th largest key itself, by counting
      uint32_t kth = 0;
      auto count = [&](auto&& pred) {
        int cnt = 0;
        for_row<DT, kRecThreads, 4>(row, sp, V,
            [&](int, const float (&x)[PER]) {
#pragma unroll
              for (int k = 0; k < PER; ++k) cnt += pred(order_key(x[k]));
            },
            [&](int, float x) { cnt += pred(order_key(x)); });
        __syncthreads();
        return cta_sum<kRecWarps>(cnt, s_i);
      };
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t t = kth | (1u << bit);
        if (count([&](uint32_t k) { return k >= t; }) >= K) kth = t;
      }
      const int above = count([&](uint32_t k) { return k > kth; });
      const int equal = count([&](uint32_t k) { return k == kth; });
      const int need = K - above;
      // all above it, then the ties in index order; s_n counts the former
      __syncthreads();
      if (tid == 0) s_n = 0;
      __syncthreads();
      below = 0.f;
      auto upper = [&](int e, float x) {
        const uint32_t k = order_key(x);
        if (k > kth) {
          const int at = atomicAdd(&s_n, 1);
          s_val[at] = x;
          s_idx[at] = e;
        } else if (k < kth) {
          below += ex2(fmaf(x, c, -ref));
        }
      };
      for_row<DT, kRecThreads, 4>(row, sp, V,
          [&](int j, const float (&x)[PER]) {
#pragma unroll
            for (int k = 0; k < PER; ++k) upper(sp.head + j * PER + k, x[k]);
          },
          upper);
      __syncthreads();
      for (int e0 = 0, got = 0; got < need && e0 < V; e0 += kRecThreads) {
        const int e = e0 + tid;
        const float x = e < V ? row_logit<DT>(row, e) : -INFINITY;
        const bool tie = e < V && order_key(x) == kth;
        const unsigned vote = __ballot_sync(0xffffffffu, tie);
        if ((tid & 31) == 0) s_i[tid >> 5] = __popc(vote);
        __syncthreads();
        int before = got, all = 0;
        for (int w = 0; w < kRecWarps; ++w) {
          if (w < (tid >> 5)) before += s_i[w];
          all += s_i[w];
        }
        before += __popc(vote & ((1u << (tid & 31)) - 1));
        if (tie && before < need) { s_val[above + before] = x; s_idx[above + before] = e; }
        got += all;
        __syncthreads();
      }
      C = K;
      if (tid == 0) {
        const uint32_t u = kth & 0x80000000u ? kth ^ 0x80000000u : ~kth;
        extra = (float)(equal - need) * ex2(fmaf(__uint_as_float(u), c, -ref));
      }
    }
    // places
    for (int i = tid; i < C; i += kRecThreads) {
      const uint32_t ki = order_key(s_val[i]);
      const int ii = s_idx[i];
      int place = 0;
      for (int j = 0; j < C; ++j) {
        const uint32_t kj = order_key(s_val[j]);
        place += (kj > ki) || (kj == ki && s_idx[j] < ii);
      }
      if (place < K) { top[place] = s_val[i]; ti[place] = ii; }
      else s_left[place] = ex2(fmaf(s_val[i], c, -ref));
    }
    for (int k = C + tid; k < K; k += kRecThreads) { top[k] = -INFINITY; ti[k] = -1; }   // fewer finite logits than K
    __syncthreads();
    for (int i = K + tid; i < C; i += kRecThreads) extra += s_left[i];
    const float tail = cta_sum<kRecWarps>(below + extra, s_f);
    if (tid == 0) {
      // the weights are 2^{x c - ref}: ref and the scale's remainder put the exponent back
      P.tail_lse[r] = tail > 0.f ? 0.693147180559945f * (ref + (log2f(tail) + m * sc.lo)) : -INFINITY;
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_record(const RecordParams& P, int nsm, cudaStream_t s) {
  const int grid = P.n < 2 * nsm ? P.n : 2 * nsm;
  if (P.dtype == SPEC_BF16) record_kernel<SPEC_BF16><<<grid, kRecThreads, 0, s>>>(P);
  else record_kernel<SPEC_F32><<<grid, kRecThreads, 0, s>>>(P);
  return cudaGetLastError();
}

}  // namespace sv
