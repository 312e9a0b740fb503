// record.cu -- the record of a teacher row: its K largest logits and the log
// mass of the rest.
//
// Per row x[V] at temperature T: the K largest logits, by value, ties to the
// lowest index, and tail = ln sum_{v not among them} e^{x_v / T}.  The tail is
// summed over the rest itself: as a difference of two full sums it would cancel
// where the K logits carry nearly all of the mass.
//
// A cluster of CS CTAs per row (one where rows fill the GPU).  Pass A keeps each
// thread's own maximum.  The K-th largest of a CTA's thread maxima is a lower
// bound of the row's K-th largest logit, since K threads each hold a logit that
// large; for random rows the logits at or above it are little more than K.
// Pass B (from L2) copies those candidates to shared memory and sums the weights
// of all others, which are in the tail for certain.  Each candidate's place is
// the number of candidates before it (value descending, index ascending: no two
// compare equal), so the order in which they were copied does not matter;
// candidates past K join the tail in that order.
// Where more than kRecCap logits reach the bound (many equal values), the K-th
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
constexpr float kLn2 = 0.693147180559945f;

// order of a float as an unsigned integer, -0 and +0 alike
__device__ __forceinline__ uint32_t order_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // order_key(-inf)

// this thread's maximum; NaN when it saw one
template <int DT>
struct ThreadMax;
template <>
struct ThreadMax<SPEC_BF16> {
  uint32_t m = 0xFF80FF80u;                  // two -inf
  __device__ __forceinline__ void add(const uint4& w) {
    m = max_nan_bf2(m, max_nan_bf2(max_nan_bf2(w.x, w.y), max_nan_bf2(w.z, w.w)));
  }
  __device__ __forceinline__ float value() const { return max_nan(bf16_lo(m), bf16_hi(m)); }
};
template <>
struct ThreadMax<SPEC_F32> {
  float m = -INFINITY;
  __device__ __forceinline__ void add(const uint4& w) {
    m = max_nan(m, max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                           max_nan(__uint_as_float(w.z), __uint_as_float(w.w))));
  }
  __device__ __forceinline__ float value() const { return m; }
};

// What the CTAs of a cluster read of one another.
struct RecShare {
  float max;                                 // of the share; NaN: one was seen
  uint32_t bound;
  int count;
  float below;
};

template <int DT, int CS>
__global__ void __launch_bounds__(kRecThreads, 2) record_kernel(const __grid_constant__ RecordParams P) {
  constexpr int PER = RowType<DT>::PER, ES = RowType<DT>::ES;
  __shared__ float s_f[kRecWarps];
  __shared__ uint32_t s_lo[kRecWarps], s_hi[kRecWarps];
  __shared__ int s_i[kRecWarps];
  __shared__ int s_n;
  __shared__ RecShare s_share;
  __shared__ unsigned long long s_cand[kRecCap];   // order key, then ~index: larger comes first
  __shared__ int s_place[kRecCap];
  __shared__ float s_left[kRecCap];                // weights of the candidates past K, by place
  const int V = P.V, K = P.K, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CS == 1 ? 0 : (int)cluster_rank();
  for (int r = blockIdx.x / CS; r < P.n; r += gridDim.x / CS) {
    const unsigned char* row = P.logits + (size_t)r * V * ES;
    const float given = P.temperature ? P.temperature[r] : 1.f, T = temperature_ok(given) ? given : 1.f;
    const RowSpan sp = row_span<DT>(row, V);
    const RowShare sh = row_share<CS>(sp, rank);
    float* top = P.top_logits + (size_t)r * K;
    int32_t* ti = P.top_index + (size_t)r * K;

    // pass A
    ThreadMax<DT> tm;
    float single = -INFINITY;
    for_row<DT, kRecThreads, 8>(row, sp, sh, V, [&](int, const uint4& w) { tm.add(w); },
                                [&](int, float x) { single = x; });
    const float mine = max_nan(tm.value(), single);
    const uint32_t key = order_key(mine);    // a NaN's does not matter
    float m = mine;
    uint32_t lo = key, hi = key;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    }
    if (lane == 0) { s_f[warp] = m; s_lo[warp] = lo; }
    if (tid == 0) s_n = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRecWarps; ++w) { m = max_nan(m, s_f[w]); lo = min(lo, s_lo[w]); }
    hi = order_key(m);
    // The largest key that K thread maxima reach, or one that few more than K do:
    // lo is reached by K or more, hi + 1 by fewer.
    uint32_t bound = kKeyNegInf + 1;         // -inf is never recorded
    if (lo <= kKeyNegInf) {
      lo = kKeyNegInf + 1;
      if (__syncthreads_count(key >= lo) < K) hi = lo;     // too few threads hold a logit: all of them
    }
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      const int reach = __syncthreads_count(key >= mid);
      if (reach >= K) {
        lo = mid;
        if (reach <= K + K / 8) break;
      } else {
        hi = mid - 1;
      }
    }
    if (lo > bound) bound = lo;
    if constexpr (CS > 1) {
      if (tid == 0) { s_share.max = m; s_share.bound = bound; }
      cluster_sync();
      float all = -INFINITY;
      uint32_t most = bound;
#pragma unroll
      for (int c = 0; c < CS; ++c) {
        all = max_nan(all, __uint_as_float(ld_cluster(map_rank(smem_u32(&s_share.max), c))));
        most = max(most, ld_cluster(map_rank(smem_u32(&s_share.bound), c)));
      }
      m = all;
      bound = most;
    }
    int st = 0;
    if (!temperature_ok(given)) st |= SPEC_ST_BAD_TEMPERATURE;
    if (!isfinite(m)) st |= SPEC_ST_NONFINITE;               // NaN, +inf, or nothing finite
    if (rank == 0 && tid == 0 && P.status) P.status[r] = st;
    if (st != 0) {                           // the same in every CTA of the cluster
      if (rank == 0) {
        for (int k = tid; k < K; k += kRecThreads) { top[k] = __int_as_float(0x7fc00000); ti[k] = -1; }
        if (tid == 0) P.tail_lse[r] = __int_as_float(0x7fc00000);
      }
      if constexpr (CS > 1) cluster_sync();
      else __syncthreads();
      continue;
    }

    // pass B: candidates, and the weights of the others
    const Scale sc = scale_split(T);
    const float c = sc.c, ref = ref_of(m, c), at_least = key_value(bound);
    const float2 C2 = make_float2(c, c), R2 = make_float2(-ref, -ref);
    float2 sum = make_float2(0.f, 0.f);
    auto take = [&](int e, float x) {
      if (x >= at_least) {
        const int at = atomicAdd(&s_n, 1);
        if (at < kRecCap) s_cand[at] = (unsigned long long)order_key(x) << 32 | (uint32_t)~e;
      } else {
        sum.x += ex2(fmaf(x, c, -ref));
      }
    };
    for_row<DT, kRecThreads, 8>(row, sp, sh, V,
        [&](int j, const uint4& w) {
          if (vec_max<DT>(w) >= at_least) {
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
              const float2 x = vec_pair<DT>(w, k);
              take(sp.head + j * PER + 2 * k, x.x);
              take(sp.head + j * PER + 2 * k + 1, x.y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
              const float2 a = __ffma2_rn(vec_pair<DT>(w, k), C2, R2);
              sum = __fadd2_rn(sum, make_float2(ex2(a.x), ex2(a.y)));
            }
          }
        },
        take);
    __syncthreads();
    float below = cta_sum<kRecWarps>(sum.x + sum.y, s_f);
    int C = s_n;
    if constexpr (CS > 1) {
      if (tid == 0) { s_share.count = C; s_share.below = below; }
      cluster_sync();                        // every share's candidates are in its shared memory
      if (rank == 0) {
        int total = C;
        for (int q = 1; q < CS; ++q) {
          const int n = (int)ld_cluster(map_rank(smem_u32(&s_share.count), q));
          below += __uint_as_float(ld_cluster(map_rank(smem_u32(&s_share.below), q)));
          if (total + n <= kRecCap) {
            const uint32_t from = map_rank(smem_u32(s_cand), q);
            uint32_t* to = reinterpret_cast<uint32_t*>(s_cand + total);
            for (int i = tid; i < 2 * n; i += kRecThreads) to[i] = ld_cluster(from + 4 * i);
          }
          total += n;
        }
        C = total;
        __syncthreads();
      }
      cluster_sync();                        // the others' shared memory is free again
      if (rank != 0) continue;
    }
    float extra = 0.f;                       // tail weights beside `below`
    if (C > kRecCap) {
      // many equal values: the K-th largest key itself, by counting
      const RowShare whole{0, sp.nvec, true};
      uint32_t kth = 0;
      auto each = [&](auto&& f) {
        for_row<DT, kRecThreads, 4>(row, sp, whole, V,
            [&](int j, const uint4& w) {
#pragma unroll
              for (int k = 0; k < PER / 2; ++k) {
                const float2 x = vec_pair<DT>(w, k);
                f(sp.head + j * PER + 2 * k, x.x);
                f(sp.head + j * PER + 2 * k + 1, x.y);
              }
            },
            f);
      };
      auto count = [&](auto&& pred) {
        int cnt = 0;
        each([&](int, float x) { cnt += pred(order_key(x)); });
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
      float less = 0.f;
      each([&](int e, float x) {
        const uint32_t k = order_key(x);
        if (k > kth) s_cand[atomicAdd(&s_n, 1)] = (unsigned long long)k << 32 | (uint32_t)~e;
        else if (k < kth) less += ex2(fmaf(x, c, -ref));
      });
      __syncthreads();
      for (int e0 = 0, got = 0; got < need && e0 < V; e0 += kRecThreads) {
        const int e = e0 + tid;
        const bool tie = e < V && order_key(row_logit<DT>(row, e)) == kth;
        const unsigned vote = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) s_i[warp] = __popc(vote);
        __syncthreads();
        int before = got, all = 0;
        for (int w = 0; w < kRecWarps; ++w) {
          if (w < warp) before += s_i[w];
          all += s_i[w];
        }
        before += __popc(vote & ((1u << lane) - 1));
        if (tie && before < need) s_cand[above + before] = (unsigned long long)kth << 32 | (uint32_t)~e;
        got += all;
        __syncthreads();
      }
      C = K;
      below = cta_sum<kRecWarps>(less, s_f) + (float)(equal - need) * ex2(fmaf(key_value(kth), c, -ref));
      __syncthreads();
    }
    // places: each candidate is compared with all by `parts` threads
    for (int i = tid; i < C; i += kRecThreads) s_place[i] = 0;
    __syncthreads();
    const int width = (C + 31) / 32 * 32, parts = width < kRecThreads ? kRecThreads / (width ? width : 32) : 1;
    if (parts > 1) {
      const int i = tid % width, part = tid / width;
      if (i < C && part < parts) {
        const int per = (C + parts - 1) / parts, j1 = min(C, (part + 1) * per);
        const unsigned long long me = s_cand[i];
        int before = 0;
        for (int j = part * per; j < j1; ++j) before += s_cand[j] > me;
        atomicAdd(&s_place[i], before);
      }
    } else {
      for (int i = tid; i < C; i += kRecThreads) {
        const unsigned long long me = s_cand[i];
        int before = 0;
        for (int j = 0; j < C; ++j) before += s_cand[j] > me;
        s_place[i] = before;
      }
    }
    __syncthreads();
    for (int i = tid; i < C; i += kRecThreads) {
      const int place = s_place[i], e = (int)~(uint32_t)s_cand[i];
      const float x = key_value((uint32_t)(s_cand[i] >> 32));
      if (place < K) {
        top[place] = x == 0.f ? row_logit<DT>(row, e) : x;   // the key has lost a zero's sign
        ti[place] = e;
      } else {
        s_left[place] = ex2(fmaf(x, c, -ref));
      }
    }
    for (int k = C + tid; k < K; k += kRecThreads) { top[k] = -INFINITY; ti[k] = -1; }   // fewer finite logits than K
    if (C > K) {
      __syncthreads();
      for (int i = K + tid; i < C; i += kRecThreads) extra += s_left[i];
      extra = cta_sum<kRecWarps>(extra, s_f);
    }
    if (tid == 0) {
      // the weights are 2^{x c - ref}: ref and the scale's remainder put the exponent back
      const float tail = below + extra;
      P.tail_lse[r] = tail > 0.f ? kLn2 * (ref + (log2f(tail) + m * sc.lo)) : -INFINITY;
    }
    __syncthreads();
  }
}

int g_clusters[kMaxDevices][2][4];           // resident at once, by device, dtype and log2 CS

template <int DT, int CS>
cudaError_t launch_as(const RecordParams& P, int dev, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int most = g_clusters[dev][DT == SPEC_BF16][log2_of(CS)];
  cfg.gridDim = dim3((P.n < most ? P.n : most) * CS);
  cfg.blockDim = dim3(kRecThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {CS, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, record_kernel<DT, CS>, P);
}

template <int DT>
cudaError_t launch_of(const RecordParams& P, int dev, int nsm, cudaStream_t s) {
  const int cs = row_cluster(P.n, P.V, RowType<DT>::ES, nsm);
  if (cs == 8) return launch_as<DT, 8>(P, dev, s);
  if (cs == 4) return launch_as<DT, 4>(P, dev, s);
  if (cs == 2) return launch_as<DT, 2>(P, dev, s);
  return launch_as<DT, 1>(P, dev, s);
}

template <int DT>
cudaError_t configure_as(int dev) {
  int* g = g_clusters[dev][DT == SPEC_BF16];
  cudaError_t e = resident_clusters(record_kernel<DT, 1>, 1, kRecThreads, 0, &g[0]);
  if (e == cudaSuccess) e = resident_clusters(record_kernel<DT, 2>, 2, kRecThreads, 0, &g[1]);
  if (e == cudaSuccess) e = resident_clusters(record_kernel<DT, 4>, 4, kRecThreads, 0, &g[2]);
  if (e == cudaSuccess) e = resident_clusters(record_kernel<DT, 8>, 8, kRecThreads, 0, &g[3]);
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
