// rows.cuh -- one logit row read by a CTA: the split into a scalar head, a body
// of 16-byte vectors and a scalar tail, and sums over the CTA in a fixed order.
#pragma once

#include "common.cuh"

namespace sv {

// Logits of a row of dtype DT; PER of them fill a 16-byte vector.
template <int DT>
struct RowType;
template <>
struct RowType<SPEC_BF16> {
  static constexpr int ES = 2, PER = 8;
  __device__ __forceinline__ static void unpack(uint4 w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) { x[2 * k] = bf16_lo(u[k]); x[2 * k + 1] = bf16_hi(u[k]); }
  }
};
template <>
struct RowType<SPEC_F32> {
  static constexpr int ES = 4, PER = 4;
  __device__ __forceinline__ static void unpack(uint4 w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
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
// 2^{x c - fl(m c)} take c alone: that scales an exponent by 1 + 2^-24 at most
// and the common offset cancels in ratios; lo enters where a sum's logarithm is
// put back into units of the logits.
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

// Calls fv(j, x) for each vector j of this thread (x its PER logits) and
// fe(e, x) for each single element e.  U vectors are loaded before any is
// used, so that a thread has that many 16-byte loads in flight.
template <int DT, int THREADS, int U, class FV, class FE>
__device__ __forceinline__ void for_row(const unsigned char* row, const RowSpan& sp, int V, FV&& fv, FE&& fe) {
  constexpr int ES = RowType<DT>::ES, PER = RowType<DT>::PER;
  const uint4* vec = reinterpret_cast<const uint4*>(row + (size_t)sp.head * ES);
  for (int j0 = threadIdx.x; j0 < sp.nvec; j0 += THREADS * U) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * THREADS;
      if (j < sp.nvec) w[u] = vec[j];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * THREADS;
      if (j < sp.nvec) {
        float x[PER];
        RowType<DT>::unpack(w[u], x);
        fv(j, x);
      }
    }
  }
  const int ends = sp.head + (V - sp.tail0);
  if ((int)threadIdx.x < ends) {
    const int e = (int)threadIdx.x < sp.head ? (int)threadIdx.x : sp.tail0 + ((int)threadIdx.x - sp.head);
    fe(e, row_logit<DT>(row, e));
  }
}

// Sum over the CTA, the same bits in every thread; `scratch` holds WARPS values
// and may be used again after the next __syncthreads.
template <int WARPS, class T>
__device__ __forceinline__ T cta_sum(T v, T* scratch) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  T t = scratch[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) t += scratch[w];
  return t;
}
template <int WARPS>
__device__ __forceinline__ float cta_max(float v, float* scratch) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = scratch[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) t = fmaxf(t, scratch[w]);
  return t;
}

}  // namespace sv
