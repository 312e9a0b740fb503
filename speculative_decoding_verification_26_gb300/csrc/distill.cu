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
// For a token outside the record it is e^{z_v / T} times one factor of the row.
//
// One CTA per row.  The recorded tokens are marked in a bit map, and the sum of
// the others leaves them out: q_r as 1 - sum q_k would cancel.  The gradient
// pass reads the row again (from L2) and writes factor times weight everywhere;
// then the K tokens and the label get their own values.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rows.cuh"

namespace sv {
namespace {

constexpr int kDisThreads = 512;
constexpr int kDisWarps = kDisThreads / 32;
constexpr float kLn2 = 0.693147180559945f;

template <int DT>
__device__ __forceinline__ void store_logit(unsigned char* row, int e, float v) {
  if constexpr (DT == SPEC_BF16) reinterpret_cast<__nv_bfloat16*>(row)[e] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(row)[e] = v;
}
template <int DT, int PER>
__device__ __forceinline__ uint4 pack_row(const float (&g)[PER]) {
  uint32_t u[4];
  if constexpr (DT == SPEC_BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(g[2 * k], g[2 * k + 1]);
      memcpy(&u[k], &b, 4);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = __float_as_uint(g[k]);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

template <int DT>
__global__ void __launch_bounds__(kDisThreads, 2) distill_kernel(const __grid_constant__ DistillParams P) {
  constexpr int PER = RowType<DT>::PER, ES = RowType<DT>::ES;
  extern __shared__ uint32_t s_bits[];       // one bit per token of the row (offset PER: see below)
  __shared__ float s_f[kDisWarps];
  __shared__ float s_g[kDisWarps];
  const int V = P.V, K = P.K, tid = threadIdx.x;
  const int words = (V + PER + 31) / 32 + 1;
  const float nan = __int_as_float(0x7fc00000);
  for (int i = tid; i < words; i += kDisThreads) s_bits[i] = 0;
  for (int r = blockIdx.x; r < P.n; r += gridDim.x) {
    const unsigned char* row = P.logits + (size_t)r * V * ES;
    unsigned char* grow = P.grad ? P.grad + (size_t)r * V * ES : nullptr;
    const RowSpan sp = row_span<DT>(row, V);
    // vectors of the gradient row start where those of the logit row do, or it is written element by element
    const bool gvec = ((reinterpret_cast<uintptr_t>(grow) ^ reinterpret_cast<uintptr_t>(row)) & 15u) == 0;
    const float w = P.row_weight ? P.row_weight[r] : 1.f;
    const float given = P.temperature ? P.temperature[r] : 1.f, T = temperature_ok(given) ? given : 1.f;
    const int y = P.label ? P.label[r] : -1;

    auto zero_grad = [&]() {
      if (!grow) return;
      if (gvec) {
        uint4* gv = reinterpret_cast<uint4*>(grow + (size_t)sp.head * ES);
        for (int j = tid; j < sp.nvec; j += kDisThreads) gv[j] = make_uint4(0, 0, 0, 0);
        const int ends = sp.head + (V - sp.tail0);
        if (tid < ends) store_logit<DT>(grow, tid < sp.head ? tid : sp.tail0 + (tid - sp.head), 0.f);
      } else {
        for (int e = tid; e < V; e += kDisThreads) store_logit<DT>(grow, e, 0.f);
      }
    };
    if (w == 0.f) {                          // a padded row: nothing of it is read
      zero_grad();
      if (tid == 0) {
        P.loss[r] = 0.f;
        if (P.parts) { P.parts[3 * (size_t)r] = 0.f; P.parts[3 * (size_t)r + 1] = 0.f; P.parts[3 * (size_t)r + 2] = 0.f; }
        if (P.status) P.status[r] = SPEC_ST_OK;
      }
      continue;
    }

    // this thread's recorded token (K <= 256 < kDisThreads), marked in the map.
    // Bit of token e: e - head + PER, so that the PER bits of vector j start at (j + 1) PER.
    int st = 0, idx = -1;
    float xk = -INFINITY, zk = -INFINITY;
    if (!temperature_ok(given)) st |= SPEC_ST_BAD_TEMPERATURE;
    if (y < -1 || y >= V) st |= SPEC_ST_BAD_TOKEN;
    __syncthreads();                         // the map is clear
    bool mine = false;
    if (tid < K) {
      idx = P.top_index[(size_t)r * K + tid];
      if (idx < -1 || idx >= V) {
        st |= SPEC_ST_BAD_TOKEN;
        idx = -1;
      }
      if (idx >= 0) {
        const int bit = idx - sp.head + PER;
        const uint32_t old = atomicOr(&s_bits[bit >> 5], 1u << (bit & 31));
        if (old >> (bit & 31) & 1) st |= SPEC_ST_BAD_TOKEN;   // recorded twice
        else mine = true;
        xk = P.top_logits[(size_t)r * K + tid];
        zk = row_logit<DT>(row, idx);
        if (xk != xk || xk == INFINITY || zk != zk || zk == INFINITY) st |= SPEC_ST_NONFINITE;
      }
    }
    const float tail = P.tail_lse ? P.tail_lse[r] : -INFINITY;
    if (tail != tail || tail == INFINITY) st |= SPEC_ST_NONFINITE;
    const float zy = y >= 0 && y < V ? row_logit<DT>(row, y) : 0.f;
    const Scale sc = scale_split(T);
    const float c = sc.c;

    // The teacher's buckets in base 2, relative to its largest logit x0: a_k =
    // (x_k - x0) c, and tail log2(e) - x0 (c + lo) with the products' roundings
    // put back (x0 c alone is off by 2^-24 |x0 c|, which the K logits share and
    // the tail does not).
    __syncthreads();                         // the map is complete
    const float xmax = cta_max<kDisWarps>(xk, s_f);
    const float x0 = xmax == -INFINITY ? 0.f : xmax;
    const float x0c = __fmul_rn(x0, c);
    const float lt = tail == -INFINITY ? -INFINITY
                                       : (fmaf(tail, kLog2eHi, -x0c) - fmaf(x0, c, -x0c)) +
                                             (tail * kLog2eLo - x0 * sc.lo);
    const float top = fmaxf(xmax == -INFINITY ? -INFINITY : 0.f, lt);
    const float ak = (xk - x0) * c - top;    // a token without mass: -inf
    const float ek = mine && xk != -INFINITY ? ex2(ak) : 0.f;
    const float er = lt != -INFINITY ? ex2(lt - top) : 0.f;
    const float Z = cta_sum<kDisWarps>(ek, s_g) + er;
    if (!(top > -INFINITY && top < INFINITY)) st |= SPEC_ST_NONFINITE;   // a record without any mass

    // the student's rest: running maximum and sum of the tokens not recorded
    float m = -INFINITY, s = 0.f;
    const unsigned char* bytes = reinterpret_cast<const unsigned char*>(s_bits);
    auto add = [&](float x) {
      if (x > m) {
        s *= m == -INFINITY ? 0.f : ex2((m - x) * c);
        m = x;
      }
      if (m != -INFINITY) s += ex2((x - m) * c);
      else if (x != x) s = x;
    };
    for_row<DT, kDisThreads, 4>(row, sp, V,
        [&](int j, float (&x)[PER]) {
          const uint32_t mark = PER == 8 ? bytes[j + 1] : (bytes[(j + 1) >> 1] >> (((j + 1) & 1) * 4)) & 15u;
          if (mark) {
#pragma unroll
            for (int k = 0; k < PER; ++k)
              if (mark >> k & 1) x[k] = -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < PER; ++k) add(x[k]);
        },
        [&](int e, float x) {
          const int bit = e - sp.head + PER;
          if (!(s_bits[bit >> 5] >> (bit & 31) & 1)) add(x);
        });
    __syncthreads();                         // s_f and s_g are read, and the map
    if (mine) atomicAnd(&s_bits[(idx - sp.head + PER) >> 5], ~(1u << ((idx - sp.head + PER) & 31)));
    const float mall = fmaxf(cta_max<kDisWarps>(fmaxf(m, zk), s_f), -INFINITY);
    const float ref = ref_of(mall, c);
    // one exponent rule for every weight from here on: 2^{x c - ref}
    const float rest = cta_sum<kDisWarps>(m == -INFINITY ? s : s * ex2(fmaf(m, c, -ref)), s_g);
    const float fk = mine ? ex2(fmaf(zk, c, -ref)) : 0.f;
    __syncthreads();
    const float S = cta_sum<kDisWarps>(fk, s_f) + rest;
    if (!isfinite(mall) || !isfinite(S)) st |= SPEC_ST_NONFINITE;
    if (__syncthreads_or(st & SPEC_ST_NONFINITE)) st |= SPEC_ST_NONFINITE;
    if (__syncthreads_or(st & SPEC_ST_BAD_TOKEN)) st |= SPEC_ST_BAD_TOKEN;
    if (st != 0) {                           // the same in every thread
      zero_grad();
      if (tid == 0) {
        P.loss[r] = nan;
        if (P.parts) { P.parts[3 * (size_t)r] = nan; P.parts[3 * (size_t)r + 1] = nan; P.parts[3 * (size_t)r + 2] = nan; }
        if (P.status) P.status[r] = st;
      }
      continue;
    }
    const float rS = 1.f / S, rZ = 1.f / Z, l2S = log2f(S), l2Z = log2f(Z);
    const float pk = ek * rZ, qk = fk * rS, pr = er * rZ, qr = rest * rS;
    // natural logarithms of p / q, term by term
    float tkl = 0.f;
    if (pk > 0.f) tkl = pk * ((ak - l2Z) - (fmaf(zk, c, -ref) - l2S)) * kLn2;
    const float sk = qk > pk ? 0.5f : qk < pk ? -0.5f : 0.f, sr = qr > pr ? 0.5f : qr < pr ? -0.5f : 0.f;
    __syncthreads();
    const float kls = cta_sum<kDisWarps>(tkl, s_f);
    const float tvs = cta_sum<kDisWarps>(mine ? fabsf(pk - qk) : 0.f, s_g);
    __syncthreads();
    const float mean = cta_sum<kDisWarps>(mine ? sk * qk : 0.f, s_f) + sr * qr;
    const float kl = kls + (pr > 0.f ? pr * ((lt - top - l2Z) - (log2f(rest) - l2S)) * kLn2 : 0.f);
    const float tv = 0.5f * (tvs + fabsf(pr - qr));
    const float ce = y >= 0 ? (l2S - fmaf(zy, c, -ref)) * kLn2 : 0.f;
    if (tid == 0) {
      float l = 0.f;
      if (P.kl != 0.f) l += P.kl * kl;
      if (P.tv != 0.f) l += P.tv * tv;
      if (P.ce != 0.f) l += P.ce * ce;
      P.loss[r] = w * l;
      if (P.parts) { P.parts[3 * (size_t)r] = kl; P.parts[3 * (size_t)r + 1] = tv; P.parts[3 * (size_t)r + 2] = ce; }
      if (P.status) P.status[r] = SPEC_ST_OK;
    }
    if (!grow) {
      __syncthreads();
      continue;
    }
    const float lce = y >= 0 ? P.ce : 0.f, wT = w / T;
    const float base = P.kl + lce - P.tv * mean;
    // q_r = 0: no token of the rest has weight, its factor does not matter
    const float rest_f = ((base + P.tv * sr) * rS - (rest > 0.f ? P.kl * pr / rest : 0.f)) * wT;
    const float gk = wT * (qk * (base + P.tv * sk) - P.kl * pk - (idx == y ? lce : 0.f));
    const float gy = ex2(fmaf(zy, c, -ref)) * rest_f - wT * lce;     // the label's, where it is not recorded
    if (gvec) {
      uint4* gv = reinterpret_cast<uint4*>(grow + (size_t)sp.head * ES);
      for_row<DT, kDisThreads, 4>(row, sp, V,
          [&](int j, float (&x)[PER]) {
#pragma unroll
            for (int k = 0; k < PER; ++k) x[k] = ex2(fmaf(x[k], c, -ref)) * rest_f;
            gv[j] = pack_row<DT, PER>(x);
          },
          [&](int e, float x) { store_logit<DT>(grow, e, ex2(fmaf(x, c, -ref)) * rest_f); });
    } else {
      for (int e = tid; e < V; e += kDisThreads)
        store_logit<DT>(grow, e, ex2(fmaf(row_logit<DT>(row, e), c, -ref)) * rest_f);
    }
    const int recorded = __syncthreads_or(mine && idx == y);   // the pass's stores come before these
    if (mine) store_logit<DT>(grow, idx, gk);
    if (tid == 0 && y >= 0 && !recorded) store_logit<DT>(grow, y, gy);
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_distill(const DistillParams& P, int nsm, cudaStream_t s) {
  const int grid = P.n < 2 * nsm ? P.n : 2 * nsm;
  const size_t smem = ((size_t)(P.V + 8 + 31) / 32 + 1) * 4;
  if (P.dtype == SPEC_BF16) distill_kernel<SPEC_BF16><<<grid, kDisThreads, smem, s>>>(P);
  else distill_kernel<SPEC_F32><<<grid, kDisThreads, smem, s>>>(P);
  return cudaGetLastError();
}

cudaError_t configure_distill() {
  const int most = ((kDistillMaxV + 8 + 31) / 32 + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(distill_kernel<SPEC_BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(distill_kernel<SPEC_F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

}  // namespace sv
