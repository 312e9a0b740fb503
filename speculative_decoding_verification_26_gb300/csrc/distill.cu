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
// A cluster of CS CTAs per row (one where rows fill the GPU).  The recorded tokens are marked in a bit map, and the sum of
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

template <int DT, int CS>
__global__ void __launch_bounds__(kDisThreads, 2) distill_kernel(const __grid_constant__ DistillParams P) {
  constexpr int PER = RowType<DT>::PER, ES = RowType<DT>::ES;
  extern __shared__ uint32_t s_bits[];       // one bit per token of the row (offset PER: see below)
  __shared__ float s_f[kDisWarps];
  __shared__ float s_g[kDisWarps];
  __shared__ float s_part[2][2];             // this CTA's maximum and sum, for the cluster (by turns)
  const int rank = CS == 1 ? 0 : (int)cluster_rank();
  int turn = 0;
  const int V = P.V, K = P.K, tid = threadIdx.x;
  const int words = (V + PER + 31) / 32 + 1;
  const float nan = __int_as_float(0x7fc00000);
  for (int i = tid; i < words; i += kDisThreads) s_bits[i] = 0;
  for (int r = blockIdx.x / CS; r < P.n; r += gridDim.x / CS) {
    const unsigned char* row = P.logits + (size_t)r * V * ES;
    unsigned char* grow = P.grad ? P.grad + (size_t)r * V * ES : nullptr;
    const RowSpan sp = row_span<DT>(row, V);
    const RowShare sh = row_share<CS>(sp, rank);
    auto my_element = [&](int e) {           // whether this CTA writes token e's gradient
      const int j = e < sp.head ? -1 : (e - sp.head) / PER;
      return j < 0 || j >= sp.nvec ? sh.ends : j >= sh.lo && j < sh.hi;
    };
    // vectors of the gradient row start where those of the logit row do, or it is written element by element
    const bool gvec = ((reinterpret_cast<uintptr_t>(grow) ^ reinterpret_cast<uintptr_t>(row)) & 15u) == 0;
    const float w = P.row_weight ? P.row_weight[r] : 1.f;
    const float given = P.temperature ? P.temperature[r] : 1.f, T = temperature_ok(given) ? given : 1.f;
    const int y = P.label ? P.label[r] : -1;

    auto zero_grad = [&]() {
      if (!grow) return;
      if (gvec) {
        uint4* gv = reinterpret_cast<uint4*>(grow + (size_t)sp.head * ES);
        for (int j = sh.lo + tid; j < sh.hi; j += kDisThreads) gv[j] = make_uint4(0, 0, 0, 0);
        const int ends = sh.ends ? sp.head + (V - sp.tail0) : 0;
        if (tid < ends) store_logit<DT>(grow, tid < sp.head ? tid : sp.tail0 + (tid - sp.head), 0.f);
      } else {
        for (int e = rank * kDisThreads + tid; e < V; e += CS * kDisThreads) store_logit<DT>(grow, e, 0.f);
      }
    };
    if (w == 0.f) {                          // a padded row: nothing of it is read
      zero_grad();
      if (rank == 0 && tid == 0) {
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
    const float2 C2 = make_float2(c, c);
    auto raise = [&](float x) {
      s *= m == -INFINITY ? 0.f : ex2(ref_of(m, c) - ref_of(x, c));
      m = x;
    };
    for_row<DT, kDisThreads, 8>(row, sp, sh, V,
        [&](int j, const uint4& w) {
          const uint32_t mark = PER == 8 ? bytes[j + 1] : (bytes[(j + 1) >> 1] >> (((j + 1) & 1) * 4)) & 15u;
          if (mark == 0) {
            const float top = vec_max<DT>(w);
            if (top > m) raise(top);
            const float nr = m == -INFINITY ? 0.f : -ref_of(m, c);       // all -inf so far: weights of 0
            const float2 R2 = make_float2(nr, nr);
            float2 t = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
              const float2 a = __ffma2_rn(vec_pair<DT>(w, k), C2, R2);
              t = __fadd2_rn(t, make_float2(ex2(a.x), ex2(a.y)));
            }
            s += t.x + t.y;
          } else {
#pragma unroll
            for (int k = 0; k < PER; ++k) {
              const float2 p = vec_pair<DT>(w, k / 2);
              const float x = k & 1 ? p.y : p.x;
              if (mark >> k & 1) continue;
              if (x > m) raise(x);
              s += ex2(fmaf(x, c, m == -INFINITY ? 0.f : -ref_of(m, c)));
            }
          }
        },
        [&](int e, float x) {
          const int bit = e - sp.head + PER;
          if (s_bits[bit >> 5] >> (bit & 31) & 1) return;
          if (x > m) raise(x);
          s += ex2(fmaf(x, c, m == -INFINITY ? 0.f : -ref_of(m, c)));
        });
    __syncthreads();                         // s_f and s_g are read, and the map
    if (mine) atomicAnd(&s_bits[(idx - sp.head + PER) >> 5], ~(1u << ((idx - sp.head + PER) & 31)));
    float mall = cta_max<kDisWarps>(fmaxf(m, zk), s_f);
    if constexpr (CS > 1) {                  // every CTA holds all zk: the maximum of both is the row's
      if (tid == 0) s_part[turn][0] = mall;
    }
    // one exponent rule for every weight from here on: 2^{x c - ref}
    auto moved = [&](float sum, float from, float to) {
      return from == -INFINITY ? sum : sum * ex2(ref_of(from, c) - ref_of(to, c));
    };
    float rest = cta_sum<kDisWarps>(moved(s, m, mall), s_g);
    if constexpr (CS > 1) {
      if (tid == 0) s_part[turn][1] = rest;
      cluster_sync();
      float pm[CS], ps[CS];
#pragma unroll
      for (int q = 0; q < CS; ++q) {
        const uint32_t from = map_rank(smem_u32(s_part[turn]), q);
        pm[q] = __uint_as_float(ld_cluster(from));
        ps[q] = __uint_as_float(ld_cluster(from + 4));
        mall = fmaxf(mall, pm[q]);
      }
      rest = 0.f;
#pragma unroll
      for (int q = 0; q < CS; ++q) rest += moved(ps[q], pm[q], mall);
      turn ^= 1;
    }
    const float ref = ref_of(mall, c);
    const float fk = mine ? ex2(fmaf(zk, c, -ref)) : 0.f;
    __syncthreads();
    const float S = cta_sum<kDisWarps>(fk, s_f) + rest;
    if (!isfinite(mall) || !isfinite(S)) st |= SPEC_ST_NONFINITE;
    if (__syncthreads_or(st & SPEC_ST_NONFINITE)) st |= SPEC_ST_NONFINITE;
    if (__syncthreads_or(st & SPEC_ST_BAD_TOKEN)) st |= SPEC_ST_BAD_TOKEN;
    if (st != 0) {                           // the same in every thread
      zero_grad();
      if (rank == 0 && tid == 0) {
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
    if (rank == 0 && tid == 0) {
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
      const float2 R2 = make_float2(-ref, -ref), F2 = make_float2(rest_f, rest_f);
      for_row<DT, kDisThreads, 4>(row, sp, sh, V,
          [&](int j, const uint4& w) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
              const float2 a = __ffma2_rn(vec_pair<DT>(w, k), C2, R2);
              const float2 g = __fmul2_rn(make_float2(ex2(a.x), ex2(a.y)), F2);
              if constexpr (DT == SPEC_BF16) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(g.x, g.y);
                memcpy(&u[k], &b, 4);
              } else {
                u[2 * k] = __float_as_uint(g.x);
                u[2 * k + 1] = __float_as_uint(g.y);
              }
            }
            __stcs(gv + j, make_uint4(u[0], u[1], u[2], u[3]));
          },
          [&](int e, float x) { store_logit<DT>(grow, e, ex2(fmaf(x, c, -ref)) * rest_f); });
    } else {
      for (int e = rank * kDisThreads + tid; e < V; e += CS * kDisThreads)
        store_logit<DT>(grow, e, ex2(fmaf(row_logit<DT>(row, e), c, -ref)) * rest_f);
      if constexpr (CS > 1) cluster_sync();  // the tokens below may be another CTA's
    }
    const int recorded = __syncthreads_or(mine && idx == y);   // the pass's stores come before these
    if (mine && my_element(idx)) store_logit<DT>(grow, idx, gk);
    if (tid == 0 && y >= 0 && !recorded && my_element(y)) store_logit<DT>(grow, y, gy);
    __syncthreads();
  }
  if constexpr (CS > 1) cluster_sync();      // no CTA leaves while its partial sums are read
}

template <int DT, int CS>
cudaError_t launch_as(const DistillParams& P, int nsm, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int most = 2 * nsm / CS;             // clusters resident at once, two CTAs per SM
  cfg.gridDim = dim3((P.n < most ? P.n : most) * CS);
  cfg.blockDim = dim3(kDisThreads);
  cfg.dynamicSmemBytes = ((size_t)(P.V + 8 + 31) / 32 + 1) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {CS, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, distill_kernel<DT, CS>, P);
}

template <int DT>
cudaError_t launch_of(const DistillParams& P, int nsm, cudaStream_t s) {
  const int cs = row_cluster(P.n, P.V, RowType<DT>::ES, nsm);
  if (cs == 8) return launch_as<DT, 8>(P, nsm, s);
  if (cs == 4) return launch_as<DT, 4>(P, nsm, s);
  if (cs == 2) return launch_as<DT, 2>(P, nsm, s);
  return launch_as<DT, 1>(P, nsm, s);
}

template <int DT>
cudaError_t configure_as() {
  const int most = ((kDistillMaxV + 8 + 31) / 32 + 1) * 4;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(distill_kernel<DT, 1>, attr, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(distill_kernel<DT, 2>, attr, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(distill_kernel<DT, 4>, attr, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(distill_kernel<DT, 8>, attr, most);
  return e;
}

}  // namespace

cudaError_t launch_distill(const DistillParams& P, int nsm, cudaStream_t s) {
  return P.dtype == SPEC_BF16 ? launch_of<SPEC_BF16>(P, nsm, s) : launch_of<SPEC_F32>(P, nsm, s);
}

cudaError_t configure_distill() {
  const cudaError_t e = configure_as<SPEC_BF16>();
  return e == cudaSuccess ? configure_as<SPEC_F32>() : e;
}

}  // namespace sv
