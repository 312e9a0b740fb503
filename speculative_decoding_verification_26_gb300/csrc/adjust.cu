// adjust.cu -- penalties for repeated tokens, biases and masks on logit rows.
//
// Row i of request b is the row after the request's history and its draft tokens
// y_0 .. y_{i-1}.  With c(v) the occurrences of v among the outputs (the history
// behind the prompt, and those drafts), and v "seen" when it occurs anywhere,
//   x <- seen ? (x > 0 ? x / rep : x rep) : x;   x <- x - c freq - [c > 0] pres;
//   x <- x + sum of the biases listed for v;     x <- -inf where the mask has 0,
// in fp32, rounded once to the row's type.  Logits that nothing touches keep their bits.
//
// A CTA takes a range of the vocabulary for all R rows of a request: it counts the
// history's tokens of its range in shared memory (whole numbers: the order of the
// atomics does not matter) and goes over its part of the rows.
#include "rows.cuh"
#include "serve.cuh"

namespace sv {
namespace {

constexpr int kAdjustThreads = 256;
constexpr int kRange = 4096;                 // tokens of a CTA
constexpr uint32_t kInPrompt = 0x80000000u;  // of a count: the token is in the prompt

template <int DT>
__device__ __forceinline__ void put_logit(unsigned char* row, int e, float x) {
  if constexpr (DT == SPEC_BF16) reinterpret_cast<__nv_bfloat16*>(row)[e] = __float2bfloat16_rn(x);
  else reinterpret_cast<float*>(row)[e] = x;
}
template <int DT>
__device__ __forceinline__ void copy_logit(unsigned char* to, const unsigned char* from, int e) {
  if constexpr (DT == SPEC_BF16) reinterpret_cast<uint16_t*>(to)[e] = reinterpret_cast<const uint16_t*>(from)[e];
  else reinterpret_cast<uint32_t*>(to)[e] = reinterpret_cast<const uint32_t*>(from)[e];
}

struct AdjustShared {
  uint32_t count[kRange];
  float bias[kRange];
  uint32_t biased[kRange / 32];
  int draft[SPEC_MAX_G + 1];
  int bad;
};

template <int DT>
__global__ void __launch_bounds__(kAdjustThreads) adjust_kernel(const AdjustParams P, int splits) {
  extern __shared__ __align__(16) unsigned char adjust_smem[];
  AdjustShared& S = *reinterpret_cast<AdjustShared*>(adjust_smem);
  const int b = blockIdx.x / splits, part = blockIdx.x % splits, t = threadIdx.x;
  const int lo = part * kRange, hi = min(P.V, lo + kRange);

  if (t == 0) S.bad = 0;
  for (int e = t; e < kRange; e += kAdjustThreads) { S.count[e] = 0; S.bias[e] = 0.f; }
  for (int e = t; e < kRange / 32; e += kAdjustThreads) S.biased[e] = 0;
  __syncthreads();

  int bad = 0;
  const int len = P.history_len ? P.history_len[b] : P.L, prompt = P.prompt_len ? P.prompt_len[b] : 0;
  if (len < 0 || len > P.L || prompt < 0 || prompt > len) bad |= SPEC_ST_BAD_LENGTH;
  else {
    const int32_t* h = P.history + (size_t)b * P.L;
    for (int e = t; e < len; e += kAdjustThreads) {
      const int v = h[e];
      if (v < -1 || v >= P.V) bad |= SPEC_ST_BAD_TOKEN;
      else if (v >= lo && v < hi) {
        if (e < prompt) atomicOr(&S.count[v - lo], kInPrompt);
        else atomicAdd(&S.count[v - lo], 1u);
      }
    }
  }
  const int most = P.D > 0 ? P.D : P.R - 1;
  int gamma = P.gamma ? P.gamma[b] : most;
  if (gamma < 0 || gamma > most) { bad |= SPEC_ST_BAD_GAMMA; gamma = most; }
  if (t < P.D) {
    const int v = t < gamma ? P.draft[(size_t)b * P.D + t] : -1;
    if (v < -1 || v >= P.V) bad |= SPEC_ST_BAD_TOKEN;
    S.draft[t] = v;
  }
  const float rep = P.repetition ? P.repetition[b] : 1.f, freq = P.frequency ? P.frequency[b] : 0.f,
              pres = P.presence ? P.presence[b] : 0.f;
  if (!(rep > 0.f) || !isfinite(rep) || !isfinite(freq) || !isfinite(pres)) bad |= SPEC_ST_BAD_PENALTY;
  if (t < 32) {
    // biases of one token are added in the order of the list: a warp takes 32 at a
    // time, the first lane of a token its sum
    for (int e0 = 0; e0 < P.biases; e0 += 32) {
      const int e = e0 + t;
      int v = -1;
      float x = 0.f;
      if (e < P.biases) {
        v = P.bias_index[(size_t)b * P.biases + e];
        x = P.bias_value[(size_t)b * P.biases + e];
        if (v < -1 || v >= P.V) bad |= SPEC_ST_BAD_TOKEN;
        if (v != -1 && !(x < INFINITY)) bad |= SPEC_ST_BAD_PENALTY;
      }
      const bool mine = v >= lo && v < hi;
      const uint32_t same = __match_any_sync(0xffffffffu, v);
      float sum = mine ? S.bias[v - lo] : 0.f;
      for (int k = 0; k < 32; ++k) {
        const float y = __shfl_sync(0xffffffffu, x, k);
        if (same >> k & 1) sum += y;
      }
      if (mine && (same & ((1u << t) - 1)) == 0) {
        S.bias[v - lo] = sum;
        atomicOr(&S.biased[(v - lo) >> 5], 1u << ((v - lo) & 31));
      }
      __syncwarp();
    }
  }
  if (bad) atomicOr(&S.bad, bad);
  __syncthreads();
  bad = S.bad;
  if (part == 0 && t == 0 && P.status) P.status[b] = bad;

  const int W = (P.V + 31) / 32, rows = min(P.R, gamma + 1);
  constexpr int ES = RowType<DT>::ES;
  for (int i = 0; i < rows; ++i) {
    const size_t r = (size_t)b * P.R + i;
    const unsigned char* in = P.in + r * P.V * ES;
    unsigned char* out = P.out + r * P.V * ES;
    for (int v = lo + t; v < hi; v += kAdjustThreads) {
      uint32_t c = S.count[v - lo];
      if (!bad) {
        for (int j = 0; j < i && j < P.D; ++j) c += S.draft[j] == v;
        if (P.mask && !(P.mask[r * W + (v >> 5)] >> (v & 31) & 1)) {
          put_logit<DT>(out, v, -INFINITY);
          continue;
        }
        const bool biased = S.biased[(v - lo) >> 5] >> ((v - lo) & 31) & 1;
        if (c != 0 || biased) {
          float x = row_logit<DT>(in, v);
          if (c != 0) {
            x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
            c &= ~kInPrompt;
            if (c != 0) x -= __fmaf_rn((float)c, freq, pres);
          }
          if (biased) x += S.bias[v - lo];
          put_logit<DT>(out, v, x);
          continue;
        }
      }
      if (out != in) copy_logit<DT>(out, in, v);
    }
  }
}

}  // namespace

cudaError_t configure_adjust() {
  const int smem = (int)sizeof(AdjustShared);
  cudaError_t e = cudaFuncSetAttribute(adjust_kernel<SPEC_BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(adjust_kernel<SPEC_F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e;
}

cudaError_t launch_adjust(const AdjustParams& P, int, cudaStream_t s) {
  const int splits = (P.V + kRange - 1) / kRange;
  const dim3 grid((unsigned)(splits * P.B));
  if (P.dtype == SPEC_BF16) adjust_kernel<SPEC_BF16><<<grid, kAdjustThreads, sizeof(AdjustShared), s>>>(P, splits);
  else adjust_kernel<SPEC_F32><<<grid, kAdjustThreads, sizeof(AdjustShared), s>>>(P, splits);
  return cudaGetLastError();
}

}  // namespace sv
