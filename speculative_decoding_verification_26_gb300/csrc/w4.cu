// w4.cu -- weights in 4 bits with a scale for each group, and read back.
//
// A row of H weights is cut into groups of 32, 64 or 128 (the last may be shorter).
// A group has a scale s (bf16) and a zero point z (0 to 15; 8 without zero points),
// and a weight is (q - z) s with q from 0 to 15.
#include "rows.cuh"
#include "serve.cuh"

namespace sv {
namespace {

constexpr int kW4Threads = 256;

// the nearest whole number to w / s, halves to even, s > 0; inv is near 1 / s.  The
// product w inv is off by a part in 2^22, so the quotient's neighbour is right but next to a
// half, where the remainder decides: it is exact (w and s q share their grid of bits).
__device__ __forceinline__ float whole_quotient(float w, float s, float inv) {
  float q = rintf(w * inv);
  const float e = __fmaf_rn(-q, s, w), half = 0.5f * s;
  if (fabsf(e) >= half && (fabsf(e) > half || ((int)q & 1))) q += copysignf(1.f, e);
  return q;
}

template <int DT>
__device__ __forceinline__ void load8(float (&w)[8], const unsigned char* p) {
  if constexpr (DT == SPEC_BF16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = vec_pair<SPEC_BF16>(v, k);
      w[2 * k] = f.x;
      w[2 * k + 1] = f.y;
    }
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}

// A warp takes a row, LANES lanes a group, a lane 8 weights.
template <int DT, int LANES>
__global__ void __launch_bounds__(kW4Threads) quantize_kernel(const W4Params P) {
  constexpr int PER = 32 / LANES, ES = RowType<DT>::ES;
  const int lane = threadIdx.x & 31, at = lane / LANES, in = lane % LANES;
  const int words = P.H / 8;
  for (long long v = (blockIdx.x * (long long)kW4Threads + threadIdx.x) / 32; v < P.V; v += gridDim.x * (kW4Threads / 32ll)) {
    const unsigned char* row = P.weight + v * P.H * ES;
    bool bad = false;
    for (int g0 = 0; g0 < P.groups; g0 += PER) {
      const int g = g0 + at, k = g * LANES + in;
      const bool live = g < P.groups && k < words;
      float w[8] = {};
      if (live) load8<DT>(w, row + (size_t)k * 8 * ES);
      float lo = 0.f, hi = 0.f;
      bool odd = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, w[j]);
        hi = fmaxf(hi, w[j]);
        odd |= !(fabsf(w[j]) < INFINITY);
      }
#pragma unroll
      for (int off = LANES / 2; off >= 1; off >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        odd |= __shfl_xor_sync(0xffffffffu, (int)odd, off) != 0;
      }
      float s, zero = 8.f;
      if (P.zero) {
        // (hi - lo) / 15 rounded to fp32 from the whole difference d + err
        const float down = hi - lo < 1e38f ? 1.f : 1.f / 256, a = hi * down, b = -lo * down;   // no overflow
        const float d = a + b, back = d - a, err = (a - (d - back)) + (b - back);
        const float q = __fdiv_rn(d, 15.f);
        s = (q + (__fmaf_rn(-q, 15.f, d) + err) / 15.f) * (1.f / down);
      } else {
        s = __fdiv_rn(fmaxf(hi, -lo), 7.f);
      }
      const __nv_bfloat16 sb = __float2bfloat16_rn(s);
      s = __bfloat162float(sb);
      const bool none = !(s > 0.f) || !(s < INFINITY) || odd;
      // scales whose reciprocal would overflow: everything times 2^64
      const float up = s < 1e-30f ? 18446744073709551616.f : 1.f, ss = s * up, inv = none ? 0.f : 1.f / ss;
      if (P.zero && !none) zero = fminf(whole_quotient(-lo * up, ss, inv), 15.f);
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = none ? zero : fminf(fmaxf(whole_quotient(w[j] * up, ss, inv) + zero, 0.f), 15.f);
        word |= (uint32_t)q << 4 * nibble_of(j);
      }
      if (live) P.packed[v * words + k] = word;
      if (live && in == 0) {
        P.scale[v * P.groups + g] = odd ? __float2bfloat16_rn(NAN) : sb;
        if (P.zero) P.zero[v * P.groups + g] = (uint8_t)zero;
      }
      bad |= odd;
    }
    if (P.status) {
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) P.status[v] = bad ? SPEC_ST_NONFINITE : SPEC_ST_OK;
    }
  }
}

__device__ __forceinline__ float weight_of(uint32_t word, int j, float z) {
  return (float)(int)(word >> 4 * nibble_of(j) & 15u) - z;
}

template <int DT>
__global__ void __launch_bounds__(kW4Threads) dequantize_kernel(const W4Params P) {
  const int lane = threadIdx.x & 31, words = P.H / 8, per = P.group / 8;
  for (long long v = (blockIdx.x * (long long)kW4Threads + threadIdx.x) / 32; v < P.V; v += gridDim.x * (kW4Threads / 32ll)) {
    for (int k = lane; k < words; k += 32) {
      const int g = k / per;
      const uint32_t word = P.packed[v * words + k];
      const float s = __bfloat162float(P.scale[v * P.groups + g]), z = P.zero ? (float)P.zero[v * P.groups + g] : 8.f;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = weight_of(word, j, z) * s;
      if constexpr (DT == SPEC_BF16) {
        uint4 o;
        uint32_t* u = &o.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
          memcpy(u + j, &p, 4);
        }
        reinterpret_cast<uint4*>(P.out)[v * words + k] = o;
      } else {
        float4* o = reinterpret_cast<float4*>(P.out) + 2 * (v * words + k);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
  }
}

int row_grid(int V, int nsm) {
  const long long most = 8ll * nsm, need = (V + kW4Threads / 32 - 1) / (kW4Threads / 32);
  return (int)(need < most ? need : most);
}

template <int LANES>
void quantize(const W4Params& P, int grid, cudaStream_t s) {
  if (P.dtype == SPEC_BF16) quantize_kernel<SPEC_BF16, LANES><<<grid, kW4Threads, 0, s>>>(P);
  else quantize_kernel<SPEC_F32, LANES><<<grid, kW4Threads, 0, s>>>(P);
}

}  // namespace

cudaError_t launch_w4_quantize(const W4Params& P, int nsm, cudaStream_t s) {
  const int grid = row_grid(P.V, nsm);
  if (P.group == 128) quantize<16>(P, grid, s);
  else if (P.group == 64) quantize<8>(P, grid, s);
  else quantize<4>(P, grid, s);
  return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(const W4Params& P, int nsm, cudaStream_t s) {
  const int grid = row_grid(P.V, nsm);
  if (P.dtype == SPEC_BF16) dequantize_kernel<SPEC_BF16><<<grid, kW4Threads, 0, s>>>(P);
  else dequantize_kernel<SPEC_F32><<<grid, kW4Threads, 0, s>>>(P);
  return cudaGetLastError();
}

}  // namespace sv
