// serve.cuh -- parameters and launches of the calls around the vocabulary rows
// of a decode step (w4.cu, adjust.cu), and what their host side (api_serve.cu)
// takes from api.cu.
#pragma once

#include "common.cuh"

namespace sv {

// ---------------------------------------------------------------------------
// 4-bit weights: row v of packed holds H / 8 words of 32 bits, word j the weights
// 8 j .. 8 j + 7 of the row, weight 8 j + i in bits 4 nibble_of(i) on, so that
// (word >> 4 p) & 0x000F000F are the weights 2 p and 2 p + 1, in the halves of a
// pair of 16-bit values.
__host__ __device__ constexpr int nibble_of(int i) { return (i >> 1) + 4 * (i & 1); }

// 128 + z as bf16 in both halves
__device__ __forceinline__ uint32_t less_of(uint32_t z) { return (0x4300u | z) * 0x10001u; }
// a word of 8 weights as bf16 pairs of q - z; less = less_of(z).  128 + q is q in the last bits of
// the mantissa; the difference is exact.
__device__ __forceinline__ void unpack8(uint32_t* out, uint32_t word, uint32_t less) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
    asm("{\n .reg .b32 u;\n lop3.b32 u, %1, 0x000F000F, 0x43004300, 0xEA;\n sub.rn.bf16x2 %0, u, %2;\n}\n"
        : "=r"(out[p])
        : "r"(word >> 4 * p), "r"(less));
}


struct W4Params {
  const unsigned char* weight;   // quantise: [V, H] of `dtype`
  int dtype, n, H, V, group, groups;     // groups of a row
  uint32_t* packed;              // [V, H / 8]
  __nv_bfloat16* scale;          // [V, groups]
  uint8_t* zero;                 // [V, groups] or null (8)
  int32_t* status;               // quantise: [V] or null
  void* out;                     // dequantise: [V, H] of `dtype`; product: [n, V] of `dtype`
  const __nv_bfloat16* hidden;   // product: [n, H]
  long long wait_limit;          // as Params::wait_limit
};
cudaError_t launch_w4_quantize(const W4Params& P, int nsm, cudaStream_t s);
cudaError_t launch_w4_dequantize(const W4Params& P, int nsm, cudaStream_t s);
cudaError_t configure_w4();            // shared-memory limits, the tensor-map encoder
cudaError_t launch_w4_linear(const W4Params& P, int nsm, cudaStream_t s);

// ---------------------------------------------------------------------------
// logit rows adjusted

struct AdjustParams {
  const unsigned char* in;       // [B, R, V]
  unsigned char* out;            // the same, or `in` itself
  int dtype, B, R, V;
  const int32_t* history;        // [B, L]
  const int32_t* history_len;    // [B] or null (= L)
  const int32_t* prompt_len;     // [B] or null (= 0)
  int L;
  const int32_t* draft;          // [B, D] or null
  const int32_t* gamma;          // [B] or null (= D)
  int D;
  const float *repetition, *frequency, *presence;   // [B] or null
  const int32_t* bias_index;     // [B, biases]
  const float* bias_value;
  int biases;
  const uint32_t* mask;          // [B, R, ceil(V / 32)] or null
  int32_t* status;               // [B] or null
};
cudaError_t configure_adjust();
cudaError_t launch_adjust(const AdjustParams& P, int nsm, cudaStream_t s);

// ---------------------------------------------------------------------------
// from api.cu

int current_device(int* dev, int* sms);      // checked to run the library's code
void count_launches(int n);                  // of this host thread
long long current_wait_limit();

}  // namespace sv
