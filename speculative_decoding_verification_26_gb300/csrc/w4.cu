// w4.cu -- weights in 4 bits with a scale for each group, and read back.
//
// A row of H weights is cut into groups of 32, 64 or 128 (the last may be shorter).
// A group has a scale s (bf16) and a zero point z (0 to 15; 8 without zero points),
// and a weight is (q - z) s with q from 0 to 15.
//
// Both kernels read and write each value once: HBM bounds them, and the instructions
// of a weight come next (4 for a bf16 weight, from its bits to its place in a word).  A
// warp takes kRows rows, 32 words of 8 weights of each at a time, so that their loads are
// on their way together.
#include "rows.cuh"
#include "serve.cuh"

namespace sv {
namespace {

constexpr int kW4Threads = 256;

// ---------------------------------------------------------------------------
// the quotient w / s as a whole number, halves to even

// Any w and s > 0; inv is near 1 / s.  The product w inv is off by a part in 2^22, so the
// neighbour is right but next to a half, where the remainder decides: it is exact (w and s q
// share their grid of bits).
__device__ __noinline__ float whole_quotient(float w, float s, float inv) {
  float q = rintf(w * inv);
  const float e = __fmaf_rn(-q, s, w), half = 0.5f * s;
  if (fabsf(e) >= half && (fabsf(e) > half || ((int)q & 1))) q += copysignf(1.f, e);
  return q;
}
// |w / s| <= 16: rounded to the grid of 2^-16 at 192, then to whole numbers at kMagic, whose last
// bits they are.  For bf16 w and s a quotient that is no half is at least 2^-13 from one (w and
// (k + 1/2) s have at most 12 bits), and a half lands on the grid exactly: the whole numbers are
// those of the exact quotient.
constexpr float kMagic = 12582912.f;         // 1.5 2^23
constexpr uint32_t kMagicBits = 0x4B400000u;
__device__ __forceinline__ float on_grid(float w, float inv) { return __fmaf_rn(w, inv, 192.f); }
__device__ __forceinline__ float at_magic(float grid) { return __fadd_rn(grid, kMagic - 192.f); }
// fp32 weights can be next to a half without being one: within 2^-14 the remainder decides
__device__ __forceinline__ bool near_half(float grid, float magic) {
  return fabsf(__fadd_rn(grid, -__fadd_rn(magic, -(kMagic - 192.f)))) > 0.5f - 1.f / 16384;
}

// a / d for d = 7 or 15, rounded to nearest: the remainder a - q d is exact, and a quotient by
// 7 or 15 that is no tie is 1/30 of a unit in the last place from one at least, where the
// correction is good to 2^-24 of it.  Not for a near the smallest numbers.
template <int D>
__device__ __forceinline__ float over(float a, float more = 0.f) {
  constexpr float c = 1.f / D;
  const float q = a * c;
  return __fmaf_rn(__fmaf_rn(-q, (float)D, a) + more, c, q);
}

// 8 weights in place k8 of a row
template <int DT>
struct Eight {
  uint4 v[DT == SPEC_BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const unsigned char* row, int k8) {
    const uint4* p = reinterpret_cast<const uint4*>(row) + (size_t)k8 * (DT == SPEC_BF16 ? 1 : 2);
#pragma unroll
    for (uint4& x : v)
      asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                   : "l"(p++));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint4& x : v) x = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (DT == SPEC_BF16) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
      return j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
    } else {
      const uint4& x = v[j / 4];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      return __uint_as_float(w[j & 3]);
    }
  }
  // the largest magnitude as bits of fp32, which order like the numbers, infinities and NaN above all
  __device__ __forceinline__ uint32_t most() const {
    if constexpr (DT == SPEC_BF16) {
      const uint32_t m = 0x7FFF7FFFu;
      const uint32_t t = __vmaxu2(__vmaxu2(v[0].x & m, v[0].y & m), __vmaxu2(v[0].z & m, v[0].w & m));
      return max(t << 16, t & 0xFFFF0000u);
    } else {
      uint32_t t = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) t = max(t, __float_as_uint(at(j)) & 0x7FFFFFFFu);
      return t;
    }
  }
};

// A group's scale, zero point and reciprocal; LANES lanes hold it.
struct Group {
  float s, zero, inv, up;                    // up: what weights and scale are multiplied by first
  bool none, odd, slow;                      // no scale; NaN or infinities; not for the quick way
};
template <int DT, int LANES, bool ZERO>
__device__ __forceinline__ Group group_of(const Eight<DT>& w) {
  Group g;
  uint32_t most = w.most();
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
  g.odd = most >= 0x7F800000u;
  const float big = __uint_as_float(most);
  const bool plain = big > 1e-25f && big < 1e37f;
  float lo = 0.f, hi = 0.f, s;
  if constexpr (ZERO) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo = fminf(lo, w.at(j));
      hi = fmaxf(hi, w.at(j));
    }
#pragma unroll
    for (int off = LANES / 2; off >= 1; off >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    // (hi - lo) / 15 rounded to fp32 from the whole difference d + err
    const float down = plain ? 1.f : big < 1e37f ? 1.f : 1.f / 256, a = hi * down, b = -lo * down;       // no overflow
    const float d = a + b, back = d - a, err = (a - (d - back)) + (b - back);
    if (plain) {
      s = over<15>(d, err);
    } else {
      const float q = __fdiv_rn(d, 15.f);
      s = (q + (__fmaf_rn(-q, 15.f, d) + err) / 15.f) * (1.f / down);
    }
  } else {
    s = plain ? over<7>(big) : __fdiv_rn(big, 7.f);
  }
  s = __bfloat162float(__float2bfloat16_rn(s));
  g.none = !(s > 0.f) || !(s < INFINITY) || g.odd;
  // scales whose reciprocal would overflow: everything times 2^64
  g.up = s < 1e-30f ? 18446744073709551616.f : 1.f;
  g.slow = !plain || g.none;
  g.s = s;
  g.inv = g.none ? 0.f : __frcp_rn(s * g.up);
  g.zero = 8.f;
  if constexpr (ZERO) {
    if (!g.none) {
      const float grid = on_grid(-lo, g.inv), m = at_magic(grid);
      g.zero = fminf(g.slow || (DT == SPEC_F32 && near_half(grid, m)) ? whole_quotient(-lo * g.up, s * g.up, g.inv) : m - kMagic, 15.f);
    }
  }
  return g;
}

// A warp takes ROWS rows, LANES lanes a group, a lane 8 weights.
template <int DT, int LANES, bool ZERO, int ROWS>
__global__ void __launch_bounds__(kW4Threads) quantize_kernel(const __grid_constant__ W4Params P) {
  constexpr int PER = 32 / LANES, ES = RowType<DT>::ES;
  const int lane = threadIdx.x & 31, words = P.H / 8;
  const long long v0 = (blockIdx.x * (long long)(kW4Threads / 32) + (threadIdx.x >> 5)) * ROWS;
  if (v0 >= P.V) return;
  const int rows = (int)min((long long)ROWS, P.V - v0);
  bool bad[ROWS] = {};
  for (int g0 = 0; g0 < P.groups; g0 += PER) {
    const int g = g0 + lane / LANES, k = g0 * LANES + lane;
    const bool live = k < words;
    Eight<DT> w[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (live && r < rows) w[r].load(P.weight + (v0 + r) * P.H * ES, k);
      else w[r].zero();
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const Group G = group_of<DT, LANES, ZERO>(w[r]);
      uint32_t word = 0;
      bool slow = G.slow;
      // sum of (kMagicBits + n) << 4 p, and of z - kMagicBits: (n + z) << 4 p
      const float least = kMagic - G.zero, most = kMagic + 15.f - G.zero;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float grid = on_grid(w[r].at(j), G.inv);
        float m = at_magic(grid);
        if constexpr (DT == SPEC_F32) slow |= near_half(grid, m);
        if constexpr (ZERO) m = fminf(fmaxf(m, least), most);
        word += __float_as_uint(m) << 4 * nibble_of(j);
      }
      word += ((uint32_t)(int)G.zero - kMagicBits) * 0x11111111u;
      if (__any_sync(0xffffffffu, slow)) {
        if (slow) {
          word = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float q = G.none ? G.zero : fminf(fmaxf(whole_quotient(w[r].at(j) * G.up, G.s * G.up, G.inv) + G.zero, 0.f), 15.f);
            word |= (uint32_t)q << 4 * nibble_of(j);
          }
        }
      }
      if (live && r < rows) {
        P.packed[(v0 + r) * words + k] = word;
        if (lane % LANES == 0) {
          P.scale[(v0 + r) * P.groups + g] = __float2bfloat16_rn(G.odd ? NAN : G.s);
          if (ZERO) P.zero[(v0 + r) * P.groups + g] = (uint8_t)G.zero;
        }
        bad[r] |= G.odd;
      }
    }
  }
  if (P.status) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const bool any = __any_sync(0xffffffffu, bad[r]);
      if (lane == 0 && r < rows) P.status[v0 + r] = any ? SPEC_ST_NONFINITE : SPEC_ST_OK;
    }
  }
}

// ---------------------------------------------------------------------------
// read back: exact whole numbers times the scale, rounded once

template <int DT, bool ZERO, int ROWS>
__global__ void __launch_bounds__(kW4Threads) dequantize_kernel(const __grid_constant__ W4Params P, int log_per) {
  const int lane = threadIdx.x & 31, words = P.H / 8;
  const long long v0 = (blockIdx.x * (long long)(kW4Threads / 32) + (threadIdx.x >> 5)) * ROWS;
  if (v0 >= P.V) return;
  const int rows = (int)min((long long)ROWS, P.V - v0);
  for (int k = lane; k < words; k += 32) {
    const int g = k >> log_per;
    uint32_t word[ROWS], s[ROWS], z[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long long v = v0 + (r < rows ? r : 0);
      word[r] = __ldg(P.packed + v * words + k);
      s[r] = __ldg(reinterpret_cast<const uint16_t*>(P.scale) + v * P.groups + g);
      z[r] = ZERO ? __ldg(P.zero + v * P.groups + g) : 8u;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (r >= rows) continue;
      uint32_t q[4];
      unpack8(q, word[r], less_of(z[r]));
      if constexpr (DT == SPEC_BF16) {
        const uint32_t both = s[r] * 0x10001u;
        uint4 o;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.x) : "r"(q[0]), "r"(both));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.y) : "r"(q[1]), "r"(both));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.z) : "r"(q[2]), "r"(both));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.w) : "r"(q[3]), "r"(both));
        reinterpret_cast<uint4*>(P.out)[(v0 + r) * words + k] = o;
      } else {
        const float f = __uint_as_float(s[r] << 16);
        float4* o = reinterpret_cast<float4*>(P.out) + 2 * ((v0 + r) * words + k);
        o[0] = make_float4(bf16_lo(q[0]) * f, bf16_hi(q[0]) * f, bf16_lo(q[1]) * f, bf16_hi(q[1]) * f);
        o[1] = make_float4(bf16_lo(q[2]) * f, bf16_hi(q[2]) * f, bf16_lo(q[3]) * f, bf16_hi(q[3]) * f);
      }
    }
  }
}

// Rows of a warp: as many as leave every SM 16 warps.
template <int MOST>
bool few(int V, int nsm) { return V < 16ll * nsm * MOST; }
int blocks(int V, int rows) { return (int)((V + (kW4Threads / 32) * (long long)rows - 1) / (kW4Threads / 32 * rows)); }

template <int DT, int LANES, bool ZERO>
void quantize(const W4Params& P, int nsm, cudaStream_t s) {
  constexpr int kRows = DT == SPEC_BF16 ? 4 : 2;
  if (few<kRows>(P.V, nsm)) quantize_kernel<DT, LANES, ZERO, 1><<<blocks(P.V, 1), kW4Threads, 0, s>>>(P);
  else quantize_kernel<DT, LANES, ZERO, kRows><<<blocks(P.V, kRows), kW4Threads, 0, s>>>(P);
}
template <int LANES>
void quantize_of(const W4Params& P, int nsm, cudaStream_t s) {
  if (P.dtype == SPEC_BF16) P.zero ? quantize<SPEC_BF16, LANES, true>(P, nsm, s) : quantize<SPEC_BF16, LANES, false>(P, nsm, s);
  else P.zero ? quantize<SPEC_F32, LANES, true>(P, nsm, s) : quantize<SPEC_F32, LANES, false>(P, nsm, s);
}
template <int DT, bool ZERO>
void dequantize(const W4Params& P, int nsm, cudaStream_t s) {
  const int log_per = P.group == 128 ? 4 : P.group == 64 ? 3 : 2;
  if (few<4>(P.V, nsm)) dequantize_kernel<DT, ZERO, 1><<<blocks(P.V, 1), kW4Threads, 0, s>>>(P, log_per);
  else dequantize_kernel<DT, ZERO, 4><<<blocks(P.V, 4), kW4Threads, 0, s>>>(P, log_per);
}

}  // namespace

cudaError_t launch_w4_quantize(const W4Params& P, int nsm, cudaStream_t s) {
  if (P.group == 128) quantize_of<16>(P, nsm, s);
  else if (P.group == 64) quantize_of<8>(P, nsm, s);
  else quantize_of<4>(P, nsm, s);
  return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(const W4Params& P, int nsm, cudaStream_t s) {
  if (P.dtype == SPEC_BF16) P.zero ? dequantize<SPEC_BF16, true>(P, nsm, s) : dequantize<SPEC_BF16, false>(P, nsm, s);
  else P.zero ? dequantize<SPEC_F32, true>(P, nsm, s) : dequantize<SPEC_F32, false>(P, nsm, s);
  return cudaGetLastError();
}

}  // namespace sv
