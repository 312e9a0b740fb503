// w4.cu -- weights in 4 bits with a scale for each group, and read back.
//
// A row of H weights is cut into groups of 32, 64 or 128 (the last may be shorter).
// A group has a scale s (bf16) and a zero point z (0 to 15; 8 without zero points),
// and a weight is (q - z) s with q from 0 to 15.
//
// Both kernels read and write each value once: HBM bounds them, and the instructions
// of a weight come next (4 for a bf16 weight, from its bits to its place in a word).  A
// warp takes several rows, or several stretches of one, so that their loads are on their way
// together.  Lanes behind the end of a row that is no multiple of 256 weights hold zeros, for which the
// warp goes the slow way of a scale of 0: 151936 x 1184 bf16 weights in groups of 128 take 89 us (67 by
// their bytes).  151936 x 2048 bf16 weights, groups of 128: 131 us (6.0 TB/s), issue 69 % busy, and 120
// us back (6.5 TB/s).
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

// a / d for d = 7 or 15, rounded to nearest, by one correction of a near quotient with its remainder
// (Markstein 1990, "Computation of elementary functions"): the remainder a - q d is exact, and a quotient by
// 7 or 15 that is no tie is 1/30 of a unit in the last place from one at least, where the
// correction is good to 2^-24 of it.  Not for a near the smallest numbers.
template <int D>
__device__ __forceinline__ float over(float a, float more = 0.f) {
  constexpr float c = 1.f / D;
  const float q = a * c;
  return __fmaf_rn(__fmaf_rn(-q, (float)D, a) + more, c, q);
}

// 8 weights of a row
template <int DT>
struct Eight {
  uint32_t w[DT == SPEC_BF16 ? 4 : 8];
  __device__ __forceinline__ void load(const unsigned char* p) {
    if constexpr (DT == SPEC_BF16)
      asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
    else if (reinterpret_cast<uintptr_t>(p) & 31) {      // the same for all: rows are whole lines
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                     : "l"(p + 4 * i));
    } else                                   // 32 bytes at once: two loads would take a sector each twice
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& x : w) x = 0;
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (DT == SPEC_BF16) return j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
    else return __uint_as_float(w[j]);
  }
  // the largest magnitude as bits of fp32, which order like the numbers, infinities and NaN above all
  __device__ __forceinline__ uint32_t most() const {
    if constexpr (DT == SPEC_BF16) {
      const uint32_t m = 0x7FFF7FFFu;
      const uint32_t t = __vmaxu2(__vmaxu2(w[0] & m, w[1] & m), __vmaxu2(w[2] & m, w[3] & m));
      return max(t << 16, t & 0xFFFF0000u);
    } else {
      uint32_t t = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) t = max(t, w[j] & 0x7FFFFFFFu);
      return t;
    }
  }
};

// What the lanes of a group agree on: the largest magnitude, and with zero points the range (then
// NaN goes through all of it).
struct Range {
  uint32_t most;
  float lo, hi;
};
__device__ __forceinline__ float least(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float greatest(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t least2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t greatest2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int DT, int LANES, bool ZERO>
__device__ __forceinline__ Range range_of(const Eight<DT>& w) {
  Range r;
  r.lo = r.hi = 0.f;
  if constexpr (!ZERO) {
    r.most = w.most();
  } else if constexpr (DT == SPEC_BF16) {
    const uint32_t lo = least2(least2(w.w[0], w.w[1]), least2(w.w[2], w.w[3]));
    const uint32_t hi = greatest2(greatest2(w.w[0], w.w[1]), greatest2(w.w[2], w.w[3]));
    r.lo = least(least(bf16_lo(lo), bf16_hi(lo)), 0.f);
    r.hi = greatest(greatest(bf16_lo(hi), bf16_hi(hi)), 0.f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r.lo = least(r.lo, w.at(j));
      r.hi = greatest(r.hi, w.at(j));
    }
  }
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1) {
    if constexpr (ZERO) {
      r.lo = least(r.lo, __shfl_xor_sync(0xffffffffu, r.lo, off));
      r.hi = greatest(r.hi, __shfl_xor_sync(0xffffffffu, r.hi, off));
    } else {
      r.most = max(r.most, __shfl_xor_sync(0xffffffffu, r.most, off));
    }
  }
  if constexpr (ZERO) r.most = __float_as_uint(greatest(-r.lo, r.hi)) & 0x7FFFFFFFu;
  return r;
}
// A group's scale and zero point, and a lane's word.
struct Coded {
  float s, zero;
  uint32_t word;
};
__device__ __forceinline__ float as_bf16(float s) { return __bfloat162float(__float2bfloat16_rn(s)); }

// Any group: magnitudes near the ends of fp32's range, scales of 0, NaN and infinities, quotients
// of fp32 weights next to a half.
template <int DT, bool ZERO>
__device__ __noinline__ Coded code_slowly(const Eight<DT> w, const Range r) {
  Coded c;
  const bool odd = r.most >= 0x7F800000u;
  c.zero = 8.f;
  if constexpr (ZERO) {
    // (hi - lo) / 15 rounded to fp32 from the whole difference d + err, without overflow
    const float down = __uint_as_float(r.most) < 1e37f ? 1.f : 1.f / 256, a = r.hi * down, b = -r.lo * down;
    const float d = a + b, back = d - a, err = (a - (d - back)) + (b - back), q = __fdiv_rn(d, 15.f);
    c.s = (q + (__fmaf_rn(-q, 15.f, d) + err) / 15.f) * (1.f / down);
  } else {
    c.s = __fdiv_rn(__uint_as_float(r.most), 7.f);
  }
  c.s = as_bf16(c.s);
  const bool none = !(c.s > 0.f) || !(c.s < INFINITY) || odd;
  // scales whose reciprocal would overflow: everything times 2^64
  const float up = c.s < 1e-30f ? 18446744073709551616.f : 1.f, s = c.s * up, inv = 1.f / s;
  if (ZERO && !none) c.zero = fminf(whole_quotient(-r.lo * up, s, inv), 15.f);
  c.word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = none ? c.zero : fminf(fmaxf(whole_quotient(w.at(j) * up, s, inv) + c.zero, 0.f), 15.f);
    c.word |= (uint32_t)q << 4 * nibble_of(j);
  }
  if (odd) c.s = NAN;
  return c;
}
// The others, 4 instructions a weight; false where the slow way has to be taken.
template <int DT, bool ZERO>
__device__ __forceinline__ bool code_quickly(const Eight<DT>& w, const Range& r, Coded& c) {
  const float big = __uint_as_float(r.most);
  bool quick = big > 1e-25f && big < 1e37f;
  if constexpr (ZERO) {
    const float b = -r.lo, d = r.hi + b, back = d - r.hi, err = (r.hi - (d - back)) + (b - back);
    c.s = over<15>(d, err);
  } else {
    c.s = over<7>(big);
  }
  c.s = as_bf16(c.s);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(c.s));
  c.zero = 8.f;
  if constexpr (ZERO) {
    const float grid = on_grid(-r.lo, inv), m = at_magic(grid);
    if constexpr (DT == SPEC_F32) quick = quick && !near_half(grid, m);
    c.zero = fminf(m - kMagic, 15.f);
  }
  // the sum of (kMagicBits + n) << 4 p, and of z - kMagicBits: (n + z) << 4 p.  With zero points n + z can be
  // 16, both rounded up, but not less than 0: of the least weight it is 0 (n = -z; -lo / s <= 15 (1 + 2^-8)
  // is rounded to 15 at most), and n does not fall with the weight.
  const float most = kMagic + 15.f - c.zero;
  uint32_t word = ZERO ? ((uint32_t)(int)c.zero - kMagicBits) * 0x11111111u : (8u - kMagicBits) * 0x11111111u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float grid = on_grid(w.at(j), inv);
    float m = at_magic(grid);
    if constexpr (DT == SPEC_F32) quick = quick && !near_half(grid, m);
    if constexpr (ZERO) m = fminf(m, most);
    word += __float_as_uint(m) << 4 * nibble_of(j);
  }
  c.word = word;
  return quick;
}

// A warp takes ROWS rows, COLS times 32 words of each at a time; LANES lanes a group, a lane 8 weights.
template <int DT, int LANES, bool ZERO, int ROWS, int COLS>
__global__ void __launch_bounds__(kW4Threads) quantize_kernel(const __grid_constant__ W4Params P) {
  constexpr int PER = 32 / LANES, BYTES = 8 * RowType<DT>::ES;
  const int lane = threadIdx.x & 31, words = P.H / 8;
  const long long v0 = (blockIdx.x * (long long)(kW4Threads / 32) + (threadIdx.x >> 5)) * ROWS;
  if (v0 >= P.V) return;
  const int rows = (int)min((long long)ROWS, P.V - v0);
  const unsigned char* from = P.weight + (v0 * words + lane) * BYTES;
  uint32_t* to = P.packed + v0 * words + lane;
  const long long at = v0 * P.groups + lane / LANES;
  const bool leads = lane % LANES == 0;
  uint32_t bad = 0;                          // a bit a row
  for (int g0 = 0; g0 < P.groups; g0 += PER * COLS, from += COLS * 32 * BYTES, to += COLS * 32) {
    Eight<DT> w[ROWS][COLS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        w[r][c].zero();
        if (g0 * LANES + c * 32 + lane < words && r < rows) w[r][c].load(from + (size_t)(r * words + c * 32) * BYTES);
      }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        if (COLS > 1 && g0 + c * PER >= P.groups) break;
        const bool live = g0 * LANES + c * 32 + lane < words;
        const Range range = range_of<DT, LANES, ZERO>(w[r][c]);
        Coded code;
        const bool quick = code_quickly<DT, ZERO>(w[r][c], range, code);
        // (the lanes of a group agree on its scale and zero point whichever way they take)
        if (!__all_sync(0xffffffffu, quick)) {
          if (!quick) code = code_slowly<DT, ZERO>(w[r][c], range);
          if (live && range.most >= 0x7F800000u) bad |= 1u << r;
        }
        if (live && r < rows) {
          to[r * words + c * 32] = code.word;
          if (leads) {
            const long long o = at + g0 + c * PER + (long long)r * P.groups;
            P.scale[o] = __float2bfloat16_rn(code.s);
            if (ZERO) P.zero[o] = (uint8_t)code.zero;
          }
        }
      }
  }
  if (P.status) {
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane < rows) P.status[v0 + lane] = bad >> lane & 1 ? SPEC_ST_NONFINITE : SPEC_ST_OK;
  }
}

// ---------------------------------------------------------------------------
// read back: exact whole numbers times the scale, rounded once

template <int DT, bool ZERO, int ROWS, int COLS>
__global__ void __launch_bounds__(kW4Threads) dequantize_kernel(const __grid_constant__ W4Params P, int log_per) {
  constexpr int EACH = DT == SPEC_BF16 ? 1 : 2;          // lanes a word: a lane writes 16 bytes
  const int lane = threadIdx.x & 31, words = P.H / 8;
  const long long v0 = (blockIdx.x * (long long)(kW4Threads / 32) + (threadIdx.x >> 5)) * ROWS;
  if (v0 >= P.V) return;
  const int rows = (int)min((long long)ROWS, P.V - v0);
  for (int k0 = lane; k0 < words * EACH; k0 += 32 * COLS) {
    uint32_t word[ROWS][COLS], s[ROWS][COLS], z[ROWS][COLS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        const long long v = v0 + (r < rows ? r : 0);
        const int at = min(k0 + 32 * c, words * EACH - 1) / EACH, g = at >> log_per;
        word[r][c] = __ldg(P.packed + v * words + at);
        s[r][c] = __ldg(reinterpret_cast<const uint16_t*>(P.scale) + v * P.groups + g);
        z[r][c] = ZERO ? __ldg(P.zero + v * P.groups + g) : 8u;
      }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        const int k = k0 + 32 * c;
        if (r >= rows || (COLS > 1 && k >= words * EACH)) continue;
        uint32_t q[4];
        uint4 o;
        if constexpr (DT == SPEC_BF16) {
          unpack8(q, word[r][c], less_of(z[r][c]));
          const uint32_t both = s[r][c] * 0x10001u;
          asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.x) : "r"(q[0]), "r"(both));
          asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.y) : "r"(q[1]), "r"(both));
          asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.z) : "r"(q[2]), "r"(both));
          asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.w) : "r"(q[3]), "r"(both));
        } else {
          unpack8(q, word[r][c] >> (k & 1) * 8, less_of(z[r][c]));       // the pairs 0 and 1, or 2 and 3
          const float f = __uint_as_float(s[r][c] << 16);
          o = make_uint4(__float_as_uint(bf16_lo(q[0]) * f), __float_as_uint(bf16_hi(q[0]) * f), __float_as_uint(bf16_lo(q[1]) * f),
                         __float_as_uint(bf16_hi(q[1]) * f));
        }
        reinterpret_cast<uint4*>(P.out)[(v0 + r) * words * EACH + k] = o;
      }
  }
}

// A warp takes kRows rows at once where that leaves every SM 16 warps, else as much of one row.
template <int MOST>
bool few(int V, int nsm) { return V < 16ll * nsm * MOST; }
int blocks(int V, int rows) { return (int)((V + (kW4Threads / 32) * (long long)rows - 1) / (kW4Threads / 32 * rows)); }

template <int DT, int LANES, bool ZERO>
void quantize(const W4Params& P, int nsm, cudaStream_t s) {
  constexpr int kRows = DT == SPEC_BF16 ? 4 : 2;
  // fp32 with zero points goes by stretches always: 20000 x 8192 weights take 142 us so and 162 by rows
  if constexpr (DT != SPEC_F32 || !ZERO) {
    if (!few<kRows>(P.V, nsm)) {
      quantize_kernel<DT, LANES, ZERO, kRows, 1><<<blocks(P.V, kRows), kW4Threads, 0, s>>>(P);
      return;
    }
  }
  quantize_kernel<DT, LANES, ZERO, 1, kRows><<<blocks(P.V, 1), kW4Threads, 0, s>>>(P);
}
template <int LANES>
void quantize_of(const W4Params& P, int nsm, cudaStream_t s) {
  if (P.dtype == SPEC_BF16) P.zero ? quantize<SPEC_BF16, LANES, true>(P, nsm, s) : quantize<SPEC_BF16, LANES, false>(P, nsm, s);
  else P.zero ? quantize<SPEC_F32, LANES, true>(P, nsm, s) : quantize<SPEC_F32, LANES, false>(P, nsm, s);
}
template <int DT, bool ZERO>
void dequantize(const W4Params& P, int nsm, cudaStream_t s) {
  const int log_per = P.group == 128 ? 4 : P.group == 64 ? 3 : 2;
  if (few<4>(P.V, nsm)) dequantize_kernel<DT, ZERO, 1, 4><<<blocks(P.V, 1), kW4Threads, 0, s>>>(P, log_per);
  else dequantize_kernel<DT, ZERO, 4, 1><<<blocks(P.V, 4), kW4Threads, 0, s>>>(P, log_per);
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
