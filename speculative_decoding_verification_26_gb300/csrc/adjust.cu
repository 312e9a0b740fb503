// adjust.cu -- penalties for repeated tokens, biases and masks on logit rows.
//
// Row i of request b is the row after the request's history and its draft tokens
// y_0 .. y_{i-1}.  With c(v) the occurrences of v among the outputs (the history
// behind the prompt, and those drafts), and v "seen" when it occurs anywhere,
//   x <- seen ? (x > 0 ? x / rep : x rep) : x;   x <- x - (c freq + pres) where c > 0;
//   x <- x + sum of the biases listed for v;     x <- -inf where the mask has 0,
// in fp32, rounded once to the row's type.  Logits that nothing touches keep their bits.
//   A sum of biases that leaves +-2^100 is held times 2^-13: there 4096 finite biases stay finite,
// so that a -inf among them stays -inf, and an fma adds it to the logit with one rounding.  (Sums in
// 64 bits cost 320 -> 430 us for 64 x 8 x 151936 bf16 logits with 4096 biases, and 67 -> 430 for
// one request whose 4096 biases are of one token.)
//
// A CTA takes a range of the vocabulary for all R rows of a request.  It counts the
// history's tokens of its range in shared memory (whole numbers: the order of the
// atomics does not matter), lists those that anything touches, and adjusts them one by one.
//   Out of place its part of the rows is copied and masked first, in 16-byte vectors (and
// copied again for a request that the counting finds at fault).
//   In place most logits are neither read nor written: vectors that the mask removes whole
// are written without a read, those that it leaves whole are left alone.
// The adjustment of a listed token stays out of the vector loops: unrolled over a vector's
// logits it did not fit the instruction cache (64 x 8 x 151936 bf16 logits: 186 us).  Rows by bulk
// copies through shared memory took 81 us, counting before copying 71 us.
//   What bounds it, in 64 x 8 x 151936 bf16 logits: the copy alone takes 51 us (6.1 TB/s), masks 3 us
// more, histories of 2048 tokens 9 to 11: counting 2, the listed tokens' logits 4, their
// stores of 2 bytes 5.  In place a mask that leaves 2 % takes 44 us, 30 of them its stores, the
// rest the vectors that it leaves in part (84 MB of reads in 64-byte pieces).
#include "rows.cuh"
#include "serve.cuh"

namespace sv {
namespace {

constexpr int kAdjustThreads = 256;
constexpr int kMaxRange = 2048, kMinRange = 1024;        // tokens of a CTA
constexpr int kRows = 2;                     // rows taken at once
constexpr uint32_t kInPrompt = 0x80000000u, kInDraft = 0x40000000u, kTouched = 0x20000000u,
                   kCount = 0x1FFFFFFFu;   // of a count word

// In shared memory: this, counts [range]; with biases their sums [range] and a bit for each that is
// held times kNarrow; the touched tokens' places in the range, and the rows' masks of the range (a
// word more each).
struct AdjustShared {
  int draft[SPEC_MAX_G + 1];
  int bad, listed;
  int pad[2];
};
__host__ __device__ constexpr size_t adjust_smem_bytes(int range, bool any, bool biases, int masked_rows) {
  return sizeof(AdjustShared) + (any ? (size_t)range * 6 + (biases ? range * 4 + range / 8 : 0) : 0) +
         ((size_t)masked_rows * (range / 8 + 4) + 15) / 16 * 16;
}
constexpr float kWide = 0x1p100f, kNarrow = 0x1p-13f;
static_assert(SPEC_MAX_BIASES <= 1 << 12, "a sum of biases");

struct Penalties {
  float rep, freq, pres;
};

// A touched logit of row i; c is its count word.
__device__ __forceinline__ float adjusted(float x, uint32_t c, int v, int i, const AdjustShared& S, const Penalties& p) {
  uint32_t n = c & kCount;
  bool seen = n != 0 || (c & kInPrompt) != 0;
  if (c & kInDraft) {
    for (int j = 0; j < i; ++j) n += S.draft[j] == v;
    seen = seen || n != 0;
  }
  if (seen) x = x > 0.f ? __fdiv_rn(x, p.rep) : x * p.rep;
  if (n != 0) x -= __fmaf_rn((float)n, p.freq, p.pres);
  return x;
}

// whether v is among the drafts before row i
__device__ __forceinline__ bool drafted(uint32_t c, int v, int i, const AdjustShared& S) {
  bool yes = false;
  if (c & kInDraft)
    for (int j = 0; j < i; ++j) yes |= S.draft[j] == v;
  return yes;
}

template <int DT>
struct Logit;
template <>
struct Logit<SPEC_BF16> {
  using Bits = uint16_t;
  static constexpr uint32_t kFull = 0xFF;
  static __device__ __forceinline__ Bits pack(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
  static __device__ __forceinline__ float value(Bits b) { return __uint_as_float((uint32_t)b << 16); }
};
template <>
struct Logit<SPEC_F32> {
  using Bits = uint32_t;
  static constexpr uint32_t kFull = 0xF;
  static __device__ __forceinline__ Bits pack(float x) { return __float_as_uint(x); }
  static __device__ __forceinline__ float value(Bits b) { return __uint_as_float(b); }
};

__device__ __forceinline__ uint4 load_vec(const unsigned char* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// a vector among others that are not read: 64 bytes from memory instead of 128
__device__ __forceinline__ uint4 load_lone_vec(const unsigned char* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::64B.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void store_vec(unsigned char* p, const uint4& v) {
  asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The bits of the PER tokens from `at` on, of a row's mask in shared memory.
template <int PER, bool ALIGNED>
__device__ __forceinline__ uint32_t allowed(const uint32_t* mask, int at, uint32_t full) {
  if constexpr (ALIGNED) {                   // `at` is a multiple of PER
    const uint32_t byte = reinterpret_cast<const uint8_t*>(mask)[at >> 3];
    return PER == 8 ? byte : byte >> (at & 4) & full;
  }
  return __funnelshift_r(mask[at >> 5], mask[(at >> 5) + 1], at & 31) & full;
}
// Logits whose bit of `keep` is 0 become -inf.  A product spreads four bits to the top bits of
// four bytes, which prmt repeats over the bytes of their logits.
__device__ __forceinline__ uint32_t spread(uint32_t four) { return four * 0x10204080u; }
template <uint32_t SELECT>
__device__ __forceinline__ uint32_t kept(uint32_t w, uint32_t bits, uint32_t gone) {
  uint32_t m;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(m) : "r"(bits), "n"(SELECT));
  return (w & m) | (gone & ~m);
}
template <int DT>
__device__ __forceinline__ void remove_others(uint4& x, uint32_t keep) {
  if constexpr (DT == SPEC_BF16) {
    const uint32_t a = spread(keep & 15u), b = spread(keep >> 4);
    x = make_uint4(kept<0x9988>(x.x, a, 0xFF80FF80u), kept<0xBBAA>(x.y, a, 0xFF80FF80u), kept<0x9988>(x.z, b, 0xFF80FF80u),
                   kept<0xBBAA>(x.w, b, 0xFF80FF80u));
  } else {
    const uint32_t a = spread(keep);
    x = make_uint4(kept<0x8888>(x.x, a, 0xFF800000u), kept<0x9999>(x.y, a, 0xFF800000u), kept<0xAAAA>(x.z, a, 0xFF800000u),
                   kept<0xBBBB>(x.w, a, 0xFF800000u));
  }
}

// ALIGNED: every row starts on a 16-byte boundary.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kAdjustThreads, 8) adjust_kernel(const __grid_constant__ AdjustParams P, int splits, int shift) {
  using Lg = Logit<DT>;
  using Bits = typename Lg::Bits;
  constexpr int ES = RowType<DT>::ES, PER = RowType<DT>::PER;
  extern __shared__ __align__(16) unsigned char adjust_smem[];
  AdjustShared& S = *reinterpret_cast<AdjustShared*>(adjust_smem);
  const int range = 1 << shift;
  uint32_t* const count = reinterpret_cast<uint32_t*>(adjust_smem + sizeof(AdjustShared));
  float* const bias = reinterpret_cast<float*>(count + range);
  uint32_t* const narrowed = count + 2 * range;
  uint16_t* const list = reinterpret_cast<uint16_t*>(P.biases > 0 ? narrowed + range / 32 : count + range);
  const int b = blockIdx.x / splits, part = blockIdx.x % splits, t = threadIdx.x;
  const int lo = part << shift, hi = min(P.V, lo + range);
  const bool counts = P.L > 0 || P.D > 0, any = counts || P.biases > 0;

  const int W = (P.V + 31) / 32, pitch = range / 32 + 1;
  uint32_t* const masks_here = reinterpret_cast<uint32_t*>(adjust_smem + adjust_smem_bytes(range, any, P.biases > 0, 0));
  const size_t first = (size_t)b * P.R * P.V + lo, row_bytes = (size_t)P.V * ES;        // element of row 0
  const unsigned char* const in0 = P.in + first * ES;
  unsigned char* const out0 = P.out + first * ES;
  const int size = hi - lo;
  const bool apart = P.out != P.in;
  const int most = P.D > 0 ? P.D : P.R - 1;
  // row i's elements [0, head) and [tail, size) are fewer than a vector each; those between start on a
  // 16-byte boundary
  const auto head_of = [&](int i) {
    return ALIGNED ? 0 : min((int)(-(reinterpret_cast<uintptr_t>(in0) + i * row_bytes) & 15) / ES, size);
  };
  const auto tail_of = [&](int i) {
    const int head = head_of(i);
    return head + (size - head) / PER * PER;
  };
  if (P.mask) {
    const uint32_t* m = P.mask + (size_t)b * P.R * W + (lo >> 5);
    const int here = min(pitch - 1, W - (lo >> 5));
    for (int e = t; e < P.R << (shift - 5); e += kAdjustThreads) {
      const int i = e >> (shift - 5), k = e & (pitch - 2);
      if (k < here) masks_here[i * pitch + k] = __ldg(m + (size_t)i * W + k);
    }
  }

  // what a request has that is out of its range; every CTA of it finds the same
  int bad = 0;
  const int len = P.history_len ? P.history_len[b] : P.L, prompt = P.prompt_len ? P.prompt_len[b] : 0;
  const bool lengths = len >= 0 && len <= P.L && prompt >= 0 && prompt <= len;
  if (!lengths) bad |= SPEC_ST_BAD_LENGTH;
  int gamma = P.gamma ? P.gamma[b] : most;
  if (gamma < 0 || gamma > most) { bad |= SPEC_ST_BAD_GAMMA; gamma = most; }
  Penalties p;
  p.rep = P.repetition ? P.repetition[b] : 1.f;
  p.freq = P.frequency ? P.frequency[b] : 0.f;
  p.pres = P.presence ? P.presence[b] : 0.f;
  if (!(p.rep > 0.f) || !isfinite(p.rep) || !isfinite(p.freq) || !isfinite(p.pres)) bad |= SPEC_ST_BAD_PENALTY;

  if (any) {
    if (t == 0) S.bad = S.listed = 0;
    // (the counts of a request without history or drafts are read for its biases)
    for (int e = t; e < range; e += kAdjustThreads) count[e] = 0;
    if (P.biases > 0)
      for (int e = t; e < range + range / 32; e += kAdjustThreads) count[range + e] = 0;      // 0.f
  }
  __syncthreads();

  const int rows = min(P.R, gamma + 1);
  const auto removed = [&](int i, int at) { return P.mask && !(masks_here[i * pitch + (at >> 5)] >> (at & 31) & 1); };
  const bool alike = ((reinterpret_cast<uintptr_t>(P.in) ^ reinterpret_cast<uintptr_t>(P.out)) & 15) == 0;
  // vectors k of kRows rows at a time; with fewer vectors than threads, rows side by side
  const int vecs = range / PER, abreast = vecs < kAdjustThreads ? vecs : kAdjustThreads;
  const int side = t / abreast * kRows, step = kAdjustThreads / abreast * kRows;
  const ptrdiff_t to_out = out0 - in0;
  const auto copy_rows = [&](bool masked) {
    if (!alike) {
      for (int i = 0; i < rows; ++i)
        for (int at = t; at < size; at += kAdjustThreads)
          reinterpret_cast<Bits*>(out0 + i * row_bytes)[at] =
              masked && removed(i, at) ? Lg::pack(-INFINITY) : reinterpret_cast<const Bits*>(in0 + i * row_bytes)[at];
      return;
    }
    for (int k = t & (abreast - 1); k * PER < size; k += abreast) {
      const unsigned char* row = in0 + side * row_bytes + k * 16;
      for (int i0 = side; i0 < rows; i0 += step, row += step * row_bytes) {
        uint4 x[kRows];
        uint32_t live = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int head = head_of(i0 + r);
          if (i0 + r < rows && head + (k + 1) * PER <= size) {
            live |= 1u << r;
            x[r] = load_vec(row + r * row_bytes + head * ES);
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (!(live >> r & 1)) continue;
          const int head = head_of(i0 + r);
          if (masked) {
            const uint32_t keep = allowed<PER, ALIGNED>(masks_here + (i0 + r) * pitch, head + k * PER, Lg::kFull);
            if (keep != Lg::kFull) remove_others<DT>(x[r], keep);
          }
          store_vec(const_cast<unsigned char*>(row) + to_out + r * row_bytes + head * ES, x[r]);
        }
      }
    }
    // the ends of a row's part
    for (int item = t; item < rows * 2 * PER; item += kAdjustThreads) {
      const int i = item / (2 * PER), e = item % (2 * PER), at = e < PER ? e : tail_of(i) + e - PER;
      if (e < PER ? e < head_of(i) : at < size)
        reinterpret_cast<Bits*>(out0 + i * row_bytes)[at] =
            masked && removed(i, at) ? Lg::pack(-INFINITY) : reinterpret_cast<const Bits*>(in0 + i * row_bytes)[at];
    }
  };
  if (apart) copy_rows(P.mask != nullptr);

  if (any) {
    const auto touch = [&](int at, uint32_t old) {       // old: its count word before
      if (old & (kTouched | kInPrompt | kInDraft | kCount)) return;
      list[atomicAdd(&S.listed, 1)] = (uint16_t)at;
    };
    if (lengths) {
      const int32_t* h = P.history + (size_t)b * P.L;
      const auto told = [&](int e, int v) {
        bad |= (unsigned)v + 1u > (unsigned)P.V;           // SPEC_ST_BAD_TOKEN is set below
        const unsigned at = (unsigned)v - (unsigned)lo;
        if (at < (unsigned)size) touch((int)at, e < prompt ? atomicOr(&count[at], kInPrompt) : atomicAdd(&count[at], 1u));
      };
      static_assert(SPEC_ST_BAD_TOKEN == 2, "bit 0 below stands for it");
      const int whole = (reinterpret_cast<uintptr_t>(h) & 15) == 0 ? len / 4 : 0;
      int e = t;
      for (; e + kAdjustThreads < whole; e += 2 * kAdjustThreads) {
        const int4 v = __ldg(reinterpret_cast<const int4*>(h) + e), w = __ldg(reinterpret_cast<const int4*>(h) + e + kAdjustThreads);
        told(4 * e, v.x); told(4 * e + 1, v.y); told(4 * e + 2, v.z); told(4 * e + 3, v.w);
        const int f = 4 * (e + kAdjustThreads);
        told(f, w.x); told(f + 1, w.y); told(f + 2, w.z); told(f + 3, w.w);
      }
      if (e < whole) {
        const int4 v = __ldg(reinterpret_cast<const int4*>(h) + e);
        told(4 * e, v.x); told(4 * e + 1, v.y); told(4 * e + 2, v.z); told(4 * e + 3, v.w);
      }
      for (e = 4 * whole + t; e < len; e += kAdjustThreads) told(e, __ldg(h + e));
      bad = (bad & ~1) | (bad & 1) * SPEC_ST_BAD_TOKEN;
    }
    if (t < P.D) {
      const int v = t < gamma ? P.draft[(size_t)b * P.D + t] : -1;
      S.draft[t] = v;
      if (v < -1 || v >= P.V) bad |= SPEC_ST_BAD_TOKEN;
      else if (v >= lo && v < hi) touch(v - lo, atomicOr(&count[v - lo], kInDraft));
    }
    if (t >= kAdjustThreads - 32) {
      // biases of one token are added in the order of the list: the last warp takes 32 at a
      // time, the first lane of a token its sum
      const int lane = t & 31;
      for (int e0 = 0; e0 < P.biases; e0 += 32) {
        const int e = e0 + lane;
        int v = -1;
        float x = 0.f;
        if (e < P.biases) {
          v = P.bias_index[(size_t)b * P.biases + e];
          x = P.bias_value[(size_t)b * P.biases + e];
          if (v < -1 || v >= P.V) bad |= SPEC_ST_BAD_TOKEN;
          if (v != -1 && !(x < INFINITY)) bad |= SPEC_ST_BAD_PENALTY;
        }
        const bool mine = v >= lo && v < hi;
        if (__any_sync(0xffffffffu, mine)) {
          const uint32_t same = __match_any_sync(0xffffffffu, mine ? v : -1 - lane);
          const bool leads = mine && (same & ((1u << lane) - 1)) == 0;
          const int at = mine ? v - lo : 0;
          const float start = bias[at];
          float sum = start + x;
          if (__any_sync(0xffffffffu, mine && same != 1u << lane)) {
            sum = start;
            for (int k = 0; k < 32; ++k) {
              const float y = __shfl_sync(0xffffffffu, x, k);
              if (same >> k & 1) sum += y;
            }
          }
          const bool held = narrowed[at >> 5] >> (at & 31) & 1, wide = leads && (held || !(fabsf(sum) <= kWide));
          if (__any_sync(0xffffffffu, wide)) {
            float narrow = held ? start : start * kNarrow;
            for (int k = 0; k < 32; ++k) {
              const float y = __shfl_sync(0xffffffffu, x, k);
              if (same >> k & 1) narrow = __fmaf_rn(y, kNarrow, narrow);
            }
            if (wide) {
              sum = narrow;
              atomicOr(&narrowed[at >> 5], 1u << (at & 31));
            }
          }
          __syncwarp();
          if (leads) {
            bias[at] = sum;
            touch(at, atomicOr(&count[at], kTouched));
          }
          __syncwarp();
        }
      }
    }
    if (bad) atomicOr(&S.bad, bad);
  }
  __syncthreads();
  if (any) bad = S.bad;
  if (part == 0 && t == 0 && P.status) P.status[b] = bad;

  if (bad) {
    if (apart && P.mask) copy_rows(false);
    return;
  }
  if (!apart && P.mask) {
    for (int k = t & (abreast - 1); k * PER < size; k += abreast) {
      unsigned char* row = out0 + side * row_bytes + k * 16;
      for (int i0 = side; i0 < rows; i0 += step, row += step * row_bytes) {
        uint4 x[kRows];
        uint32_t keep[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int head = head_of(i0 + r);
          keep[r] = Lg::kFull;
          if (i0 + r < rows && head + (k + 1) * PER <= size)
            keep[r] = allowed<PER, ALIGNED>(masks_here + (i0 + r) * pitch, head + k * PER, Lg::kFull);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          x[r] = make_uint4(0, 0, 0, 0);
          if (keep[r] != Lg::kFull && keep[r] != 0) x[r] = load_lone_vec(row + r * row_bytes + head_of(i0 + r) * ES);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (keep[r] == Lg::kFull) continue;
          remove_others<DT>(x[r], keep[r]);
          store_vec(row + r * row_bytes + head_of(i0 + r) * ES, x[r]);
        }
      }
    }
    for (int item = t; item < rows * 2 * PER; item += kAdjustThreads) {
      const int i = item / (2 * PER), e = item % (2 * PER), at = e < PER ? e : tail_of(i) + e - PER;
      if ((e < PER ? e < head_of(i) : at < size) && removed(i, at))
        reinterpret_cast<Bits*>(out0 + i * row_bytes)[at] = Lg::pack(-INFINITY);
    }
    __syncthreads();                         // vectors with listed tokens have been written
  }
  const int listed = any ? S.listed : 0;
  for (int item = t; item < listed * rows; item += kAdjustThreads) {
    const int i = item / listed, at = list[item - i * listed];
    if (removed(i, at)) continue;
    const uint32_t c = count[at];
    Bits* const to = reinterpret_cast<Bits*>(out0 + i * row_bytes) + at;       // the logit, copied: it is in L2
    float x = adjusted(Lg::value(*to), c, lo + at, i, S, p);
    if (P.biases > 0 && (c & kTouched)) x = __fmaf_rn(bias[at], narrowed[at >> 5] >> (at & 31) & 1 ? 1.f / kNarrow : 1.f, x);
    else if ((c & (kInPrompt | kCount)) == 0 && !drafted(c, lo + at, i, S)) continue;       // a draft of a later row alone
    *to = Lg::pack(x);
  }
}

}  // namespace

template <int DT, bool ALIGNED>
static cudaError_t allow() {
  return cudaFuncSetAttribute(adjust_kernel<DT, ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)adjust_smem_bytes(kMaxRange, true, true, SPEC_MAX_G + 1));
}
cudaError_t configure_adjust() {
  cudaError_t e = allow<SPEC_BF16, true>();
  if (e == cudaSuccess) e = allow<SPEC_BF16, false>();
  if (e == cudaSuccess) e = allow<SPEC_F32, true>();
  if (e == cudaSuccess) e = allow<SPEC_F32, false>();
  return e;
}

cudaError_t launch_adjust(const AdjustParams& P, int nsm, cudaStream_t s) {
  // the largest range that still gives every SM four CTAs
  int shift = 11;
  static_assert(kMaxRange == 1 << 11 && kMinRange == 1 << 10, "ranges");
  const auto splits_of = [&](int sh) { return (P.V + (1ll << sh) - 1) >> sh; };
  while (shift > 10 && splits_of(shift) * P.B < 4ll * nsm) --shift;
  const int splits = (int)splits_of(shift);
  const size_t smem = adjust_smem_bytes(1 << shift, P.L > 0 || P.D > 0 || P.biases > 0, P.biases > 0, P.mask ? P.R : 0);
  const unsigned grid = (unsigned)(splits * (long long)P.B);
  const int es = P.dtype == SPEC_BF16 ? 2 : 4;
  const bool aligned = ((size_t)P.V * es) % 16 == 0 && reinterpret_cast<uintptr_t>(P.in) % 16 == 0 && reinterpret_cast<uintptr_t>(P.out) % 16 == 0;
  if (P.dtype == SPEC_BF16) {
    if (aligned) adjust_kernel<SPEC_BF16, true><<<grid, kAdjustThreads, smem, s>>>(P, splits, shift);
    else adjust_kernel<SPEC_BF16, false><<<grid, kAdjustThreads, smem, s>>>(P, splits, shift);
  } else {
    if (aligned) adjust_kernel<SPEC_F32, true><<<grid, kAdjustThreads, smem, s>>>(P, splits, shift);
    else adjust_kernel<SPEC_F32, false><<<grid, kAdjustThreads, smem, s>>>(P, splits, shift);
  }
  return cudaGetLastError();
}

}  // namespace sv
