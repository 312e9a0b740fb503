// linear_ce.cu -- softmax cross entropy of a vocabulary projection, in pieces
// of the vocabulary, without keeping the logits; and its gradients.
//
//   l = h W^T, lse_i = ln sum_v e^{l_iv}, loss_i = lse_i - l_{i, y_i};
//   G_iv = g_i (e^{l_iv - lse_i} - [v = y_i]),  dh = G W,  dW = G^T h.
//
// Rows without a label (and in the backward pass rows of weight 0) take no part:
// gather_rows copies the rows that count to the front of a compact matrix, so
// that a masked row costs nothing and a NaN in it reaches nothing; for the
// backward pass, zero rows fill its last stage of 64.
// Forward: the label's logit apart (gather_rows), one maximum and sum of the
// others per row and vocabulary tile, merged by merge_rows.  Backward, for each piece of the vocabulary: G of the piece (the
// logits again, softmax in the epilogue), dW of the piece, and the piece's part
// of dh, summed in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "rows.cuh"
#include "tc_gemm.cuh"

namespace sv {
namespace {

constexpr int kGatherThreads = 256;
// Rows of a CTA: one per warp; 64 past 32768 rows, where each CTA's pass over all
// labels would cost more than the copies.
constexpr int kGatherFew = 8, kGatherMany = 64;

// The rows that count, in order: row_of, their labels, and their hidden states.
template <bool BWD, int kGatherRows>
__global__ void __launch_bounds__(kGatherThreads) gather_rows(const __grid_constant__ CeParams P) {
  griddep_launch();                          // the next kernel's set-up needs nothing of this one
  __shared__ int s_before[kGatherThreads / 32], s_all[kGatherThreads / 32];
  __shared__ int s_row[kGatherRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = blockIdx.x * kGatherRows;
  auto counts = [&](int r) {
    const int y = P.label[r];
    if (y < 0 || y >= P.V) return false;
    if (!BWD) return true;
    const float g = P.grad_loss ? P.grad_loss[r] : 1.f;
    return g != 0.f && isfinite(P.lse_in[r]);
  };
  int before = 0, all = 0;
  for (int r = tid; r < P.n; r += kGatherThreads) {
    const bool v = counts(r);
    all += v;
    before += v && r < r0;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, off);
    all += __shfl_xor_sync(0xffffffffu, all, off);
  }
  if (lane == 0) { s_before[warp] = before; s_all[warp] = all; }
  __syncthreads();
  before = 0;
  all = 0;
  for (int w = 0; w < kGatherThreads / 32; ++w) { before += s_before[w]; all += s_all[w]; }
  if (warp == 0) {
    for (int i0 = 0, base = before; i0 < kGatherRows; i0 += 32) {
      const int i = i0 + lane, r = r0 + i;
      const bool v = i < kGatherRows && r < P.n && counts(r);
      const unsigned vote = __ballot_sync(0xffffffffu, v);
      const int at = base + __popc(vote & ((1u << lane) - 1));
      base += __popc(vote);
      if (i < kGatherRows) s_row[i] = v ? at : -1;
      if (v) {
        P.row_of[at] = r;
        P.lab[at] = P.label[r];
        if (BWD) {
          P.lse_c[at] = P.lse_in[r];
          P.g_c[at] = P.grad_loss ? P.grad_loss[r] : 1.f;
        }
      }
      if (i >= kGatherRows || r >= P.n) continue;
      if (BWD) P.pos_of[r] = v ? at : -1;
      if (!BWD && !v) {
        const int y = P.label[r];
        const float z = y == -1 ? 0.f : __int_as_float(0x7fc00000);
        P.loss[r] = z;
        P.lse[r] = z;
        if (P.status) P.status[r] = y == -1 ? SPEC_ST_OK : SPEC_ST_BAD_TOKEN;
      }
    }
    if (blockIdx.x == 0 && lane == 0) { P.count[0] = all; P.count[1] = 0; }
  }
  __syncthreads();
  const int nv = P.H / 8;
  for (int i = warp; i < kGatherRows; i += kGatherThreads / 32) {
    if (s_row[i] >= 0) {
      const uint4* src = reinterpret_cast<const uint4*>(P.hidden + (size_t)(r0 + i) * P.H);
      uint4* dst = reinterpret_cast<uint4*>(P.rows + (size_t)s_row[i] * P.row_stride);
      // the label's logit on the way: products of bf16 are exact in fp32, and the sums are
      // rounded to nearest (the tensor cores' are not, see ForwardWork)
      const uint4* wl = reinterpret_cast<const uint4*>(P.weight + (size_t)P.label[r0 + i] * P.H);
      float a = 0.f, b = 0.f;
#pragma unroll 4
      for (int k = lane; k < nv; k += 32) {
        const uint4 x = src[k], w = wl[k];
        dst[k] = x;
        a = fmaf(bf16_lo(x.x), bf16_lo(w.x), a);
        b = fmaf(bf16_hi(x.x), bf16_hi(w.x), b);
        a = fmaf(bf16_lo(x.y), bf16_lo(w.y), a);
        b = fmaf(bf16_hi(x.y), bf16_hi(w.y), b);
        a = fmaf(bf16_lo(x.z), bf16_lo(w.z), a);
        b = fmaf(bf16_hi(x.z), bf16_hi(w.z), b);
        a = fmaf(bf16_lo(x.w), bf16_lo(w.w), a);
        b = fmaf(bf16_hi(x.w), bf16_hi(w.w), b);
      }
      a += b;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
      if (lane == 0) {
        if (BWD) P.label_g[s_row[i]] = P.g_c[s_row[i]] * expm1f(a - P.lse_in[r0 + i]);
        else P.label_logit[s_row[i]] = a;
      }
    }
    // places past the last row that counts: dW sums over whole stages of rows, and a
    // stage's last rows are zero; what lies behind them only reaches rows of its own
    const int at = r0 + i;
    if (at >= all) {
      if (BWD && at < (all + kTcK - 1) / kTcK * kTcK) {
        uint4* dst = reinterpret_cast<uint4*>(P.rows + (size_t)at * P.row_stride);
        for (int k = lane; k < nv; k += 32) dst[k] = make_uint4(0, 0, 0, 0);
      }
      if (lane == 0) {
        P.lab[at] = -1;
        if (BWD) { P.lse_c[at] = 0.f; P.g_c[at] = 0.f; P.label_g[at] = 0.f; }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The three products, as work of tc_run (see tc_gemm.cuh).

struct CeMaps {
  // k inner: boxes of 64 k x 128 rows; k outer: 64 columns x 64 k
  CUtensorMap rows, weight, soft, rows_t, weight_t, soft_t;
  CUtensorMap soft_out, grad_weight;         // stores: boxes of 64 columns x 32 rows
};

// Tiles of logits: rows x vocabulary.  Groups of kGroup row tiles (4096 rows),
// within a group the vocabulary outer and the rows inner: the pairs at work read
// few vocabulary tiles and one group's rows, both from L2, and the weights come
// from HBM once a group.
constexpr int kGroup = 16;
struct LogitTiles {
  int row_tiles, vocab_tiles, rows;          // rows that count
  __device__ __forceinline__ int index(int l, int pair, int pairs) const {
    const int t = pair + l * pairs;
    return t < row_tiles * vocab_tiles ? t : -1;
  }
  __device__ __forceinline__ void at(int t, int& mb, int& vt) const {
    const int per = kGroup * vocab_tiles, g = t / per, first = g * kGroup;
    const int size = row_tiles - first < kGroup ? row_tiles - first : kGroup;
    const int u = t - g * per;
    vt = u / size;
    mb = first + u - vt * size;
  }
};

// Forward: a tile's maximum and sum of each row, without the label.  The tensor cores
// cut their sums off (about 1e-5 of a logit of 16 over H = 2048), and where the label
// has nearly all of the mass its loss is as small as that: the label's logit is summed
// apart (gather_rows), the loss is ln(1 + the others' weights beside the label's), and
// the others' logits are sums of parts of kChunk stages, 1024 of H (H = 2048: the loss off
// by 5.8e-6 of itself at most, 1e-5 with whole sums and 3.8e-6 with parts of 512; one row
// 115.4, 115.2 and 117.9 us; 4096 rows 1.26, 1.25 and 1.34 ms in short runs, and 1.40 ms
// with parts of 1024 where the power cap holds).
constexpr int kChunk = 16;
struct ForwardWork {
  const CeParams& P;
  const CeMaps& M;
  LogitTiles lt;
  __device__ __forceinline__ int index(int l, int pair, int pairs) const { return lt.index(l, pair, pairs); }
  __device__ __forceinline__ TcTile tile(int t) const {
    int mb, vt;
    lt.at(t, mb, vt);
    return {{&M.rows, true, mb * kTcTile, 0}, {&M.weight, true, vt * kTcTile, 0}, (P.H + kTcK - 1) / kTcK};
  }
  __device__ __forceinline__ bool counts(int t, const TcHalfRow& e) const {      // the same for the warp
    int mb, vt;
    lt.at(t, mb, vt);
    return mb * kTcTile + e.row - (int)(threadIdx.x & 31) < lt.rows;
  }
  __device__ __forceinline__ void epilogue(int t, TcHalfRow& e, float (&x)[kTcHalf]) const {
    int mb, vt;
    lt.at(t, mb, vt);
    const int i = mb * kTcTile + e.row, v0 = vt * kTcTile + e.col;
    const int at = P.lab[i] - v0, left = P.V - v0;           // the label's column; columns of the vocabulary
    if ((at >= 0 && at < kTcHalf) || left < kTcHalf) {
#pragma unroll
      for (int c = 0; c < kTcHalf; ++c)
        if (c == at || c >= left) x[c] = -INFINITY;
    }
    float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int c = 4; c < kTcHalf; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
    const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    // x - m first: m log2(e) of logits masked with the type's lowest value would overflow
    const float ref = m == -INFINITY ? 0.f : -m;             // a half past the vocabulary: weights of 0
    const float2 R2 = make_float2(ref, ref), K2 = make_float2(kLog2eHi, kLog2eHi);
    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < kTcHalf; c += 2) {
      const float2 a = __fmul2_rn(__fadd2_rn(make_float2(x[c], x[c + 1]), R2), K2);
      part[c >> 1 & 1] = __fadd2_rn(part[c >> 1 & 1], make_float2(ex2(a.x), ex2(a.y)));
    }
    part[0] = __fadd2_rn(part[0], part[1]);
    float s = part[0].x + part[0].y;
    const float2 other = e.join(make_float2(m, s));
    if (e.col != 0) return;
    const float both = fmaxf(m, other.x);    // a NaN sum stays
    // a half without a finite logit has a sum of 0 (or NaN)
    s = (m == -INFINITY ? s : s * ex2((m - both) * kLog2eHi)) +
        (other.x == -INFINITY ? other.y : other.y * ex2((other.x - both) * kLog2eHi));
    P.part[(size_t)vt * P.n_pad + i] = make_float2(both, s);
  }
};

__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    memcpy(&u[k], &b, 4);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// 32 columns from c0 of a half row: in tensor memory, or joined from parts
__device__ __forceinline__ void columns(float (&v)[32], const TcHalfRow& e, int c0) { tc_load32(v, e.tmem + c0); }
__device__ __forceinline__ void columns(float (&v)[32], const float (&x)[kTcHalf], int c0) {
#pragma unroll
  for (int c = 0; c < 32; ++c) v[c] = x[c0 + c];
}

// backward: G of a piece as bf16, its one rounding before the two products that
// read it; the logits and the softmax are fp32.  Past kWholeLogits stages (H = 2048) the
// logits are sums of the same parts as the forward call's, to match the lse that they are
// taken beside: with whole sums and an offset l that all logits of a row share, the rows of
// G sum to -2e-6 l at H = 2048 (below its rounding while l < 1000), to -4e-5 l at 8192 and
// -4e-4 l at 65536.  Parts cost 140 us for 135 at H = 1160, where whole sums are used, and
// nothing to speak of at 2048 and more (4.43 ms for 4.41).
constexpr int kWholeLogits = 32;
struct SoftWork {
  const CeParams& P;
  const CeMaps& M;
  LogitTiles lt;
  int v_begin;
  __device__ __forceinline__ int index(int l, int pair, int pairs) const { return lt.index(l, pair, pairs); }
  __device__ __forceinline__ TcTile tile(int t) const {
    int mb, vt;
    lt.at(t, mb, vt);
    return {{&M.rows, true, mb * kTcTile, 0}, {&M.weight, true, v_begin + vt * kTcTile, 0}, (P.H + kTcK - 1) / kTcK};
  }
  // a stage's last rows are zero (G sums over rows in whole stages); later ones are not read
  __device__ __forceinline__ bool counts(int t, const TcHalfRow& e) const {      // the same for the warp
    int mb, vt;
    lt.at(t, mb, vt);
    return mb * kTcTile + e.row - (int)(threadIdx.x & 31) < (lt.rows + kTcK - 1) / kTcK * kTcK;
  }
  __device__ __forceinline__ void epilogue(int t, TcHalfRow& e) const {
    if (counts(t, e)) store<1>(t, e, e);
  }
  __device__ __forceinline__ void epilogue(int t, TcHalfRow& e, float (&x)[kTcHalf]) const { store<2>(t, e, x); }
  template <int UNROLL, class From>
  __device__ __forceinline__ void store(int t, TcHalfRow& e, const From& from) const {
    int mb, vt;
    lt.at(t, mb, vt);
    const int i = mb * kTcTile + e.row, first = i - (int)(threadIdx.x & 31), v0 = v_begin + vt * kTcTile + e.col;
    const int at = P.lab[i] - v0;
    const float g = P.g_c[i], gy = P.label_g[i], lse = P.lse_c[i];
    const float2 L2 = make_float2(-lse, -lse), K2 = make_float2(kLog2eHi, kLog2eHi);    // l - lse first, as in the forward pass
#pragma unroll UNROLL
    for (int c0 = 0; c0 < kTcHalf; c0 += 64) {
      uint4 out[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[32];
        columns(x, from, c0 + 32 * h);
        const int left = P.V - v0 - c0 - 32 * h, mark = at - c0 - 32 * h;
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 a = __fmul2_rn(__fadd2_rn(make_float2(x[c], x[c + 1]), L2), K2);
          x[c] = c < left && g != 0.f ? g * ex2(a.x) : 0.f;
          x[c + 1] = c + 1 < left && g != 0.f ? g * ex2(a.y) : 0.f;
          if (c == mark) x[c] = gy;
          if (c + 1 == mark) x[c + 1] = gy;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) out[4 * h + c] = pack8(x + 8 * c);
      }
      e.store.put(&M.soft_out, vt * kTcTile + e.col + c0, first, out);
    }
  }
};

// The gradients' sums are whole up to kWholeSteps stages and joined from parts of kGradChunk
// beyond (rows for dW, a piece's vocabulary for dh).  The tensor cores cut off at every
// addition of 16 k, and sums of one sign drift: dW of 131072 rows was off by 2.8e-4, of 2^20
// rows by 4.4e-3, past its rounding to bf16 (2^-8).  Parts cost 194 us for 183 where tiles
// are many and short (64 x 1024 x 128256), 132.5 for 134.6 at 333 x 1160 x 40001, and the
// same at 4096 rows.
constexpr int kWholeSteps = 512, kGradChunk = 256;

// Stages of k that a tile of dW takes at least: the time to write it.
constexpr int kStoreSteps = 6;

// backward: a piece's part of dh (k: the piece's vocabulary, in `splits` parts
// of `per` stages) and its rows of dW (k: the rows that count)
struct GradWork {
  const CeParams& P;
  const CeMaps& M;
  int v_begin, rows, row_tiles, col_tiles, steps_x, steps_w, hidden_tiles, weight_tiles;
  // The long tiles of dh first, round robin.  Pairs that have one less of them take
  // `lead` tiles of dW in its place before the others join: a pair's tiles of dh are
  // few (120 for 4096 rows), and one more is a third of its work.
  __device__ __forceinline__ int index(int l, int pair, int pairs) const {
    const int more = hidden_tiles % pairs, own = hidden_tiles / pairs + (pair < more);
    if (l < own) return pair + l * pairs;
    l -= own;
    const int light = pairs - more;
    int lead = 0;
    if (more != 0 && steps_w > 0) {
      const int w = steps_w > kStoreSteps ? steps_w : kStoreSteps;
      lead = (P.split_steps + w / 2) / w;
      if (lead > weight_tiles / light) lead = weight_tiles / light;
    }
    int t;
    if (pair >= more) {
      t = l < lead ? l * light + (pair - more) : lead * light + (l - lead) * pairs + pair;
    } else {
      t = lead * light + l * pairs + pair;
    }
    return t < weight_tiles ? hidden_tiles + t : -1;
  }
  __device__ __forceinline__ void hidden_at(int t, int& mb, int& nb, int& sp) const {
    nb = t % col_tiles;
    mb = t / col_tiles % row_tiles;
    sp = t / (col_tiles * row_tiles);
  }
  __device__ __forceinline__ TcTile tile(int t) const {
    if (t < hidden_tiles) {
      int mb, nb, sp;
      hidden_at(t, mb, nb, sp);
      const int first = sp * P.split_steps, left = steps_x - first;
      return {{&M.soft, true, mb * kTcTile, first * kTcK},
              {&M.weight_t, false, nb * kTcTile, v_begin + first * kTcK},
              left < 0 ? 0 : left < P.split_steps ? left : P.split_steps};
    }
    t -= hidden_tiles;
    const int vb = t / col_tiles, nb = t % col_tiles;
    return {{&M.soft_t, false, vb * kTcTile, 0}, {&M.rows_t, false, nb * kTcTile, 0}, steps_w};
  }
  __device__ __forceinline__ bool counts(int t, const TcHalfRow& e) const {      // the same for the warp
    const int first = e.row - (int)(threadIdx.x & 31);
    if (t < hidden_tiles) {
      int mb, nb, sp;
      hidden_at(t, mb, nb, sp);
      return mb * kTcTile + first < rows;
    }
    return v_begin + (t - hidden_tiles) / col_tiles * kTcTile + first < P.V;
  }
  __device__ __forceinline__ void epilogue(int t, TcHalfRow& e) const {
    if (counts(t, e)) store<1>(t, e, e, e.any);
  }
  __device__ __forceinline__ void epilogue(int t, TcHalfRow& e, float (&x)[kTcHalf]) const { store<4>(t, e, x, true); }
  template <int UNROLL, class From>
  __device__ __forceinline__ void store(int t, TcHalfRow& e, const From& from, bool any) const {
    const int lane = threadIdx.x & 31;
    if (t < hidden_tiles) {
      int mb, nb, sp;
      hidden_at(t, mb, nb, sp);
      const int i = mb * kTcTile + e.row, j0 = nb * kTcTile + e.col;
      float* out = P.acc + ((size_t)sp * P.n_pad + i) * P.H + j0;
#pragma unroll UNROLL
      for (int c0 = 0; c0 < kTcHalf; c0 += 32) {
        if (j0 + c0 >= P.H) break;
        float x[32];
        if (any) {
          columns(x, from, c0);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = 0.f;
        }
        if (i >= rows) continue;
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          if (j0 + c0 + c >= P.H) break;     // H is a multiple of 8
          float4* at = reinterpret_cast<float4*>(out + c0 + c);
          float4 v = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
          if (v_begin != 0) {
            const float4 o = *at;
            v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
          }
          *at = v;
        }
      }
      return;
    }
    t -= hidden_tiles;
    const int vb = t / col_tiles, nb = t % col_tiles, first = v_begin + vb * kTcTile + e.row - lane;
    const int j0 = nb * kTcTile + e.col;
#pragma unroll (UNROLL / 2 > 1 ? UNROLL / 2 : 1)
    for (int c0 = 0; c0 < kTcHalf; c0 += 64) {
      if (j0 + c0 >= P.H) break;
      uint4 out[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (any) {
          float x[32];
          columns(x, from, c0 + 32 * h);
#pragma unroll
          for (int c = 0; c < 4; ++c) out[4 * h + c] = pack8(x + 8 * c);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) out[4 * h + c] = make_uint4(0, 0, 0, 0);
        }
      }
      e.store.put(&M.grad_weight, j0 + c0, first, out);
    }
  }
};

__device__ __forceinline__ int piece_len(const CeParams& P, int v_begin) {
  return P.V - v_begin < P.piece ? P.V - v_begin : P.piece;
}
// Each kernel's work is made after tc_run's set-up, which waits for the kernel before.
__global__ void __cluster_dims__(2) __launch_bounds__(kTcThreads, 1)
    ce_forward(const __grid_constant__ CeParams P, const __grid_constant__ CeMaps M) {
  tc_run<kChunk>([&] {
    const int count = *P.count;
    return ForwardWork{P, M, {(count + kTcTile - 1) / kTcTile, (P.V + kTcTile - 1) / kTcTile, count}};
  }, P.wait_limit, P.count + 1);
}
template <int CHUNK>
__global__ void __cluster_dims__(2) __launch_bounds__(kTcThreads, 1)
    ce_softmax(const __grid_constant__ CeParams P, const __grid_constant__ CeMaps M, int v_begin) {
  tc_run<CHUNK>([&] {
    const int count = *P.count;
    return SoftWork{P, M, {(count + kTcTile - 1) / kTcTile, (piece_len(P, v_begin) + kTcTile - 1) / kTcTile, count},
                    v_begin};
  }, P.wait_limit, P.count + 1);
}
template <int CHUNK>
__global__ void __cluster_dims__(2) __launch_bounds__(kTcThreads, 1)
    ce_grads(const __grid_constant__ CeParams P, const __grid_constant__ CeMaps M, int v_begin) {
  tc_run<CHUNK>([&] {
    const int len = piece_len(P, v_begin), count = *P.count;
    const int rt = (count + kTcTile - 1) / kTcTile, ct = (P.H + kTcTile - 1) / kTcTile;
    const int ht = P.grad_hidden ? rt * ct * P.splits : 0;
    const int wt = P.grad_weight ? (len + kTcTile - 1) / kTcTile * ct : 0;
    return GradWork{P, M, v_begin, count, rt, ct, (len + kTcK - 1) / kTcK, (count + kTcK - 1) / kTcK, ht, wt};
  }, P.wait_limit, P.count + 1);
}

// lse and loss of the rows that count: the tiles' maxima and sums, each warp a
// share of the tiles of 32 rows.  20 loads in flight spill 10 words a thread.
constexpr int kMergeThreads = 1024, kMergeWarps = kMergeThreads / 32;
__global__ void __launch_bounds__(kMergeThreads) merge_rows(const __grid_constant__ CeParams P) {
  __shared__ float2 s_part[kMergeWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  griddep_launch();
  griddep_wait();
  if (blockIdx.x * 32 >= *P.count) return;
  const int tiles = (P.V + kTcTile - 1) / kTcTile;
  // the maximum of several parts first, then their sums beside it; parts without a finite
  // logit hold 0 or NaN
  float m = -INFINITY, s = 0.f;
  auto beside = [](float2 p, float top) { return p.x == -INFINITY ? p.y : p.y * ex2((p.x - top) * kLog2eHi); };
  constexpr int U = 20;                      // loads in flight: a vocabulary of 163840 in one go
  for (int t0 = warp; t0 < tiles; t0 += U * kMergeWarps) {
    float2 p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * kMergeWarps;
      p[u] = t < tiles ? P.part[(size_t)t * P.n_pad + i] : make_float2(-INFINITY, 0.f);
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, p[u].x);
    s = beside(make_float2(m, s), top);
#pragma unroll
    for (int u = 0; u < U; ++u) s += beside(p[u], top);
    m = top;
  }
  s_part[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp != 0 || i >= *P.count) return;
  float all = m;
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) all = fmaxf(all, s_part[w][lane].x);
  s = beside(make_float2(m, s), all);
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) s += beside(s_part[w][lane], all);
  m = all;
  // with the label: lse - z = ln(1 + others / e^z), where z is the larger without lse's rounding
  const float z = P.label_logit[i], top = fmaxf(m, z), nan = __int_as_float(0x7fc00000);
  const float others = m == -INFINITY ? s : s * ex2((m - top) * kLog2eHi);
  const float own = ex2((z - top) * kLog2eHi);
  const float loss = z >= m ? log1pf(others) : (top - z) + kLn2 * log2f(others + own);
  const float lse = top + kLn2 * log2f(others + own);
  const int failed = P.count[1], r = P.row_of[i];
  const bool ok = isfinite(top) && isfinite(lse) && !failed;
  P.lse[r] = ok ? lse : nan;
  P.loss[r] = ok ? loss : nan;
  if (P.status) P.status[r] = failed ? SPEC_ST_TIMEOUT : ok ? SPEC_ST_OK : SPEC_ST_NONFINITE;
}

// Every row of dh: the sum of its parts, or zeros where the row took no part.
// After a wait that ran out (no healthy call) both gradients are NaN.
__global__ void __launch_bounds__(256) finish_grads(const __grid_constant__ CeParams P) {
  griddep_wait();
  const long long me = blockIdx.x * 256ll + threadIdx.x, all = gridDim.x * 256ll;
  const bool failed = P.count[1] != 0;
  const uint4 nans = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
  const int nv = P.H / 8;
  if (failed && P.grad_weight)
    for (long long t = me; t < (long long)P.V * nv; t += all) reinterpret_cast<uint4*>(P.grad_weight)[t] = nans;
  if (!P.grad_hidden) return;
  const int nq = P.H / 4;
  for (long long t = me; t < (long long)P.n * nq; t += all) {
    const int r = (int)(t / nq), j = (int)(t % nq) * 4, pos = P.pos_of[r];
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pos >= 0) {
      const float* a = P.acc + (size_t)pos * P.H + j;
      const size_t stride = (size_t)P.n_pad * P.H;
#pragma unroll 8
      for (int sp = 0; sp < P.splits; ++sp) {
        const float4 u = *reinterpret_cast<const float4*>(a + sp * stride);
        s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w;
      }
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    uint2 o;
    memcpy(&o.x, &lo, 4);
    memcpy(&o.y, &hi, 4);
    reinterpret_cast<uint2*>(P.grad_hidden)[t] = failed ? make_uint2(nans.x, nans.x) : o;
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;              // set once by configure_linear_ce

// bf16 matrix of `height` rows of `width`, `stride` apart, boxes of 64 columns x `box` rows
bool encode(CUtensorMap* map, const void* p, uint64_t width, uint64_t stride, uint64_t height, uint32_t box) {
  const cuuint64_t dims[2] = {width, height}, strides[1] = {stride * 2};
  const cuuint32_t boxes[2] = {(cuuint32_t)kTcK, box}, ones[2] = {1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BWD>
void launch_gather(const CeParams& P, cudaStream_t s) {
  if (P.n <= 32768) gather_rows<BWD, kGatherFew><<<P.n_pad / kGatherFew, kGatherThreads, 0, s>>>(P);
  else gather_rows<BWD, kGatherMany><<<P.n_pad / kGatherMany, kGatherThreads, 0, s>>>(P);
}

}  // namespace

cudaError_t configure_linear_ce() {
  cudaDriverEntryPointQueryResult found;
  void* f = nullptr;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return e;
  if (found != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
  g_encode = reinterpret_cast<EncodeTiled>(f);
  const int smem = (int)kTcSmem;
  e = cudaFuncSetAttribute(ce_forward, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(ce_softmax<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(ce_softmax<kChunk>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(ce_grads<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(ce_grads<kGradChunk>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e;
}

// A kernel after another of the call: its set-up may overlap the end of that one.
template <class K, class... A>
cudaError_t launch_after(K kernel, int grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The maps of rows and G end with the last stage of rows: what lies behind it is zeros
// without a read (64 rows of a tile of 256, G read once for each tile of H: 186 us with
// all of them, 181 without; a map that ends at row n itself is slow, 176 us for 115 of
// one row).
static int rows_read(const CeParams& P) { return (P.n + kTcK - 1) / kTcK * kTcK; }

cudaError_t launch_ce_forward(const CeParams& P, int nsm, cudaStream_t s, int* launches) {
  CeMaps M;
  memset(&M, 0, sizeof M);
  if (!encode(&M.rows, P.rows, P.H, P.row_stride, rows_read(P), kTcHalf) ||
      !encode(&M.weight, P.weight, P.H, P.H, P.V, kTcHalf))
    return cudaErrorInvalidValue;
  launch_gather<false>(P, s);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_after(ce_forward, nsm / 2 * 2, kTcThreads, kTcSmem, s, P, M);
  if (e == cudaSuccess) e = launch_after(merge_rows, P.n_pad / 32, kMergeThreads, 0, s, P);
  *launches = 3;
  return e;
}

cudaError_t launch_ce_backward(const CeParams& P, int nsm, cudaStream_t s, int* launches) {
  CeMaps M;
  memset(&M, 0, sizeof M);
  if (!encode(&M.rows, P.rows, P.H, P.row_stride, rows_read(P), kTcHalf) ||
      !encode(&M.weight, P.weight, P.H, P.H, P.V, kTcHalf) ||
      !encode(&M.soft, P.soft, P.piece, P.piece, rows_read(P), kTcHalf) ||
      !encode(&M.rows_t, P.rows, P.H, P.row_stride, rows_read(P), kTcK) ||
      !encode(&M.weight_t, P.weight, P.H, P.H, P.V, kTcK) ||
      !encode(&M.soft_t, P.soft, P.piece, P.piece, rows_read(P), kTcK) ||
      !encode(&M.soft_out, P.soft, P.piece, P.piece, P.n_pad, 32) ||
      (P.grad_weight && !encode(&M.grad_weight, P.grad_weight, P.H, P.H, P.V, 32)))
    return cudaErrorInvalidValue;
  const auto softmax = P.H <= kWholeLogits * kTcK ? ce_softmax<0> : ce_softmax<kChunk>;
  const bool whole = P.split_steps <= kWholeSteps && P.n <= kWholeSteps * kTcK;
  const auto grads = whole ? ce_grads<0> : ce_grads<kGradChunk>;
  launch_gather<true>(P, s);
  cudaError_t e = cudaGetLastError();
  int n = 2;
  for (long long v = 0; v < P.V && e == cudaSuccess; v += P.piece, n += 2) {
    e = launch_after(softmax, nsm / 2 * 2, kTcThreads, kTcSmem, s, P, M, (int)v);
    if (e == cudaSuccess) e = launch_after(grads, nsm / 2 * 2, kTcThreads, kTcSmem, s, P, M, (int)v);
  }
  if (e == cudaSuccess) e = launch_after(finish_grads, 4 * nsm, 256, 0, s, P);
  *launches = n;
  return e;
}

size_t ce_layout(CeParams& P, bool backward, void* base) {
  unsigned char* b = static_cast<unsigned char*>(base);
  size_t at = 0;
  auto place = [&](size_t bytes) {
    unsigned char* p = b ? b + at : nullptr;
    at = (at + bytes + 255) / 256 * 256;
    return p;
  };
  P.n_pad = (P.n + kTcTile - 1) / kTcTile * kTcTile;
  P.count = reinterpret_cast<int*>(place(256));
  P.row_of = reinterpret_cast<int*>(place(4ull * P.n_pad));
  P.lab = reinterpret_cast<int*>(place(4ull * P.n_pad));
  // rows start on 128-byte lines: a box row of 64 columns that straddles two takes
  // twice the L2 requests
  P.row_stride = (P.H + kTcK - 1) / kTcK * kTcK;
  P.rows = reinterpret_cast<__nv_bfloat16*>(place(2ull * P.n_pad * P.row_stride));
  if (!backward) {
    P.label_logit = reinterpret_cast<float*>(place(4ull * P.n_pad));
    P.part = reinterpret_cast<float2*>(place(8ull * P.n_pad * ((P.V + kTcTile - 1) / kTcTile)));
    return at;
  }
  // G of a piece takes at most 256 MB, and a piece is a whole number of tiles: past 2^19
  // rows one, and up to 512 MB
  const long long all = (P.V + kTcTile - 1ll) / kTcTile * kTcTile;
  long long piece = (128ll << 20) / P.n_pad / kTcTile * kTcTile;
  if (piece < kTcTile) piece = kTcTile;
  P.piece = (int)(piece < all ? piece : all);
  // dh = G W sums over the whole piece, dW = G^T h over the rows: where few rows
  // make the former the longer chain, its k is split so that no tile has more than
  // about half of a pair's share of all stages (76 pairs)
  const long long rt = P.n_pad / kTcTile, ct = (P.H + kTcTile - 1) / kTcTile;
  const long long steps_x = P.piece / kTcK, rows_w = (P.n + kTcK - 1) / kTcK;
  const long long steps_w = rows_w > kStoreSteps ? rows_w : kStoreSteps;
  const long long share = (rt * ct * steps_x + P.piece / kTcTile * ct * steps_w) / 76;
  long long most = share / 2 < 8 ? 8 : share / 2;
  if (most < (steps_x + 63) / 64) most = (steps_x + 63) / 64;
  if (most > steps_x) most = steps_x;
  P.split_steps = (int)most;
  P.splits = (int)((steps_x + most - 1) / most);
  P.pos_of = reinterpret_cast<int*>(place(4ull * P.n));
  P.lse_c = reinterpret_cast<float*>(place(4ull * P.n_pad));
  P.g_c = reinterpret_cast<float*>(place(4ull * P.n_pad));
  P.label_g = reinterpret_cast<float*>(place(4ull * P.n_pad));
  P.soft = reinterpret_cast<__nv_bfloat16*>(place(2ull * P.n_pad * P.piece));
  P.acc = reinterpret_cast<float*>(place(4ull * P.splits * P.n_pad * P.H));
  return at;
}

}  // namespace sv
