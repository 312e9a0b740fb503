// linear_ce.cu -- softmax cross entropy of a vocabulary projection, in pieces
// of the vocabulary, without keeping the logits; and its gradients.
//
//   l = h W^T, lse_i = ln sum_v e^{l_iv}, loss_i = lse_i - l_{i, y_i};
//   G_iv = g_i (e^{l_iv - lse_i} - [v = y_i]),  dh = G W,  dW = G^T h.
//
// Rows without a label (and in the backward pass rows of weight 0) take no part:
// gather_rows copies the rows that count to the front of a compact matrix, so
// that a masked row costs nothing and a NaN in it reaches nothing, and fills it
// up with zero rows to a whole tile.
// Forward: one maximum and sum per row and vocabulary tile, merged by
// merge_rows.  Backward, for each piece of the vocabulary: G of the piece (the
// logits again, softmax in the epilogue), dW of the piece, and the piece's part
// of dh, summed in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rows.cuh"

namespace sv {
namespace {

constexpr int kGatherThreads = 256, kGatherRows = 32;

// The rows that count, in order: row_of, their labels, and their hidden states.
template <bool BWD>
__global__ void __launch_bounds__(kGatherThreads) gather_rows(const __grid_constant__ CeParams P) {
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
    const int r = r0 + lane;
    const bool v = r < P.n && counts(r);
    const unsigned vote = __ballot_sync(0xffffffffu, v);
    const int at = before + __popc(vote & ((1u << lane) - 1));
    s_row[lane] = v ? at : -1;
    if (v) {
      const int y = P.label[r];
      P.row_of[at] = r;
      P.lab[at] = y;
      if (BWD) {
        P.lse_c[at] = P.lse_in[r];
        P.g_c[at] = P.grad_loss ? P.grad_loss[r] : 1.f;
      }
    }
    if (BWD && r < P.n) P.pos_of[r] = v ? at : -1;
    if (!BWD && r < P.n && !v) {
      const int y = P.label[r];
      const float z = y == -1 ? 0.f : __int_as_float(0x7fc00000);
      P.loss[r] = z;
      P.lse[r] = z;
      if (P.status) P.status[r] = y == -1 ? SPEC_ST_OK : SPEC_ST_BAD_TOKEN;
    }
    if (blockIdx.x == 0 && lane == 0) *P.count = all;
  }
  __syncthreads();
  const int nv = P.H / 8;
  for (int i = warp; i < kGatherRows; i += kGatherThreads / 32) {
    if (s_row[i] >= 0) {
      const uint4* src = reinterpret_cast<const uint4*>(P.hidden + (size_t)(r0 + i) * P.H);
      uint4* dst = reinterpret_cast<uint4*>(P.rows + (size_t)s_row[i] * P.H);
      for (int k = lane; k < nv; k += 32) dst[k] = src[k];
    }
    const int at = r0 + i;                   // places past the last row that counts
    if (at >= all) {
      uint4* dst = reinterpret_cast<uint4*>(P.rows + (size_t)at * P.H);
      for (int k = lane; k < nv; k += 32) dst[k] = make_uint4(0, 0, 0, 0);
      if (lane == 0) {
        P.lab[at] = -1;
        if (BWD) { P.lse_c[at] = 0.f; P.g_c[at] = 0.f; }
      }
    }
  }
}

// 64 x 64 tile of sum_k A(i, k) B(j, k), 256 threads, 4 x 4 sums each.
struct Operand {
  const __nv_bfloat16* p;
  long long outer, inner;                    // strides of i (or j) and of k
  int limit;                                 // i (or j) below it
};
constexpr int kTile = 64, kStep = 16, kCeThreads = 256;

__device__ __forceinline__ void tile_product(const Operand& A, const Operand& B, int i0, int j0, int K,
                                             float (&acc)[4][4]) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  const int tid = threadIdx.x, ti = tid >> 4, tj = tid & 15;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = 0.f;
  for (int k0 = 0; k0 < K; k0 += kStep) {
    for (int t = tid; t < kTile * kStep; t += kCeThreads) {
      // neighbours along the operand's unit stride
      const int ia = A.inner == 1 ? t / kStep : t % kTile, ka = A.inner == 1 ? t % kStep : t / kTile;
      const int jb = B.inner == 1 ? t / kStep : t % kTile, kb = B.inner == 1 ? t % kStep : t / kTile;
      sa[ka][ia] = i0 + ia < A.limit && k0 + ka < K
                       ? __bfloat162float(A.p[(i0 + ia) * A.outer + (k0 + ka) * A.inner]) : 0.f;
      sb[kb][jb] = j0 + jb < B.limit && k0 + kb < K
                       ? __bfloat162float(B.p[(j0 + jb) * B.outer + (k0 + kb) * B.inner]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      float x[4], y[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) { x[a] = sa[k][ti * 4 + a]; y[a] = sb[k][tj * 4 + a]; }
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(x[a], y[b], acc[a][b]);
    }
    __syncthreads();
  }
}

// one vocabulary tile's maximum and sum of each row, and the label's logit
__global__ void __launch_bounds__(kCeThreads) ce_forward(const __grid_constant__ CeParams P) {
  const int i0 = blockIdx.y * kTile, v0 = blockIdx.x * kTile, count = *P.count;
  if (i0 >= count) return;
  float acc[4][4];
  tile_product({P.rows, P.H, 1, P.n_pad}, {P.weight, P.H, 1, P.V}, i0, v0, P.H, acc);
  const int ti = threadIdx.x >> 4, tj = threadIdx.x & 15;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = i0 + ti * 4 + a, y = P.lab[i];
    float m = -INFINITY;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int v = v0 + tj * 4 + b;
      if (v < P.V) {
        m = acc[a][b] != acc[a][b] ? INFINITY : fmaxf(m, acc[a][b]);   // a NaN makes the row's sum NaN below
        if (v == y) P.label_logit[i] = acc[a][b];
      }
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float s = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (v0 + tj * 4 + b < P.V) s += ex2((acc[a][b] - m) * kLog2eHi);
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (tj == 0) P.part[(size_t)blockIdx.x * P.n_pad + i] = make_float2(m, s);
  }
}

__global__ void __launch_bounds__(256) merge_rows(const __grid_constant__ CeParams P) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= *P.count) return;
  const int tiles = (P.V + kTile - 1) / kTile;
  float m = -INFINITY, s = 0.f;
  for (int t = 0; t < tiles; ++t) m = fmaxf(m, P.part[(size_t)t * P.n_pad + i].x);
  for (int t = 0; t < tiles; ++t) {
    const float2 p = P.part[(size_t)t * P.n_pad + i];
    s += p.y * ex2((p.x - m) * kLog2eHi);
  }
  const float lse = m + 0.693147180559945f * log2f(s);
  const bool ok = isfinite(m) && isfinite(lse);
  const int r = P.row_of[i];
  P.lse[r] = ok ? lse : __int_as_float(0x7fc00000);
  P.loss[r] = ok ? lse - P.label_logit[i] : __int_as_float(0x7fc00000);
  if (P.status) P.status[r] = ok ? SPEC_ST_OK : SPEC_ST_NONFINITE;
}

// G of vocabulary rows [v_begin, v_begin + piece) as bf16: the one rounding of G
// before the products that read it; the logits and the softmax are fp32
__global__ void __launch_bounds__(kCeThreads) ce_softmax(const __grid_constant__ CeParams P, int v_begin) {
  const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
  if (i0 >= P.n_pad) return;
  float acc[4][4];
  tile_product({P.rows, P.H, 1, P.n_pad}, {P.weight + (size_t)v_begin * P.H, P.H, 1, P.V - v_begin}, i0, j0, P.H, acc);
  const int ti = threadIdx.x >> 4, tj = threadIdx.x & 15;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int i = i0 + ti * 4 + a, y = P.lab[i];
    const float g = P.g_c[i], lse = P.lse_c[i];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int j = j0 + tj * 4 + b, v = v_begin + j;
      const float p = v < P.V && g != 0.f ? g * (ex2((acc[a][b] - lse) * kLog2eHi) - (v == y ? 1.f : 0.f)) : 0.f;
      P.soft[(size_t)i * P.piece + j] = __float2bfloat16_rn(p);
    }
  }
}

__global__ void __launch_bounds__(kCeThreads) ce_grad_weight(const __grid_constant__ CeParams P, int v_begin) {
  const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
  const int len = P.V - v_begin < P.piece ? P.V - v_begin : P.piece;
  if (i0 >= len) return;
  float acc[4][4];
  tile_product({P.soft, 1, P.piece, len}, {P.rows, 1, P.H, P.H}, i0, j0, *P.count, acc);
  const int ti = threadIdx.x >> 4, tj = threadIdx.x & 15;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int i = i0 + ti * 4 + a, j = j0 + tj * 4 + b;
      if (i < len && j < P.H) P.grad_weight[(size_t)(v_begin + i) * P.H + j] = __float2bfloat16_rn(acc[a][b]);
    }
}

__global__ void __launch_bounds__(kCeThreads) ce_grad_hidden(const __grid_constant__ CeParams P, int v_begin) {
  const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
  const int len = P.V - v_begin < P.piece ? P.V - v_begin : P.piece;
  if (i0 >= *P.count) return;
  float acc[4][4];
  tile_product({P.soft, P.piece, 1, P.n_pad}, {P.weight + (size_t)v_begin * P.H, 1, P.H, P.H}, i0, j0, len, acc);
  const int ti = threadIdx.x >> 4, tj = threadIdx.x & 15;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int i = i0 + ti * 4 + a, j = j0 + tj * 4 + b;
      if (j < P.H) {
        float* at = P.acc + (size_t)i * P.H + j;
        *at = v_begin == 0 ? acc[a][b] : *at + acc[a][b];
      }
    }
}

// every row of dh: its sum, or zeros where the row took no part
__global__ void __launch_bounds__(256) scatter_rows(const __grid_constant__ CeParams P) {
  const long long total = (long long)P.n * P.H;
  for (long long t = blockIdx.x * 256ll + threadIdx.x; t < total; t += gridDim.x * 256ll) {
    const int r = (int)(t / P.H), pos = P.pos_of[r];
    P.grad_hidden[t] = __float2bfloat16_rn(pos < 0 ? 0.f : P.acc[(size_t)pos * P.H + t % P.H]);
  }
}

}  // namespace

cudaError_t launch_ce_forward(const CeParams& P, int nsm, cudaStream_t s, int* launches) {
  gather_rows<false><<<P.n_pad / kGatherRows, kGatherThreads, 0, s>>>(P);
  ce_forward<<<dim3((P.V + kTile - 1) / kTile, P.n_pad / kTile), kCeThreads, 0, s>>>(P);
  merge_rows<<<(P.n_pad + 255) / 256, 256, 0, s>>>(P);
  *launches = 3;
  return cudaGetLastError();
}

cudaError_t launch_ce_backward(const CeParams& P, int nsm, cudaStream_t s, int* launches) {
  gather_rows<true><<<P.n_pad / kGatherRows, kGatherThreads, 0, s>>>(P);
  int n = 1;
  const int hb = (P.H + kTile - 1) / kTile;
  for (int v = 0; v < P.V; v += P.piece) {
    ce_softmax<<<dim3(P.piece / kTile, P.n_pad / kTile), kCeThreads, 0, s>>>(P, v);
    ++n;
    if (P.grad_weight) { ce_grad_weight<<<dim3(hb, P.piece / kTile), kCeThreads, 0, s>>>(P, v); ++n; }
    if (P.grad_hidden) { ce_grad_hidden<<<dim3(hb, P.n_pad / kTile), kCeThreads, 0, s>>>(P, v); ++n; }
    if (v > P.V - P.piece) break;            // the last piece (v + piece may pass 2^31 - 1)
  }
  if (P.grad_hidden) { scatter_rows<<<4 * nsm, 256, 0, s>>>(P); ++n; }
  *launches = n;
  return cudaGetLastError();
}

size_t ce_layout(CeParams& P, bool backward, void* base) {
  unsigned char* b = static_cast<unsigned char*>(base);
  size_t at = 0;
  auto place = [&](size_t bytes) {
    unsigned char* p = b ? b + at : nullptr;
    at = (at + bytes + 255) / 256 * 256;
    return p;
  };
  P.n_pad = (P.n + kCeRowTile - 1) / kCeRowTile * kCeRowTile;
  P.count = reinterpret_cast<int*>(place(256));
  P.row_of = reinterpret_cast<int*>(place(4ull * P.n_pad));
  P.lab = reinterpret_cast<int*>(place(4ull * P.n_pad));
  P.rows = reinterpret_cast<__nv_bfloat16*>(place(2ull * P.n_pad * P.H));
  if (!backward) {
    P.label_logit = reinterpret_cast<float*>(place(4ull * P.n_pad));
    P.part = reinterpret_cast<float2*>(place(8ull * P.n_pad * ((P.V + kTile - 1) / kTile)));
    return at;
  }
  // G of a piece takes at most about 256 MB, and a piece is a whole number of tiles
  const long long all = (P.V + kCeVocabTile - 1ll) / kCeVocabTile * kCeVocabTile;
  long long piece = (128ll << 20) / P.n_pad / kCeVocabTile * kCeVocabTile;
  if (piece < kCeVocabTile) piece = kCeVocabTile;
  P.piece = (int)(piece < all ? piece : all);
  P.pos_of = reinterpret_cast<int*>(place(4ull * P.n));
  P.lse_c = reinterpret_cast<float*>(place(4ull * P.n_pad));
  P.g_c = reinterpret_cast<float*>(place(4ull * P.n_pad));
  P.soft = reinterpret_cast<__nv_bfloat16*>(place(2ull * P.n_pad * P.piece));
  P.acc = reinterpret_cast<float*>(place(4ull * P.n_pad * P.H));
  return at;
}

}  // namespace sv
