// api_serve.cu -- host side of the calls around the vocabulary rows of a decode
// step: argument checks and launches on the caller's stream.
#include <atomic>
#include <mutex>

#include "serve.cuh"

using namespace sv;

namespace {

// Kernels are configured on the first call that needs them, on each device.
enum Family { kW4, kAdjust, kFamilies };
bool g_ready[kFamilies][kMaxDevices];
std::mutex g_serve_mu;

int serving_state(Family f, int* sms) {
  int dev = 0;
  const int rc = current_device(&dev, sms);
  if (rc != SPEC_OK) return rc;
  std::lock_guard<std::mutex> lk(g_serve_mu);
  if (!g_ready[f][dev]) {
    if ((f == kW4 ? configure_w4() : configure_adjust()) != cudaSuccess) return SPEC_ERR_CUDA;
    g_ready[f][dev] = true;
  }
  return SPEC_OK;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + bn && y < x + an;
}
size_t size_of(int dtype) { return dtype == SPEC_BF16 ? 2 : 4; }
bool logit_type(int dtype) { return dtype == SPEC_F32 || dtype == SPEC_BF16; }

bool w4_ok(W4Params& P, int H, int V, int group, const void* packed, const void* scale, const void* zero) {
  if (V < 1 || V >= (1 << 28) || H < 32 || H > 65536 || H % 32 || (group != 32 && group != 64 && group != 128)) return false;
  if (!packed || !scale || !aligned(packed, 16) || !aligned(scale, 2)) return false;
  P.H = H; P.V = V; P.group = group; P.groups = (H + group - 1) / group;
  P.packed = static_cast<uint32_t*>(const_cast<void*>(packed));
  P.scale = static_cast<__nv_bfloat16*>(const_cast<void*>(scale));
  P.zero = static_cast<uint8_t*>(const_cast<void*>(zero));
  return true;
}
// whether [p, p + bytes) overlaps the packed weights, their scales or zero points
bool on_weights(const W4Params& P, const void* p, size_t bytes) {
  const size_t per = (size_t)P.V * P.groups;
  return overlap(p, bytes, P.packed, (size_t)P.V * P.H / 2) || overlap(p, bytes, P.scale, 2 * per) ||
         overlap(p, bytes, P.zero, per);
}
int after(cudaError_t e) {
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  count_launches(1);
  return SPEC_OK;
}

}  // namespace

extern "C" {

int spec_w4_quantize(const void* weight, int dtype, int V, int H, int group, uint8_t* packed, void* scale, uint8_t* zero,
                     int32_t* status, spec_stream_t stream) {
  W4Params P{};
  if (!w4_ok(P, H, V, group, packed, scale, zero) || !weight || !logit_type(dtype)) return SPEC_ERR_INVALID_ARG;
  const size_t per = (size_t)V * P.groups, bytes = size_of(dtype) * (size_t)V * H;
  if (!aligned(weight, 16) || !aligned(status, 4)) return SPEC_ERR_INVALID_ARG;
  if (on_weights(P, weight, bytes) || on_weights(P, status, 4 * (size_t)V) || overlap(status, 4 * (size_t)V, weight, bytes) ||
      overlap(packed, (size_t)V * H / 2, scale, 2 * per) || overlap(packed, (size_t)V * H / 2, zero, per) ||
      overlap(scale, 2 * per, zero, per))
    return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = serving_state(kW4, &sms);
  if (rc != SPEC_OK) return rc;
  P.weight = static_cast<const unsigned char*>(weight);
  P.dtype = dtype; P.status = status;
  return after(launch_w4_quantize(P, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int spec_w4_dequantize(const uint8_t* packed, const void* scale, const uint8_t* zero, int V, int H, int group, void* weight,
                       int dtype, spec_stream_t stream) {
  W4Params P{};
  if (!w4_ok(P, H, V, group, packed, scale, zero) || !weight || !logit_type(dtype)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(weight, 16) || on_weights(P, weight, size_of(dtype) * (size_t)V * H)) return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = serving_state(kW4, &sms);
  if (rc != SPEC_OK) return rc;
  P.out = weight; P.dtype = dtype;
  return after(launch_w4_dequantize(P, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int spec_linear_w4(const void* hidden, int dtype, int n, const uint8_t* packed, const void* scale, const uint8_t* zero, int V,
                   int H, int group, void* logits, int logits_dtype, spec_stream_t stream) {
  W4Params P{};
  if (!w4_ok(P, H, V, group, packed, scale, zero) || !hidden || !logits || dtype != SPEC_BF16 || !logit_type(logits_dtype))
    return SPEC_ERR_INVALID_ARG;
  // tiles of 16 rows and 128 columns or more are counted in 32 bits
  if (n < 1 || n > (1 << 20) || ((n + 15ll) / 16) * ((V + 127ll) / 128) >= (1ll << 30)) return SPEC_ERR_INVALID_ARG;
  const size_t bytes = size_of(logits_dtype) * (size_t)n * V;
  if (!aligned(hidden, 16) || !aligned(logits, size_of(logits_dtype))) return SPEC_ERR_INVALID_ARG;
  if (on_weights(P, logits, bytes) || overlap(logits, bytes, hidden, 2 * (size_t)n * H)) return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = serving_state(kW4, &sms);
  if (rc != SPEC_OK) return rc;
  P.hidden = static_cast<const __nv_bfloat16*>(hidden);
  P.n = n; P.out = logits; P.dtype = logits_dtype;
  P.wait_limit = current_wait_limit();
  return after(launch_w4_linear(P, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int spec_adjust_logits(const void* logits, void* out, int dtype, int B, int R, int V, const int32_t* history, int L,
                       const int32_t* history_len, const int32_t* prompt_len, const int32_t* draft_tokens, int D,
                       const int32_t* gamma, const float* repetition, const float* frequency, const float* presence,
                       const int32_t* bias_index, const float* bias_value, int biases, const uint32_t* mask, int32_t* status,
                       spec_stream_t stream) {
  if (B < 1 || B > SPEC_MAX_B || R < 1 || R > SPEC_MAX_G + 1 || V < 2 || V >= (1 << 28) || !logits || !out || !logit_type(dtype))
    return SPEC_ERR_INVALID_ARG;
  if (L < 0 || L > SPEC_MAX_HISTORY || (L > 0 && !history) || D < 0 || D > SPEC_MAX_G + 1 || (D > 0 && !draft_tokens) ||
      biases < 0 || biases > SPEC_MAX_BIASES || (biases > 0 && (!bias_index || !bias_value)))
    return SPEC_ERR_INVALID_ARG;
  if (D > 0 && D < R - 1) return SPEC_ERR_INVALID_ARG;               // row i sees y_0 .. y_{i - 1}
  const size_t es = size_of(dtype), bytes = es * (size_t)B * R * V;
  if (!aligned(logits, es) || !aligned(out, es)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {history, history_len, prompt_len, draft_tokens, gamma, repetition, frequency, presence, bias_index,
                         bias_value, mask, status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  if (out != logits && overlap(logits, bytes, out, bytes)) return SPEC_ERR_INVALID_ARG;
  // what a CTA reads, another may not write
  const size_t b4 = 4 * (size_t)B;
  const struct { const void* p; size_t bytes; } read[] = {
      {history, b4 * L}, {history_len, b4}, {prompt_len, b4}, {draft_tokens, b4 * D}, {gamma, b4}, {repetition, b4},
      {frequency, b4}, {presence, b4}, {bias_index, b4 * biases}, {bias_value, b4 * biases},
      {mask, b4 * R * ((V + 31ll) / 32)}};
  for (const auto& r : read)
    if (overlap(out, bytes, r.p, r.bytes) || overlap(status, b4, r.p, r.bytes)) return SPEC_ERR_INVALID_ARG;
  if (overlap(status, b4, logits, bytes) || overlap(status, b4, out, bytes)) return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = serving_state(kAdjust, &sms);
  if (rc != SPEC_OK) return rc;
  AdjustParams P{};
  P.in = static_cast<const unsigned char*>(logits);
  P.out = static_cast<unsigned char*>(out);
  P.dtype = dtype; P.B = B; P.R = R; P.V = V;
  P.history = history; P.history_len = history_len; P.prompt_len = prompt_len; P.L = L;
  P.draft = draft_tokens; P.gamma = gamma; P.D = D;
  P.repetition = repetition; P.frequency = frequency; P.presence = presence;
  P.bias_index = bias_index; P.bias_value = bias_value; P.biases = biases;
  P.mask = mask; P.status = status;
  return after(launch_adjust(P, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
