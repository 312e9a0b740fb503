// api.cu -- the C ABI declared in include/spec_verify.h.
//
// Host side only: argument checks, workspace layout, and the two launches of
// one call on the caller's stream:
//   plan_kernel    (1 CTA)        resets counters, settles requests with bad
//                                 arguments, builds the row schedule;
//   verify_kernel  (persistent)   streams the needed logit rows, decides each
//                                 position as soon as its rows are in, and
//                                 runs each request's final draw.
// The second launch uses programmatic dependent launch, so its start-up
// overlaps the plan kernel; it waits on griddepcontrol.wait before reading
// the schedule.  The plan kernel is launched without it, so it starts only
// after all earlier work on the stream (which may be producing the inputs).
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "common.cuh"

using namespace sv;

namespace {

thread_local uint64_t g_launches = 0;
std::atomic<long long> g_wait_limit{kWaitLimitCycles};   // spec_set_wait_limit
thread_local cudaEvent_t g_prof_begin = nullptr, g_prof_end = nullptr;

// Kernels configured together, on the first call that needs them: what one family asks of
// the device does not hold up, or fail, the calls of another.
enum Family { kVerification, kRecord, kDistill, kLinearCe, kFamilies };

struct DevState {
  bool known = false;
  int sms = 0;        // multiprocessors
  int ctas = 0;       // resident verify CTAs on the device (SMs x CTAs per SM, at most 2 per SM)
  int status = SPEC_OK;                    // whether the device runs the library's code
  bool ready[kFamilies] = {};
  int verification = SPEC_OK;              // of a ready kVerification
};
DevState g_dev[kMaxDevices];
std::mutex g_mu;

cudaError_t configure(Family f, int dev) {
  switch (f) {
    case kRecord: return configure_record(dev);
    case kDistill: return configure_distill(dev);
    case kLinearCe: return configure_linear_ce();
    default: return configure_kernels();
  }
}

// The current device, with the kernels of `f` configured.
int device_for(Family f, int* device, DevState** state) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPEC_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return SPEC_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_mu);
  DevState& d = g_dev[dev];
  *device = dev;
  *state = &d;
  if (!d.known) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SPEC_ERR_CUDA;
    if (major != 10 || minor != 3) d.status = SPEC_ERR_UNSUPPORTED;   // the library carries sm_103a code only
    d.known = true;
  }
  if (d.status != SPEC_OK) return d.status;
  if (!d.ready[f]) {
    if (configure(f, dev) != cudaSuccess) return SPEC_ERR_CUDA;
    if (f == kVerification) {
      int per_sm = 0;
      if (verify_blocks_per_sm(&per_sm) != cudaSuccess) return SPEC_ERR_CUDA;
      d.verification = per_sm < 1 ? SPEC_ERR_UNSUPPORTED : SPEC_OK;
      d.ctas = d.sms * (per_sm < 2 ? per_sm : 2);
    }
    d.ready[f] = true;
  }
  return f == kVerification ? d.verification : SPEC_OK;
}

// For the verification calls and those beside them: resident verify CTAs.
int device_state(int* ctas) {
  int dev = 0;
  DevState* d = nullptr;
  const int rc = device_for(kVerification, &dev, &d);
  if (rc == SPEC_OK) *ctas = d->ctas;
  return rc;
}

// For the drafter-training calls: the device and its multiprocessors.
int training_state(Family f, int* dev, int* sms) {
  DevState* d = nullptr;
  const int rc = device_for(f, dev, &d);
  if (rc == SPEC_OK) *sms = d->sms;
  return rc;
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + bn && y < x + an;
}

bool ce_sizes_ok(int n, int H, int V) {
  // tiles of 256 x 256 logits are counted in 32 bits
  return n >= 1 && n <= (1 << 20) && H >= 8 && H <= 65536 && H % 8 == 0 && V >= 2 && V < (1 << 28) &&
         ((n + 255ll) / 256) * ((V + 255ll) / 256) < (1ll << 30);
}

bool sizes_ok(int B, int G, int V) {
  if (B < 1 || B > SPEC_MAX_B || G < 0 || G > SPEC_MAX_G || V < 2 || V >= (1 << 28)) return false;
  // work items, draw-queue and deferred-queue entries are counted in 32 bits
  const long long ce = chunk_elems(SPEC_F32), se = stage_elems(SPEC_F32);
  const long long rows = (long long)B * (2 * G + 1);
  const long long nch = (V + ce - 1) / ce, nres = (V + se - 1) / se;
  return rows * nch < (1ll << 31) && (long long)B * (kMaxDrawRounds * nres + 2 * G * nch + 2) < (1ll << 31);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Call {
  int mode;
  const void* target;
  const void* draft;
  int dtype, B, G, V;
  const int32_t* draft_tokens;
  const int32_t* gamma;
  const float* temperature;
  const float* uniforms;
  int32_t* accept_len;
  int32_t* tokens;
  int32_t* status;
  float* signals;
  float* row_signals;
  float* accept_prob;
  void* workspace;
  size_t workspace_bytes;
  cudaStream_t stream;
};

int run(const Call& c) {
  if (!sizes_ok(c.B, c.G, c.V) || (c.dtype != SPEC_F32 && c.dtype != SPEC_BF16)) return SPEC_ERR_INVALID_ARG;
  const size_t es = c.dtype == SPEC_BF16 ? 2 : 4;
  const bool greedy = c.mode == MODE_GREEDY, sample = c.mode == MODE_SAMPLE, sig = c.mode == MODE_SIGNALS;
  // required pointers
  if (!sig && (!c.target || !c.accept_len || !c.tokens)) return SPEC_ERR_INVALID_ARG;
  if (!sig && c.G > 0 && !c.draft_tokens) return SPEC_ERR_INVALID_ARG;
  if ((sample || sig) && c.G > 0 && !c.draft) return SPEC_ERR_INVALID_ARG;
  if (!greedy && !c.temperature) return SPEC_ERR_INVALID_ARG;
  if ((sample || c.mode == MODE_ONEHOT) && !c.uniforms) return SPEC_ERR_INVALID_ARG;
  if (sig && !c.signals) return SPEC_ERR_INVALID_ARG;
  if (!aligned(c.target, es) || !aligned(c.draft, es)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {c.draft_tokens, c.gamma, c.temperature, c.uniforms, c.accept_len, c.tokens,
                         c.status, c.signals, c.row_signals, c.accept_prob};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  const Layout L = make_layout(c.B, c.G, c.V, c.dtype);
  if (!c.workspace || c.workspace_bytes < L.total) return SPEC_ERR_WORKSPACE;
  if (!aligned(c.workspace, 256)) return SPEC_ERR_INVALID_ARG;
  int ctas = 0;
  const int ds = device_state(&ctas);
  if (ds != SPEC_OK) return ds;

  unsigned char* ws = static_cast<unsigned char*>(c.workspace);
  Params P{};
  P.target = static_cast<const unsigned char*>(c.target);
  P.draft = static_cast<const unsigned char*>(c.draft);
  P.dtype = c.dtype; P.B = c.B; P.G = c.G; P.V = c.V; P.mode = c.mode;
  P.signals_on = sig ? 1 : (sample && c.signals ? 1 : 0);
  P.draft_tokens = c.draft_tokens; P.gamma = c.gamma; P.temperature = c.temperature; P.uniforms = c.uniforms;
  P.accept_len = c.accept_len; P.tokens = c.tokens; P.status = c.status;
  P.signals = c.signals; P.row_signals = c.row_signals; P.accept_prob = c.accept_prob;
  P.hdr = reinterpret_cast<Header*>(ws + L.hdr);
  P.req_flags = reinterpret_cast<int*>(ws + L.req_flags);
  P.known_reject = reinterpret_cast<int*>(ws + L.known_reject);
  P.row_list = reinterpret_cast<int*>(ws + L.row_list);
  P.req_scale = reinterpret_cast<float*>(ws + L.req_scale);
  P.req_scale_lo = reinterpret_cast<float*>(ws + L.req_scale_lo);
  P.req_ks = reinterpret_cast<float*>(ws + L.req_ks);
  P.req_gam = reinterpret_cast<int*>(ws + L.req_gam);
  P.req_status = reinterpret_cast<int*>(ws + L.req_status);
  P.req_fin = reinterpret_cast<unsigned*>(ws + L.req_fin);
  P.cparts = reinterpret_cast<tword*>(ws + L.cparts);
  P.dsum = reinterpret_cast<tword*>(ws + L.dsum);
  P.gsum = reinterpret_cast<tword*>(ws + L.gsum);
  P.dd = reinterpret_cast<tword*>(ws + L.dd);
  P.dq = reinterpret_cast<tword*>(ws + L.dq);
  P.claim = reinterpret_cast<tword*>(ws + L.claim);
  P.defq = reinterpret_cast<tword*>(ws + L.defq);
  P.nrows = L.nrows; P.nch = L.nch; P.nres = L.nres; P.dq_cap = L.dq_cap; P.def_cap = L.def_cap;
  // Lookahead: greedy and sample calls read every row in position-major order
  // and skip the rows past a decided reject (a dependency per position, a
  // read issued only once the position before is accepted, would put a full
  // pipeline latency on every step of a long chain).  A one-hot call reads
  // the target rows of positions 0 and 1 up front and the row of position
  // i + 2 once position i is accepted (its drafts are rejected early: most
  // later rows are not needed).
  P.lookahead = c.mode == MODE_ONEHOT ? 2 : c.G + 1;
  P.aligned_rows = ((size_t)c.V * es) % 16 == 0 && aligned(c.target, 16) && aligned(c.draft, 16);
  P.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  // Rows a draw may read again (positions 0 .. keep_pos, both models in the
  // full-q mode) are loaded with an evict-last L2 policy, as long as they
  // fill at most 3/4 of the 129 MB L2 of a GB300; the draw then reads them
  // from L2.  Calls without draws keep nothing.
  P.keep_pos = -1;
  if (sample || c.mode == MODE_ONEHOT) {
    const double per_pos = (double)c.B * (sample ? 2 : 1) * c.V * es;
    const double budget = 0.75 * 129.0 * 1024 * 1024;
    for (int j = 0; j <= c.G && (j + 1) * per_pos <= budget; ++j) P.keep_pos = j;
  }

  // persistent grid: every CTA resident at once (two per SM), never more
  // CTAs than work items
  const long long max_items = (long long)c.B * (2 * c.G + 1) * L.nch;
  const int grid1 = (int)(max_items < (long long)ctas ? max_items : (long long)ctas);
  const cudaEvent_t pb = g_prof_begin, pe = g_prof_end;
  g_prof_begin = g_prof_end = nullptr;
  cudaError_t e = launch_plan(P, c.stream);
  if (e == cudaSuccess) {
    ++g_launches;
    if (pb) e = cudaEventRecord(pb, c.stream);
  }
  if (e == cudaSuccess) e = launch_verify(P, grid1 > 0 ? grid1 : 1, c.stream, pb == nullptr);
  if (e == cudaSuccess) {
    ++g_launches;
    if (pe) e = cudaEventRecord(pe, c.stream);
  }
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// Library-owned scratch of spec_verify_sample_static (one per device: a
// __device__ variable lives in each context that loads the module).
static __device__ __align__(256) unsigned char g_static_ws[SPEC_STATIC_WORKSPACE_BYTES];

// Device address of g_static_ws on the current device, looked up once per
// device with that device current.
void* g_static_addr[kMaxDevices] = {};

int static_workspace(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPEC_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return SPEC_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_static_addr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_static_ws) != cudaSuccess || p == nullptr) return SPEC_ERR_CUDA;
    g_static_addr[dev] = p;
  }
  *out = g_static_addr[dev];
  return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_workspace_bytes(int B, int G, int V) {
  if (!sizes_ok(B, G, V)) return 0;
  const Layout a = make_layout(B, G, V, SPEC_F32), b = make_layout(B, G, V, SPEC_BF16);
  return a.total > b.total ? a.total : b.total;
}

const char* spec_status_string(int code) {
  switch (code) {
    case SPEC_OK: return "ok";
    case SPEC_ERR_INVALID_ARG: return "invalid argument";
    case SPEC_ERR_WORKSPACE: return "workspace missing or too small";
    case SPEC_ERR_CUDA: return "CUDA launch or runtime error";
    case SPEC_ERR_UNSUPPORTED: return "device is not sm_103";
    default: break;
  }
  return "unknown code";
}

const char* spec_request_status_string(int bit) {
  switch (bit) {
    case SPEC_ST_OK: return "ok";
    case SPEC_ST_NONFINITE: return "non-finite logits in a row that was read";
    case SPEC_ST_BAD_TOKEN: return "draft token outside [0, V)";
    case SPEC_ST_BAD_GAMMA: return "gamma outside [0, G]";
    case SPEC_ST_ZERO_RESIDUAL: return "residual mass rounded to zero; drew from p";
    case SPEC_ST_GUARDED: return "near-tie draw taken again in extended precision (informational)";
    case SPEC_ST_TIMEOUT: return "internal wait timed out";
    case SPEC_ST_BAD_TEMPERATURE: return "temperature not positive and finite";
    case SPEC_ST_BAD_UNIFORM: return "uniform outside [0, 1)";
    default: break;
  }
  return "unknown status bit";
}

uint64_t spec_launch_count(void) { return g_launches; }

int spec_set_wait_limit(long long cycles) {
  g_wait_limit.store(cycles > 0 ? cycles : kWaitLimitCycles, std::memory_order_relaxed);
  return SPEC_OK;
}

int spec_profile_next_call(void* begin_event, void* end_event) {
  g_prof_begin = static_cast<cudaEvent_t>(begin_event);
  g_prof_end = static_cast<cudaEvent_t>(end_event);
  return SPEC_OK;
}

int spec_verify_greedy(const void* target_logits, int dtype, int B, int G, int V, const int32_t* draft_tokens,
                       const int32_t* gamma, int32_t* accept_len, int32_t* tokens, int32_t* status,
                       void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  Call c{MODE_GREEDY, target_logits, nullptr, dtype, B, G, V, draft_tokens, gamma, nullptr, nullptr,
         accept_len, tokens, status, nullptr, nullptr, nullptr, workspace, workspace_bytes,
         reinterpret_cast<cudaStream_t>(stream)};
  return run(c);
}

int spec_verify_sample(const void* target_logits, const void* draft_logits, int dtype, int B, int G, int V,
                       const int32_t* draft_tokens, const int32_t* gamma, const float* temperature,
                       const float* uniforms, int32_t* accept_len, int32_t* tokens, float* signals,
                       float* accept_prob, int32_t* status, void* workspace, size_t workspace_bytes,
                       spec_stream_t stream) {
  Call c{MODE_SAMPLE, target_logits, draft_logits, dtype, B, G, V, draft_tokens, gamma, temperature, uniforms,
         accept_len, tokens, status, signals, nullptr, accept_prob, workspace, workspace_bytes,
         reinterpret_cast<cudaStream_t>(stream)};
  return run(c);
}

int spec_verify_sample_static(const void* target_logits, const void* draft_logits, int dtype, int B, int G,
                              int V, const int32_t* draft_tokens, const int32_t* gamma, const float* temperature,
                              const float* uniforms, int32_t* accept_len, int32_t* tokens, float* signals,
                              float* accept_prob, int32_t* status, spec_stream_t stream) {
  // size checks first: nothing touches the device when they fail
  const size_t need = spec_workspace_bytes(B, G, V);
  if (need == 0) return SPEC_ERR_INVALID_ARG;
  if (need > (size_t)SPEC_STATIC_WORKSPACE_BYTES) return SPEC_ERR_WORKSPACE;
  void* ws = nullptr;
  const int rc = static_workspace(&ws);
  if (rc != SPEC_OK) return rc;
  Call c{MODE_SAMPLE, target_logits, draft_logits, dtype, B, G, V, draft_tokens, gamma, temperature, uniforms,
         accept_len, tokens, status, signals, nullptr, accept_prob, ws, (size_t)SPEC_STATIC_WORKSPACE_BYTES,
         reinterpret_cast<cudaStream_t>(stream)};
  return run(c);
}

int spec_verify_onehot(const void* target_logits, int dtype, int B, int G, int V, const int32_t* draft_tokens,
                       const int32_t* gamma, const float* temperature, const float* uniforms, int32_t* accept_len,
                       int32_t* tokens, float* accept_prob, int32_t* status, void* workspace,
                       size_t workspace_bytes, spec_stream_t stream) {
  Call c{MODE_ONEHOT, target_logits, nullptr, dtype, B, G, V, draft_tokens, gamma, temperature, uniforms,
         accept_len, tokens, status, nullptr, nullptr, accept_prob, workspace, workspace_bytes,
         reinterpret_cast<cudaStream_t>(stream)};
  return run(c);
}

int spec_divergence_stats(const void* target_logits, const void* draft_logits, int dtype, int B, int G, int V,
                          const int32_t* gamma, const float* temperature, float* stats, int32_t* status,
                          spec_stream_t stream) {
  if (!sizes_ok(B, G, V) || (dtype != SPEC_F32 && dtype != SPEC_BF16)) return SPEC_ERR_INVALID_ARG;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (!temperature || (G > 0 && (!target_logits || !draft_logits || !stats))) return SPEC_ERR_INVALID_ARG;
  if (!aligned(target_logits, es) || !aligned(draft_logits, es)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {gamma, temperature, stats, status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  int ctas = 0;
  const int ds = device_state(&ctas);
  if (ds != SPEC_OK) return ds;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (status && cudaMemsetAsync(status, 0, sizeof(int32_t) * (size_t)B, s) != cudaSuccess) return SPEC_ERR_CUDA;
  if (G == 0) return SPEC_OK;
  int dev = 0, nsm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SPEC_ERR_CUDA;
  DivParams P{};
  P.target = static_cast<const unsigned char*>(target_logits);
  P.draft = static_cast<const unsigned char*>(draft_logits);
  P.dtype = dtype; P.B = B; P.G = G; P.V = V;
  P.aligned = ((size_t)V * es) % 16 == 0 && aligned(target_logits, 16) && aligned(draft_logits, 16);
  P.gamma = gamma; P.temperature = temperature; P.stats = stats; P.status = status;
  const long long pairs = (long long)B * G;
  const int grid = (int)(pairs < (long long)nsm ? pairs : (long long)nsm);
  if (launch_divergence(P, grid, s) != cudaSuccess) return SPEC_ERR_CUDA;
  ++g_launches;
  return SPEC_OK;
}

int spec_filter_top_k_top_p(void* logits, int dtype, int n, int V, const int32_t* top_k, const float* top_p,
                            const float* temperature, int32_t* status, spec_stream_t stream) {
  if (n < 1 || V < 2 || V >= (1 << 28) || !logits || (dtype != SPEC_F32 && dtype != SPEC_BF16))
    return SPEC_ERR_INVALID_ARG;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (!aligned(logits, es)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {top_k, top_p, temperature, status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  int ctas = 0;
  const int ds = device_state(&ctas);
  if (ds != SPEC_OK) return ds;
  FiltParams P{};
  P.logits = static_cast<unsigned char*>(logits);
  P.dtype = dtype; P.n = n; P.V = V;
  P.top_k = top_k; P.top_p = top_p; P.temperature = temperature; P.status = status;
  const int grid = n < ctas ? n : ctas;   // one row per resident CTA at a time (two per SM)
  if (launch_filter(P, grid > 0 ? grid : 1, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return SPEC_ERR_CUDA;
  ++g_launches;
  return SPEC_OK;
}

int spec_gamma_select(const float* signals, const float* comp, const float* model, int B, int32_t* gamma_star,
                      float* expected, spec_stream_t stream) {
  if (B < 1 || B > SPEC_MAX_B || !signals || !model || !gamma_star) return SPEC_ERR_INVALID_ARG;
  if (!aligned(signals, 16)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {comp, model, gamma_star, expected};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  int ctas = 0;
  const int ds = device_state(&ctas);
  if (ds != SPEC_OK) return ds;
  if (launch_gamma_select(signals, comp, model, B, gamma_star, expected, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return SPEC_ERR_CUDA;
  ++g_launches;
  return SPEC_OK;
}

int spec_topk_logits(const void* logits, int dtype, int n, int V, int K, const float* temperature, float* top_logits,
                     int32_t* top_index, float* tail_lse, int32_t* status, spec_stream_t stream) {
  if (n < 1 || n > (1 << 30) || V < 2 || V >= (1 << 28) || K < 1 || K > SPEC_MAX_TOPK || K > V) return SPEC_ERR_INVALID_ARG;
  if (!logits || !top_logits || !top_index || !tail_lse || (dtype != SPEC_F32 && dtype != SPEC_BF16))
    return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {temperature, top_logits, top_index, tail_lse, status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(logits, dtype == SPEC_BF16 ? 2 : 4)) return SPEC_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  const int ds = training_state(kRecord, &dev, &sms);
  if (ds != SPEC_OK) return ds;
  RecordParams P{};
  P.logits = static_cast<const unsigned char*>(logits);
  P.dtype = dtype; P.n = n; P.V = V; P.K = K;
  P.temperature = temperature;
  P.top_logits = top_logits; P.top_index = top_index; P.tail_lse = tail_lse; P.status = status;
  P.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  if (launch_record(P, dev, sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return SPEC_ERR_CUDA;
  ++g_launches;
  return SPEC_OK;
}

int spec_distill_topk(const void* logits, int dtype, int n, int V, int K, const float* top_logits,
                      const int32_t* top_index, const float* tail_lse, const int32_t* label, const float* row_weight,
                      const float* temperature, float kl, float tv, float ce, float* loss, float* parts,
                      void* grad_logits, int32_t* status, spec_stream_t stream) {
  if (n < 1 || n > (1 << 30) || V < 2 || V > SPEC_DISTILL_MAX_V || K < 1 || K > SPEC_MAX_TOPK) return SPEC_ERR_INVALID_ARG;
  if (!logits || !top_logits || !top_index || !loss || (dtype != SPEC_F32 && dtype != SPEC_BF16))
    return SPEC_ERR_INVALID_ARG;
  if (!std::isfinite(kl) || !std::isfinite(tv) || !std::isfinite(ce)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {top_logits, top_index, tail_lse, label, row_weight, temperature, loss, parts, status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (!aligned(logits, es) || !aligned(grad_logits, es)) return SPEC_ERR_INVALID_ARG;
  if (grad_logits && grad_logits != logits) {        // in place, or apart
    if (overlap(logits, (size_t)n * V * es, grad_logits, (size_t)n * V * es)) return SPEC_ERR_INVALID_ARG;
  }
  int dev = 0, sms = 0;
  const int ds = training_state(kDistill, &dev, &sms);
  if (ds != SPEC_OK) return ds;
  DistillParams P{};
  P.logits = static_cast<const unsigned char*>(logits);
  P.dtype = dtype; P.n = n; P.V = V; P.K = K;
  P.top_logits = top_logits; P.top_index = top_index; P.tail_lse = tail_lse;
  P.label = label; P.row_weight = row_weight; P.temperature = temperature;
  P.kl = kl; P.tv = tv; P.ce = ce;
  P.loss = loss; P.parts = parts; P.status = status;
  P.grad = static_cast<unsigned char*>(grad_logits);
  P.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  if (launch_distill(P, dev, sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return SPEC_ERR_CUDA;
  ++g_launches;
  return SPEC_OK;
}

size_t spec_linear_ce_workspace_bytes(int n, int H, int V, int backward) {
  if (!ce_sizes_ok(n, H, V)) return 0;
  CeParams P{};
  P.n = n; P.H = H; P.V = V;
  return ce_layout(P, backward != 0, nullptr);
}

int spec_linear_ce_forward(const void* hidden, const void* weight, int dtype, int n, int H, int V,
                           const int32_t* label, float* loss, float* lse, int32_t* status, void* workspace,
                           size_t workspace_bytes, spec_stream_t stream) {
  if (!ce_sizes_ok(n, H, V) || dtype != SPEC_BF16 || !hidden || !weight || !label || !loss || !lse)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(weight, 16)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {label, loss, lse, status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  CeParams P{};
  P.n = n; P.H = H; P.V = V;
  if (!workspace || workspace_bytes < ce_layout(P, false, workspace)) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SPEC_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  const int ds = training_state(kLinearCe, &dev, &sms);
  if (ds != SPEC_OK) return ds;
  P.hidden = static_cast<const __nv_bfloat16*>(hidden);
  P.weight = static_cast<const __nv_bfloat16*>(weight);
  P.label = label; P.loss = loss; P.lse = lse; P.status = status;
  P.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  int launches = 0;
  const cudaError_t e = launch_ce_forward(P, sms, reinterpret_cast<cudaStream_t>(stream), &launches);
  g_launches += launches;
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

int spec_linear_ce_backward(const void* hidden, const void* weight, int dtype, int n, int H, int V,
                            const int32_t* label, const float* lse, const float* grad_loss, void* grad_hidden,
                            void* grad_weight, void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  if (!ce_sizes_ok(n, H, V) || dtype != SPEC_BF16 || !hidden || !weight || !label || !lse)
    return SPEC_ERR_INVALID_ARG;
  if (!grad_hidden && !grad_weight) return SPEC_ERR_INVALID_ARG;
  const void* ptrs16[] = {hidden, weight, grad_hidden, grad_weight};
  for (const void* p : ptrs16)
    if (!aligned(p, 16)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs4[] = {label, lse, grad_loss};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  // rows of grad_weight are written while others of weight are still to be read
  const size_t nh = 2 * (size_t)n * H, vh = 2 * (size_t)V * H;
  if (overlap(grad_weight, vh, weight, vh) || overlap(grad_weight, vh, hidden, nh) ||
      overlap(grad_hidden, nh, weight, vh) || overlap(grad_hidden, nh, grad_weight, vh) ||
      (grad_hidden != hidden && overlap(grad_hidden, nh, hidden, nh)))
    return SPEC_ERR_INVALID_ARG;
  CeParams P{};
  P.n = n; P.H = H; P.V = V;
  if (!workspace || workspace_bytes < ce_layout(P, true, workspace)) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SPEC_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  const int ds = training_state(kLinearCe, &dev, &sms);
  if (ds != SPEC_OK) return ds;
  P.hidden = static_cast<const __nv_bfloat16*>(hidden);
  P.weight = static_cast<const __nv_bfloat16*>(weight);
  P.label = label; P.lse_in = lse; P.grad_loss = grad_loss;
  P.grad_hidden = static_cast<__nv_bfloat16*>(grad_hidden);
  P.grad_weight = static_cast<__nv_bfloat16*>(grad_weight);
  P.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  int launches = 0;
  const cudaError_t e = launch_ce_backward(P, sms, reinterpret_cast<cudaStream_t>(stream), &launches);
  g_launches += launches;
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

int spec_draft_signals(const void* draft_logits, int dtype, int B, int G, int V, const int32_t* gamma,
                       const float* temperature, float* signals, float* row_signals, int32_t* status,
                       void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  Call c{MODE_SIGNALS, nullptr, draft_logits, dtype, B, G, V, nullptr, gamma, temperature, nullptr,
         nullptr, nullptr, status, signals, row_signals, nullptr, workspace, workspace_bytes,
         reinterpret_cast<cudaStream_t>(stream)};
  return run(c);
}

}  // extern "C"
