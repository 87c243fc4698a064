// C ABI of the library (declared in include/grpo.h): argument validation on
// the host, then the launches on the caller's stream.  Nothing here allocates
// device memory or synchronises, except grpo_check_error.
#include <math.h>
#include <stdlib.h>

#include <algorithm>
#include <atomic>
#include <map>
#include <memory>
#include <mutex>
#include <new>
#include <utility>

#include "common.cuh"
#include "host_ctx.cuh"
#include "lmhead.cuh"
#include "ops.cuh"
#include "host_rows.cuh"
#include "selftest.cuh"
#include "grpo.h"

namespace grpo {

int row_split(int64_t row_bytes, const char* env, int max_split) {
  if (env != nullptr) {
    if (const char* s = getenv(env)) {
      const int k = atoi(s);
      if (k == 1 || k == 2 || k == 4 || k == 8) return k;
    }
  }
  int k = 1;
  while (k < max_split && row_bytes / (2 * k) >= 32768) k *= 2;
  return k;
}

int lse_split(int64_t row_bytes, int64_t rows_max, int sms, const char* env) {
  int k = 1;
  while (k < 8 && rows_max * k < 4 * (int64_t)sms) k *= 2;
  return row_split(row_bytes, env, k);
}

int grid_mult(const char* env, int def) {
  if (const char* s = getenv(env)) {
    const int k = atoi(s);
    if (k > 0 && k <= 4096) return k;
  }
  return def;
}

namespace {

// SM count per device ordinal (ordinals below 64; others are asked each time)
std::atomic<int> g_sms[64] = {};

cudaError_t current_device(DeviceInfo* d) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  d->device = dev;
  int n = dev >= 0 && dev < 64 ? g_sms[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) g_sms[dev].store(n, std::memory_order_relaxed);
  }
  d->sms = n;
  return cudaSuccess;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// What the library enqueued last on a stream, and which memory it touches.
// Two launches may touch memory before waiting on the kernel before them,
// when the host knows that kernel: the backward, right after the loss
// forward, writes the rows that score nothing (it reads only the lengths and
// writes only dlogits before its wait); the advantage, right after the mask,
// computes its groups (it reads the rewards and writes the advantages).  Each
// may do so only when its own buffers are disjoint from those of the call
// before it (what that call writes must not be read or written, what it
// reads must not be written); otherwise it waits first as every launch does.
// So every entry point that enqueues work calls stream_take_last() first, and
// a successful loss forward or mask call records itself and its buffers.
// Calls from several host threads on one stream are ordered as their launches
// are only if the caller orders them.
enum LastCall { kLastOther = 0, kLastLossFwd = 1, kLastMask = 2 };

struct Span {  // [lo, hi) in the process's (unified) address space
  uintptr_t lo = 0, hi = 0;
};
Span span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return p == nullptr ? Span{} : Span{a, a + bytes};
}
struct CallRecord {
  int kind = kLastOther;
  Span writes[5];
  Span reads[6];
};
bool overlaps(const Span* set, int n, Span x) {
  if (x.lo == x.hi) return false;
  for (int k = 0; k < n; ++k)
    if (set[k].lo < x.hi && x.lo < set[k].hi) return true;
  return false;
}
// Whether a launch that writes `w` and reads `r` before its wait may follow
// the recorded call without waiting on it.
bool disjoint_from(const CallRecord& c, Span w, Span r) {
  return !overlaps(c.writes, 5, w) && !overlaps(c.reads, 6, w) && !overlaps(c.writes, 5, r);
}

std::mutex g_order_mutex;
std::map<std::pair<unsigned long long, cudaStream_t>, CallRecord> g_last_call;

// A stream handle names a stream of the current context (the legacy default
// stream 0 is a different stream in each), so records are kept per context.
std::pair<unsigned long long, cudaStream_t> order_key(cudaStream_t st) {
  unsigned long long ctx = 0;
  if (current_context_id(&ctx) != cudaSuccess) (void)cudaGetLastError();
  return {ctx, st};
}

// grpo_set_early_start(0) turns the two early starts off process-wide.
std::atomic<int> g_early_start{1};

// The library's last call on `st` (kind kLastOther if not recorded, or if
// early starts are off); forgets it.
CallRecord stream_take_last(cudaStream_t st) {
  const auto key = order_key(st);
  std::lock_guard<std::mutex> lk(g_order_mutex);
  const auto it = g_last_call.find(key);
  if (it == g_last_call.end()) return CallRecord{};
  const CallRecord last = it->second;
  g_last_call.erase(it);
  return g_early_start.load() ? last : CallRecord{};
}
void stream_take_after_fwd(cudaStream_t st) { (void)stream_take_last(st); }

void stream_mark_last(cudaStream_t st, const CallRecord& rec) {
  const auto key = order_key(st);
  std::lock_guard<std::mutex> lk(g_order_mutex);
  g_last_call[key] = rec;
}

// a*b*c without int64 overflow, or -1
int64_t mul3(int64_t a, int64_t b, int64_t c) {
  if (a < 0 || b < 0 || c < 0) return -1;
  if (a == 0 || b == 0 || c == 0) return 0;
  if (a > INT64_MAX / b) return -1;
  const int64_t ab = a * b;
  if (ab > INT64_MAX / c) return -1;
  return ab * c;
}

grpo_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA; }

// Shape checks shared by the loss calls.
grpo_status check_shapes(grpo_dtype dtype, int64_t N, int64_t P, int64_t C, int64_t V) {
  if (dtype != GRPO_F32 && dtype != GRPO_BF16) return GRPO_ERR_UNSUPPORTED;
  if (N < 0 || P < 1 || C < 0 || V < 1) return GRPO_ERR_INVALID_ARG;
  if (P > INT64_MAX - C) return GRPO_ERR_UNSUPPORTED;  // P + C is formed below
  if (N > 0 && C > 0 && N > (int64_t)INT32_MAX / C) return GRPO_ERR_UNSUPPORTED;  // N*C < 2^31
  const int64_t elems = mul3(N, P + C, V);
  if (elems < 0 || elems > INT64_MAX / 4) return GRPO_ERR_UNSUPPORTED;
  return GRPO_OK;
}

}  // namespace
}  // namespace grpo

using namespace grpo;

extern "C" {

const char* grpo_status_string(grpo_status s) {
  switch (s) {
    case GRPO_OK:
      return "ok";
    case GRPO_ERR_INVALID_ARG:
      return "invalid argument";
    case GRPO_ERR_UNSUPPORTED:
      return "unsupported dtype or size";
    case GRPO_ERR_WORKSPACE:
      return "workspace missing or too small";
    case GRPO_ERR_MISALIGNED:
      return "pointer misaligned";
    case GRPO_ERR_CUDA:
      return "CUDA runtime error";
    case GRPO_ERR_TOKEN_RANGE:
      return "a scored token id is outside [0, V)";
    case GRPO_ERR_LENGTH_RANGE:
      return "a completion length is outside [0, C]";
    case GRPO_ERR_TIMEOUT:
      return "a device-side wait timed out";
    case GRPO_ERR_VALUE:
      return "a norm is not finite, or a row of probabilities is undefined";
  }
  return "unknown status";
}

grpo_status grpo_mask(const int64_t* input_ids, int64_t N, int64_t P, int64_t C, int64_t eos_id,
                      uint8_t* mask, int32_t* len, grpo_stream_t stream) {
  if (N < 0 || P < 0 || C < 0) return GRPO_ERR_INVALID_ARG;
  if (N == 0) return GRPO_OK;
  if (len == nullptr || (C > 0 && input_ids == nullptr)) return GRPO_ERR_INVALID_ARG;
  if (P > INT64_MAX - C || mul3(N, P + C, 8) < 0 || C > INT32_MAX) return GRPO_ERR_UNSUPPORTED;
  if (!aligned(input_ids, 8) || !aligned(len, 4)) return GRPO_ERR_MISALIGNED;
  stream_take_last(stream);
  const cudaError_t e = launch_mask(input_ids, N, P, C, eos_id, mask, len, (cudaStream_t)stream);
  if (e == cudaSuccess) {
    CallRecord rec;
    rec.kind = kLastMask;
    rec.writes[0] = span(mask, (size_t)(N * C));
    rec.writes[1] = span(len, sizeof(int32_t) * (size_t)N);
    rec.reads[0] = span(input_ids, sizeof(int64_t) * (size_t)(N * (P + C)));
    stream_mark_last(stream, rec);
  }
  return from_cuda(e);
}

grpo_status grpo_advantage(const float* rewards, int64_t B, int64_t G, float* adv,
                           grpo_stream_t stream) {
  if (B < 0 || G < 1) return GRPO_ERR_INVALID_ARG;
  if (B == 0) return GRPO_OK;
  if (rewards == nullptr || adv == nullptr) return GRPO_ERR_INVALID_ARG;
  if (mul3(B, G, 4) < 0 || B > INT32_MAX) return GRPO_ERR_UNSUPPORTED;
  if (!aligned(rewards, 4) || !aligned(adv, 4)) return GRPO_ERR_MISALIGNED;
  const CallRecord last = stream_take_last(stream);
  const bool after_mask =
      last.kind == kLastMask && disjoint_from(last, span(adv, sizeof(float) * (size_t)(B * G)),
                                              span(rewards, sizeof(float) * (size_t)(B * G)));
  return from_cuda(
      launch_advantage(rewards, B, G, 0, 0.f, adv, nullptr, (cudaStream_t)stream, after_mask));
}

grpo_status grpo_advantage_ex(const float* rewards, int64_t B, int64_t G, grpo_adv_mode mode,
                              float std_eps, float* adv, int32_t* n_contrast,
                              grpo_stream_t stream) {
  if (B < 0 || G < 1) return GRPO_ERR_INVALID_ARG;
  if (mode != GRPO_ADV_DR && mode != GRPO_ADV_STD) return GRPO_ERR_UNSUPPORTED;
  if (!(std_eps >= 0.f) || isinf(std_eps)) return GRPO_ERR_INVALID_ARG;
  if (B > 0 && (rewards == nullptr || adv == nullptr)) return GRPO_ERR_INVALID_ARG;
  if (mul3(B, G, 4) < 0 || B > INT32_MAX) return GRPO_ERR_UNSUPPORTED;
  if (!aligned(rewards, 4) || !aligned(adv, 4) || !aligned(n_contrast, 4))
    return GRPO_ERR_MISALIGNED;
  const CallRecord last = stream_take_last(stream);
  const bool after_mask =
      last.kind == kLastMask && disjoint_from(last, span(adv, sizeof(float) * (size_t)(B * G)),
                                              span(rewards, sizeof(float) * (size_t)(B * G)));
  return from_cuda(launch_advantage(rewards, B, G, (int)mode, std_eps, adv, n_contrast,
                                    (cudaStream_t)stream, after_mask));
}

grpo_status grpo_workspace_size(int64_t N, int64_t C, int64_t V, size_t* bytes) {
  if (bytes == nullptr || N < 0 || C < 0 || V < 1) return GRPO_ERR_INVALID_ARG;
  if (N > 0 && C > 0 && N > (int64_t)INT32_MAX / C) return GRPO_ERR_UNSUPPORTED;
  *bytes = ws_layout(N).total;
  return GRPO_OK;
}

}  // extern "C"

namespace {

// mode 0: full forward; 1: log-probs only (no loss, w or adv needed).
grpo_status loss_fwd_impl(const void* logits, grpo_dtype dtype, int64_t N, int64_t P, int64_t C,
                          int64_t V, const int64_t* input_ids, const int32_t* len,
                          const float* adv, const float* old_logp, const float* ref_logp,
                          float eps, float beta, float norm, int agg, float* logp, float* lse,
                          float* w, float* loss, void* workspace, size_t workspace_bytes,
                          grpo_stream_t stream, int mode) {
  grpo_status s = check_shapes(dtype, N, P, C, V);
  if (s != GRPO_OK) return s;
  if (!(eps >= 0.f && eps < 1.f) || !(beta >= 0.f) || isinf(beta) || isnan(norm) || isinf(norm))
    return GRPO_ERR_INVALID_ARG;
  if (agg != 0 && agg != 1) return GRPO_ERR_UNSUPPORTED;
  if ((mode == 0 && loss == nullptr) || workspace == nullptr) return GRPO_ERR_INVALID_ARG;
  if (N > 0 && (len == nullptr || (mode == 0 && adv == nullptr))) return GRPO_ERR_INVALID_ARG;
  if (N > 0 && C > 0 &&
      (logits == nullptr || input_ids == nullptr || logp == nullptr || lse == nullptr ||
       (mode == 0 && w == nullptr)))
    return GRPO_ERR_INVALID_ARG;
  if (mode == 0 && beta != 0.f && ref_logp == nullptr && N > 0 && C > 0)
    return GRPO_ERR_INVALID_ARG;
  const size_t esize = dtype == GRPO_F32 ? 4 : 2;
  if (!aligned(logits, esize) || !aligned(input_ids, 8) || !aligned(len, 4) ||
      !aligned(adv, 4) || !aligned(old_logp, 4) || !aligned(ref_logp, 4) || !aligned(logp, 4) ||
      !aligned(lse, 4) || !aligned(w, 4) || !aligned(loss, 4) || !aligned(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < ws_layout(N).total) return GRPO_ERR_WORKSPACE;

  FwdArgs a;
  a.logits = logits;
  a.dtype = dtype == GRPO_F32 ? 0 : 1;
  a.N = N;
  a.P = P;
  a.C = C;
  a.V = V;
  a.ids = input_ids;
  a.len = len;
  a.adv = adv;
  a.old_logp = old_logp;
  a.ref_logp = beta != 0.f ? ref_logp : nullptr;
  a.eps = eps;
  a.beta = beta;
  a.norm = norm;
  a.agg = agg;
  a.logp = logp;
  a.lse = lse;
  a.w = w;
  a.loss = loss;
  a.ws = workspace;
  const cudaStream_t st = (cudaStream_t)stream;
  DeviceInfo d;
  cudaError_t e = current_device(&d);
  if (e != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_after_fwd(st);
  // the prep kernel also resets the error flags and the reduction ticket
  if ((e = launch_prep(a, st)) != cudaSuccess) return GRPO_ERR_CUDA;
  if (N == 0 || C == 0)
    return mode == 0 ? from_cuda(cudaMemsetAsync(loss, 0, sizeof(float), st)) : GRPO_OK;
  if ((e = launch_lse_gather(a, d, st, true)) != cudaSuccess) return GRPO_ERR_CUDA;
  if (mode == 1) return GRPO_OK;  // the log-sum-exp kernel zeroed the masked positions
  if ((e = launch_surrogate(a, st)) != cudaSuccess) return GRPO_ERR_CUDA;
  CallRecord rec;
  rec.kind = kLastLossFwd;
  const size_t nc4 = sizeof(float) * (size_t)(N * C);
  rec.writes[0] = span(logp, nc4);
  rec.writes[1] = span(lse, nc4);
  rec.writes[2] = span(w, nc4);
  rec.writes[3] = span(loss, sizeof(float));
  rec.writes[4] = span(workspace, workspace_bytes);
  rec.reads[0] = span(logits, (size_t)mul3(N, P + C, V) * (dtype == GRPO_F32 ? 4 : 2));
  rec.reads[1] = span(input_ids, sizeof(int64_t) * (size_t)(N * (P + C)));
  rec.reads[2] = span(len, sizeof(int32_t) * (size_t)N);
  rec.reads[3] = span(adv, sizeof(float) * (size_t)N);
  rec.reads[4] = span(old_logp, nc4);
  rec.reads[5] = span(a.ref_logp, nc4);
  stream_mark_last(st, rec);
  return GRPO_OK;
}

}  // namespace

extern "C" {

grpo_status grpo_loss_fwd(const void* logits, grpo_dtype dtype, int64_t N, int64_t P, int64_t C,
                          int64_t V, const int64_t* input_ids, const int32_t* len,
                          const float* adv, const float* old_logp, const float* ref_logp,
                          float eps, float beta, float norm, float* logp, float* lse, float* w,
                          float* loss, void* workspace, size_t workspace_bytes,
                          grpo_stream_t stream) {
  return loss_fwd_impl(logits, dtype, N, P, C, V, input_ids, len, adv, old_logp, ref_logp, eps,
                       beta, norm, 0, logp, lse, w, loss, workspace, workspace_bytes, stream, 0);
}

grpo_status grpo_loss_fwd_ex(const void* logits, grpo_dtype dtype, int64_t N, int64_t P,
                             int64_t C, int64_t V, const int64_t* input_ids, const int32_t* len,
                             const float* adv, const float* old_logp, const float* ref_logp,
                             float eps, float beta, float norm, grpo_aggregation agg,
                             float* logp, float* lse, float* w, float* loss, void* workspace,
                             size_t workspace_bytes, grpo_stream_t stream) {
  return loss_fwd_impl(logits, dtype, N, P, C, V, input_ids, len, adv, old_logp, ref_logp, eps,
                       beta, norm, (int)agg, logp, lse, w, loss, workspace, workspace_bytes,
                       stream, 0);
}

grpo_status grpo_logprobs(const void* logits, grpo_dtype dtype, int64_t N, int64_t P, int64_t C,
                          int64_t V, const int64_t* input_ids, const int32_t* len, float* logp,
                          float* lse, void* workspace, size_t workspace_bytes,
                          grpo_stream_t stream) {
  return loss_fwd_impl(logits, dtype, N, P, C, V, input_ids, len, nullptr, nullptr, nullptr, 0.f,
                       0.f, 0.f, 0, logp, lse, nullptr, nullptr, workspace, workspace_bytes,
                       stream, 1);
}

grpo_status grpo_loss_bwd_ex(const void* logits, grpo_dtype dtype, int64_t N, int64_t P,
                             int64_t C, int64_t V, const int64_t* input_ids, const int32_t* len,
                             const float* lse, const float* w, const float* grad_loss,
                             void* dlogits, uint32_t flags, grpo_stream_t stream) {
  if (flags & ~(uint32_t)GRPO_BWD_SKIP_ZERO_WEIGHT) return GRPO_ERR_UNSUPPORTED;
  grpo_status s = check_shapes(dtype, N, P, C, V);
  if (s != GRPO_OK) return s;
  if (N == 0) return GRPO_OK;
  if (dlogits == nullptr || len == nullptr) return GRPO_ERR_INVALID_ARG;
  if (C > 0 && (logits == nullptr || input_ids == nullptr || lse == nullptr || w == nullptr))
    return GRPO_ERR_INVALID_ARG;
  const size_t esize = dtype == GRPO_F32 ? 4 : 2;
  if (!aligned(logits, esize) || !aligned(dlogits, esize) || !aligned(input_ids, 8) ||
      !aligned(len, 4) || !aligned(lse, 4) || !aligned(w, 4) || !aligned(grad_loss, 4))
    return GRPO_ERR_MISALIGNED;
  const size_t bytes = (size_t)mul3(N, P + C, V) * esize;
  const char* lo = static_cast<const char*>(logits);
  const char* dl = static_cast<const char*>(dlogits);
  if (logits != nullptr && dl < lo + bytes && lo < dl + bytes) return GRPO_ERR_INVALID_ARG;

  BwdArgs a;
  a.logits = logits;
  a.dtype = dtype == GRPO_F32 ? 0 : 1;
  a.N = N;
  a.P = P;
  a.C = C;
  a.V = V;
  a.ids = input_ids;
  a.len = len;
  a.lse = lse;
  a.w = w;
  a.grad = grad_loss;
  a.dlogits = dlogits;
  a.skip_zero_weight = (flags & GRPO_BWD_SKIP_ZERO_WEIGHT) != 0;
  DeviceInfo d;
  if (current_device(&d) != cudaSuccess) return GRPO_ERR_CUDA;
  {
    // before its wait the backward writes dlogits (zero rows) and reads len
    const CallRecord last = stream_take_last(stream);
    a.after_fwd = last.kind == kLastLossFwd &&
                  disjoint_from(last, span(dlogits, bytes), span(len, sizeof(int32_t) * (size_t)N));
  }
  return from_cuda(launch_dlogits(a, d, (cudaStream_t)stream));
}

grpo_status grpo_loss_bwd(const void* logits, grpo_dtype dtype, int64_t N, int64_t P, int64_t C,
                          int64_t V, const int64_t* input_ids, const int32_t* len,
                          const float* lse, const float* w, const float* grad_loss,
                          void* dlogits, grpo_stream_t stream) {
  return grpo_loss_bwd_ex(logits, dtype, N, P, C, V, input_ids, len, lse, w, grad_loss, dlogits, 0u,
                          stream);
}

}  // extern "C"

namespace {

// Launches prep and the gather of the scored rows from host memory (through
// the buffer's device mapping `host_src`) into the same rows of `staging`.
grpo_status launch_host_gather(const void* host_src, void* staging, size_t esize, int64_t N,
                               int64_t P, int64_t C, int64_t V, const int32_t* len,
                               void* workspace, const DeviceInfo& d, cudaStream_t st) {
  FwdArgs a = {};
  a.N = N;
  a.P = P;
  a.C = C;
  a.V = V;
  a.len = len;
  a.ws = workspace;
  if (launch_prep(a, st) != cudaSuccess) return GRPO_ERR_CUDA;
  return from_cuda(launch_gather_host_rows(host_src, staging, esize, a, d, st));
}

// grpo_loss_fwd_bwd_ex; with host_src (the device mapping of page-locked
// host logits, validated by the caller) the scored rows are first gathered
// from it into `logits`, the staging buffer.
grpo_status fwd_bwd_impl(const void* logits, grpo_dtype dtype, int64_t N, int64_t P, int64_t C,
                         int64_t V, const int64_t* input_ids, const int32_t* len,
                         const float* adv, const float* old_logp, const float* ref_logp,
                         float eps, float beta, float norm, grpo_aggregation agg,
                         const float* grad_loss, float* logp, float* lse, float* w, float* loss,
                         void* dlogits, void* workspace, size_t workspace_bytes,
                         grpo_stream_t stream, const void* host_src) {
  if (agg != GRPO_AGG_TOKEN_SUM && agg != GRPO_AGG_SEQ_MEAN) return GRPO_ERR_UNSUPPORTED;
  grpo_status s = check_shapes(dtype, N, P, C, V);
  if (s != GRPO_OK) return s;
  const size_t esize = dtype == GRPO_F32 ? 4 : 2;
  if (N > 0 && dlogits == nullptr) return GRPO_ERR_INVALID_ARG;
  if (!aligned(dlogits, esize) || !aligned(grad_loss, 4)) return GRPO_ERR_MISALIGNED;
  if (N > 0 && logits != nullptr) {
    const size_t bytes = (size_t)mul3(N, P + C, V) * esize;
    const char* lo = static_cast<const char*>(logits);
    const char* dl = static_cast<const char*>(dlogits);
    if (dl < lo + bytes && lo < dl + bytes) return GRPO_ERR_INVALID_ARG;
  }
  const bool same_phase = ((reinterpret_cast<uintptr_t>(logits) ^
                            reinterpret_cast<uintptr_t>(dlogits)) & 15u) == 0;
  if (N > 0 && C > 0) {
    // the forward's validation (pointers, eps, beta, norm, workspace), before
    // anything is enqueued
    if (!(eps >= 0.f && eps < 1.f) || !(beta >= 0.f) || isinf(beta) || isnan(norm) ||
        isinf(norm))
      return GRPO_ERR_INVALID_ARG;
    if (loss == nullptr || workspace == nullptr || len == nullptr || adv == nullptr ||
        logits == nullptr || input_ids == nullptr || logp == nullptr || lse == nullptr ||
        w == nullptr)
      return GRPO_ERR_INVALID_ARG;
    if (beta != 0.f && ref_logp == nullptr) return GRPO_ERR_INVALID_ARG;
    if (!aligned(logits, esize) || !aligned(input_ids, 8) || !aligned(len, 4) ||
        !aligned(adv, 4) || !aligned(old_logp, 4) || !aligned(ref_logp, 4) ||
        !aligned(logp, 4) || !aligned(lse, 4) || !aligned(w, 4) || !aligned(loss, 4) ||
        !aligned(workspace, 256))
      return GRPO_ERR_MISALIGNED;
    if (workspace_bytes < ws_layout(N).total) return GRPO_ERR_WORKSPACE;
  }
  if (N == 0 || C == 0 || !same_phase) {  // nothing to fuse, or no common vector grid
    if (host_src != nullptr && N > 0 && C > 0) {
      DeviceInfo d;
      if (current_device(&d) != cudaSuccess) return GRPO_ERR_CUDA;
      stream_take_after_fwd((cudaStream_t)stream);
      s = launch_host_gather(host_src, const_cast<void*>(logits), esize, N, P, C, V, len,
                             workspace, d, (cudaStream_t)stream);
      if (s != GRPO_OK) return s;
    }
    s = grpo_loss_fwd_ex(logits, dtype, N, P, C, V, input_ids, len, adv, old_logp, ref_logp, eps,
                         beta, norm, agg, logp, lse, w, loss, workspace, workspace_bytes, stream);
    if (s != GRPO_OK) return s;
    return grpo_loss_bwd(logits, dtype, N, P, C, V, input_ids, len, lse, w, grad_loss, dlogits,
                         stream);
  }

  FwdArgs a;
  a.logits = logits;
  a.dtype = dtype == GRPO_F32 ? 0 : 1;
  a.N = N;
  a.P = P;
  a.C = C;
  a.V = V;
  a.ids = input_ids;
  a.len = len;
  a.adv = adv;
  a.old_logp = old_logp;
  a.ref_logp = beta != 0.f ? ref_logp : nullptr;
  a.eps = eps;
  a.beta = beta;
  a.norm = norm;
  a.agg = (int)agg;
  a.logp = logp;
  a.lse = lse;
  a.w = w;
  a.loss = loss;
  a.ws = workspace;
  BwdArgs b;
  b.logits = logits;
  b.dtype = a.dtype;
  b.N = N;
  b.P = P;
  b.C = C;
  b.V = V;
  b.ids = input_ids;
  b.len = len;
  b.lse = lse;
  b.w = w;
  b.grad = grad_loss;
  b.dlogits = dlogits;
  b.skip_zero_weight = false;
  b.after_fwd = false;
  const cudaStream_t st = (cudaStream_t)stream;
  DeviceInfo d;
  if (current_device(&d) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_after_fwd(st);
  if (host_src != nullptr && ((reinterpret_cast<uintptr_t>(host_src) ^
                               reinterpret_cast<uintptr_t>(logits)) & 15u) == 0) {
    // The gradient kernel reads the scored rows from host memory itself
    // (writing them to the staging buffer for its second pass), so its
    // arithmetic runs while the rows cross the host link; the zero writer
    // runs beside it (this variant holds no head slots in shared memory).
    FwdArgs ah = a;
    ah.logits = host_src;
    if (launch_prep(ah, st) != cudaSuccess) return GRPO_ERR_CUDA;
    if (launch_lse_grad_host(ah, b, const_cast<void*>(logits), d, st) != cudaSuccess)
      return GRPO_ERR_CUDA;
    return from_cuda(launch_zero_rows(b, d, st, logp, lse, w));
  }
  if (host_src != nullptr) {
    // Host rows in another 16-byte phase than the staging buffer: gather them
    // first.  The zero writer goes between the gather and the gradient kernel:
    // it needs no logits, so it writes while the gather waits on the host link
    // (it does not wait on the gather; its CTA 0 waits before exiting, so the
    // gradient kernel, which waits on it, sees the gathered rows).
    grpo_status g = launch_host_gather(host_src, const_cast<void*>(logits), esize, N, P, C, V,
                                       len, workspace, d, st);
    if (g != GRPO_OK) return g;
    if (launch_zero_rows(b, d, st, logp, lse, w) != cudaSuccess) return GRPO_ERR_CUDA;
    return from_cuda(launch_lse_grad(a, b, d, st));
  }
  if (launch_prep(a, st) != cudaSuccess) return GRPO_ERR_CUDA;
  if (launch_lse_grad(a, b, d, st) != cudaSuccess) return GRPO_ERR_CUDA;
  return from_cuda(launch_zero_rows(b, d, st, logp, lse, w));
}

}  // namespace

extern "C" {

grpo_status grpo_loss_fwd_bwd_ex(const void* logits, grpo_dtype dtype, int64_t N, int64_t P,
                                 int64_t C, int64_t V, const int64_t* input_ids,
                                 const int32_t* len, const float* adv, const float* old_logp,
                                 const float* ref_logp, float eps, float beta, float norm,
                                 grpo_aggregation agg, const float* grad_loss, float* logp,
                                 float* lse, float* w, float* loss, void* dlogits, void* workspace,
                                 size_t workspace_bytes, grpo_stream_t stream) {
  return fwd_bwd_impl(logits, dtype, N, P, C, V, input_ids, len, adv, old_logp, ref_logp, eps,
                      beta, norm, agg, grad_loss, logp, lse, w, loss, dlogits, workspace,
                      workspace_bytes, stream, nullptr);
}

// [p, p + bytes) must be page-locked host memory the device can address:
// its first and its last byte both registered host memory, mapped by the
// device `bytes - 1` apart (a buffer pinned or registered shorter than the
// array fails the second test).  *dev_ptr receives the device address of p.
static grpo_status host_range(const void* p, size_t bytes, void** dev_ptr) {
  cudaPointerAttributes first, last;
  if (cudaPointerGetAttributes(&first, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return GRPO_ERR_INVALID_ARG;
  }
  if (first.type != cudaMemoryTypeHost || first.devicePointer == nullptr)
    return GRPO_ERR_INVALID_ARG;
  const char* end = static_cast<const char*>(p) + (bytes - 1);
  if (cudaPointerGetAttributes(&last, end) != cudaSuccess) {
    (void)cudaGetLastError();
    return GRPO_ERR_INVALID_ARG;
  }
  if (last.type != cudaMemoryTypeHost ||
      static_cast<const char*>(last.devicePointer) !=
          static_cast<const char*>(first.devicePointer) + (bytes - 1))
    return GRPO_ERR_INVALID_ARG;
  *dev_ptr = first.devicePointer;
  return GRPO_OK;
}

grpo_status grpo_loss_fwd_bwd_host(const void* host_logits, grpo_dtype dtype, int64_t N,
                                   int64_t P, int64_t C, int64_t V, const int64_t* input_ids,
                                   const int32_t* len, const float* adv, const float* old_logp,
                                   const float* ref_logp, float eps, float beta, float norm,
                                   const float* grad_loss, float* logp, float* lse, float* w,
                                   float* loss, void* dlogits, void* staging, void* workspace,
                                   size_t workspace_bytes, grpo_stream_t stream) {
  grpo_status s = check_shapes(dtype, N, P, C, V);
  if (s != GRPO_OK) return s;
  const size_t esize = dtype == GRPO_F32 ? 4 : 2;
  const size_t bytes = (size_t)mul3(N, P + C, V) * esize;
  // dlogits: device memory, or page-locked host memory (all of it) that the
  // kernels write through its device mapping, across the host link
  void* dl_dev = dlogits;
  bool dl_host = false;
  if (dlogits != nullptr && bytes > 0) {
    cudaPointerAttributes da;
    if (cudaPointerGetAttributes(&da, dlogits) != cudaSuccess) {
      (void)cudaGetLastError();
      return GRPO_ERR_INVALID_ARG;
    }
    if (da.type == cudaMemoryTypeUnregistered) return GRPO_ERR_INVALID_ARG;  // pageable
    if (da.type == cudaMemoryTypeHost) {
      s = host_range(dlogits, bytes, &dl_dev);
      if (s != GRPO_OK) return s;
      dl_host = true;
    }
  }
  if (N == 0 || C == 0)
    return grpo_loss_fwd_bwd(staging, dtype, N, P, C, V, input_ids, len, adv, old_logp, ref_logp,
                             eps, beta, norm, grad_loss, logp, lse, w, loss, dl_dev, workspace,
                             workspace_bytes, stream);
  if (host_logits == nullptr || staging == nullptr || len == nullptr || workspace == nullptr)
    return GRPO_ERR_INVALID_ARG;
  if (!aligned(host_logits, esize) || !aligned(staging, esize) || !aligned(len, 4) ||
      !aligned(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < ws_layout(N).total) return GRPO_ERR_WORKSPACE;
  // the logits must be page-locked host memory the device can address, all
  // of it: the kernels read any scored row, up to the last byte
  void* host_dev = nullptr;
  s = host_range(host_logits, bytes, &host_dev);
  if (s != GRPO_OK) return s;
  // dlogits overlaps neither the logits nor the staging buffer
  const char* dl = static_cast<const char*>(dlogits);
  const char* other = dl_host ? static_cast<const char*>(host_logits)
                              : static_cast<const char*>(staging);
  if (dlogits != nullptr && dl < other + bytes && other < dl + bytes) return GRPO_ERR_INVALID_ARG;
  return fwd_bwd_impl(staging, dtype, N, P, C, V, input_ids, len, adv, old_logp, ref_logp, eps,
                      beta, norm, GRPO_AGG_TOKEN_SUM, grad_loss, logp, lse, w, loss, dl_dev,
                      workspace, workspace_bytes, stream, host_dev);
}

grpo_status grpo_loss_fwd_bwd(const void* logits, grpo_dtype dtype, int64_t N, int64_t P,
                              int64_t C, int64_t V, const int64_t* input_ids, const int32_t* len,
                              const float* adv, const float* old_logp, const float* ref_logp,
                              float eps, float beta, float norm, const float* grad_loss,
                              float* logp, float* lse, float* w, float* loss, void* dlogits,
                              void* workspace, size_t workspace_bytes, grpo_stream_t stream) {
  return grpo_loss_fwd_bwd_ex(logits, dtype, N, P, C, V, input_ids, len, adv, old_logp, ref_logp,
                              eps, beta, norm, GRPO_AGG_TOKEN_SUM, grad_loss, logp, lse, w, loss,
                              dlogits, workspace, workspace_bytes, stream);
}

grpo_status grpo_lmhead_workspace_size(int64_t N, int64_t C, int64_t V, int64_t d,
                                       size_t* bytes) {
  if (bytes == nullptr || N < 0 || C < 0 || V < 1) return GRPO_ERR_INVALID_ARG;
  if (d < 128 || d % 128 != 0) return GRPO_ERR_UNSUPPORTED;
  if (N > 0 && C > 0 && N > (int64_t)INT32_MAX / C) return GRPO_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  *bytes = lm_layout(N, C, d, dev.sms).total;
  return GRPO_OK;
}

}  // extern "C"

namespace {

// Checks shared by the LM-head calls (bf16 hidden [N, P+C, d], weight [V, d]).
grpo_status lmhead_check(const void* hidden, const void* weight, int64_t N, int64_t P, int64_t C,
                         int64_t V, int64_t d, const int64_t* input_ids, const int32_t* len,
                         const void* workspace) {
  grpo_status s = check_shapes(GRPO_BF16, N, P, C, V);
  if (s != GRPO_OK) return s;
  if (d < 128 || d % 128 != 0) return GRPO_ERR_UNSUPPORTED;
  if (V > (int64_t)INT32_MAX - 256 || mul3(N, P + C, d) < 0) return GRPO_ERR_UNSUPPORTED;
  if (workspace == nullptr || (N > 0 && len == nullptr)) return GRPO_ERR_INVALID_ARG;
  if (N > 0 && C > 0 && (hidden == nullptr || weight == nullptr || input_ids == nullptr))
    return GRPO_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(input_ids, 8) || !aligned(len, 4) ||
      !aligned(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  return GRPO_OK;
}

// mode 0: log-probs only; 1: log-probs, then the loss.
grpo_status lmhead_fwd_impl(const void* hidden, const void* weight, int64_t N, int64_t P, int64_t C,
                            int64_t V, int64_t d, const int64_t* input_ids, const int32_t* len,
                            const float* adv, const float* old_logp, const float* ref_logp,
                            float eps, float beta, float norm, int agg, float* logp, float* lse,
                            float* w, float* loss, void* workspace, size_t workspace_bytes,
                            grpo_stream_t stream, int mode) {
  if (agg != GRPO_AGG_TOKEN_SUM && agg != GRPO_AGG_SEQ_MEAN) return GRPO_ERR_UNSUPPORTED;
  grpo_status s = lmhead_check(hidden, weight, N, P, C, V, d, input_ids, len, workspace);
  if (s != GRPO_OK) return s;
  if (N > 0 && C > 0 && (logp == nullptr || lse == nullptr)) return GRPO_ERR_INVALID_ARG;
  if (mode == 1) {
    if (!(eps >= 0.f && eps < 1.f) || !(beta >= 0.f) || isinf(beta) || isnan(norm) ||
        isinf(norm))
      return GRPO_ERR_INVALID_ARG;
    if (loss == nullptr || (N > 0 && adv == nullptr) || (N > 0 && C > 0 && w == nullptr))
      return GRPO_ERR_INVALID_ARG;
    if (beta != 0.f && ref_logp == nullptr && N > 0 && C > 0) return GRPO_ERR_INVALID_ARG;
  }
  if (!aligned(logp, 4) || !aligned(lse, 4) || !aligned(adv, 4) || !aligned(old_logp, 4) ||
      !aligned(ref_logp, 4) || !aligned(w, 4) || !aligned(loss, 4))
    return GRPO_ERR_MISALIGNED;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  if (workspace_bytes < lm_layout(N, C, d, dev.sms).total) return GRPO_ERR_WORKSPACE;
  stream_take_after_fwd(stream);
  FwdArgs a = {};
  a.dtype = 1;
  a.N = N;
  a.P = P;
  a.C = C;
  a.V = V;
  a.ids = input_ids;
  a.len = len;
  a.adv = adv;
  a.old_logp = old_logp;
  a.ref_logp = beta != 0.f ? ref_logp : nullptr;
  a.eps = eps;
  a.beta = beta;
  a.norm = norm;
  a.agg = agg;
  a.logp = logp;
  a.lse = lse;
  a.w = w;
  a.loss = loss;
  a.ws = workspace;
  const cudaStream_t st = (cudaStream_t)stream;
  if (launch_prep(a, st) != cudaSuccess) return GRPO_ERR_CUDA;
  if (N == 0 || C == 0)
    return mode == 1 ? from_cuda(cudaMemsetAsync(loss, 0, sizeof(float), st)) : GRPO_OK;
  cudaError_t e = launch_lmhead(hidden, weight, a, d, dev, st);
  if (e != cudaSuccess || mode == 0) return from_cuda(e);
  return from_cuda(launch_surrogate(a, st));
}

}  // namespace

extern "C" {

grpo_status grpo_lmhead_logprobs(const void* hidden, const void* weight, int64_t N, int64_t P,
                                 int64_t C, int64_t V, int64_t d, const int64_t* input_ids,
                                 const int32_t* len, float* logp, float* lse, void* workspace,
                                 size_t workspace_bytes, grpo_stream_t stream) {
  return lmhead_fwd_impl(hidden, weight, N, P, C, V, d, input_ids, len, nullptr, nullptr, nullptr,
                         0.f, 0.f, 0.f, GRPO_AGG_TOKEN_SUM, logp, lse, nullptr, nullptr, workspace,
                         workspace_bytes, stream, 0);
}

grpo_status grpo_lmhead_loss_fwd(const void* hidden, const void* weight, int64_t N, int64_t P,
                                 int64_t C, int64_t V, int64_t d, const int64_t* input_ids,
                                 const int32_t* len, const float* adv, const float* old_logp,
                                 const float* ref_logp, float eps, float beta, float norm,
                                 float* logp, float* lse, float* w, float* loss, void* workspace,
                                 size_t workspace_bytes, grpo_stream_t stream) {
  return lmhead_fwd_impl(hidden, weight, N, P, C, V, d, input_ids, len, adv, old_logp, ref_logp,
                         eps, beta, norm, GRPO_AGG_TOKEN_SUM, logp, lse, w, loss, workspace,
                         workspace_bytes, stream, 1);
}

grpo_status grpo_lmhead_loss_fwd_ex(const void* hidden, const void* weight, int64_t N, int64_t P,
                                    int64_t C, int64_t V, int64_t d, const int64_t* input_ids,
                                    const int32_t* len, const float* adv, const float* old_logp,
                                    const float* ref_logp, float eps, float beta, float norm,
                                    grpo_aggregation agg, float* logp, float* lse, float* w,
                                    float* loss, void* workspace, size_t workspace_bytes,
                                    grpo_stream_t stream) {
  return lmhead_fwd_impl(hidden, weight, N, P, C, V, d, input_ids, len, adv, old_logp, ref_logp,
                         eps, beta, norm, (int)agg, logp, lse, w, loss, workspace, workspace_bytes,
                         stream, 1);
}

grpo_status grpo_lmhead_bwd_workspace_size_rows(int64_t N, int64_t C, int64_t V, int64_t d,
                                                int64_t rows_per_pass, size_t* bytes) {
  if (bytes == nullptr || N < 0 || C < 0 || V < 1 || rows_per_pass < 0)
    return GRPO_ERR_INVALID_ARG;
  if (d < 128 || d % 128 != 0) return GRPO_ERR_UNSUPPORTED;
  if (N > 0 && C > 0 && N > (int64_t)INT32_MAX / C) return GRPO_ERR_UNSUPPORTED;
  if (V > (int64_t)INT32_MAX - 256) return GRPO_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  *bytes = lm_bwd_layout(N, C, V, d, dev.sms, rows_per_pass).total;
  return GRPO_OK;
}

grpo_status grpo_lmhead_bwd_workspace_size(int64_t N, int64_t C, int64_t V, int64_t d,
                                           size_t* bytes) {
  return grpo_lmhead_bwd_workspace_size_rows(N, C, V, d, 0, bytes);
}

grpo_status grpo_lmhead_loss_bwd(const void* hidden, const void* weight, int64_t N, int64_t P,
                                 int64_t C, int64_t V, int64_t d, const int64_t* input_ids,
                                 const int32_t* len, const float* lse, const float* w,
                                 const float* grad_loss, float* dhidden, float* dweight,
                                 void* workspace, size_t workspace_bytes, grpo_stream_t stream) {
  return grpo_lmhead_loss_bwd_ex(hidden, weight, N, P, C, V, d, input_ids, len, lse, w, grad_loss,
                                 dhidden, dweight, 0u, workspace, workspace_bytes, stream);
}

grpo_status grpo_lmhead_loss_bwd_ex(const void* hidden, const void* weight, int64_t N, int64_t P,
                                    int64_t C, int64_t V, int64_t d, const int64_t* input_ids,
                                    const int32_t* len, const float* lse, const float* w,
                                    const float* grad_loss, float* dhidden, float* dweight,
                                    uint32_t flags, void* workspace, size_t workspace_bytes,
                                    grpo_stream_t stream) {
  if (flags & ~GRPO_BWD_SKIP_ZERO_WEIGHT) return GRPO_ERR_UNSUPPORTED;
  grpo_status s = lmhead_check(hidden, weight, N, P, C, V, d, input_ids, len, workspace);
  if (s != GRPO_OK) return s;
  if (dweight == nullptr || (N > 0 && dhidden == nullptr)) return GRPO_ERR_INVALID_ARG;
  if (N > 0 && C > 0 && (lse == nullptr || w == nullptr)) return GRPO_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(w, 4) || !aligned(grad_loss, 4) || !aligned(dhidden, 16) ||
      !aligned(dweight, 16))
    return GRPO_ERR_MISALIGNED;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  // rows per pass: as many as the workspace holds (every possible row when it
  // is grpo_lmhead_bwd_workspace_size bytes), at least one block of 256
  const int64_t blocks = (N * C + 255) / 256;
  int64_t lo = 1, hi = blocks > 0 ? blocks : 1;
  if (workspace_bytes < lm_bwd_layout(N, C, V, d, dev.sms, 256).total) return GRPO_ERR_WORKSPACE;
  while (lo < hi) {  // the layout grows with the rows per pass
    const int64_t mid = (lo + hi + 1) / 2;
    if (lm_bwd_layout(N, C, V, d, dev.sms, mid * 256).total <= workspace_bytes)
      lo = mid;
    else
      hi = mid - 1;
  }
  const LmBwdLayout bl = lm_bwd_layout(N, C, V, d, dev.sms, lo * 256);
  stream_take_after_fwd(stream);
  FwdArgs f = {};
  f.N = N;
  f.P = P;
  f.C = C;
  f.V = V;
  f.len = len;
  f.ws = workspace;
  const cudaStream_t st = (cudaStream_t)stream;
  if (launch_prep(f, st) != cudaSuccess) return GRPO_ERR_CUDA;
  if (N == 0 || C == 0) {  // nothing is scored: both gradients are zero
    if (cudaMemsetAsync(dweight, 0, (size_t)V * (size_t)d * 4, st) != cudaSuccess)
      return GRPO_ERR_CUDA;
    const int64_t nh = mul3(N, P + C, d);
    return nh == 0 ? GRPO_OK : from_cuda(cudaMemsetAsync(dhidden, 0, (size_t)nh * 4, st));
  }
  LmBwdArgs a;
  a.hidden = hidden;
  a.weight = weight;
  a.N = N;
  a.P = P;
  a.C = C;
  a.V = V;
  a.d = d;
  a.ids = input_ids;
  a.lse = lse;
  a.w = w;
  a.grad = grad_loss;
  a.dhidden = dhidden;
  a.dweight = dweight;
  a.ws = workspace;
  a.rows_pass = bl.rows_pass;
  a.skip_zero_weight = (flags & GRPO_BWD_SKIP_ZERO_WEIGHT) != 0;
  if (launch_lmhead_bwd_rows(a, dev, st) != cudaSuccess) return GRPO_ERR_CUDA;
  for (int64_t pass = 0; pass < bl.npass; ++pass) {
    if (launch_lmhead_dz(a, pass, dev, st) != cudaSuccess) return GRPO_ERR_CUDA;
    cudaError_t e = launch_lmhead_grads(a, pass, dev, st);
    if (e != cudaSuccess) return from_cuda(e);
  }
  return GRPO_OK;
}

// ---- the operators around the loss ----------------------------------------------

}  // extern "C"

namespace {

// A matrix of `rows` rows of d elements, `ld` apart: fits int64 bytes.
bool matrix_fits(int64_t rows, int64_t ld) { return mul3(rows, ld, 8) >= 0; }
size_t matrix_bytes(int64_t rows, int64_t d, int64_t ld, grpo_dtype t) {
  return rows < 1 ? 0 : ((size_t)(rows - 1) * (size_t)ld + (size_t)d) * (t == GRPO_F32 ? 4 : 2);
}
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}
bool known_dtype(grpo_dtype t) { return t == GRPO_F32 || t == GRPO_BF16; }
size_t esize_of(grpo_dtype t) { return t == GRPO_F32 ? 4 : 2; }

// Rows of a verification: a grid of up to 32 CTAs per row stays below 2^31.
bool verify_fits(int64_t N, int64_t K) {
  return K <= (int64_t)1 << 20 && N <= ((int64_t)1 << 26) / (K + 1);
}

// Rows of logits of a token statistics call.
bool rows_fit(int64_t N, int64_t R) {
  return N == 0 || R == 0 || N <= ((int64_t)1 << 26) / R;
}
// Checks shared by those calls: rows of V elements at i * seq + j * row.
grpo_status check_rows(grpo_dtype dtype, int64_t N, int64_t R, int64_t V, int64_t seq,
                       int64_t row) {
  if (!known_dtype(dtype)) return GRPO_ERR_UNSUPPORTED;
  if (N < 0 || R < 0 || V < 1) return GRPO_ERR_INVALID_ARG;
  if (!rows_fit(N, R) || V > INT32_MAX - 65536) return GRPO_ERR_UNSUPPORTED;
  if (row < 0 || seq < 0) return GRPO_ERR_INVALID_ARG;
  const int64_t across = mul3(N, seq, 16), along = mul3(R, row, 16);
  if (across < 0 || along < 0 || across > INT64_MAX / 2 || along > INT64_MAX / 2)
    return GRPO_ERR_UNSUPPORTED;
  return GRPO_OK;
}
// Whether no two of them share an element: sequences behind one another, or rows.
bool rows_apart(int64_t N, int64_t R, int64_t V, int64_t seq, int64_t row) {
  if (N < 1 || R < 1) return true;
  if ((R > 1 && row < V) || (N > 1 && seq < V)) return false;
  return N == 1 || R == 1 || seq >= (R - 1) * row + V || row >= (N - 1) * seq + V;
}
bool tokens_fit(int64_t N, int64_t R, int64_t seq, int64_t row) {
  const int64_t across = mul3(N, seq, 16), along = mul3(R, row, 16);
  return across >= 0 && along >= 0 && across <= INT64_MAX / 2 && along <= INT64_MAX / 2;
}
// (of one row or more)
size_t rows_bytes(int64_t N, int64_t R, int64_t V, int64_t seq, int64_t row, grpo_dtype t) {
  return ((size_t)(N - 1) * (size_t)seq + (size_t)(R - 1) * (size_t)row + (size_t)V) * esize_of(t);
}
Span token_span(const int64_t* tokens, int64_t N, int64_t R, int64_t seq, int64_t row) {
  return span(tokens, 8 * (size_t)((N - 1) * seq + (R - 1) * row + 1));
}

constexpr int64_t kMaxEmbedDim = (int64_t)1 << 24;

// Shape checks shared by the embedding calls.
grpo_status check_embed(int64_t n, int64_t V, int64_t d, int64_t ldw, int64_t ldx) {
  if (n < 0 || V < 1 || d < 1 || ldw < d || ldx < d) return GRPO_ERR_INVALID_ARG;
  if (n > INT32_MAX - 65536 || V > INT32_MAX - 65536 || d > kMaxEmbedDim ||
      !matrix_fits(V, ldw) || !matrix_fits(n, ldx))
    return GRPO_ERR_UNSUPPORTED;
  return GRPO_OK;
}

}  // namespace

extern "C" {

grpo_status grpo_embed_fwd(const int64_t* ids, int64_t n, const void* weight, grpo_dtype wdtype,
                           int64_t V, int64_t d, int64_t ldw, float scale, void* out,
                           grpo_dtype odtype, int64_t ldo, grpo_stream_t stream) {
  if (!known_dtype(wdtype) || !known_dtype(odtype)) return GRPO_ERR_UNSUPPORTED;
  const grpo_status s = check_embed(n, V, d, ldw, ldo);
  if (s != GRPO_OK) return s;
  if (isnan(scale) || isinf(scale)) return GRPO_ERR_INVALID_ARG;
  if (n == 0) return GRPO_OK;
  if (ids == nullptr || weight == nullptr || out == nullptr) return GRPO_ERR_INVALID_ARG;
  if (!aligned(ids, 8) || !aligned(weight, esize_of(wdtype)) || !aligned(out, esize_of(odtype)))
    return GRPO_ERR_MISALIGNED;
  const size_t ob = matrix_bytes(n, d, ldo, odtype);
  if (overlap(out, ob, weight, matrix_bytes(V, d, ldw, wdtype)) ||
      overlap(out, ob, ids, 8 * (size_t)n))
    return GRPO_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_last(stream);
  EmbedFwdArgs a;
  a.ids = ids;
  a.n = n;
  a.weight = weight;
  a.wdtype = wdtype == GRPO_F32 ? 0 : 1;
  a.V = V;
  a.d = d;
  a.ldw = ldw;
  a.scale = scale;
  a.out = out;
  a.odtype = odtype == GRPO_F32 ? 0 : 1;
  a.ldo = ldo;
  return from_cuda(launch_embed_fwd(a, dev, (cudaStream_t)stream));
}

grpo_status grpo_embed_workspace_size(int64_t n, int64_t V, int64_t d, size_t* bytes) {
  if (bytes == nullptr) return GRPO_ERR_INVALID_ARG;
  const grpo_status s = check_embed(n, V, d, d, d);
  if (s != GRPO_OK) return s;
  *bytes = embed_workspace_bytes(n, V, d);
  return GRPO_OK;
}

grpo_status grpo_embed_bwd(const int64_t* ids, int64_t n, const void* dout, grpo_dtype ddtype,
                           int64_t V, int64_t d, int64_t ldd, float scale, int64_t pad_id,
                           void* dweight, grpo_dtype wdtype, int64_t ldw, int accumulate,
                           void* workspace, size_t workspace_bytes, grpo_stream_t stream) {
  if (!known_dtype(ddtype) || !known_dtype(wdtype)) return GRPO_ERR_UNSUPPORTED;
  const grpo_status s = check_embed(n, V, d, ldw, ldd);
  if (s != GRPO_OK) return s;
  if (isnan(scale) || isinf(scale)) return GRPO_ERR_INVALID_ARG;
  if (dweight == nullptr || workspace == nullptr) return GRPO_ERR_INVALID_ARG;
  if (n > 0 && (ids == nullptr || dout == nullptr)) return GRPO_ERR_INVALID_ARG;
  if (!aligned(ids, 8) || !aligned(dout, esize_of(ddtype)) ||
      !aligned(dweight, esize_of(wdtype)) || !aligned(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < embed_workspace_bytes(n, V, d)) return GRPO_ERR_WORKSPACE;
  const size_t wb = matrix_bytes(V, d, ldw, wdtype);
  const size_t db = matrix_bytes(n, d, ldd, ddtype);
  if (overlap(dweight, wb, dout, db) || overlap(dweight, wb, ids, 8 * (size_t)n) ||
      overlap(dweight, wb, workspace, workspace_bytes) ||
      overlap(workspace, workspace_bytes, dout, db) ||
      overlap(workspace, workspace_bytes, ids, 8 * (size_t)n))
    return GRPO_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_last(stream);
  EmbedBwdArgs a;
  a.ids = ids;
  a.n = n;
  a.dout = dout;
  a.ddtype = ddtype == GRPO_F32 ? 0 : 1;
  a.V = V;
  a.d = d;
  a.ldd = ldd;
  a.scale = scale;
  a.pad_id = pad_id;
  a.dweight = dweight;
  a.wdtype = wdtype == GRPO_F32 ? 0 : 1;
  a.ldw = ldw;
  a.accumulate = accumulate != 0;
  a.ws = workspace;
  return from_cuda(launch_embed_bwd(a, dev, (cudaStream_t)stream));
}

grpo_status grpo_grad_norm_workspace_size(int64_t count, size_t* bytes) {
  if (bytes == nullptr || count < 0) return GRPO_ERR_INVALID_ARG;
  if (count > INT32_MAX) return GRPO_ERR_UNSUPPORTED;
  *bytes = grad_norm_workspace_bytes(count);
  return GRPO_OK;
}

}  // extern "C"

namespace {

grpo_status clip_impl(const grpo_tensor* tensors, int64_t count, grpo_norm_type type,
                      float max_norm, float eps, bool norm_only, float* stats, void* workspace,
                      size_t workspace_bytes, grpo_stream_t stream) {
  if (type != GRPO_NORM_L2 && type != GRPO_NORM_MAX) return GRPO_ERR_UNSUPPORTED;
  if (count < 0 || !(max_norm >= 0.f) || !(eps >= 0.f) || isinf(eps)) return GRPO_ERR_INVALID_ARG;
  if (count > INT32_MAX) return GRPO_ERR_UNSUPPORTED;
  if ((count > 0 && tensors == nullptr) || stats == nullptr || workspace == nullptr)
    return GRPO_ERR_INVALID_ARG;
  if (!aligned(stats, 4) || !aligned(workspace, 256)) return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < grad_norm_workspace_bytes(count)) return GRPO_ERR_WORKSPACE;
  GradTensor* g = nullptr;
  GradTensor few[64];
  std::unique_ptr<GradTensor[]> many;
  if (count <= 64) {
    g = few;
  } else {
    many.reset(new (std::nothrow) GradTensor[(size_t)count]);
    if (!many) return GRPO_ERR_UNSUPPORTED;
    g = many.get();
  }
  int64_t all = 0;
  for (int64_t k = 0; k < count; ++k) {
    const grpo_tensor& t = tensors[k];
    if (!known_dtype(t.dtype) || !known_dtype(t.out_dtype)) return GRPO_ERR_UNSUPPORTED;
    if (t.numel < 0 || (t.numel > 0 && t.data == nullptr)) return GRPO_ERR_INVALID_ARG;
    if (t.numel == 0) {  // nothing behind its pointers
      g[k].data = g[k].out = nullptr;
      g[k].numel = 0;
      g[k].dt = 0;
      continue;
    }
    if (t.numel > INT64_MAX / 16 - all) return GRPO_ERR_UNSUPPORTED;
    all += t.numel;
    void* out = t.out == nullptr ? const_cast<void*>(t.data) : t.out;
    // in place: no other type; elsewhere: not over part of the input
    if (out == t.data && t.out_dtype != t.dtype) return GRPO_ERR_INVALID_ARG;
    if (!aligned(t.data, esize_of(t.dtype)) || !aligned(out, esize_of(t.out_dtype)))
      return GRPO_ERR_MISALIGNED;
    const size_t nb = (size_t)t.numel * esize_of(t.dtype);
    const size_t no = (size_t)t.numel * esize_of(t.out_dtype);
    if (!norm_only && ((out != t.data && overlap(out, no, t.data, nb)) ||
                       overlap(out, no, workspace, workspace_bytes)))
      return GRPO_ERR_INVALID_ARG;
    g[k].data = t.data;
    g[k].out = out;
    g[k].numel = t.numel;
    g[k].dt = (t.dtype == GRPO_BF16 ? 1 : 0) | (t.out_dtype == GRPO_BF16 ? 2 : 0);
  }
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_last(stream);
  ClipArgs a;
  a.tensors = g;
  a.count = count;
  a.type = type == GRPO_NORM_L2 ? 0 : 1;
  a.max_norm = max_norm;
  a.eps = eps;
  a.norm_only = norm_only;
  a.stats = stats;
  a.ws = workspace;
  return from_cuda(launch_clip(a, dev, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

grpo_status grpo_clip_grad_norm(const grpo_tensor* tensors, int64_t count, grpo_norm_type type,
                                float max_norm, float eps, float* stats, void* workspace,
                                size_t workspace_bytes, grpo_stream_t stream) {
  return clip_impl(tensors, count, type, max_norm, eps, false, stats, workspace, workspace_bytes,
                   stream);
}

grpo_status grpo_grad_norm(const grpo_tensor* tensors, int64_t count, grpo_norm_type type,
                           float* stats, void* workspace, size_t workspace_bytes,
                           grpo_stream_t stream) {
  return clip_impl(tensors, count, type, INFINITY, 0.f, true, stats, workspace, workspace_bytes,
                   stream);
}

grpo_status grpo_verify_workspace_size(int64_t N, int64_t K, size_t* bytes) {
  if (bytes == nullptr || N < 0 || K < 0) return GRPO_ERR_INVALID_ARG;
  if (!verify_fits(N, K)) return GRPO_ERR_UNSUPPORTED;
  *bytes = verify_workspace_bytes(N, K);
  return GRPO_OK;
}

grpo_status grpo_verify_drafts(const void* target_logits, const void* draft_logits,
                               grpo_dtype dtype, int64_t N, int64_t K, int64_t V,
                               int64_t target_seq, int64_t target_row, int64_t draft_seq,
                               int64_t draft_row, const int64_t* draft_tokens,
                               const int32_t* draft_len, const float* u, const float* noise,
                               int64_t noise_row, const float* temperature, int64_t* tokens,
                               int32_t* n_accepted, float* logp, void* workspace,
                               size_t workspace_bytes, grpo_stream_t stream) {
  if (!known_dtype(dtype)) return GRPO_ERR_UNSUPPORTED;
  if (N < 0 || K < 0 || V < 1) return GRPO_ERR_INVALID_ARG;
  if (!verify_fits(N, K) || V >= (int64_t)1 << 29) return GRPO_ERR_UNSUPPORTED;
  const bool has_draft = draft_logits != nullptr && K > 0;
  if (target_row < V || target_seq < 0 || noise_row < V) return GRPO_ERR_INVALID_ARG;
  if (mul3(K + 1, target_row, 8) < 0 || mul3(N, target_seq, 8) < 0 || mul3(N, noise_row, 8) < 0)
    return GRPO_ERR_UNSUPPORTED;
  if (N > 1 && target_seq < K * target_row + V) return GRPO_ERR_INVALID_ARG;
  if (has_draft) {
    if (draft_row < V || draft_seq < 0) return GRPO_ERR_INVALID_ARG;
    if (mul3(K, draft_row, 8) < 0 || mul3(N, draft_seq, 8) < 0) return GRPO_ERR_UNSUPPORTED;
    if (N > 1 && draft_seq < (K - 1) * draft_row + V) return GRPO_ERR_INVALID_ARG;
  }
  if (workspace == nullptr) return GRPO_ERR_INVALID_ARG;
  if (N > 0) {
    if (target_logits == nullptr || noise == nullptr || tokens == nullptr ||
        n_accepted == nullptr || logp == nullptr)
      return GRPO_ERR_INVALID_ARG;
    if (K > 0 && (draft_tokens == nullptr || u == nullptr)) return GRPO_ERR_INVALID_ARG;
  }
  if (!aligned(target_logits, esize_of(dtype)) || !aligned(draft_logits, esize_of(dtype)) ||
      !aligned(draft_tokens, 8) || !aligned(draft_len, 4) || !aligned(u, 4) ||
      !aligned(noise, 4) || !aligned(temperature, 4) || !aligned(tokens, 8) ||
      !aligned(n_accepted, 4) || !aligned(logp, 4) || !aligned(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < verify_workspace_bytes(N, K)) return GRPO_ERR_WORKSPACE;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_last(stream);
  VerifyArgs a;
  a.target = target_logits;
  a.draft = has_draft ? draft_logits : nullptr;
  a.dtype = dtype == GRPO_F32 ? 0 : 1;
  a.N = N;
  a.K = K;
  a.V = V;
  a.tld = target_row;
  a.tls = target_seq;
  a.dld = has_draft ? draft_row : 0;
  a.dls = has_draft ? draft_seq : 0;
  a.tokens = draft_tokens;
  a.lens = draft_len;
  a.u = u;
  a.noise = noise;
  a.nld = noise_row;
  a.temperature = temperature;
  a.out_tokens = tokens;
  a.n_accepted = n_accepted;
  a.logp = logp;
  a.ws = workspace;
  return from_cuda(launch_verify(a, dev, (cudaStream_t)stream));
}

grpo_status grpo_token_stats_workspace_size(int64_t N, int64_t R, size_t* bytes) {
  if (bytes == nullptr || N < 0 || R < 0) return GRPO_ERR_INVALID_ARG;
  if (!rows_fit(N, R)) return GRPO_ERR_UNSUPPORTED;
  *bytes = token_stats_workspace_bytes(N, R);
  return GRPO_OK;
}

grpo_status grpo_token_stats(const void* logits, grpo_dtype dtype, int64_t N, int64_t R, int64_t V,
                             int64_t logits_seq, int64_t logits_row, const int64_t* tokens,
                             int64_t token_seq, int64_t token_row, const int32_t* len,
                             const float* temperature, int64_t top, float* logp, float* entropy,
                             float* norm, int64_t* top_tokens, float* top_logp, void* workspace,
                             size_t workspace_bytes, grpo_stream_t stream) {
  const grpo_status s = check_rows(dtype, N, R, V, logits_seq, logits_row);
  if (s != GRPO_OK) return s;
  if (token_seq < 0 || token_row < 0 || top < 0 || top > V) return GRPO_ERR_INVALID_ARG;
  if (top > kMaxTop || !tokens_fit(N, R, token_seq, token_row)) return GRPO_ERR_UNSUPPORTED;
  if (workspace == nullptr) return GRPO_ERR_INVALID_ARG;
  const int64_t rows = N * R;
  if (rows > 0) {
    if (logits == nullptr || tokens == nullptr || logp == nullptr || entropy == nullptr ||
        norm == nullptr)
      return GRPO_ERR_INVALID_ARG;
    if (top > 0 && (top_tokens == nullptr || top_logp == nullptr)) return GRPO_ERR_INVALID_ARG;
  }
  if (!aligned(logits, esize_of(dtype)) || !aligned(tokens, 8) || !aligned(len, 4) ||
      !aligned(temperature, 4) || !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(norm, 8) ||
      (top > 0 && (!aligned(top_tokens, 8) || !aligned(top_logp, 4))) || !aligned(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < token_stats_workspace_bytes(N, R)) return GRPO_ERR_WORKSPACE;
  if (rows > 0) {
    const size_t n = (size_t)rows, alternatives = n * (size_t)top;
    const Span writes[6] = {span(workspace, token_stats_workspace_bytes(N, R)), span(logp, 4 * n),
                            span(entropy, 4 * n), span(norm, 8 * n),
                            span(top_tokens, 8 * alternatives), span(top_logp, 4 * alternatives)};
    for (int k = 1; k < 6; ++k)
      if (overlaps(writes, k, writes[k])) return GRPO_ERR_INVALID_ARG;
    const Span reads[4] = {span(logits, rows_bytes(N, R, V, logits_seq, logits_row, dtype)),
                           token_span(tokens, N, R, token_seq, token_row),
                           span(len, 4 * (size_t)N), span(temperature, 4 * (size_t)N)};
    for (const Span& r : reads)
      if (overlaps(writes, 6, r)) return GRPO_ERR_INVALID_ARG;
  }
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_last(stream);
  TokenStatsArgs a;
  a.logits = logits;
  a.dtype = dtype == GRPO_F32 ? 0 : 1;
  a.N = N;
  a.R = R;
  a.V = V;
  a.seq = logits_seq;
  a.row = logits_row;
  a.tokens = tokens;
  a.token_seq = token_seq;
  a.token_row = token_row;
  a.lens = len;
  a.temperature = temperature;
  a.top = (int)top;
  a.logp = logp;
  a.entropy = entropy;
  a.norm = norm;
  a.top_tokens = top_tokens;
  a.top_logp = top_logp;
  a.ws = workspace;
  return from_cuda(launch_token_stats(a, dev, (cudaStream_t)stream));
}

grpo_status grpo_token_stats_bwd(const void* logits, grpo_dtype dtype, int64_t N, int64_t R,
                                 int64_t V, int64_t logits_seq, int64_t logits_row,
                                 const int64_t* tokens, int64_t token_seq, int64_t token_row,
                                 const int32_t* len, const float* temperature, const float* norm,
                                 const float* entropy, const float* grad_logp,
                                 const float* grad_entropy, void* dlogits, int64_t dlogits_seq,
                                 int64_t dlogits_row, grpo_stream_t stream) {
  grpo_status s = check_rows(dtype, N, R, V, logits_seq, logits_row);
  if (s == GRPO_OK) s = check_rows(dtype, N, R, V, dlogits_seq, dlogits_row);
  if (s != GRPO_OK) return s;
  if (token_seq < 0 || token_row < 0 || !rows_apart(N, R, V, dlogits_seq, dlogits_row))
    return GRPO_ERR_INVALID_ARG;
  if (!tokens_fit(N, R, token_seq, token_row)) return GRPO_ERR_UNSUPPORTED;
  const int64_t rows = N * R;
  if (rows == 0) return GRPO_OK;
  if (logits == nullptr || norm == nullptr || dlogits == nullptr ||
      (grad_logp != nullptr && tokens == nullptr) ||
      (grad_entropy != nullptr && entropy == nullptr))
    return GRPO_ERR_INVALID_ARG;
  if (!aligned(logits, esize_of(dtype)) || !aligned(dlogits, esize_of(dtype)) ||
      !aligned(tokens, 8) || !aligned(len, 4) || !aligned(temperature, 4) || !aligned(norm, 8) ||
      !aligned(entropy, 4) || !aligned(grad_logp, 4) || !aligned(grad_entropy, 4))
    return GRPO_ERR_MISALIGNED;
  const Span out = span(dlogits, rows_bytes(N, R, V, dlogits_seq, dlogits_row, dtype));
  const size_t n = (size_t)rows;
  const Span reads[8] = {span(logits, rows_bytes(N, R, V, logits_seq, logits_row, dtype)),
                         token_span(tokens, N, R, token_seq, token_row),
                         span(len, 4 * (size_t)N),
                         span(temperature, 4 * (size_t)N),
                         span(norm, 8 * n),
                         span(entropy, 4 * n),
                         span(grad_logp, 4 * n),
                         span(grad_entropy, 4 * n)};
  if (overlaps(reads, 8, out)) return GRPO_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_last(stream);
  TokenStatsBwdArgs a;
  a.logits = logits;
  a.dtype = dtype == GRPO_F32 ? 0 : 1;
  a.N = N;
  a.R = R;
  a.V = V;
  a.seq = logits_seq;
  a.row = logits_row;
  a.tokens = tokens;
  a.token_seq = token_seq;
  a.token_row = token_row;
  a.lens = len;
  a.temperature = temperature;
  a.norm = norm;
  a.entropy = entropy;
  a.grad_logp = grad_logp;
  a.grad_entropy = grad_entropy;
  a.dlogits = dlogits;
  a.dseq = dlogits_seq;
  a.drow = dlogits_row;
  return from_cuda(launch_token_stats_bwd(a, dev, (cudaStream_t)stream));
}

grpo_status grpo_adamw_step(const grpo_adamw_tensor* tensors, int64_t count, int state_bits,
                            const grpo_adamw_hyper* hyper, grpo_stream_t stream) {
  if (state_bits != 8 && state_bits != 32) return GRPO_ERR_UNSUPPORTED;
  if (count < 0 || hyper == nullptr || (count > 0 && tensors == nullptr))
    return GRPO_ERR_INVALID_ARG;
  if (count > INT32_MAX) return GRPO_ERR_UNSUPPORTED;
  const grpo_adamw_hyper& h = *hyper;
  const auto size = [](double x) { return x >= 0.0 && x <= 3e38; };  // a float32 magnitude
  if (!(h.beta1 >= 0.0 && h.beta1 < 1.0) || !(h.beta2 >= 0.0 && h.beta2 < 1.0) ||
      !(h.eps >= 0.0 && h.eps <= 0x1p126) ||  // (its reciprocal is a normal number)
      !size(h.weight_decay) || (h.lr_dev == nullptr && !size(h.lr)) ||
      (h.step_dev == nullptr && h.step < 1))
    return GRPO_ERR_INVALID_ARG;
  if (h.norm != nullptr && (!(h.max_norm >= 0.0) || !size(h.norm_eps))) return GRPO_ERR_INVALID_ARG;
  if (!aligned(h.step_dev, 8) || !aligned(h.lr_dev, 4) || !aligned(h.norm, 4))
    return GRPO_ERR_MISALIGNED;
  const bool eight = state_bits == 8;
  const size_t state = eight ? 1 : 4;
  // (room for the table and for the order of its params)
  std::unique_ptr<AdamwTensor[]> table(new (std::nothrow) AdamwTensor[(size_t)count + 1]);
  std::unique_ptr<Span[]> spans(new (std::nothrow) Span[(size_t)count + 1]);
  if (!table || !spans) return GRPO_ERR_UNSUPPORTED;
  int64_t n = 0, all = 0;
  for (int64_t k = 0; k < count; ++k) {
    const grpo_adamw_tensor& t = tensors[k];
    if (!known_dtype(t.param_dtype) || !known_dtype(t.grad_dtype)) return GRPO_ERR_UNSUPPORTED;
    if (t.numel < 0) return GRPO_ERR_INVALID_ARG;
    if (t.numel == 0 || t.grad == nullptr) continue;  // left as it is
    if (t.param == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr ||
        (eight != (t.scales != nullptr)) ||
        (t.master != nullptr && t.param_dtype != GRPO_BF16))
      return GRPO_ERR_INVALID_ARG;
    if (t.numel > INT64_MAX / 16 - all) return GRPO_ERR_UNSUPPORTED;
    all += t.numel;
    if (!aligned(t.param, esize_of(t.param_dtype)) || !aligned(t.grad, esize_of(t.grad_dtype)) ||
        !aligned(t.exp_avg, state) || !aligned(t.exp_avg_sq, state) || !aligned(t.scales, 8) ||
        !aligned(t.master, 4))
      return GRPO_ERR_MISALIGNED;
    const size_t e = (size_t)t.numel;
    const Span own[6] = {span(t.param, e * esize_of(t.param_dtype)), span(t.exp_avg, e * state),
                         span(t.exp_avg_sq, e * state), span(t.master, 4 * e),
                         span(t.scales, 8 * ((e + kStateBlock - 1) / kStateBlock)),
                         span(t.grad, e * esize_of(t.grad_dtype))};
    for (int x = 1; x < 6; ++x)
      if (overlaps(own, x, own[x])) return GRPO_ERR_INVALID_ARG;
    spans[(size_t)n] = own[0];
    AdamwTensor& o = table[(size_t)n++];
    o.param = t.param;
    o.master = t.master;
    o.grad = t.grad;
    o.avg = t.exp_avg;
    o.sq = t.exp_avg_sq;
    o.scales = t.scales;
    o.numel = t.numel;
    o.dt = (t.param_dtype == GRPO_BF16 ? 1 : 0) | (t.grad_dtype == GRPO_BF16 ? 2 : 0);
  }
  if (n == 0) return GRPO_OK;
  // a param listed twice (tied weights) would be updated twice, by blocks that run
  // at the same time
  std::sort(spans.get(), spans.get() + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  for (int64_t k = 1; k < n; ++k)
    if (spans[(size_t)k].lo < spans[(size_t)k - 1].hi) return GRPO_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (current_device(&dev) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_last(stream);
  AdamwArgs a;
  a.tensors = table.get();
  a.count = n;
  a.eight = eight;
  a.step = h.step;
  a.step_dev = h.step_dev;
  a.lr = h.lr;
  a.lr_dev = h.lr_dev;
  a.beta1 = h.beta1;
  a.beta2 = h.beta2;
  a.eps = h.eps;
  a.decay = h.weight_decay;
  a.norm = h.norm;
  a.max_norm = h.max_norm;
  a.norm_eps = h.norm_eps;
  return from_cuda(launch_adamw(a, dev, (cudaStream_t)stream));
}

grpo_status grpo_check_error(const void* workspace, grpo_stream_t stream) {
  if (workspace == nullptr) return GRPO_ERR_INVALID_ARG;
  WsHeader hdr = {};
  const cudaStream_t st = (cudaStream_t)stream;
  stream_take_after_fwd(st);
  if (cudaMemcpyAsync(&hdr, workspace, sizeof hdr, cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return GRPO_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return GRPO_ERR_CUDA;
  uint32_t flags = hdr.flags;
  if (flags == kFlagIndirect && hdr.status_check == ~hdr.status_count) {
    // the flags of every item, a block at a time
    const uint32_t n = hdr.status_count;
    uint32_t buf[1024];
    const char* ws = static_cast<const char*>(workspace);
    flags = 0;
    for (uint32_t k = 0; k < n; k += 1024) {
      const uint32_t c = n - k < 1024 ? n - k : 1024;
      if (cudaMemcpyAsync(buf, ws + 256 + 4 * (size_t)k, 4 * (size_t)c, cudaMemcpyDeviceToHost,
                          st) != cudaSuccess ||
          cudaStreamSynchronize(st) != cudaSuccess)
        return GRPO_ERR_CUDA;
      for (uint32_t j = 0; j < c; ++j) flags |= buf[j];
    }
  }
  if (flags & kFlagTokenRange) return GRPO_ERR_TOKEN_RANGE;
  if (flags & kFlagLengthRange) return GRPO_ERR_LENGTH_RANGE;
  if (flags & kFlagTimeout) return GRPO_ERR_TIMEOUT;
  if (flags & kFlagValue) return GRPO_ERR_VALUE;
  return GRPO_OK;
}

void grpo_set_early_start(int enable) { g_early_start.store(enable != 0 ? 1 : 0); }

grpo_status grpo_selftest_timeout(void* workspace, grpo_stream_t stream) {
  if (workspace == nullptr) return GRPO_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return GRPO_ERR_MISALIGNED;
  stream_take_after_fwd(stream);
  return from_cuda(launch_selftest_timeout(workspace, (cudaStream_t)stream));
}

grpo_status grpo_copy(void* dst, const void* src, size_t bytes, grpo_stream_t stream) {
  if (bytes == 0) return GRPO_OK;
  if (dst == nullptr || src == nullptr) return GRPO_ERR_INVALID_ARG;
  if (!aligned(dst, 16) || !aligned(src, 16) || bytes % 16 != 0) return GRPO_ERR_MISALIGNED;
  const char* d8 = static_cast<const char*>(dst);
  const char* s8 = static_cast<const char*>(src);
  if (d8 < s8 + bytes && s8 < d8 + bytes) return GRPO_ERR_INVALID_ARG;
  DeviceInfo d;
  if (current_device(&d) != cudaSuccess) return GRPO_ERR_CUDA;
  stream_take_after_fwd(stream);
  return from_cuda(launch_copy(dst, src, bytes, d, (cudaStream_t)stream));
}

}  // extern "C"
