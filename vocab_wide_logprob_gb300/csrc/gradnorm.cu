// Global norm of many gradient tensors, and clipping.
//
//   norm = sqrt(sum over all tensors and elements of g^2)   (or max |g|)
//   coef = min(1, max_norm / (norm + eps))
//   out  = coef * g                                          (per element)
//
// Two launches, or three: the norm kernel reads every element once and leaves
// one float64 partial per CTA; they are added in a fixed order; the
// scaling kernel scales.  The table of tensors travels in the kernels'
// parameters (kMaxTensors of them a launch), so a call needs no copy, no device
// table and no synchronisation, and can be captured.
//
// HBM-bound: the norm of 988 MB reads at 7.0 TB/s (141 us), the scaling of it
// into another buffer moves 7.1 TB/s (279 us); a call on 290 tensors takes 435
// us, the norm of 64 MB 10.8 us, 26 small tensors 9 us (8 of it the host's).
#include <math.h>

#include "ops.cuh"

namespace grpo {
namespace {

constexpr int kVecs = 8;  // 16-byte loads in flight per thread
constexpr int64_t kChunkBytes = (int64_t)kThreads * kVecs * 16;  // 32 KiB of one tensor

// What a launch knows about its tensors.  first[k] is the chunk that tensor k
// begins with; first[count] the number of chunks.
template <int CAP>
struct Table {
  const void* data[CAP];
  void* out[CAP];
  int64_t numel[CAP];
  int64_t first[CAP + 1];
  uint8_t dt[CAP];  // bit 0: data is bf16, bit 1: out is bf16
  int count;
};

template <int CAP>
__device__ __forceinline__ int find_tensor(const Table<CAP>& t, int64_t chunk) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// norm
// ---------------------------------------------------------------------------

// A sum of squares, or a maximum.  This GPU has few float64 units (a warp's
// float64 instruction holds the pipe for 16 cycles), so sums are kept as an
// unevaluated pair of floats, hi + lo, exact to 2^-47 of themselves; float64
// takes the batches whose squares leave float32's range, and the CTAs' totals.
struct Acc {
  float hi, lo;  // kMax: hi alone
  double rare;
};
// hi + lo += x (x of any size): the rounding error of each sum is kept.
__device__ __forceinline__ void pair_add(float& hi, float& lo, float x) {
  const float s = hi + x, t = s - hi;
  lo += (hi - (s - t)) + (x - t);
  hi = s;
}
// Squares of values above 2^40 or (all of a batch) below 2^-50 are taken
// apart: scaled by a power of two, which is exact.
template <int N>
__device__ __forceinline__ void add_squares(Acc& a, const float* x, float top) {
  if (top > 0x1p40f || (top < 0x1p-50f && top > 0.f)) {
    const float sc = top > 1.f ? 0x1p-80f : 0x1p100f;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) s = fmaf(x[k] * sc, x[k] * sc, s);
    a.rare += (double)s * (top > 1.f ? 0x1p160 : 0x1p-200);
    return;
  }
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    s0 = fmaf(x[k], x[k], s0);
    s1 = fmaf(x[k + 1], x[k + 1], s1);
    s2 = fmaf(x[k + 2], x[k + 2], s2);
    s3 = fmaf(x[k + 3], x[k + 3], s3);
  }
  pair_add(a.hi, a.lo, (s0 + s1) + (s2 + s3));
}

// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  return a != a ? a : (b != b ? b : fmaxf(a, b));
}

template <typename T, bool kMax>
__device__ __forceinline__ void chunk_norm(Acc& acc, const T* data, int64_t numel, int64_t e0) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec;
  constexpr int kElems = (int)(kChunkBytes / sizeof(T));
  const int64_t e1 = min(e0 + kElems, numel);
  const int tid = threadIdx.x;
  // 16-byte aligned interior [a, b); ragged ends are scalar
  const uintptr_t addr = reinterpret_cast<uintptr_t>(data + e0);
  const int64_t a = min(e0 + (int64_t)(((16u - (unsigned)(addr & 15u)) & 15u) / sizeof(T)), e1);
  const int nvec = (int)((e1 - a) / EPV);
  const int64_t b = a + (int64_t)nvec * EPV;
  uint4 d[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int k = tid + u * kThreads;
    d[u] = k < nvec ? ld_stream(data + a + (int64_t)k * EPV) : make_uint4(0, 0, 0, 0);
  }
  float edge = 0.f;
  if (tid < a - e0) edge = E::load1(data + e0 + tid);
  if (tid >= 32 && tid - 32 < e1 - b) edge = E::load1(data + b + tid - 32);
  if (kMax) {
    acc.hi = max_nan(acc.hi, fabsf(edge));
  } else if (edge != 0.f) {
    const float ed[4] = {edge, 0.f, 0.f, 0.f};
    add_squares<4>(acc, ed, fabsf(edge));
  }
  // halves of the loads at a time, to bound the registers
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[kVecs / 2 * EPV];
#pragma unroll
    for (int u = 0; u < kVecs / 2; ++u) E::unpack(d[h * (kVecs / 2) + u], x + u * EPV);
    if (kMax) {
#pragma unroll
      for (int k = 0; k < kVecs / 2 * EPV; ++k) acc.hi = max_nan(acc.hi, fabsf(x[k]));
    } else {
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < kVecs / 2 * EPV; ++k) top = fmaxf(top, fabsf(x[k]));
      add_squares<kVecs / 2 * EPV>(acc, x, top);
    }
  }
}

__device__ __forceinline__ double combine(double a, double b, bool is_max) {
  if (!is_max) return a + b;
  return a != a ? a : (b != b ? b : fmax(a, b));
}

// Sum (or maximum) over the CTA in a fixed tree, in thread 0.
template <bool kMax>
__device__ __forceinline__ double block_total(Acc a) {
  __shared__ float s_hi[kWarps], s_lo[kWarps];
  __shared__ double s_rare[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto tree = [&](int width) {
    for (int o = width / 2; o > 0; o >>= 1) {
      const float hi = __shfl_xor_sync(0xffffffffu, a.hi, o);
      const float lo = __shfl_xor_sync(0xffffffffu, a.lo, o);
      if (kMax) {
        a.hi = max_nan(a.hi, hi);
      } else {
        // (the smaller lane's value first in both, so that both get the same bits)
        float h = (lane & o) ? hi : a.hi, l = ((lane & o) ? lo : a.lo) + ((lane & o) ? a.lo : lo);
        pair_add(h, l, (lane & o) ? a.hi : hi);
        a.hi = h;
        a.lo = l;
      }
    }
  };
  tree(32);
  // (0, or not a number: the rare batches of any thread)
  const bool rare = !kMax && __any_sync(0xffffffffu, !(a.rare == 0.0));
  if (rare)
    for (int o = 16; o > 0; o >>= 1) a.rare += __shfl_xor_sync(0xffffffffu, a.rare, o);
  if (lane == 0) {
    s_hi[warp] = a.hi;
    s_lo[warp] = a.lo;
    s_rare[warp] = a.rare;
  }
  __syncthreads();
  if (warp != 0) return 0.0;
  a.hi = lane < kWarps ? s_hi[lane] : 0.f;
  a.lo = lane < kWarps ? s_lo[lane] : 0.f;
  a.rare = lane < kWarps ? s_rare[lane] : 0.0;
  tree(kWarps);
  if (!kMax && __any_sync(0xffffffffu, !(a.rare == 0.0)))
    for (int o = kWarps / 2; o > 0; o >>= 1) a.rare += __shfl_xor_sync(0xffffffffu, a.rare, o);
  return kMax ? (double)a.hi : (double)a.hi + (double)a.lo + a.rare;
}

template <int CAP, bool kMax>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Table<CAP> t,
                                                             double* partial) {
  pdl_wait();
  pdl_trigger();
  const int64_t chunks = t.first[t.count];
  Acc a = {0.f, 0.f, 0.0};
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int k = find_tensor(t, c);
    if (t.dt[k] & 1)
      chunk_norm<uint16_t, kMax>(a, static_cast<const uint16_t*>(t.data[k]), t.numel[k],
                                 (c - t.first[k]) * (kChunkBytes / 2));
    else
      chunk_norm<float, kMax>(a, static_cast<const float*>(t.data[k]), t.numel[k],
                              (c - t.first[k]) * (kChunkBytes / 4));
  }
  const double total = block_total<kMax>(a);
  if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

// ---------------------------------------------------------------------------
// clip
// ---------------------------------------------------------------------------

template <typename TI, typename TO>
__device__ __forceinline__ void chunk_scale(const void* data_, void* out_, int64_t numel,
                                            int64_t chunk, float coef) {
  constexpr int kElems = (int)(kChunkBytes / sizeof(TI));
  constexpr int kUnits = kElems / 8 / kThreads;  // of 8 elements, per thread
  const int64_t e0 = chunk * kElems;
  const TI* data = static_cast<const TI*>(data_) + e0;
  TO* out = static_cast<TO*>(out_) + e0;
  const int n = (int)min((int64_t)kElems, numel - e0);
  const int tid = threadIdx.x;
  const bool vec = (reinterpret_cast<uintptr_t>(data) | reinterpret_cast<uintptr_t>(out)) % 16 == 0;
  int done = 0;
  if (vec && n == kElems) {
    constexpr int U = kUnits < 4 ? kUnits : 4;  // units in flight
    const TI* p = data + 8 * tid;
    TO* q = out + 8 * tid;
#pragma unroll
    for (int h = 0; h < kUnits; h += U) {
      Vec8<TI> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u].load(p + (h + u) * kThreads * 8);
#pragma unroll
      for (int u = 0; u < U; ++u) v[u].template store<true>(q + (h + u) * kThreads * 8, coef);
    }
    return;
  }
  if (vec) {
    const int n8 = n / 8;
#pragma unroll 1
    for (int k = tid; k < n8; k += kThreads) {
      Vec8<TI> v;
      v.load(data + 8 * k);
      v.template store<true>(out + 8 * k, coef);
    }
    done = 8 * n8;
  }
#pragma unroll 4
  for (int e = done + tid; e < n; e += kThreads) {
    float x;
    if constexpr (sizeof(TI) == 4)
      x = data[e];
    else
      x = bf16_bits_to_float(data[e]);
    Elt<TO>::store1(out + e, x * coef);
  }
}

// The partials added by kW warps in a fixed order, and the coefficient from
// their sum, in the first warp.  Where every CTA does this it is one warp (a
// float64 instruction occupies its pipe for many cycles here, and the CTAs of
// an SM share it); where it is done once, eight.
template <bool kMax, int kW>
__device__ __forceinline__ float coefficient(const double* partial, int npartial, float max_norm,
                                             float eps, float* stats, WsHeader* hdr) {
  double s = 0.0;
#pragma unroll 8
  for (int k = threadIdx.x; k < npartial; k += 32 * kW) s = combine(s, partial[k], kMax);
  for (int o = 16; o > 0; o >>= 1) s = combine(s, __shfl_xor_sync(0xffffffffu, s, o), kMax);
  if (kW > 1) {
    __shared__ double warp_sum[kW];
    if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = s;
    __syncthreads();
    s = warp_sum[0];
    for (int w = 1; w < kW; ++w) s = combine(s, warp_sum[w], kMax);
  }
  const double norm = kMax ? s : sqrt(s);
  double c = (double)max_norm / (norm + (double)eps);
  c = c > 1.0 ? 1.0 : c;         // keeps NaN
  if (isinf(max_norm)) c = 1.0;  // no limit
  if (stats != nullptr && threadIdx.x == 0) {
    stats[0] = (float)norm;
    stats[1] = (float)c;
    hdr->flags = isfinite((float)norm) ? 0u : kFlagValue;
  }
  return (float)c;
}

// The norm and the coefficient alone: the whole second step of
// grpo_grad_norm, and for many chunks the scaling kernel's first.
template <bool kMax>
__global__ void __launch_bounds__(kThreads) grad_coef_kernel(const double* partial, int npartial,
                                                       float max_norm, float eps, float* stats,
                                                       WsHeader* hdr) {
  pdl_wait();
  pdl_trigger();
  coefficient<kMax, kWarps>(partial, npartial, max_norm, eps, stats, hdr);
}

// Scales the chunks last to first (what the norm kernel read last may still be
// in L2: of 988 MB 1% is; keeping more of it by the loads' eviction priorities
// made this kernel slower than it saved).  In place and under the limit there is nothing
// to write.  npartial: the partials to form the coefficient from (the same sum
// in every CTA), or 0: it is in stats already.
template <int CAP, bool kMax>
__global__ void __launch_bounds__(kThreads, 4) grad_scale_kernel(const __grid_constant__ Table<CAP> t,
                                                              const double* partial, int npartial,
                                                              float max_norm, float eps,
                                                              int copies, float* stats,
                                                              WsHeader* hdr, int first) {
  __shared__ float s_coef;
  pdl_wait();
  pdl_trigger();
  float coef;
  if (npartial == 0) {
    coef = stats[1];
  } else {
    if (threadIdx.x < 32) {
      const float c = coefficient<kMax, 1>(partial, npartial, max_norm, eps,
                                        first && blockIdx.x == 0 ? stats : nullptr, hdr);
      if (threadIdx.x == 0) s_coef = c;
    }
    __syncthreads();
    coef = s_coef;
  }
  if (coef == 1.f && !copies) return;
  const int64_t chunks = t.first[t.count];
  for (int64_t r = blockIdx.x; r < chunks; r += gridDim.x) {
    const int64_t ch = chunks - 1 - r;
    const int k = find_tensor(t, ch);
    if (coef == 1.f && t.out[k] == t.data[k]) continue;
    const int64_t n = t.numel[k], j = ch - t.first[k];
    switch (t.dt[k]) {
      case 0:
        chunk_scale<float, float>(t.data[k], t.out[k], n, j, coef);
        break;
      case 1:
        chunk_scale<uint16_t, float>(t.data[k], t.out[k], n, j, coef);
        break;
      case 2:
        chunk_scale<float, uint16_t>(t.data[k], t.out[k], n, j, coef);
        break;
      default:
        chunk_scale<uint16_t, uint16_t>(t.data[k], t.out[k], n, j, coef);
    }
  }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------

constexpr int kMaxTensors = 768;     // tensors of one launch: the parameters stay below 32 KiB
constexpr int kMaxPartials = kPlanSms * 8;  // CTAs of one norm launch
static_assert(sizeof(Table<kMaxTensors>) < 32000, "kernel parameters");

template <int CAP>
void fill(Table<CAP>* t, const GradTensor* g, int count) {
  t->count = count;
  int64_t at = 0;
  for (int k = 0; k < count; ++k) {
    t->data[k] = g[k].data;
    t->out[k] = g[k].out;
    t->numel[k] = g[k].numel;
    t->dt[k] = (uint8_t)g[k].dt;
    t->first[k] = at;
    const int64_t per = kChunkBytes / ((g[k].dt & 1) ? 2 : 4);
    at += (g[k].numel + per - 1) / per;
  }
  t->first[count] = at;
}

int64_t chunks_of(const GradTensor& g) {
  const int64_t per = kChunkBytes / ((g.dt & 1) ? 2 : 4);
  return (g.numel + per - 1) / per;
}

// One group of tensors.  step 0: its norm kernel, nparts partials from part0
// on; step 2: its scaling kernel (nparts partials in all, or 0 when the
// coefficient is known).
template <int CAP, bool kMax>
cudaError_t clip_launch(const ClipArgs& a, const GradTensor* g, int count, int part0, int nparts,
                        int step, bool first, const DeviceInfo& d, cudaStream_t st) {
  Table<CAP> t;
  fill(&t, g, count);
  double* partial = reinterpret_cast<double*>(static_cast<char*>(a.ws) + 256);
  if (step == 0)
    return launch_pdl(grad_norm_kernel<CAP, kMax>, dim3((unsigned)nparts), dim3(kThreads), 0, st,
                      1, t, partial + part0);
  bool copies = false;
  for (int k = 0; k < count; ++k) copies |= g[k].out != g[k].data;
  // into other tensors a CTA per chunk (1 GiB in 460 us, norm included; 64 CTAs
  // per SM, 471); in place, where there may be nothing to do, those that are
  // resident at once (1 GiB under the limit 154 us, over it 480; a CTA per chunk
  // 186 and 466)
  const int64_t chunks = t.first[count];
  int64_t grid = 4 * (int64_t)d.sms;
  if (grid > chunks || copies) grid = chunks;
  if (grid < 1) grid = 1;
  return launch_pdl(grad_scale_kernel<CAP, kMax>, dim3((unsigned)grid), dim3(kThreads), 0, st, 1,
                    t, (const double*)partial, nparts, a.max_norm, a.eps, (int)copies, a.stats,
                    static_cast<WsHeader*>(a.ws), (int)first);
}

template <bool kMax>
cudaError_t clip_run(const ClipArgs& a, const DeviceInfo& d, cudaStream_t st) {
  // the norm of every group of tensors, the coefficient, the scaling of every
  // group.  With few chunks the scaling kernel's CTAs form the coefficient
  // themselves (a launch less: 8 MiB into a copy 8.5 us, against 9.7); with many a
  // kernel of its own does it once (64 MiB 30 us, against 41; 16 MiB 13.2 either way).
  int64_t all = 0;
  for (int64_t k = 0; k < a.count; ++k) all += chunks_of(a.tensors[k]);
  const bool apart = a.norm_only || all > 4 * (int64_t)d.sms;
  int parts = 0;
  cudaError_t e = cudaSuccess;
  for (int step = 0; step < 3; ++step) {
    if (step == 1) {
      if (apart)
        e = launch_pdl(grad_coef_kernel<kMax>, dim3(1), dim3(kThreads), 0, st, 1,
                       (const double*)(static_cast<char*>(a.ws) + 256), parts, a.max_norm, a.eps,
                       a.stats, static_cast<WsHeader*>(a.ws));
      if (e != cudaSuccess || a.norm_only) return e;
      continue;
    }
    int part0 = 0;
    for (int64_t k = 0; k == 0 || k < a.count; k += kMaxTensors) {
      const int cnt = (int)(a.count - k < kMaxTensors ? a.count - k : kMaxTensors);
      const GradTensor* g = a.tensors + k;
      int64_t np = 0;
      for (int j = 0; j < cnt; ++j) np += chunks_of(g[j]);
      if (np > 8 * (int64_t)d.sms) np = 8 * (int64_t)d.sms;
      if (np > kMaxPartials) np = kMaxPartials;
      if (np < 1) np = 1;
      const int n = step == 0 ? (int)np : (apart ? 0 : parts);
      if (cnt <= 32)
        e = clip_launch<32, kMax>(a, g, cnt, part0, n, step, k == 0, d, st);
      else if (cnt <= 192)
        e = clip_launch<192, kMax>(a, g, cnt, part0, n, step, k == 0, d, st);
      else
        e = clip_launch<kMaxTensors, kMax>(a, g, cnt, part0, n, step, k == 0, d, st);
      if (e != cudaSuccess) return e;
      part0 += (int)np;
    }
    if (step == 0) parts = part0;
  }
  return e;
}

}  // namespace

size_t grad_norm_workspace_bytes(int64_t count) {
  const size_t groups = count < 1 ? 1 : (size_t)((count + kMaxTensors - 1) / kMaxTensors);
  return 256 + align_up(groups * kMaxPartials * sizeof(double), 256);
}

cudaError_t launch_clip(const ClipArgs& a, const DeviceInfo& d, cudaStream_t st) {
  return a.type == 0 ? clip_run<false>(a, d, st) : clip_run<true>(a, d, st);
}

}  // namespace grpo
