// AdamW over many tensors in one launch, with states in float32 or in 8 bits.
//
//   g  = c grad,  m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2
//   w' = w - lr (m' / (1 - b1^t) / (sqrt(v' / (1 - b2^t)) + eps) + decay w)
//
// in float32 per element; w is the float32 master where there is one.  The
// decay is added to the update before lr multiplies both: 1 - lr decay would
// round to 1 for the learning rates of policy updates.
//
// States in 8 bits: a warp holds a block of 256 elements, 8 per lane, so that the
// block's largest |m'| and sqrt(v') are two warp reductions.  e4m3 keeps 3 bits
// after the leading one over 2^18 of range: rounding to nearest is off by up to 2^-4 of
// a value, which the step itself never sees (it uses the unrounded m' and v').
// A value next to a border between codes goes to one or the other by its last bit, so
// everything up to the codes is rounded as the formula is written, operation by
// operation (no fused products, the root and the quotients correctly rounded): the codes
// are those of the same float32 formula anywhere.
#include <math.h>

#include <type_traits>

#include "ops.cuh"

namespace grpo {
namespace {

constexpr int kChunk = 2048;  // elements of a thread block's piece of a tensor
constexpr int kUnits = kChunk / 8 / kThreads;  // of 8 elements, per thread
constexpr float kF8Max = 448.f;                // e4m3's largest value
constexpr float kF8Tiny = 0x1p-9f;             // and its smallest positive one
constexpr float kNothing = 0x1p-80f;           // a block of smaller |m| is stored as 0
static_assert(kChunk % kStateBlock == 0 && kStateBlock == 8 * 32, "a warp holds a block");

template <int CAP>
struct Table {
  void* param[CAP];
  float* master[CAP];
  const void* grad[CAP];
  void* avg[CAP];
  void* sq[CAP];
  float* scales[CAP];
  int64_t numel[CAP];
  int64_t first[CAP + 1];  // the chunk that a tensor begins with
  uint8_t dt[CAP];         // bit 0: param is bf16, bit 1: grad is bf16
  int count;
};

struct Hyper {
  float lr, beta1, beta2, one_minus1, one_minus2, eps, decay;
  float inv_c1, inv_root_c2;  // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float ln_beta1, ln_beta2;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* norm;
  float max_norm, norm_eps;
};

// What a step takes from device memory where the caller has it there.
struct Now {
  float coef, lr, inv_c1, inv_root_c2;
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

// ---- 8 consecutive elements ------------------------------------------------------

__device__ __forceinline__ void ld8(const float* p, float* x) {
  if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]),
                   "=f"(x[6]), "=f"(x[7])
                 : "l"(p));
    return;
  }
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void ld8(const uint16_t* p, float* x) {
  Elt<uint16_t>::unpack(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void st8(float* p, const float* x) {
  if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
    st_32bytes<false>(p, x);
    return;
  }
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void st8(uint16_t* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = Elt<uint16_t>::pack(x);
}

// e4m3 codes
struct F8 {
  uint8_t bits;
};
__device__ __forceinline__ uint32_t f8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void f8_unpack2(uint32_t w, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}
__device__ __forceinline__ void ld8(const F8* p, float* x) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  f8_unpack2(w.x & 0xffffu, x[0], x[1]);
  f8_unpack2(w.x >> 16, x[2], x[3]);
  f8_unpack2(w.y & 0xffffu, x[4], x[5]);
  f8_unpack2(w.y >> 16, x[6], x[7]);
}
__device__ __forceinline__ void st8(F8* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(f8_pack2(x[0], x[1]) | f8_pack2(x[2], x[3]) << 16,
                                            f8_pack2(x[4], x[5]) | f8_pack2(x[6], x[7]) << 16);
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const uint16_t* p) { return bf16_bits_to_float(*p); }
__device__ __forceinline__ float ld1(const F8* p) {
  float x, y;
  f8_unpack2(p->bits, x, y);
  return x;
}
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(uint16_t* p, float x) { Elt<uint16_t>::store1(p, x); }
__device__ __forceinline__ void st1(F8* p, float x) { p->bits = (uint8_t)f8_pack2(x, 0.f); }

// n of 8 elements (zeros behind them); wide: all 8, aligned
template <typename T>
__device__ __forceinline__ void load(const T* p, float* x, bool wide, int n) {
  if (wide) {
    ld8(p, x);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = k < n ? ld1(p + k) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store(T* p, const float* x, bool wide, int n) {
  if (wide) {
    st8(p, x);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) st1(p + k, x[k]);
}

__device__ __forceinline__ float max_keep_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The block's scale from a lane's largest value, and its reciprocal, rounded.
__device__ __forceinline__ float block_scale(float largest, float& inverse) {
  for (int o = 16; o > 0; o >>= 1)
    largest = max_keep_nan(largest, __shfl_xor_sync(0xffffffffu, largest, o));
  const bool any = largest > kNothing;
  const float scale = any ? __fmul_rn(largest, 1.f / kF8Max) : (largest != largest ? NAN : 0.f);
  inverse = any ? __frcp_rn(scale) : 0.f;
  return scale;
}
// x / s correctly rounded, from the correctly rounded 1 / s (P. Markstein's
// theorem: an estimate within one step, its remainder by a fused product, one correction).
// s is above 2^-89, so that the remainder of a quotient that has a code is exact.
__device__ __forceinline__ float quotient(float x, float s, float inverse) {
  const float q = __fmul_rn(x, inverse);
  return __fmaf_rn(__fmaf_rn(-q, s, x), inverse, q);
}

// ---- the step ------------------------------------------------------------------------

// One chunk of one tensor.  W: param, G: grad, kMaster: bf16 param with a master.
template <typename W, typename G, bool kMaster, bool kEight>
__device__ __forceinline__ void chunk_step(W* param, float* master, const G* grad, void* avg_,
                                           void* sq_, float* scales, int64_t numel, int64_t e0,
                                           const Hyper& h, const Now& now) {
  using State = std::conditional_t<kEight, F8, float>;
  State* avg = static_cast<State*>(avg_);
  State* sq = static_cast<State*>(sq_);
  const int lane = threadIdx.x & 31;
  const uintptr_t states = reinterpret_cast<uintptr_t>(avg) | reinterpret_cast<uintptr_t>(sq);
  const uintptr_t others = reinterpret_cast<uintptr_t>(param) | reinterpret_cast<uintptr_t>(grad) |
                           (kMaster ? reinterpret_cast<uintptr_t>(master) : 0);
  const bool aligned = (others & 15) == 0 && (states & (kEight ? 7 : 15)) == 0;
  float g[kUnits][8], m[kUnits][8], v[kUnits][8], w[kUnits][8];
  float2 sc[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t e = e0 + (int64_t)(u * kThreads + threadIdx.x) * 8;
    const int n = (int)min((int64_t)8, numel - e);  // (none or fewer behind the end)
    const bool wide = aligned && n == 8;
    load(grad + e, g[u], wide, n);
    load(avg + e, m[u], wide, n);
    load(sq + e, v[u], wide, n);
    if (kMaster)
      load(master + e, w[u], wide, n);
    else
      load(param + e, w[u], wide, n);
    if (kEight) {
      const int64_t block = (e - lane * 8) / kStateBlock;
      sc[u] = block * kStateBlock < numel ? make_float2(scales[2 * block], scales[2 * block + 1])
                                          : make_float2(0.f, 0.f);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t e = e0 + (int64_t)(u * kThreads + threadIdx.x) * 8;
    const int n = (int)min((int64_t)8, numel - e);
    const bool wide = aligned && n == 8;
    float most_m = 0.f, most_r = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gk = __fmul_rn(g[u][k], now.coef);
      float mk = m[u][k], vk = v[u][k];
      if (kEight) {
        mk = __fmul_rn(mk, sc[u].x);
        vk = __fmul_rn(vk, sc[u].y);
        vk = __fmul_rn(vk, vk);
      }
      mk = __fadd_rn(__fmul_rn(mk, h.beta1), __fmul_rn(gk, h.one_minus1));
      vk = __fadd_rn(__fmul_rn(vk, h.beta2), __fmul_rn(__fmul_rn(gk, gk), h.one_minus2));
      const float root = __fsqrt_rn(vk);
      const float up = __fdividef(mk * now.inv_c1, fmaf(root, now.inv_root_c2, h.eps));
      w[u][k] = fmaf(-now.lr, fmaf(h.decay, w[u][k], up), w[u][k]);
      m[u][k] = mk;
      v[u][k] = kEight ? root : vk;
      if (kEight) {
        most_m = max_keep_nan(most_m, fabsf(mk));
        most_r = max_keep_nan(most_r, root);
      }
    }
    if (kEight) {
      float im, ir;
      const float sm = block_scale(most_m, im), sr = block_scale(most_r, ir);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[u][k] = quotient(m[u][k], sm, im);
        const float r = quotient(v[u][k], sr, ir);
        v[u][k] = r > 0.f ? fmaxf(r, kF8Tiny) : r;
      }
      if (lane == 0 && n > 0) {
        const int64_t block = e / kStateBlock;
        scales[2 * block] = sm;
        scales[2 * block + 1] = sr;
      }
    }
    store(avg + e, m[u], wide, n);
    store(sq + e, v[u], wide, n);
    if (kMaster) store(master + e, w[u], wide, n);
    store(param + e, w[u], wide, n);
  }
}

template <int CAP, bool kEight>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ Table<CAP> t,
                                                            const __grid_constant__ Hyper h) {
  pdl_wait();
  pdl_trigger();
  Now now = {1.f, h.lr, h.inv_c1, h.inv_root_c2};
  if (h.norm != nullptr) {
    const float norm = *h.norm;
    if (!(fabsf(norm) < INFINITY)) return;  // the step is skipped
    now.coef = fminf(__fmul_rn(h.max_norm, __frcp_rn(norm + h.norm_eps)), 1.f);
  }
  if (h.lr_dev != nullptr) now.lr = *h.lr_dev;
  if (h.step_dev != nullptr) {
    const float step = (float)*h.step_dev;
    now.inv_c1 = 1.f / -expm1f(step * h.ln_beta1);
    now.inv_root_c2 = 1.f / sqrtf(-expm1f(step * h.ln_beta2));
  }
  const int64_t chunk = blockIdx.x;
  const int k = find_tensor(t, chunk);
  const int64_t e0 = (chunk - t.first[k]) * kChunk, n = t.numel[k];
  const int dt = t.dt[k] | (t.master[k] != nullptr ? 4 : 0);
  using B = uint16_t;
#define STEP(W, G, MASTER)                                                                 \
  chunk_step<W, G, MASTER, kEight>(static_cast<W*>(t.param[k]), t.master[k],               \
                                   static_cast<const G*>(t.grad[k]), t.avg[k], t.sq[k],    \
                                   t.scales[k], n, e0, h, now)
  switch (dt) {
    case 0:
      STEP(float, float, false);
      break;
    case 1:
      STEP(B, float, false);
      break;
    case 2:
      STEP(float, B, false);
      break;
    case 3:
      STEP(B, B, false);
      break;
    case 5:
      STEP(B, float, true);
      break;
    default:
      STEP(B, B, true);
  }
#undef STEP
}

// ---- launch ------------------------------------------------------------------------------

constexpr int kMaxTensors = 480;  // of one launch: the parameters stay below 32 KiB
static_assert(sizeof(Table<kMaxTensors>) + sizeof(Hyper) < 32000, "kernel parameters");

int64_t chunks_of(const AdamwTensor& t) { return (t.numel + kChunk - 1) / kChunk; }

template <int CAP>
cudaError_t launch_group(const AdamwTensor* g, int count, bool eight, const Hyper& h,
                         cudaStream_t st) {
  Table<CAP> t;
  t.count = count;
  int64_t at = 0;
  for (int k = 0; k < count; ++k) {
    t.param[k] = g[k].param;
    t.master[k] = g[k].master;
    t.grad[k] = g[k].grad;
    t.avg[k] = g[k].avg;
    t.sq[k] = g[k].sq;
    t.scales[k] = g[k].scales;
    t.numel[k] = g[k].numel;
    t.dt[k] = (uint8_t)g[k].dt;
    t.first[k] = at;
    at += chunks_of(g[k]);
  }
  t.first[count] = at;
  const dim3 grid((unsigned)at), block(kThreads);
  return eight ? launch_pdl(adamw_kernel<CAP, true>, grid, block, 0, st, 1, t, h)
               : launch_pdl(adamw_kernel<CAP, false>, grid, block, 0, st, 1, t, h);
}

}  // namespace

cudaError_t launch_adamw(const AdamwArgs& a, const DeviceInfo&, cudaStream_t st) {
  Hyper h;
  h.lr = (float)a.lr;
  h.beta1 = (float)a.beta1;
  h.beta2 = (float)a.beta2;
  h.one_minus1 = (float)(1.0 - a.beta1);
  h.one_minus2 = (float)(1.0 - a.beta2);
  h.eps = (float)a.eps;
  h.decay = (float)a.decay;
  h.ln_beta1 = (float)log(a.beta1);
  h.ln_beta2 = (float)log(a.beta2);
  h.inv_c1 = (float)(1.0 / -expm1((double)a.step * log(a.beta1)));
  h.inv_root_c2 = (float)(1.0 / sqrt(-expm1((double)a.step * log(a.beta2))));
  h.step_dev = a.step_dev;
  h.lr_dev = a.lr_dev;
  h.norm = a.norm;
  h.max_norm = (float)a.max_norm;
  h.norm_eps = (float)a.norm_eps;
  // tensors in launches of at most kMaxTensors and 2^30 chunks
  int64_t k = 0;
  while (k < a.count) {
    int n = 0;
    int64_t chunks = 0;
    while (k + n < a.count && n < kMaxTensors &&
           (n == 0 || chunks + chunks_of(a.tensors[k + n]) < (int64_t)1 << 30))
      chunks += chunks_of(a.tensors[k + n++]);
    const AdamwTensor* g = a.tensors + k;
    const cudaError_t e = n <= 32    ? launch_group<32>(g, n, a.eight, h, st)
                          : n <= 128 ? launch_group<128>(g, n, a.eight, h, st)
                                     : launch_group<kMaxTensors>(g, n, a.eight, h, st);
    if (e != cudaSuccess) return e;
    k += n;
  }
  return cudaSuccess;
}

}  // namespace grpo
