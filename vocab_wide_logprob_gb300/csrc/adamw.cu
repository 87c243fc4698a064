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
// operation: no fused products, the quotients correctly rounded, the root but in one of a
// million cases, c and the scales as products with rounded reciprocals.  So the codes are
// those of the same float32 formula anywhere, but for about as few.
#include <math.h>

#include <type_traits>

#include "ops.cuh"

namespace grpo {
namespace {

constexpr int kUnit = 8 * kThreads;  // elements that a thread block takes at once
constexpr float kF8Max = 448.f;                // e4m3's largest value
constexpr float kNothing = 0x1p-80f;           // a block of smaller |m| is stored as 0
constexpr float kMaxRoot = 0x1.fffffep63f;     // of the largest float
static_assert(kUnit % kStateBlock == 0 && kStateBlock == 8 * 32, "a warp holds a block");

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
  int units;  // of a chunk
};

struct Hyper {
  float lr, beta1, beta2, one_minus1, one_minus2, eps, decay;
  float inv_c1, inv_root_c2;  // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float ln_beta1, ln_beta2;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* norm;
  float max_norm, norm_eps;
  float minus_zero;
};

// What a step takes from device memory where the caller has it there.
struct Now {
  float coef, lr, inv_c1, inv_root_c2;
};

// ---- 8 consecutive elements ------------------------------------------------------

// As they are stored, in registers.
template <typename T>
struct Raw8;

template <>
struct Raw8<float> {
  float x[8];
  __device__ __forceinline__ void load(const float* p) {
    if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
      asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]),
                     "=f"(x[6]), "=f"(x[7])
                   : "l"(p));
      return;
    }
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void load_some(const float* p, int n) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? p[k] : 0.f;
  }
  __device__ __forceinline__ uint64_t pair(int k) const { return f2_pack(x[2 * k], x[2 * k + 1]); }
  __device__ __forceinline__ void set(int k, uint64_t v) { f2_unpack(v, x[2 * k], x[2 * k + 1]); }
  __device__ __forceinline__ void store(float* p) const {
    if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
      st_32bytes<false>(p, x);
      return;
    }
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void store_some(float* p, int n) const {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = x[k];
  }
};

template <>
struct Raw8<uint16_t> {  // bfloat16
  uint32_t w[4];
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ __forceinline__ void load_some(const uint16_t* p, int n) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (2 * k < n ? (uint32_t)p[2 * k] : 0u) |
             (2 * k + 1 < n ? (uint32_t)p[2 * k + 1] << 16 : 0u);
  }
  __device__ __forceinline__ uint64_t pair(int k) const {
    return f2_pack(bf16_lo(w[k]), bf16_hi(w[k]));
  }
  __device__ __forceinline__ void set(int k, uint64_t v) {
    float a, b;
    f2_unpack(v, a, b);
    w[k] = pack_bf16x2(a, b);
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store_some(uint16_t* p, int n) const {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = (uint16_t)(w[k / 2] >> (k % 2 * 16));
  }
};

template <>
struct Raw8<uint8_t> {  // e4m3 codes
  uint32_t w[2];
  __device__ __forceinline__ void load(const uint8_t* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
  __device__ __forceinline__ void load_some(const uint8_t* p, int n) {
    w[0] = w[1] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) w[k / 4] |= (uint32_t)p[k] << (k % 4 * 8);
  }
  __device__ __forceinline__ uint64_t pair(int k) const {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[k / 2] >> (k % 2 * 16))));
    float a, b;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(h));
    return f2_pack(a, b);
  }
  __device__ __forceinline__ void set(int k, uint64_t v) {  // k in order
    float a, b;
    f2_unpack(v, a, b);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    w[k / 2] = k % 2 == 0 ? (uint32_t)r : w[k / 2] | (uint32_t)r << 16;
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ void store_some(uint8_t* p, int n) const {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = (uint8_t)(w[k / 4] >> (k % 4 * 8));
  }
};

template <typename T>
__device__ __forceinline__ void load(Raw8<T>& r, const T* p, bool wide, int n) {
  if (wide)
    r.load(p);
  else
    r.load_some(p, n);
}
template <typename T>
__device__ __forceinline__ void store(const Raw8<T>& r, T* p, bool wide, int n) {
  if (wide)
    r.store(p);
  else
    r.store_some(p, n);
}

// The block's scale from a lane's largest value (not negative: its bits are ordered
// as it is, NaN above all), and its reciprocal by one Newton step.
__device__ __forceinline__ float block_scale(float largest, float& inverse) {
  const float all = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(largest)));
  const bool any = all > kNothing;
  const float scale = any ? __fmul_rn(all, 1.f / kF8Max) : (all != all ? NAN : 0.f);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(scale));
  inverse = any ? fmaf(fmaf(-y, scale, 1.f), y, y) : 0.f;
  return scale;
}
__device__ __forceinline__ uint64_t both(float x) { return f2_pack(x, x); }

// Products that stay products: an addition behind f2_mul becomes one fused
// instruction with it (seen in the sums' last bits); behind x y + z, with a z that is -0
// but not known to be when this is compiled, it cannot.
__device__ __forceinline__ uint64_t product(uint64_t x, uint64_t y, const Hyper& h) {
  return f2_fma(x, y, both(h.minus_zero));
}

// |x| / s correctly rounded, for x that is all -|x| (sign -1) or any x (sign 1), from the
// correctly rounded 1 / s (P. Markstein's theorem: an estimate within one step, its
// remainder by a fused product, one correction).  s is above 2^-89, so that the remainder
// of a quotient that has a code is exact.  minus_s: -s, or s for sign -1; inverse: with
// the sign.
__device__ __forceinline__ uint64_t quotient(uint64_t x, uint64_t minus_s, uint64_t inverse) {
  const uint64_t q = f2_mul(x, inverse);
  return f2_fma(f2_fma(q, minus_s, x), inverse, q);
}
// -sqrt(v) from -v, by one Newton step (Heron's, on the reciprocal root's
// estimate y): v y = sqrt(v) (1 + d) with |d| below 2^-22, and the remainder (v y)^2 - v is
// exact, so that what is rounded at the end is off by 2^-44: the nearest float32 but in one of a
// million cases.  For v that is 0 or from 2^-126 to the largest float: infinity gives NaN here,
// and below 2^-126, where the estimate is held, the root comes out too small.
__device__ __forceinline__ uint64_t minus_root(uint64_t minus_v) {
  float a, b, ya, yb;
  f2_unpack(minus_v, a, b);
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(ya) : "f"(max_keep_nan(-a, 0x1p-126f)));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(yb) : "f"(max_keep_nan(-b, 0x1p-126f)));
  const uint64_t y = f2_pack(ya, yb), s = f2_mul(minus_v, y);
  return f2_fma(f2_fma(s, s, minus_v), f2_mul(y, both(0.5f)), s);
}
// Whether one of the two v is none of those.
__device__ __forceinline__ bool outside(uint64_t minus_v, uint64_t root) {
  float a, b;
  f2_unpack(minus_v, a, b);
  // (below 2^23 - 1 where v lies between 0 and 2^-126; 0 is the largest number)
  const uint32_t least = min(__float_as_uint(a) - 0x80000001u, __float_as_uint(b) - 0x80000001u);
  f2_unpack(root, a, b);
  int nan;  // (of either, in one instruction)
  asm("{\n\t.reg .pred p;\n\tsetp.nan.f32 p, %1, %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(nan)
      : "f"(a), "f"(b));
  return least < 0x7fffffu || nan != 0;
}
// The same for any v: below 2^-126 it is scaled by 2^100, the root of infinity is infinity.
__device__ __forceinline__ uint64_t minus_root_any(uint64_t minus_v) {
  float v[2], up[2], r[2];
  f2_unpack(minus_v, v[0], v[1]);
#pragma unroll
  for (int k = 0; k < 2; ++k) up[k] = v[k] > -0x1p-126f ? 0x1p50f : 1.f;
  const uint64_t by = f2_pack(up[0], up[1]);
  f2_unpack(minus_root(f2_mul(f2_mul(minus_v, by), by)), r[0], r[1]);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (up[k] != 1.f) r[k] *= 0x1p-50f;
    if (v[k] == -INFINITY) r[k] = v[k];
  }
  return f2_pack(r[0], r[1]);
}
// -sqrt(v') as 8-bit states store it: an infinite one beside a finite m' as the largest float's
// (the block keeps a scale), or |m'| if that is more (the next steps stay of lr's size).
__device__ __forceinline__ uint64_t stored_roots(uint64_t root, uint64_t m) {
  float a, b, c, d;
  f2_unpack(root, a, b);
  f2_unpack(m, c, d);
  if (a == -INFINITY && fabsf(c) < INFINITY) a = fminf(-kMaxRoot, -fabsf(c));
  if (b == -INFINITY && fabsf(d) < INFINITY) b = fminf(-kMaxRoot, -fabsf(d));
  return f2_pack(a, b);
}
__device__ __forceinline__ uint64_t reciprocals(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return f2_pack(a, b);
}

// ---- the step ------------------------------------------------------------------------

// One tensor's arrays from a chunk's first element on.
template <typename W, typename G, typename State, typename Value>
struct Arrays {
  W* param;
  Value* value;  // the master, or the param
  const G* grad;
  State *avg, *sq;
  float2* scales;
  int left;      // elements from here on (of the chunk)
  bool aligned;  // all of them
};

// What 8 elements' step reads.
template <typename G, typename State, typename Value>
struct In {
  Raw8<G> g;
  Raw8<State> m, v;
  Raw8<Value> w;
  float2 sc;
  template <typename W>
  __device__ __forceinline__ void fetch(const Arrays<W, G, State, Value>& t, int e) {
    const int n = max(0, min(8, t.left - e));
    const bool wide = t.aligned && n == 8;
    load(g, t.grad + e, wide, n);
    load(m, t.avg + e, wide, n);
    load(v, t.sq + e, wide, n);
    load(w, t.value + e, wide, n);
    const int block = e / kStateBlock;  // one of the warp's
    sc = sizeof(State) == 1 && block * kStateBlock < t.left ? t.scales[block]
                                                            : make_float2(0.f, 0.f);
  }
};

// 8 elements' step, from what was fetched.
template <typename W, typename G, typename State, typename Value>
__device__ __forceinline__ void step8(const Arrays<W, G, State, Value>& t, int e,
                                      In<G, State, Value>& x, const Hyper& h, const Now& now) {
  constexpr bool kEight = sizeof(State) == 1;
  const int n = max(0, min(8, t.left - e));
  const bool wide = t.aligned && n == 8;
  uint64_t new_m[4], new_v[4];  // m', and -v' or (as 8-bit states store it) -sqrt(v')
  float most_m = 0.f, most_r = 0.f;
  // (two pairs at a time, looked at together for v' that minus_root does not take: 494 M elements
  // with 8-bit states 1,002 us, pair by pair 1,016; 1,032 without the look)
#pragma unroll
  for (int k0 = 0; k0 < 4; k0 += 2) {
    uint64_t mk[2], vk[2], root[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = k0 + j;
      const uint64_t gk = f2_mul(x.g.pair(k), both(now.coef));
      mk[j] = x.m.pair(k), vk[j] = x.v.pair(k);
      if (kEight) {
        mk[j] = f2_mul(mk[j], both(x.sc.x));
        vk[j] = f2_mul(vk[j], both(x.sc.y));
        vk[j] = f2_mul(vk[j], vk[j]);
      }
      mk[j] = f2_add(product(mk[j], both(h.beta1), h), product(gk, both(h.one_minus1), h));
      vk[j] = f2_add(product(vk[j], both(-h.beta2), h),
                    product(f2_mul(gk, gk), both(-h.one_minus2), h));
      root[j] = minus_root(vk[j]);
      new_v[k] = kEight ? root[j] : vk[j];
    }
    if (outside(vk[0], root[0]) || outside(vk[1], root[1])) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        root[j] = minus_root_any(vk[j]);
        if (kEight) new_v[k0 + j] = stored_roots(root[j], mk[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = k0 + j;
      const uint64_t over = reciprocals(f2_fma(root[j], both(-now.inv_root_c2), both(h.eps)));
      const uint64_t wk = x.w.pair(k);
      // lr (m' / c1 / (..) + decay w)
      const uint64_t change = f2_fma(f2_mul(mk[j], both(now.inv_c1)), over, f2_mul(wk, both(h.decay)));
      x.w.set(k, f2_fma(change, both(-now.lr), wk));
      new_m[k] = mk[j];
      if (kEight) {
        float a, b;
        f2_unpack(mk[j], a, b);
        most_m = max_keep_nan(most_m, max_keep_nan(fabsf(a), fabsf(b)));
        f2_unpack(new_v[k], a, b);
        most_r = max_keep_nan(most_r, max_keep_nan(fabsf(a), fabsf(b)));
      }
    }
  }
  if constexpr (kEight) {
    float im, ir;
    const float sm = block_scale(most_m, im), sr = block_scale(most_r, ir);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x.m.set(k, quotient(new_m[k], both(-sm), both(im)));
      x.v.set(k, quotient(new_v[k], both(sr), both(-ir)));
    }
    // a positive root stays positive: a code that is 0 becomes 1 (a root of 0 has the code of
    // -0 this far, which its sign gives away)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t& w = x.v.w[j];
      // (0x80 in the bytes that are 0: no byte's sum passes into the next)
      const uint32_t zero = ~(((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w) & 0x80808080u;
      w = (w & 0x7f7f7f7fu) | zero >> 7;
    }
    if ((threadIdx.x & 31) == 0) t.scales[e / kStateBlock] = make_float2(sm, sr);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x.m.set(k, new_m[k]);
      float a, b;
      f2_unpack(new_v[k], a, b);
      x.v.set(k, f2_pack(fabsf(a), fabsf(b)));
    }
  }
  store(x.m, t.avg + e, wide, n);
  store(x.v, t.sq + e, wide, n);
  store(x.w, t.value + e, wide, n);
  if constexpr (!std::is_same_v<W, Value>) {
    Raw8<W> rounded;
#pragma unroll
    for (int k = 0; k < 4; ++k) rounded.set(k, x.w.pair(k));
    store(rounded, t.param + e, wide, n);
  }
}

// One chunk of one tensor.  W: param, G: grad, kMaster: bf16 param with a master.
template <typename W, typename G, bool kMaster, bool kEight>
__device__ __forceinline__ void chunk_step(W* param, float* master, const G* grad, void* avg_,
                                           void* sq_, float* scales, int64_t numel, int64_t e0,
                                           int units, const Hyper& h, const Now& now) {
  using State = std::conditional_t<kEight, uint8_t, float>;
  using Value = std::conditional_t<kMaster, float, W>;
  Arrays<W, G, State, Value> t;
  t.param = param + e0;
  if constexpr (kMaster)
    t.value = master + e0;
  else
    t.value = t.param;
  t.grad = grad + e0;
  t.avg = static_cast<State*>(avg_) + e0;
  t.sq = static_cast<State*>(sq_) + e0;
  t.scales = reinterpret_cast<float2*>(scales) + e0 / kStateBlock;
  t.left = (int)min(numel - e0, (int64_t)units * kUnit);
  const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  t.aligned = ((at(t.param) | at(t.grad) | at(t.value)) & 15) == 0 &&
              ((at(t.avg) | at(t.sq)) & (kEight ? 7 : 15)) == 0;
  // (a warp that has elements stays whole: it shares a block's scales)
  int e = threadIdx.x * 8;
  const int warp_left = t.left + (threadIdx.x & 31) * 8;
  if (e >= warp_left) return;
  // (a fetch at the loop's head instead of its end costs the 8-bit kernel a quarter: the
  // compiler then orders the loads behind the spilled registers)
  In<G, State, Value> x;
  x.fetch(t, e);
#pragma unroll 1
  for (;;) {
    step8(t, e, x, h, now);
    e += kUnit;
    if (e >= warp_left) break;
    x.fetch(t, e);
  }
}

// Thread blocks per SM: with 8-bit states the arithmetic (53 to 73 instructions an element,
// by the types) fills 60 to 70% of the issue slots, and what hides the loads and the two reductions is other
// warps: 494 M elements take 994 us with six blocks (some registers spilled), 1,155 with
// five, 1,263 with four (with masters five and six are within 2%).  Loads ahead of their use cost
// more than they hide: before the root took any v', 1,084 us with four blocks that fetch a unit
// ahead and 1,245 with a ring of asynchronous copies, where six blocks took 1,035.  With 32-bit
// states four blocks keep HBM busy.
template <int CAP, bool kEight>
__global__ void __launch_bounds__(kThreads, kEight ? 6 : 4) adamw_kernel(const __grid_constant__ Table<CAP> t,
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
  const int64_t e0 = (chunk - t.first[k]) * t.units * kUnit, n = t.numel[k];
  const int dt = t.dt[k] | (t.master[k] != nullptr ? 4 : 0);
  using B = uint16_t;
#define STEP(W, G, MASTER)                                                                 \
  chunk_step<W, G, MASTER, kEight>(static_cast<W*>(t.param[k]), t.master[k],               \
                                   static_cast<const G*>(t.grad[k]), t.avg[k], t.sq[k],    \
                                   t.scales[k], n, e0, t.units, h, now)
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

int64_t chunks_of(const AdamwTensor& t, int units) {
  const int64_t size = (int64_t)units * kUnit;
  return (t.numel + size - 1) / size;
}

template <int CAP>
cudaError_t launch_group(const AdamwTensor* g, int count, int units, bool eight, const Hyper& h,
                         cudaStream_t st) {
  Table<CAP> t;
  t.count = count;
  t.units = units;
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
    at += chunks_of(g[k], units);
  }
  t.first[count] = at;
  const dim3 grid((unsigned)at), block(kThreads);
  return eight ? launch_pdl(adamw_kernel<CAP, true>, grid, block, 0, st, 1, t, h)
               : launch_pdl(adamw_kernel<CAP, false>, grid, block, 0, st, 1, t, h);
}

}  // namespace

cudaError_t launch_adamw(const AdamwArgs& a, const DeviceInfo& d, cudaStream_t st) {
  Hyper h;
  h.lr = (float)a.lr;
  h.beta1 = (float)a.beta1;
  h.beta2 = (float)a.beta2;
  h.one_minus1 = (float)(1.0 - a.beta1);
  h.one_minus2 = (float)(1.0 - a.beta2);
  // (what is below float32's normal numbers would be 0 to the reciprocal, and 0 / 0 a NaN)
  h.eps = a.eps > 0.0 ? fmaxf((float)a.eps, 0x1p-126f) : 0.f;
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
  h.minus_zero = -0.f;
  // Chunks of two units, which find their tensor and their numbers once, where params and
  // gradients are of different types and no master is kept (8-bit states, 494 M elements:
  // float32 params 988 us, 1,008 with one unit; bfloat16 931 and 961), and one for the others
  // (float32 alone 1,127 us, 1,266 with two; bfloat16 alone 946 and 984; masters 1,262 and 1,432,
  // 1,175 and 1,329; 32-bit states 1,941 and 1,964).  Where that leaves fewer than 64 chunks per
  // SM, one: 11.6 M elements 29.0 us, 30.1 with two.
  int64_t all = 0;
  bool differ = true;
  for (int64_t k = 0; k < a.count; ++k) {
    const AdamwTensor& t = a.tensors[k];
    all += t.numel;
    differ = differ && t.master == nullptr && (t.dt == 1 || t.dt == 2);
  }
  const int units = a.eight && differ && all / (2 * kUnit) >= 64 * (int64_t)d.sms ? 2 : 1;
  // tensors in launches of at most kMaxTensors and 2^30 chunks
  int64_t k = 0;
  while (k < a.count) {
    int n = 0;
    int64_t chunks = 0;
    while (k + n < a.count && n < kMaxTensors &&
           (n == 0 || chunks + chunks_of(a.tensors[k + n], units) < (int64_t)1 << 30))
      chunks += chunks_of(a.tensors[k + n++], units);
    const AdamwTensor* g = a.tensors + k;
    const cudaError_t e = n <= 32    ? launch_group<32>(g, n, units, a.eight, h, st)
                          : n <= 128 ? launch_group<128>(g, n, units, a.eight, h, st)
                                     : launch_group<kMaxTensors>(g, n, units, a.eight, h, st);
    if (e != cudaSuccess) return e;
    k += n;
  }
  return cudaSuccess;
}

}  // namespace grpo
