// Verification of drafted tokens against the target's probabilities.
//
// Per sequence, with z_j the target's logits that follow j drafted tokens,
// p_j = softmax(z_j / T), q_j = softmax(y_j / T) the draft's distribution that
// token x_j was drawn from (all mass on x_j when there are no draft logits),
// u_j uniform and e_v exponential random numbers given by the caller:
//   x_j is accepted while u_j * q_j(x_j) < p_j(x_j);
//   at the first rejection a the emitted token is
//       argmax_v max(p_a(v) - q_a(v), 0) / e_v        (the residual's race),
//   and argmax_v p_a(v) / e_v on the row after the last drafted token;
//   with T = 0: x_j is accepted while it is argmax z_j, and argmax z_a emitted.
//
// One thread block cluster walks one sequence: every CTA streams its slice of
// a row and keeps a running (max, sum of exponentials), the cluster's CTAs
// exchange their partials through distributed shared memory, and all of them
// take the same decision from the same bits.  Rows after the first rejection
// are never read; the rejected row's second reading (for the race) comes out
// of L2.  One launch, no atomics between sequences.
//
// Whole-number outputs must not depend on float32 rounding where a decision
// is close, so the tests are made in float64 from float32 sums, and the race
// keeps in float32 only bounds: the candidates whose upper bound reaches the
// best lower bound (a handful of a row) are compared in float64.
#include <math.h>

#include <map>
#include <mutex>
#include <tuple>

#include "host_ctx.cuh"
#include "ops.cuh"

namespace grpo {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kCandidates = 1024;      // race candidates a CTA can hold
constexpr float kMinTemperature = 1e-6f;  // below it a temperature counts as 0
constexpr float kBig = 1e30f;          // maxima beyond it take the subtracting form below
constexpr double kLn2 = 0.69314718055994530942;
// relative error bound of the float32 probabilities in the race (about 2^-22
// from the exponent's rounding at 60 bits, ex2 and the products), with room
constexpr float kRaceMargin = 1e-5f;

// exp(x / T) = 2^(x c), c = log2(e) / T kept as c_hi + c_lo with c_lo > 0 (so
// that -inf stays -inf in both steps).
struct Temper {
  float hi, lo;
  double c;
};
__device__ __forceinline__ Temper temper(float T) {
  Temper t;
  t.c = 1.4426950408889634074 / (double)T;
  t.hi = __double2float_rd(t.c);
  t.lo = fmaxf((float)(t.c - (double)t.hi), 1e-37f);
  return t;
}

// Reference exponent of a row (or part of one) with maximum m: weights are
// 2^(x c - r).  With r the rounded product, x c - r is rounded once, at its
// own size: near the maximum, where the weights matter, it is exact to 2^-24.
// Where the product would leave float32's range, weights are 2^((x - m) c).
__device__ __forceinline__ float ref_of(float m, const Temper& t) { return m * t.hi; }
__device__ __forceinline__ bool is_big(float m) { return !(fabsf(m) < kBig); }
__device__ __forceinline__ float exponent(float x, float m, float r, bool big, const Temper& t) {
  if (big) {
    const float s = x - m;
    return fmaf(s, t.hi, s * t.lo);
  }
  return fmaf(x, t.lo, fmaf(x, t.hi, -r));
}
// 2^(reference m1 - reference m2): moves a sum from one reference to a larger one
__device__ __forceinline__ float rescale(float m1, float m2, const Temper& t) {
  if (m1 == m2) return 1.f;
  if (m1 == -INFINITY) return 0.f;
  if (is_big(m1) || is_big(m2)) return ex2((m1 - m2) * t.hi);
  return ex2(ref_of(m1, t) - ref_of(m2, t));
}
__device__ __forceinline__ void merge(float& m, float& s, float m2, float s2, const Temper& t) {
  const float M = fmaxf(m, m2);
  // a NaN sum stays; an empty part (max -inf) has sum 0 or NaN
  s = s * rescale(m, M, t) + s2 * rescale(m2, M, t);
  m = M;
}
// natural log of p(x) in float64
__device__ __forceinline__ double log_prob(float x, float m, double s, const Temper& t) {
  const double e = is_big(m) ? ((double)x - (double)m) * t.c
                             : (double)x * t.c - (double)ref_of(m, t);
  return e * kLn2 - log(s);
}

struct VerifyParams {
  int64_t N, K, V, tld, tls, dld, dls, nld;
  const int64_t* tokens;
  const int32_t* lens;
  const float* u;
  const float* noise;
  const float* temperature;
  int64_t* out_tokens;
  int32_t* n_accepted;
  float* logp;
  WsHeader* hdr;
  uint32_t* status;  // [N]
  int64_t chunk;     // elements of a row per CTA of the cluster
};

// What a CTA tells the others about its slice of a row (rank 0 adds what the
// decision needs, so that every CTA decides from the same bits).
struct Part {
  float mt, st, md, sd;      // target and draft: max, sum
  int64_t arg;               // lowest index of the target's maximum (T = 0)
  float u, temperature;
  float xt, xd;              // logits of the drafted token
  int64_t token;
  int32_t bonus, flags, pad[2];
};
static_assert(sizeof(Part) == 64, "four 16-byte stores");

struct Decision {
  int accept, emit;  // go on; or emit by race (1), argmax (2), nothing (3)
  float mt, md;
  double st, sd;
  int64_t arg, token;
  double lp;  // log-prob of the drafted token
  uint32_t flags;
};

struct RowStat {
  float m, s;
  int64_t arg;
};

// (max, sum) of one CTA's slice [v0, v1) of a row, per thread; with kArg also
// where the thread saw its maximum first.
template <typename T, bool kArg>
__device__ __forceinline__ RowStat row_stats(const T* row, int64_t v0, int64_t v1,
                                             const Temper& t) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec;
  constexpr int U = 4;
  const int tid = threadIdx.x;
  RowStat r;
  r.m = -INFINITY;
  r.s = 0.f;
  r.arg = INT64_MAX;
  if (v0 >= v1) return r;
  const uintptr_t addr = reinterpret_cast<uintptr_t>(row + v0);
  const int64_t a =
      min(v0 + (int64_t)(((16u - (unsigned)(addr & 15u)) & 15u) / sizeof(T)), v1);
  const int64_t nvec = (v1 - a) / EPV;
  const int64_t b = a + nvec * EPV;
  float m = -INFINITY, edge_s = 0.f;
  int64_t where = -1;  // first vector of the batch that holds the maximum
  uint64_t acc01 = f2_pack(0.f, 0.f), acc23 = f2_pack(0.f, 0.f);
  const uint64_t hi2 = f2_pack(t.hi, t.hi), lo2 = f2_pack(t.lo, t.lo);
  // the ragged head and tail, at most one element of each per thread
  int64_t he = -1, te = -1;
  if (tid < a - v0) he = v0 + tid;
  if (tid < v1 - b) te = b + tid;
  auto one = [&](int64_t e) {
    const float x = E::load1(row + e);
    if (x > m) {
      const float sc = rescale(m, x, t);
      const uint64_t sc2 = f2_pack(sc, sc);
      acc01 = f2_mul(acc01, sc2);
      acc23 = f2_mul(acc23, sc2);
      edge_s *= sc;
      m = x;
      if (kArg) r.arg = e;
      where = -1;
    }
    if (x != -INFINITY) edge_s += ex2(exponent(x, m, ref_of(m, t), is_big(m), t));
  };
  if (he >= 0) one(he);
  for (int64_t base = tid; base < nvec; base += kThreads * U) {
    uint4 d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = base + u * kThreads;
      d[u] = k < nvec ? ld_stream(row + a + k * EPV)
                      : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
    }
    const float bm = E::template batch_max<U>(d);
    if (bm > m) {
      const float sc = rescale(m, bm, t);
      const uint64_t sc2 = f2_pack(sc, sc);
      acc01 = f2_mul(acc01, sc2);
      acc23 = f2_mul(acc23, sc2);
      edge_s *= sc;
      m = bm;
      where = base;
    }
    float x[U * EPV];
#pragma unroll
    for (int u = 0; u < U; ++u) E::unpack(d[u], x + u * EPV);
    if (!is_big(m)) {
      const float nr = -ref_of(m, t);
      const uint64_t nr2 = f2_pack(nr, nr);
#pragma unroll
      for (int k = 0; k < U * EPV; k += 4) {
        const uint64_t x01 = f2_pack(x[k], x[k + 1]), x23 = f2_pack(x[k + 2], x[k + 3]);
        acc01 = f2_add(acc01, f2_ex2(f2_fma(x01, lo2, f2_fma(x01, hi2, nr2))));
        acc23 = f2_add(acc23, f2_ex2(f2_fma(x23, lo2, f2_fma(x23, hi2, nr2))));
      }
    } else if (m == -INFINITY) {  // nothing but -inf so far, or NaN
#pragma unroll
      for (int k = 0; k < U * EPV; ++k)
        if (x[k] != x[k]) edge_s = x[k];
    } else {
#pragma unroll
      for (int k = 0; k < U * EPV; ++k) edge_s += ex2(exponent(x[k], m, 0.f, true, t));
    }
  }
  if (te >= 0) one(te);
  if (kArg && where >= 0) {  // the batch's first element at the maximum
    r.arg = INT64_MAX;
    for (int u = U - 1; u >= 0; --u) {
      const int64_t k = where + u * kThreads;
      if (k < nvec)
        for (int e = EPV - 1; e >= 0; --e)
          if (E::load1(row + a + k * EPV + e) == m) r.arg = a + k * EPV + e;
    }
  }
  float a0, a1, a2, a3;
  f2_unpack(acc01, a0, a1);
  f2_unpack(acc23, a2, a3);
  r.m = m;
  r.s = edge_s + ((a0 + a1) + (a2 + a3));
  return r;
}

struct Shared {
  Part part[2][kMaxCluster];
  float4 red[kWarps];     // (mt, st, md, sd) per warp
  int64_t red_arg[kWarps];
  Decision dec;
  double win[2][kMaxCluster];
  int64_t win_at[2][kMaxCluster];
  double wred[kWarps];
  int64_t wred_at[kWarps];
  int best, count;
  int32_t cand[kCandidates];
  float cand_hi[kCandidates];
};

// The CTA's statistic of a row, left per warp in sh.red (x, y or z, w).
template <bool kArg>
__device__ __forceinline__ void warp_stats(RowStat r, const Temper& t, Shared& sh, bool draft) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, r.m, o);
    const float s2 = __shfl_xor_sync(0xffffffffu, r.s, o);
    if (kArg) {
      const int64_t a2 = __shfl_xor_sync(0xffffffffu, r.arg, o);
      r.arg = m2 > r.m ? a2 : (m2 == r.m ? min(r.arg, a2) : r.arg);
    }
    merge(r.m, r.s, m2, s2, t);
  }
  if (lane == 0) {
    if (draft) {
      sh.red[warp].z = r.m;
      sh.red[warp].w = r.s;
    } else {
      sh.red[warp].x = r.m;
      sh.red[warp].y = r.s;
      sh.red_arg[warp] = r.arg;
    }
  }
}

// The row's race in this CTA's slice: best score and its lowest index.
struct Racer {
  Temper t;
  float mt, rt, it, md, rd, id;  // max, reference exponent, 1 / sum
  double st, sd;
  bool bigt, bigd, has_draft;
  int64_t skip;  // token without mass in the residual (drafts without logits), or -1
};

template <typename T>
__device__ __forceinline__ double race_score64(const Racer& c, const T* tr, const T* dr,
                                               const float* nr, int64_t v) {
  if (v == c.skip) return 0.0;
  double p = exp(log_prob(Elt<T>::load1(tr + v), c.mt, c.st, c.t));
  if (c.has_draft) p -= exp(log_prob(Elt<T>::load1(dr + v), c.md, c.sd, c.t));
  return p > 0.0 ? p / (double)__ldg(nr + v) : 0.0;
}

__device__ __forceinline__ void better(double& s, int64_t& at, double s2, int64_t at2) {
  if (s2 > s || (s2 == s && at2 < at)) {
    s = s2;
    at = at2;
  }
}

// lower and upper bound of a score
__device__ __forceinline__ void race_bounds(const Racer& c, float x, float y, float e, float& lo,
                                            float& hi) {
  const float p = ex2(exponent(x, c.mt, c.rt, c.bigt, c.t)) * c.it;
  const float q = c.has_draft ? ex2(exponent(y, c.md, c.rd, c.bigd, c.t)) * c.id : 0.f;
  const float w = __fdividef(1.f, e), d = p - q, b = kRaceMargin * (p + q);
  lo = (d - b) * w;
  hi = (d + b) * w;
}

template <typename T>
__device__ void race(const Racer& c, const T* tr, const T* dr, const float* nr, int64_t v0,
                     int64_t v1, Shared& sh, double& score, int64_t& at) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    sh.best = 0;
    sh.count = 0;
  }
  __syncthreads();
  // one batch of a warp: raise the CTA's best lower bound, keep the elements
  // that may still beat it
  auto batch = [&](const float* lo, const float* hi, const int64_t* v, int n) {
    float top = 0.f;
    for (int k = 0; k < n; ++k) top = fmaxf(top, lo[k]);
    const unsigned wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    float bar = __int_as_float(*(volatile int*)&sh.best);
    if (__uint_as_float(wtop) > bar) {
      if (lane == 0) atomicMax(&sh.best, (int)wtop);
      bar = __uint_as_float(wtop);
    }
    for (int k = 0; k < n; ++k)
      if (hi[k] >= bar && hi[k] > 0.f && bar > 0.f) {
        const int s = atomicAdd(&sh.count, 1);
        if (s < kCandidates) {
          sh.cand[s] = (int32_t)v[k];
          sh.cand_hi[s] = hi[k];
        }
      }
  };
  const bool vec = reinterpret_cast<uintptr_t>(tr) % 16 == 0 && v0 % EPV == 0 &&
                   reinterpret_cast<uintptr_t>(nr) % 16 == 0 &&
                   (!c.has_draft || reinterpret_cast<uintptr_t>(dr) % 16 == 0);
  int64_t from = v0;
  if (vec) {
    const int64_t nvec = (v1 - v0) / EPV;
    for (int64_t base = 0; base < nvec; base += kThreads) {
      const int64_t k = base + tid;
      float lo[EPV], hi[EPV];
      int64_t v[EPV];
#pragma unroll
      for (int j = 0; j < EPV; ++j) {
        lo[j] = hi[j] = 0.f;
        v[j] = v0 + k * EPV + j;
      }
      if (k < nvec) {
        float x[EPV], y[EPV], e[EPV];
        E::unpack(ld_stream(tr + v0 + k * EPV), x);
        if (c.has_draft) E::unpack(ld_stream(dr + v0 + k * EPV), y);
#pragma unroll
        for (int j = 0; j < EPV; j += 4)
          Elt<float>::unpack(ld_stream(nr + v0 + k * EPV + j), e + j);
#pragma unroll
        for (int j = 0; j < EPV; ++j) {
          race_bounds(c, x[j], c.has_draft ? y[j] : 0.f, e[j], lo[j], hi[j]);
          if (v[j] == c.skip) lo[j] = hi[j] = 0.f;
        }
      }
      batch(lo, hi, v, EPV);
    }
    from = v0 + nvec * EPV;
  }
  for (int64_t base = from; base < v1; base += kThreads) {
    float lo = 0.f, hi = 0.f;
    const int64_t v = base + tid;
    if (v < v1 && v != c.skip)
      race_bounds(c, E::load1(tr + v), c.has_draft ? E::load1(dr + v) : 0.f, __ldg(nr + v), lo,
                  hi);
    batch(&lo, &hi, &v, 1);
  }
  __syncthreads();
  const float bar = __int_as_float(sh.best);
  const int count = sh.count;
  score = 0.0;
  at = INT64_MAX;
  if (bar > 0.f && count <= kCandidates) {
    for (int k = tid; k < count; k += kThreads)
      if (sh.cand_hi[k] >= bar)
        better(score, at, race_score64(c, tr, dr, nr, sh.cand[k]), sh.cand[k]);
  } else {
    // bounds that do not separate anything (residuals at the level of the
    // rounding): every element in float64
    for (int64_t v = v0 + tid; v < v1; v += kThreads)
      better(score, at, race_score64(c, tr, dr, nr, v), v);
  }
  for (int o = 16; o > 0; o >>= 1) {
    const double s2 = __shfl_xor_sync(0xffffffffu, score, o);
    const int64_t a2 = __shfl_xor_sync(0xffffffffu, at, o);
    better(score, at, s2, a2);
  }
  if (lane == 0) {
    sh.wred[warp] = score;
    sh.wred_at[warp] = at;
  }
  __syncthreads();
  score = sh.wred[0];
  at = sh.wred_at[0];
  for (int k = 1; k < kWarps; ++k) better(score, at, sh.wred[k], sh.wred_at[k]);
}

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_s64(uint32_t addr, int64_t v) {
  asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Thread 0 of each CTA: merge the ranks' parts in rank order and decide.
__device__ __forceinline__ void decide(const Part* part, int ranks, bool has_draft, Decision& d) {
  const Part& h = part[0];
  d.flags = (uint32_t)h.flags;
  d.token = h.token;
  d.accept = 0;
  d.lp = 0.0;
  const bool greedy = h.temperature < kMinTemperature;
  const Temper t = temper(greedy ? 1.f : h.temperature);
  float mt = h.mt, st = h.st, md = h.md, sd = h.sd;
  int64_t arg = h.arg;
  for (int k = 1; k < ranks; ++k) {
    const Part& o = part[k];
    arg = o.mt > mt ? o.arg : (o.mt == mt ? min(arg, o.arg) : arg);
    merge(mt, st, o.mt, o.st, t);
    if (has_draft) merge(md, sd, o.md, o.sd, t);
  }
  d.mt = mt;
  d.st = (double)st;
  d.md = md;
  d.sd = (double)sd;
  d.arg = arg;
  const bool use_draft = has_draft && !h.bonus && !greedy;
  bool defined = h.temperature >= 0.f && h.temperature <= 3.4e38f && mt > -INFINITY &&
                 mt < INFINITY && st > 0.f && st < INFINITY;
  if (use_draft) defined = defined && md > -INFINITY && md < INFINITY && sd > 0.f && sd < INFINITY;
  if (!defined) {
    d.emit = 3;
    d.flags |= kFlagValue;
    return;
  }
  d.emit = greedy ? 2 : 1;
  if (h.bonus || d.token < 0) return;  // (-1: a drafted token outside [0, V) is not accepted)
  d.lp = log_prob(h.xt, mt, d.st, t);
  if (greedy) {
    d.accept = d.token == arg;
  } else {
    const double lq = use_draft ? log_prob(h.xd, md, d.sd, t) : 0.0;
    d.accept = h.xt > -INFINITY && (double)h.u * exp(lq - d.lp) < 1.0;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) verify_kernel(const VerifyParams p,
                                                             const T* __restrict__ target,
                                                             const T* __restrict__ draft) {
  __shared__ __align__(16) Shared sh;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_ctarank(), ranks = cluster_size();
  const bool has_draft = draft != nullptr;
  pdl_wait();
  pdl_trigger();
  // every CTA of the cluster runs before the first distributed store
  if (ranks > 1) cluster_sync();
  if (blockIdx.x == 0 && tid == 0) {
    p.hdr->flags = kFlagIndirect;
    p.hdr->status_count = (uint32_t)p.N;
    p.hdr->status_check = ~(uint32_t)p.N;
  }
  const int64_t v0 = min(p.V, (int64_t)rank * p.chunk), v1 = min(p.V, v0 + p.chunk);
  int slot = 0, wslot = 0;
  for (int64_t i = cluster_id_x(); i < p.N; i += nclusters_x()) {
    int32_t len = p.lens != nullptr ? p.lens[i] : (int32_t)p.K;
    uint32_t flags = 0;
    if (len < 0 || len > p.K) {
      flags = kFlagLengthRange;
      len = len < 0 ? 0 : (int32_t)p.K;
    }
    const float Ti = p.temperature != nullptr ? p.temperature[i] : 1.f;
    const bool greedy = Ti < kMinTemperature;
    const Temper t = temper(greedy ? 1.f : Ti);
    int64_t j = 0;
    const T* trow = nullptr;
    const T* drow = nullptr;
    for (;; ++j) {
      const bool bonus = j >= len;
      trow = target + i * p.tls + j * p.tld;
      drow = has_draft && !bonus ? draft + i * p.dls + j * p.dld : nullptr;
      if (greedy)
        warp_stats<true>(row_stats<T, true>(trow, v0, v1, t), t, sh, false);
      else
        warp_stats<false>(row_stats<T, false>(trow, v0, v1, t), t, sh, false);
      const bool read_draft = drow != nullptr && !greedy;
      if (read_draft)
        warp_stats<false>(row_stats<T, false>(drow, v0, v1, t), t, sh, true);
      __syncthreads();
      if (tid < (int)ranks) {
        union {
          Part part;
          float4 f[4];
        } o;
        Part& a = o.part;
        a.mt = sh.red[0].x;
        a.st = sh.red[0].y;
        a.arg = sh.red_arg[0];
        a.md = read_draft ? sh.red[0].z : -INFINITY;
        a.sd = read_draft ? sh.red[0].w : 0.f;
        for (int k = 1; k < kWarps; ++k) {
          const float4 r = sh.red[k];
          a.arg = r.x > a.mt ? sh.red_arg[k] : (r.x == a.mt ? min(a.arg, sh.red_arg[k]) : a.arg);
          merge(a.mt, a.st, r.x, r.y, t);
          if (read_draft) merge(a.md, a.sd, r.z, r.w, t);
        }
        a.u = 0.f;
        a.temperature = Ti;
        a.xt = a.xd = 0.f;
        a.token = -1;
        a.bonus = bonus;
        a.flags = 0;
        a.pad[0] = a.pad[1] = 0;
        if (rank == 0) {
          a.flags = (int32_t)flags;
          if (!bonus) {
            const int64_t x = p.tokens[i * p.K + j];
            a.u = p.u[i * p.K + j];
            if (x >= 0 && x < p.V) {
              a.token = x;
              a.xt = Elt<T>::load1(trow + x);
              if (read_draft) a.xd = Elt<T>::load1(drow + x);
            } else {
              a.flags |= (int32_t)kFlagTokenRange;
            }
          }
        }
        const uint32_t dst = map_to_rank(smem_u32(&sh.part[slot][rank]), (uint32_t)tid);
#pragma unroll
        for (int k = 0; k < 4; ++k) st_cluster_f32x4(dst + 16 * k, o.f[k]);
      }
      __syncwarp();  // the cluster barrier instructions are warp-aligned
      if (ranks > 1)
        cluster_sync();
      else
        __syncthreads();
      if (tid == 0) decide(sh.part[slot], (int)ranks, has_draft, sh.dec);
      __syncthreads();
      // (the part slots alternate: this one is rewritten two rows on, after a
      // barrier that every CTA reaches only when it has decided here)
      slot ^= 1;
      flags |= sh.dec.flags;
      // (a row after the last drafted token is never accepted: rank 0 says so)
      if (!sh.dec.accept || j >= p.K) break;
      if (rank == 0 && tid == 0) {
        p.out_tokens[i * (p.K + 1) + j] = sh.dec.token;
        p.logp[i * (p.K + 1) + j] = (float)sh.dec.lp;
      }
    }
    // the emitted token
    const Decision d = sh.dec;
    int64_t token = -1;
    if (d.emit == 2) {
      token = d.arg;
    } else if (d.emit == 1) {
      Racer c;
      c.t = t;
      c.mt = d.mt;
      c.rt = ref_of(d.mt, t);
      c.bigt = is_big(d.mt);
      c.it = (float)(1.0 / d.st);
      c.st = d.st;
      c.md = d.md;
      c.rd = ref_of(d.md, t);
      c.bigd = is_big(d.md);
      c.sd = d.sd;
      c.id = d.sd > 0.0 ? (float)(1.0 / d.sd) : 0.f;
      const bool bonus = sh.part[slot ^ 1][0].bonus != 0;
      c.has_draft = has_draft && !bonus;
      c.skip = !has_draft && !bonus ? d.token : -1;
      for (int mode = 0; mode < 2; ++mode) {
        double s;
        int64_t at;
        race(c, trow, drow, p.noise + i * p.nld, v0, v1, sh, s, at);
        if (tid < (int)ranks) {
          st_cluster_f64(map_to_rank(smem_u32(&sh.win[wslot][rank]), (uint32_t)tid), s);
          st_cluster_s64(map_to_rank(smem_u32(&sh.win_at[wslot][rank]), (uint32_t)tid), at);
        }
        __syncwarp();
        if (ranks > 1)
          cluster_sync();
        else
          __syncthreads();
        s = sh.win[wslot][0];
        at = sh.win_at[wslot][0];
        for (uint32_t k = 1; k < ranks; ++k) better(s, at, sh.win[wslot][k], sh.win_at[wslot][k]);
        wslot ^= 1;
        token = s > 0.0 ? at : -1;
        // nothing left in the residual (p = q up to rounding): the target's own race
        if (s > 0.0 || (!c.has_draft && c.skip < 0)) break;
        c.has_draft = false;
        c.skip = -1;
      }
      if (token < 0) flags |= kFlagValue;  // no positive finite score
    }
    if (rank == 0) {
      const int64_t o = i * (p.K + 1);
      if (tid == 0) {
        p.out_tokens[o + j] = token;
        p.logp[o + j] = token >= 0 ? (float)log_prob(Elt<T>::load1(trow + token), d.mt, d.st, t)
                                   : __int_as_float(0x7fc00000);
        p.n_accepted[i] = (int32_t)j;
        p.status[i] = flags & ~kFlagIndirect;
      }
      for (int64_t k = j + 1 + tid; k <= p.K; k += kThreads) {
        p.out_tokens[o + k] = -1;
        p.logp[o + k] = 0.f;
      }
    }
    __syncthreads();  // sh.dec and the race's arrays are free
  }
  // no CTA leaves while another may still store into it
  if (ranks > 1) cluster_sync();
}

std::mutex g_occ_mutex;
std::map<std::tuple<int, int, int>, int> g_occ;  // (device, dtype, cluster) -> clusters at once

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, const DeviceInfo& d, cudaStream_t st) {
  constexpr int EPV = Elt<T>::kPerVec;
  const int K = lse_split(a.V * (int64_t)sizeof(T), a.N, d.sms, "GRPO_VERIFY_CLUSTER");
  VerifyParams p;
  p.N = a.N;
  p.K = a.K;
  p.V = a.V;
  p.tld = a.tld;
  p.tls = a.tls;
  p.dld = a.dld;
  p.dls = a.dls;
  p.nld = a.nld;
  p.tokens = a.tokens;
  p.lens = a.lens;
  p.u = a.u;
  p.noise = a.noise;
  p.temperature = a.temperature;
  p.out_tokens = a.out_tokens;
  p.n_accepted = a.n_accepted;
  p.logp = a.logp;
  p.hdr = static_cast<WsHeader*>(a.ws);
  p.status = reinterpret_cast<uint32_t*>(static_cast<char*>(a.ws) + 256);
  p.chunk = ((a.V + K - 1) / K + EPV - 1) / EPV * EPV;
  auto kern = verify_kernel<T>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = K;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(K);
  int clusters = 0;
  const auto key = std::make_tuple(d.device, (int)sizeof(T), K);
  {
    std::lock_guard<std::mutex> g(g_occ_mutex);
    const auto it = g_occ.find(key);
    if (it != g_occ.end()) clusters = it->second;
  }
  if (clusters == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) clusters = 1;
    std::lock_guard<std::mutex> g(g_occ_mutex);
    g_occ[key] = clusters;
  }
  const int64_t nq = clusters < a.N ? clusters : a.N;
  cfg.gridDim = dim3((unsigned)(nq * K));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p, static_cast<const T*>(a.target),
                            static_cast<const T*>(a.draft));
}

}  // namespace

size_t verify_workspace_bytes(int64_t N) {
  return 256 + align_up(sizeof(uint32_t) * (size_t)(N < 1 ? 1 : N), 256);
}

cudaError_t launch_verify(const VerifyArgs& a, const DeviceInfo& d, cudaStream_t st) {
  if (a.N == 0) return cudaMemsetAsync(a.ws, 0, sizeof(WsHeader), st);
  return a.dtype == 0 ? launch_t<float>(a, d, st) : launch_t<uint16_t>(a, d, st);
}

}  // namespace grpo
