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
// Two kernels.  verify_rows_kernel computes (max, sum of exponentials) of every
// target and draft row, each row split over CTAs that work on their own; where
// the rows are many bytes it runs position by position and leaves out rows
// behind a rejection that is already known (the last CTA of a
// position's rows decides it and publishes it; nothing waits for anything, and
// a row that was read in vain changes no result).  verify_emit_kernel, one
// thread block cluster per sequence, takes every position's decision at once,
// one position per warp, and runs the race over the row that the sequence
// stops at.
//
// Whole-number outputs must not depend on float32 rounding where a decision
// is close, so the tests are made in float64 from float32 sums, and the race
// keeps in float32 only bounds: the candidates whose upper bound reaches the
// best lower bound (a handful of a row) are compared in float64.
#include <math.h>
#include <stddef.h>

#include <atomic>

#include "host_ctx.cuh"
#include "ops.cuh"

namespace grpo {
namespace {

constexpr int kRaceThreads = 512;
constexpr int kRaceWarps = kRaceThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSplit = 32;          // CTAs per row of the rows kernel (one lane each when merged)
constexpr int64_t kMinPartBytes = 8192;  // of a row, when it is split
constexpr int kCandidates = 1024;      // race candidates a CTA can hold
constexpr float kMinTemperature = 1e-6f;  // below it a temperature counts as 0
constexpr float kFar = 0x1p24f;        // |exponents| from it on take the subtracting form below
constexpr double kLn2 = 0.69314718055994530942;
// Relative error bound of the float32 probabilities in the race.  An exponent
// between 0 and -126 (ex2 gives 0 beyond) is rounded once, by 2^-18 at most: 2.6e-6
// of the weight.  ex2 adds 2^-22 of its own, the quotients, the products and
// the noise's reciprocal (2^-23) less than 6e-7 together: 3.5e-6 of 1e-5.
constexpr float kRaceMargin = 1e-5f;

// 1 / x on the special-function unit (2^-23; infinite for 0).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(x / T) = 2^(x c) with c = log2(e) / T rounded to float32 once, for the
// target and the draft alike and in every step: the distributions are those of
// a temperature that differs from T by at most 2^-23 of itself, which moves a
// ratio p / q by 2^-23 of its own logarithm.
struct Temper {
  float c;
};
__device__ __forceinline__ Temper temper(float T) { return {__fdiv_rn(1.44269504f, T)}; }

// Weights of a row (or part of one) with maximum m.  Near rows: 2^(x c - r) with
// r the product m c rounded.  x c - r is rounded once, at its own size: near the
// maximum, where the weights matter, it is exact to 2^-24 but for the rounding of
// r, which all the weights and the sum share.  That is half a step of r: 1/2 below
// 2^24, but beyond 2^31 more than ex2's range, and the weight of the maximum
// itself would be infinite or 0.  So rows whose |m c| reaches 2^24 are far:
// 2^((x - m) c), where x - m is exact for every x that has a weight.
__device__ __forceinline__ float ref_of(float m, const Temper& t) { return m * t.c; }
__device__ __forceinline__ bool is_far(float m, const Temper& t) {
  return !(fabsf(ref_of(m, t)) < kFar);  // (also m = +-inf)
}
__device__ __forceinline__ float exponent(float x, float m, float r, bool far, const Temper& t) {
  if (far) {
    return (x - m) * t.c;
  }
  return fmaf(x, t.c, -r);
}
// 2^(reference of m1 - reference of m2), m1 <= m2: moves a sum from one reference
// to a larger one.  A far row's reference is m c itself, a near one's the rounded
// product: between the two the product is taken exactly.
__device__ __forceinline__ float rescale(float m1, float m2, const Temper& t) {
  if (m1 == m2) return 1.f;
  if (m1 == -INFINITY) return 0.f;
  const bool f1 = is_far(m1, t), f2 = is_far(m2, t);
  if (f1 && f2) return ex2((m1 - m2) * t.c);
  if (f1) return ex2(fmaf(m1, t.c, -ref_of(m2, t)));
  if (f2) return ex2(fmaf(-m2, t.c, ref_of(m1, t)));
  return ex2(ref_of(m1, t) - ref_of(m2, t));
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ int64_t warp_min(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = min(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
// The lanes' parts (m, s) of a row as one, in every lane.  A NaN sum stays; an
// empty part has m = -inf and s = 0.
__device__ __forceinline__ void warp_merge(float& m, float& s, const Temper& t) {
  const float M = warp_max(m);
  s = warp_sum(s * rescale(m, M, t));
  m = M;
}
// natural log of a weight in float64 (p is weight / sum)
__device__ __forceinline__ double log_weight(float x, float m, const Temper& t) {
  const double c = (double)t.c;
  const double e =
      is_far(m, t) ? ((double)x - (double)m) * c : (double)x * c - (double)ref_of(m, t);
  return e * kLn2;
}
// Acceptance and log-probs within this of a border are looked at in float64
// (logf and the differences of float32 logs are good to about 2e-6 here).
constexpr float kClose = 1e-4f;

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
  uint32_t* status;   // [N]
  // (reference, sum) of part s of target row (j, i) at [(j * N + i) * split + s];
  // the draft rows' after all of those.  top, arg: a greedy target row's
  // maximum and where it is first.
  float2* part;
  float* top;
  int64_t* arg;
  float* picked;      // the drafted tokens' logits, in the order of the rows
  int32_t* rejected;  // [N]: a position at which the sequence is known to stop
  uint32_t* ticket;   // [K * N]: CTAs done with a position's rows
  int split, split_log2;  // CTAs per row, a power of two
  int64_t part_elems; // elements of a row per CTA
  int lazy;           // rows behind a known rejection are left out
  int64_t chunk;      // elements of a row per CTA of the emitting cluster
};

__device__ __forceinline__ int32_t clamped_len(const VerifyParams& p, int64_t i, uint32_t* flags) {
  const int32_t len = p.lens != nullptr ? p.lens[i] : (int32_t)p.K;
  if (len >= 0 && len <= p.K) return len;
  *flags |= kFlagLengthRange;
  return len < 0 ? 0 : (int32_t)p.K;
}
__device__ __forceinline__ float temperature_of(const VerifyParams& p, int64_t i) {
  return p.temperature != nullptr ? p.temperature[i] : 1.f;
}

struct Decision {
  int accept, emit;  // go on; or emit by race (1), argmax (2), nothing (3)
  float mt, md, st, sd;  // maxima and sums of the rows
  int64_t arg, token;
  float lp;  // log-prob of the drafted token
  uint32_t flags;
};

// The rows kernel streams a row through shared memory: every thread copies its
// own 16-byte vectors kRowStages batches ahead (asynchronous copies, read back
// by the thread that issued them: no barrier, no registers).  The ring alone
// reads 6.2 TB/s; with the exponentials 4.8 TB/s (247 MB in 51 us at 128
// sequences of 5 rows of 151,936 bfloat16 and their drafts), bound by issue
// slots: one unpack, half a packed FMA and one ex2 per element, and some 600
// instructions per warp and part around them.
constexpr int kRowVecs = 4;  // vectors of a batch, per thread
constexpr int kRowStages = 3;
constexpr size_t kRowRing = (size_t)kRowStages * kRowVecs * kThreads * 16;
// A warp's reference follows its maximum only when a value is this much above
// it (as an exponent of 2: weights up to 16, no loss): nearly never after the
// first batch.
constexpr float kRefSlack = 4.f;

// One warp's share of a row: reference m and sum, in every lane; with kArg
// also the exact maximum and its lowest index.
struct RowStat {
  float m, s, top;
  int64_t arg;
};

// Over the slice [v0, v1) of a row, by all warps of the CTA; also the logit x,
// where the slice holds it.
template <typename T, bool kArg>
__device__ __forceinline__ RowStat row_stats(const T* row, int64_t v0, int64_t v1,
                                             const Temper& t, uint32_t ring, bool holds,
                                             int64_t x, float& picked) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec;
  constexpr int U = kRowVecs;
  constexpr uint32_t kAll = 0xffffffffu;
  const int tid = threadIdx.x;
  const uintptr_t addr = reinterpret_cast<uintptr_t>(row + v0);
  const int64_t a =
      min(v0 + (int64_t)(((16u - (unsigned)(addr & 15u)) & 15u) / sizeof(T)), max(v0, v1));
  const int nvec = (int)((max(a, v1) - a) / EPV);
  const int64_t b = a + (int64_t)nvec * EPV;
  const int batches = (nvec + kThreads * U - 1) / (kThreads * U);

  float m = -INFINITY, above = -INFINITY;  // the warp's reference; what moves it
  float edge_s = 0.f, top = -INFINITY;
  int where = -1;  // first vector of the batch that holds the thread's maximum
  uint64_t acc01 = f2_pack(0.f, 0.f), acc23 = f2_pack(0.f, 0.f);
  const uint64_t c2 = f2_pack(t.c, t.c);
  auto adopt = [&](float x) {  // the whole warp
    const float M = warp_max(fmaxf(x, m));
    const float sc = rescale(m, M, t);
    acc01 = f2_mul(acc01, f2_pack(sc, sc));
    acc23 = f2_mul(acc23, f2_pack(sc, sc));
    edge_s *= sc;
    m = M;
    above = is_far(M, t) ? M : M + __fdividef(kRefSlack, t.c);
  };
  auto consume = [&](const uint4* d, int base) {
    const float bm = E::template batch_max<U>(d);
    if (__any_sync(kAll, bm > above)) adopt(bm);
    if (kArg && bm > top) {
      top = bm;
      where = base;
    }
    if (!is_far(m, t)) {
      const float nr = -ref_of(m, t);
      const uint64_t nr2 = f2_pack(nr, nr);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[EPV];
        E::unpack(d[u], x);
#pragma unroll
        for (int k = 0; k < EPV; k += 4) {
          const uint64_t x01 = f2_pack(x[k], x[k + 1]), x23 = f2_pack(x[k + 2], x[k + 3]);
          acc01 = f2_add(acc01, f2_ex2(f2_fma(x01, c2, nr2)));
          acc23 = f2_add(acc23, f2_ex2(f2_fma(x23, c2, nr2)));
        }
      }
    } else {  // (nothing but -inf and NaN so far: any reference gives 0 and NaN)
      const float nm = m == -INFINITY ? 0.f : -m;
      const uint64_t nm2 = f2_pack(nm, nm);
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        float x[EPV];
        E::unpack(u == 0 ? d[0] : u == 1 ? d[1] : u == 2 ? d[2] : d[3], x);
#pragma unroll
        for (int k = 0; k < EPV; k += 2)
          acc01 = f2_add(acc01, f2_ex2(f2_mul(f2_add(f2_pack(x[k], x[k + 1]), nm2), c2)));
      }
    }
  };
  static_assert(U == 4, "the far rows' path names the vectors");

  const uint32_t mine = ring + 16 * tid;  // vector u of stage s: + (s * U + u) * kThreads * 16
  const T* src = row + a + (int64_t)tid * EPV;
  int ahead = 0;  // batches issued
  auto issue = [&](int stage) {
    const int base = ahead * (kThreads * U) + tid;
    const T* q = src + (int64_t)ahead * (kThreads * U * EPV);
    const uint32_t to = mine + stage * (U * kThreads * 16);
    if (base - tid + kThreads * U <= nvec) {
#pragma unroll
      for (int u = 0; u < U; ++u) cp_async16(to + u * (kThreads * 16), q + u * (kThreads * EPV));
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (base + u * kThreads < nvec) cp_async16(to + u * (kThreads * 16), q + u * (kThreads * EPV));
    }
    cp_async_commit();
    ++ahead;
  };
#pragma unroll
  for (int k = 0; k < kRowStages; ++k) issue(k);
  if (holds) picked = E::load1(row + x);
  int stage = 0;
  for (int n = 0; n < batches; ++n) {
    cp_async_wait<kRowStages - 1>();
    const int base = n * (kThreads * U) + tid;
    const uint32_t at = mine + stage * (U * kThreads * 16);
    uint4 d[U];
    if (base - tid + kThreads * U <= nvec) {
#pragma unroll
      for (int u = 0; u < U; ++u) d[u] = ld_shared_v4(at + u * (kThreads * 16));
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        d[u] = base + u * kThreads < nvec
                   ? ld_shared_v4(at + u * (kThreads * 16))
                   : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
    }
    consume(d, base);
    issue(stage);  // (the batch was in registers)
    stage = stage + 1 == kRowStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();

  // the ragged ends: the first warp, at most one element of each per lane
  float xh = -INFINITY, xt = -INFINITY;
  if (tid < 32) {
    if (v0 + tid < a) xh = E::load1(row + v0 + tid);
    if (b + tid < v1) xt = E::load1(row + b + tid);
    const float bm = fmaxf(xh, xt);
    if (__any_sync(kAll, bm > above)) adopt(bm);
    const float r = ref_of(m, t);
    const bool far = is_far(m, t);
    if (xh != -INFINITY) edge_s += ex2(exponent(xh, m, r, far, t));
    if (xt != -INFINITY) edge_s += ex2(exponent(xt, m, r, far, t));
  }
  RowStat out;
  out.arg = INT64_MAX;
  out.top = top;
  if (kArg) {
    out.top = warp_max(fmaxf(top, fmaxf(xh, xt)));
    if (out.top > -INFINITY) {  // the thread's first element at the maximum
      if (xt == out.top) out.arg = b + tid;
      if (where >= 0 && top == out.top)
        for (int u = U - 1; u >= 0; --u) {
          const int k = where + u * kThreads;
          if (k < nvec)
            for (int e = EPV - 1; e >= 0; --e)
              if (E::load1(row + a + (int64_t)k * EPV + e) == out.top)
                out.arg = a + (int64_t)k * EPV + e;
        }
      if (xh == out.top) out.arg = v0 + tid;
    }
    out.arg = warp_min(out.arg);
  }
  float a0, a1, a2, a3;
  f2_unpack(acc01, a0, a1);
  f2_unpack(acc23, a2, a3);
  out.m = m;
  out.s = warp_sum(edge_s + ((a0 + a1) + (a2 + a3)));
  return out;
}

// Position j of sequence i, by one warp: the lanes take the parts of the
// target's and the draft's row, a tree of shuffles merges them, and every lane
// decides.  The results are every lane's.
__device__ __forceinline__ void decide(const VerifyParams& p, bool has_draft, int64_t i, int64_t j,
                                       int32_t len, float Ti, Decision& d) {
  const int lane = threadIdx.x & 31;
  const bool greedy = Ti < kMinTemperature, bonus = j >= len;
  const bool use_draft = has_draft && !bonus && !greedy;
  const Temper t = temper(greedy ? 1.f : Ti);
  d.flags = 0;
  d.accept = 0;
  d.lp = 0.f;
  d.token = -1;
  const int64_t trow = j * p.N + i, drow = (p.K + 1 + j) * p.N + i;
  d.mt = d.md = -INFINITY;
  d.st = d.sd = 0.f;
  d.arg = INT64_MAX;
  float top = -INFINITY;
  if (lane < p.split) {
    const float2 v = __ldcg(p.part + trow * p.split + lane);
    d.mt = v.x;
    d.st = v.y;
    if (use_draft) {
      const float2 w = __ldcg(p.part + drow * p.split + lane);
      d.md = w.x;
      d.sd = w.y;
    }
    if (greedy) {
      top = __ldcg(p.top + trow * p.split + lane);
      d.arg = __ldcg(p.arg + trow * p.split + lane);
    }
  }
  float xt = 0.f, xd = 0.f, u = 0.f;
  if (!bonus) {
    const int64_t x = p.tokens[i * p.K + j];
    u = p.u[i * p.K + j];
    xt = __ldcg(p.picked + trow);
    if (use_draft) xd = __ldcg(p.picked + drow);
    if (x >= 0 && x < p.V)
      d.token = x;
    else
      d.flags |= kFlagTokenRange;
  }
  warp_merge(d.mt, d.st, t);
  if (use_draft) warp_merge(d.md, d.sd, t);
  if (greedy) d.arg = warp_min(top == warp_max(top) ? d.arg : INT64_MAX);
  bool defined = Ti >= 0.f && Ti <= 3.4e38f && d.mt > -INFINITY && d.mt < INFINITY &&
                 d.st > 0.f && d.st < INFINITY;
  if (use_draft)
    defined = defined && d.md > -INFINITY && d.md < INFINITY && d.sd > 0.f && d.sd < INFINITY;
  if (!defined) {
    d.emit = 3;
    d.flags |= kFlagValue;
    return;
  }
  d.emit = greedy ? 2 : 1;
  if (d.token < 0) return;  // after the last draft, or an id outside [0, V)
  // (differences of the exponents in float64, the sums' logs in float32)
  const double wt = log_weight(xt, d.mt, t);
  d.lp = (float)(wt - (double)logf(d.st));
  if (greedy) {
    d.accept = d.token == d.arg;
    return;
  }
  if (!(xt > -INFINITY)) return;
  const double wd = use_draft ? log_weight(xd, d.md, t) : 0.0;
  // log(q / p) and its border -log(u)
  const float ratio = (float)(wd - wt) + (logf(d.st) - (use_draft ? logf(d.sd) : 0.f));
  const float border = -logf(u);
  if (fabsf(ratio - border) > kClose * fmaxf(1.f, fabsf(border))) {
    d.accept = ratio < border;
  } else {  // also NaN, u = 0 against q = 0 and u < 0
    const double lq = use_draft ? wd - log((double)d.sd) : 0.0;
    d.accept = (double)u * exp(lq - (wt - log((double)d.st))) < 1.0;
  }
}

// One row part per CTA.  Grid order: positions, then sequences, then kinds
// (target, draft), then parts, so that a position's decision is known before
// most of the next position's CTAs begin: 247 of 350 MB are read at 128 x 4
// drafts of which 73% are accepted, where 207 MB are needed.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) verify_rows_kernel(const VerifyParams p,
                                                                  const T* __restrict__ target,
                                                                  const T* __restrict__ draft) {
  extern __shared__ __align__(16) unsigned char row_ring[];
  __shared__ float2 s_red[kWarps];
  __shared__ float s_top[kWarps];
  __shared__ int64_t s_arg[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  unsigned q = blockIdx.x;
  const int s = (int)(q & (unsigned)(p.split - 1));  // (a power of two)
  q >>= p.split_log2;
  bool is_draft = false;
  if (draft != nullptr) {
    // (the last position has no draft rows)
    const unsigned pairs = (unsigned)(2 * p.N * p.K);
    if (q < pairs) {
      is_draft = q & 1;
      q >>= 1;
    } else {
      q -= pairs / 2;
    }
  }
  const unsigned jq = q / (unsigned)p.N;
  const int64_t j = jq, i = q - jq * (unsigned)p.N;
  // (loads that are in flight together: each costs a CTA's start its latency)
  uint32_t flags = 0;
  // (one thread reads it for all: other CTAs lower it meanwhile)
  int32_t stop = INT32_MAX;
  if (p.lazy && tid == 0) stop = *(volatile int32_t*)(p.rejected + i);
  int64_t x = -1;  // the drafted token
  if (tid == 0 && j < p.K) x = p.tokens[i * p.K + j];
  const float Ti = temperature_of(p, i);
  const int32_t len = clamped_len(p, i, &flags);
  const bool greedy = Ti < kMinTemperature;
  if (j > len || (is_draft && (j == len || greedy))) return;
  if (p.lazy && __syncthreads_or(stop < j)) return;
  const Temper t = temper(greedy ? 1.f : Ti);
  const int64_t v0 = min(p.V, s * p.part_elems), v1 = min(p.V, v0 + p.part_elems);
  const T* row = is_draft ? draft + i * p.dls + j * p.dld : target + i * p.tls + j * p.tld;
  const bool holds = j < len && x >= v0 && x < v1;  // its logit (thread 0)
  const uint32_t ring = smem_u32(row_ring);
  float picked = 0.f;
  const RowStat r = greedy ? row_stats<T, true>(row, v0, v1, t, ring, holds, x, picked)
                           : row_stats<T, false>(row, v0, v1, t, ring, holds, x, picked);
  if (lane == 0) {
    s_red[warp] = make_float2(r.m, r.s);
    s_top[warp] = r.top;
    s_arg[warp] = r.arg;
  }
  __syncthreads();
  if (warp != 0) return;
  float m = lane < kWarps ? s_red[lane].x : -INFINITY;
  float sum = lane < kWarps ? s_red[lane].y : 0.f;
  warp_merge(m, sum, t);
  const int64_t row_at = ((is_draft ? p.K + 1 : 0) + j) * p.N + i;
  const int64_t at = (row_at << p.split_log2) + s;
  if (greedy) {
    const float top = lane < kWarps ? s_top[lane] : -INFINITY, M = warp_max(top);
    const int64_t arg = warp_min(lane < kWarps && top == M ? s_arg[lane] : INT64_MAX);
    if (lane == 0) {
      p.top[at] = M;
      p.arg[at] = arg;
    }
  }
  uint32_t last = 0;
  if (lane == 0) {
    p.part[at] = make_float2(m, sum);
    if (holds) p.picked[row_at] = picked;
    if (p.lazy && j < len) {
      const uint32_t expect = (uint32_t)(p.split * (draft != nullptr && !greedy ? 2 : 1));
      __threadfence();
      last = atomicAdd(p.ticket + j * p.N + i, 1u) + 1u == expect;
      __threadfence();
    }
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  Decision d;
  decide(p, draft != nullptr, i, j, len, Ti, d);
  if (lane == 0 && !d.accept) atomicMin(p.rejected + i, (int32_t)j);
}

__global__ void __launch_bounds__(kThreads) verify_init_kernel(int32_t* rejected, int64_t n,
                                                               uint32_t* ticket, int64_t m) {
  pdl_wait();
  pdl_trigger();
  const int64_t all = (int64_t)gridDim.x * kThreads;
  for (int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x; k < n; k += all)
    rejected[k] = INT32_MAX;
  for (int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x; k < m; k += all) ticket[k] = 0;
}

// What the float32 bounds say about a slice: its best lower bound, and the
// largest upper bound and the token of the elements that reach it.
struct __align__(16) Bounds {  // (one 16-byte store into another CTA)
  float lo, hi;
  int32_t token, count;  // count: elements that reach the lower bound; -1: not separated
};

struct Shared {
  Decision dec;
  int stop;  // the position that the sequence stops at
  uint32_t flags;
  // what the CTAs of the cluster tell one another, per round
  Bounds bounds[2][kMaxCluster];
  double win[2][kMaxCluster];
  int64_t win_at[2][kMaxCluster];
  int again[2][kMaxCluster];  // rank 0's: 1 a race is run, 2 and a second one may follow; + 4: a wait gave up
  double wred[kRaceWarps];
  int64_t wred_at[kRaceWarps];
  int best, top, count;
  float off[2], low[2];  // of the race's rows: offsets, factors of the lower bounds
  int abort;        // a bounded wait gave up
  uint32_t issued;  // steps of the ring that were copied
  uint64_t full[3], empty[3];
  int32_t cand[kCandidates];
  float cand_hi[kCandidates];
};

// The rows of a race: their maxima and sums.
struct Racer {
  Temper t;
  float mt, md, st, sd;
  bool has_draft;
  int64_t skip;  // token without mass in the residual (drafts without logits), or -1
};

template <typename T>
__device__ __forceinline__ double race_score64(const Racer& c, const T* tr, const T* dr,
                                               const float* nr, int64_t v) {
  if (v == c.skip) return 0.0;
  double p = exp(log_weight(Elt<T>::load1(tr + v), c.mt, c.t)) / (double)c.st;
  if (c.has_draft) p -= exp(log_weight(Elt<T>::load1(dr + v), c.md, c.t)) / (double)c.sd;
  return p > 0.0 ? p / (double)__ldg(nr + v) : 0.0;
}

__device__ __forceinline__ void better(double& s, int64_t& at, double s2, int64_t at2) {
  if (s2 > s || (s2 == s && at2 < at)) {
    s = s2;
    at = at2;
  }
}

// Lower and upper bounds of scores, from exponents (x - o) c - r: o = 0 and the
// rounded reference for a near row, the maximum and r = 0 for a far one.  The
// sums are divided out after the exponentials: taken into the exponents, their
// logarithms would be rounded at the size of the references, which may be
// thousands.  What is rarely asked for (the offsets of far rows, the lower bounds'
// factors) waits in shared memory: with an offset subtracted from every element
// 128 sequences of 9 rows took 7 us more, by its registers.
struct RaceBounds {
  float c, rt, rd;   // exponents: x c - r
  float t_up, d_up;  // (1 + margin) / the target's sum, (margin - 1) / the draft's
  bool far;          // one of the rows is
};
// By every thread, before a barrier: thread 0 leaves the shared part.
__device__ __forceinline__ RaceBounds race_bounds_for(const Racer& c, Shared& sh) {
  const float it = rcp(c.st), id = c.has_draft ? rcp(c.sd) : 0.f;
  const bool ft = is_far(c.mt, c.t), fd = c.has_draft && is_far(c.md, c.t);
  if (threadIdx.x == 0) {
    sh.off[0] = ft ? c.mt : 0.f;
    sh.off[1] = fd ? c.md : 0.f;
    sh.low[0] = (1.f - kRaceMargin) * it;
    sh.low[1] = (-kRaceMargin - 1.f) * id;
  }
  return {c.t.c,
          ft ? 0.f : ref_of(c.mt, c.t),
          c.has_draft && !fd ? ref_of(c.md, c.t) : 0.f,
          (1.f + kRaceMargin) * it,
          (kRaceMargin - 1.f) * id,
          ft || fd};
}
template <bool kDraft, int N>
__device__ __forceinline__ void race_offsets(const Shared& sh, float (&x)[N], float (&y)[N]) {
  const float ot = sh.off[0], od = sh.off[1];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    x[q] -= ot;
    if (kDraft) y[q] -= od;
  }
}
template <bool kDraft>
__device__ __forceinline__ void race_bounds(const RaceBounds& c, float t_lo, float d_lo, float x,
                                            float y, float e, float& lo, float& hi) {
  const float p = ex2(fmaf(x, c.c, -c.rt)), q = kDraft ? ex2(fmaf(y, c.c, -c.rd)) : 0.f;
  const float w = rcp(e);
  lo = fmaf(q, d_lo, p * t_lo) * w;
  hi = fmaf(q, c.d_up, p * c.t_up) * w;
}
// The upper bounds of a pair of elements.
template <bool kDraft>
__device__ __forceinline__ uint64_t race_upper2(const RaceBounds& c, float x0, float x1, float y0,
                                                float y1, float e0, float e1) {
  const uint64_t c2 = f2_pack(c.c, c.c);
  const uint64_t p = f2_ex2(f2_fma(f2_pack(x0, x1), c2, f2_pack(-c.rt, -c.rt)));
  const uint64_t w = f2_pack(rcp(e0), rcp(e1));
  uint64_t h = f2_mul(p, f2_pack(c.t_up, c.t_up));
  if (kDraft) {
    const uint64_t q = f2_ex2(f2_fma(f2_pack(y0, y1), c2, f2_pack(-c.rd, -c.rd)));
    h = f2_fma(q, f2_pack(c.d_up, c.d_up), h);
  }
  return f2_mul(h, w);
}

// The race streams its rows in steps of 8 elements per thread of target, draft
// and noise: bulk copies (TMA), race_stages() steps ahead, issued by thread 0
// when every warp has released the stage.  Copies begin at the 16-byte boundary
// at or before an array's first element.  156 MB in the emitting kernel's 41 us,
// decisions included (128 sequences); with per-thread copies the call took 5 us
// more.
constexpr int kRaceElems = 8 * kRaceThreads;
template <typename T>
__host__ __device__ constexpr int race_stages() {
  return sizeof(T) == 4 ? 2 : 3;
}
template <typename T>
__host__ __device__ constexpr uint32_t race_stage_bytes() {
  return (uint32_t)kRaceElems * (2 * (uint32_t)sizeof(T) + 4) + 3 * 16;
}
template <typename T>
__host__ __device__ constexpr size_t race_ring() {
  return (size_t)race_stages<T>() * race_stage_bytes<T>();
}

// The CTA's best lower bound, raised by this warp's.
__device__ __forceinline__ float race_raise(Shared& sh, float top) {
  const unsigned wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  const float bar = __int_as_float(*(volatile int*)&sh.best);
  if (__uint_as_float(wtop) <= bar) return bar;
  if ((threadIdx.x & 31) == 0) atomicMax(&sh.best, (int)wtop);
  return __uint_as_float(wtop);
}
__device__ __forceinline__ void race_keep(Shared& sh, float hi, float bar, int64_t v) {
  // (with no lower bound yet, everything that may have mass: its own lower
  // bound may be 0 where p and q are close, and its score still the largest)
  if (hi >= bar && hi > 0.f) {
    const int s = atomicAdd(&sh.count, 1);
    if (s < kCandidates) {
      sh.cand[s] = (int32_t)v;
      sh.cand_hi[s] = hi;
    }
  }
}

// n8 groups of 8 elements from v0 on, pairs of them through packed arithmetic.
// kAligned: all three arrays are 16-byte aligned at v0, and a thread takes 8
// neighbours as vectors; otherwise it takes elements kRaceThreads apart (and
// the row goes on for 8 elements either side, which the copies may read).  `used`
// counts the ring's steps over all calls (every thread the same).  Returns the
// largest upper bound.
template <typename T, bool kDraft, bool kAligned>
__device__ __forceinline__ float race_stream(const RaceBounds& rb, int64_t left_out, const T* tr,
                                             const T* dr, const float* nr, int64_t v0, int n8,
                                             Shared& sh, uint32_t ring, uint32_t& used) {
  using E = Elt<T>;
  constexpr int W = E::kPerVec == 8 ? 1 : 2;  // vectors of 8 logits
  constexpr uint32_t S = race_stages<T>(), kLogits = kRaceElems * sizeof(T) + 16;
  const int tid = threadIdx.x, lane = tid & 31;
  const int steps = (n8 + kRaceThreads - 1) / kRaceThreads;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (*(volatile int*)&sh.abort) return;
    if (!mbar_wait(smem_u32(bar), parity)) *(volatile int*)&sh.abort = 1;
  };
  auto past = [](const void* q) {  // bytes behind a 16-byte boundary
    return kAligned ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(q) & 15u);
  };
  const uint32_t ot = past(tr + v0), od = kDraft ? past(dr + v0) : 0u, on = past(nr + v0);
  auto issue = [&](int step) {  // thread 0
    const uint32_t n = used + (uint32_t)step, st = n % S;
    wait(&sh.empty[st], ((n / S) & 1u) ^ 1u);
    if (*(volatile int*)&sh.abort) return;
    const uint32_t to = ring + st * race_stage_bytes<T>(), full = smem_u32(&sh.full[st]);
    const uint32_t count = (uint32_t)min(kRaceElems, 8 * (n8 - step * kRaceThreads));
    const int64_t v = v0 + (int64_t)step * kRaceElems;
    auto bytes = [&](uint32_t off, uint32_t size) { return (off + count * size + 15u) & ~15u; };
    const uint32_t bt = bytes(ot, sizeof(T)), bd = kDraft ? bytes(od, sizeof(T)) : 0u,
                   bn = bytes(on, 4);
    mbar_arrive_expect_tx(full, bt + bd + bn);
    bulk_g2s(to, reinterpret_cast<const char*>(tr + v) - ot, bt, full);
    if (kDraft) bulk_g2s(to + kLogits, reinterpret_cast<const char*>(dr + v) - od, bd, full);
    bulk_g2s(to + 2 * kLogits, reinterpret_cast<const char*>(nr + v) - on, bn, full);
    sh.issued = n + 1;
  };
  if (tid == 0)
    for (int k = 0; k < (int)S && k < steps; ++k) issue(k);
  const int64_t in = left_out - v0;  // the token left out, if it is here
  const int skip = left_out >= 0 && in >= 0 && in < 8 * (int64_t)n8 ? (int)in : -1;
  float bar = 0.f, largest = 0.f;
#pragma unroll 1
  for (int step = 0, k = tid; step < steps; ++step, k += kRaceThreads) {
    const uint32_t n = used + (uint32_t)step, st = n % S;
    // the stage of the step before, once every warp has released it
    if (tid == 0 && step > 0 && step - 1 + (int)S < steps) issue(step - 1 + (int)S);
    __syncwarp();
    wait(&sh.full[st], (n / S) & 1u);
    float most = 0.f;
    float x[8], y[8], e[8];
    const uint32_t at = ring + st * race_stage_bytes<T>();
    // element q of the thread is number first + q * apart from v0 on
    const int first = kAligned ? 8 * k : step * kRaceElems + tid;
    constexpr int apart = kAligned ? 1 : kRaceThreads;
    if (!kAligned) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t o = (uint32_t)(tid + q * kRaceThreads);
        const bool in = first + q * apart < 8 * n8;
        x[q] = in ? lds_elt(at + ot + o * (uint32_t)sizeof(T), T()) : -INFINITY;
        y[q] = kDraft && in ? lds_elt(at + kLogits + od + o * (uint32_t)sizeof(T), T()) : -INFINITY;
        e[q] = in ? lds_elt(at + 2 * kLogits + on + o * 4, float()) : 1.f;
      }
    } else if (k < n8) {
      if (W == 1) {
        E::unpack(ld_shared_v4(at + 16 * tid), x);
        if (kDraft) E::unpack(ld_shared_v4(at + kLogits + 16 * tid), y);
      } else {
#pragma unroll
        for (int q = 0; q < W; ++q) {
          E::unpack(ld_shared_v4(at + 32 * tid + 16 * q), x + q * E::kPerVec);
          if (kDraft) E::unpack(ld_shared_v4(at + kLogits + 32 * tid + 16 * q), y + q * E::kPerVec);
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
        Elt<float>::unpack(ld_shared_v4(at + 2 * kLogits + 32 * tid + 16 * q), e + 4 * q);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.empty[st]));
    if (rb.far) race_offsets<kDraft>(sh, x, y);
    if (!kAligned || k < n8) {
#pragma unroll
      for (int q = 0; q < 8; q += 2) {
        const uint64_t h =
            kDraft ? race_upper2<true>(rb, x[q], x[q + 1], y[q], y[q + 1], e[q], e[q + 1])
                   : race_upper2<false>(rb, x[q], x[q + 1], 0.f, 0.f, e[q], e[q + 1]);
        float h0, h1;
        f2_unpack(h, h0, h1);
        most = fmaxf(most, fmaxf(h0, h1));
      }
      largest = fmaxf(largest, most);
    }
    // an upper bound above everything so far: both bounds, one by one
    bar = fmaxf(bar, __int_as_float(*(volatile int*)&sh.best));
    if (__any_sync(0xffffffffu, most > 0.f && most >= bar)) {
      float hi[8], top = 0.f;
      const float t_lo = sh.low[0], d_lo = sh.low[1];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        hi[q] = 0.f;
        if ((!kAligned || k < n8) && first + q * apart != skip) {
          float lo;
          race_bounds<kDraft>(rb, t_lo, d_lo, x[q], kDraft ? y[q] : 0.f, e[q], lo, hi[q]);
          top = fmaxf(top, lo);
        }
      }
      bar = race_raise(sh, top);
#pragma unroll
      for (int q = 0; q < 8; ++q) race_keep(sh, hi[q], bar, v0 + first + q * apart);
    }
  }
  used += (uint32_t)steps;
  return largest;
}

template <typename T, bool kAligned>
__device__ Bounds race_bounds_of(const Racer& c, const T* tr, const T* dr, const float* nr,
                                 int64_t v0, int64_t v1, Shared& sh, uint32_t ring,
                                 uint32_t& used) {
  using E = Elt<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RaceBounds rb = race_bounds_for(c, sh);
  if (tid == 0) {
    sh.best = 0;
    sh.top = 0;
    sh.count = 0;
  }
  __syncthreads();
  // upper bound (that of a skipped token too: it only asks for the exact race)
  float largest = 0.f;
  // [v0, head) and [tail, v1) are left to single loads
  int64_t head = v0, tail = v0;
  if constexpr (kAligned) {
    const int n8 = (int)((v1 - v0) / 8);
    largest = c.has_draft ? race_stream<T, true, true>(rb, c.skip, tr, dr, nr, v0, n8, sh, ring, used)
                          : race_stream<T, false, true>(rb, c.skip, tr, dr, nr, v0, n8, sh, ring, used);
    tail = v0 + (int64_t)n8 * 8;
  } else if (v1 - v0 >= 32) {
    head = v0 + 8;
    const int n8 = (int)((v1 - 8 - head) / 8);
    largest = c.has_draft ? race_stream<T, true, false>(rb, c.skip, tr, dr, nr, head, n8, sh, ring, used)
                          : race_stream<T, false, false>(rb, c.skip, tr, dr, nr, head, n8, sh, ring, used);
    tail = head + (int64_t)n8 * 8;
  }
  constexpr int M = 4;
  const float t_lo = sh.low[0], d_lo = sh.low[1];
  const int64_t singles = (head - v0) + (v1 - tail);
  auto single = [&](int64_t k) { return k < head - v0 ? v0 + k : tail + (k - (head - v0)); };
  for (int64_t base = 0; base < singles; base += kRaceThreads * M) {
    float hi[M], top = 0.f, x[M], y[M], e[M];
#pragma unroll
    for (int w = 0; w < M; ++w) {
      const int64_t k = base + w * kRaceThreads + tid, v = single(k);
      if (k < singles) {
        x[w] = E::load1(tr + v);
        y[w] = c.has_draft ? E::load1(dr + v) : 0.f;
        e[w] = __ldg(nr + v);
      }
    }
    if (rb.far) race_offsets<true>(sh, x, y);
#pragma unroll
    for (int w = 0; w < M; ++w) {
      const int64_t k = base + w * kRaceThreads + tid;
      hi[w] = 0.f;
      if (k < singles && single(k) != c.skip) {
        float lo;
        if (c.has_draft)
          race_bounds<true>(rb, t_lo, d_lo, x[w], y[w], e[w], lo, hi[w]);
        else
          race_bounds<false>(rb, t_lo, d_lo, x[w], 0.f, e[w], lo, hi[w]);
        top = fmaxf(top, lo);
      }
      largest = fmaxf(largest, hi[w]);
    }
    const float bar = race_raise(sh, top);
#pragma unroll
    for (int w = 0; w < M; ++w) race_keep(sh, hi[w], bar, single(base + w * kRaceThreads + tid));
  }
  const unsigned wlargest = __reduce_max_sync(0xffffffffu, __float_as_uint(largest));
  if (lane == 0) atomicMax(&sh.top, (int)wlargest);
  __syncthreads();
  Bounds r;
  r.lo = __int_as_float(sh.best);
  r.hi = __int_as_float(sh.top);
  r.token = -1;
  r.count = r.hi > 0.f ? -1 : 0;  // nothing with mass here, or nothing separated (yet)
  if (*(volatile int*)&sh.abort) {  // a wait gave up: the exact race, which needs no ring
    r.lo = 0.f;
    r.hi = INFINITY;
    r.count = -1;
    return r;
  }
  const int count = sh.count;
  if (warp == 0 && r.lo > 0.f && count <= kCandidates) {
    // the candidates that reach the final bound, to the front of the list
    int kept = 0;
    float hi = 0.f;
    for (int k0 = 0; k0 < count; k0 += 32) {
      const int k = k0 + lane;
      const float h = k < count ? sh.cand_hi[k] : 0.f;
      const int32_t v = k < count ? sh.cand[k] : 0;
      const uint32_t in = __ballot_sync(0xffffffffu, k < count && h >= r.lo);
      if (k < count && h >= r.lo) {
        sh.cand[kept + __popc(in & ((1u << lane) - 1u))] = v;
        hi = fmaxf(hi, h);
      }
      kept += __popc(in);
      __syncwarp();
    }
    r.hi = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(hi)));
    r.count = kept;
    r.token = sh.cand[0];
    if (lane == 0) sh.count = kept;
  }
  return r;  // warp 0's
}

// The slice's best score in float64 and its lowest index: of the candidates
// kept, or (bounds that do not separate anything, residuals at the level of
// the rounding) of every element.
template <typename T>
__device__ void race_exact(const Racer& c, const T* tr, const T* dr, const float* nr, int64_t v0,
                           int64_t v1, bool separated, Shared& sh, double& score, int64_t& at) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  score = 0.0;
  at = INT64_MAX;
  if (separated) {
    if (warp == 0)
      for (int k = lane; k < sh.count; k += 32)
        better(score, at, race_score64(c, tr, dr, nr, sh.cand[k]), sh.cand[k]);
  } else {
    for (int64_t v = v0 + tid; v < v1; v += kRaceThreads)
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
  for (int k = 1; k < kRaceWarps; ++k) better(score, at, sh.wred[k], sh.wred_at[k]);
}

// A line on its way into L2.
__device__ __forceinline__ void prefetch_l2(const void* q) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
}
__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_s64(uint32_t addr, int64_t v) {
  asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_s32(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

static_assert(sizeof(Bounds) == 16 && offsetof(Shared, bounds) % 16 == 0, "16-byte stores");
static_assert(offsetof(Shared, win) % 8 == 0 && offsetof(Shared, win_at) % 8 == 0 &&
                  offsetof(Shared, again) % 4 == 0,
              "stores into other CTAs");

__device__ __forceinline__ void cluster_or_cta_sync(uint32_t ranks) {
  __syncwarp();  // the cluster barrier instructions are warp-aligned
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
}

// kAligned: every row of the three arrays, and every slice of one, begins at a
// 16-byte boundary.  (Two kernels: with both loops in one 102 us instead of 90 at
// 128 sequences.  At two CTAs per SM there are 64 registers per thread; the
// aligned rows' kernel keeps 120 bytes on its stack, the other 8 to 16.)
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kRaceThreads, 2) verify_emit_kernel(
    const VerifyParams p, const T* __restrict__ target, const T* __restrict__ draft) {
  extern __shared__ __align__(16) unsigned char emit_ring[];
  __shared__ __align__(16) Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank(), ranks = cluster_size();
  const int64_t i = cluster_id_x();
  const int64_t v0 = min(p.V, (int64_t)rank * p.chunk), v1 = min(p.V, v0 + p.chunk);
  const float* noise = p.noise + i * p.nld;
  // The kernel before this one waited before it let this one start, so the
  // caller's inputs are complete: the lengths, temperatures and the noise (on
  // its way into L2) need no wait.
  uint32_t flags = 0;
  const int32_t len = clamped_len(p, i, &flags);
  const float Ti = temperature_of(p, i);
  const bool greedy = Ti < kMinTemperature;
  if (!greedy)
    for (int64_t v = v0 + 32 * (int64_t)tid; v < v1; v += 32 * kRaceThreads) prefetch_l2(noise + v);
  const Temper t = temper(greedy ? 1.f : Ti);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && tid == 0) {
    p.hdr->flags = kFlagIndirect;
    p.hdr->status_count = (uint32_t)p.N;
    p.hdr->status_check = ~(uint32_t)p.N;
  }
  // every position's decision, one per warp; the first that is not accepted
  // is where the sequence stops (a row that was left out lies behind it, and
  // a published rejection is taken over as it is)
  const int32_t known = p.lazy ? p.rejected[i] : INT32_MAX;
  if (tid == 0) {
    sh.stop = INT32_MAX;
    sh.flags = flags;
    sh.abort = 0;
    sh.issued = 0;
    for (int k = 0; k < 3; ++k) {
      mbar_init(smem_u32(&sh.full[k]), 1);
      mbar_init(smem_u32(&sh.empty[k]), kRaceWarps);
    }
    mbar_init_fence();
  }
  for (int64_t base = 0; base <= len; base += kRaceWarps) {
    __syncthreads();
    const int64_t j = base + warp;
    Decision d;
    d.accept = 0;
    if (j <= len && j <= known) {
      decide(p, draft != nullptr, i, j, len, Ti, d);
      if (j == known) d.accept = 0;
      if (lane == 0 && !d.accept) atomicMin(&sh.stop, (int)j);
    }
    __syncthreads();
    const int stop = sh.stop;
    if (lane == 0 && j <= stop && j <= len) {
      if (d.flags) atomicOr(&sh.flags, d.flags);
      if (j == stop) {
        sh.dec = d;
      } else if (rank == 0) {
        p.out_tokens[i * (p.K + 1) + j] = d.token;
        p.logp[i * (p.K + 1) + j] = d.lp;
      }
    }
    if (stop != INT32_MAX) break;
  }
  // (also: every CTA of the cluster runs before the first distributed store)
  cluster_or_cta_sync(ranks);
  const Decision d = sh.dec;
  const int64_t j = sh.stop;
  const bool bonus = j >= len;
  flags = sh.flags;
  const T* trow = target + i * p.tls + j * p.tld;
  const T* drow = draft != nullptr && !bonus ? draft + i * p.dls + j * p.dld : nullptr;
  Racer c;
  c.t = t;
  c.mt = d.mt;
  c.st = d.st;
  c.md = d.md;
  c.sd = d.sd;
  c.has_draft = drow != nullptr;
  c.skip = draft == nullptr && !bonus ? d.token : -1;
  int64_t token = d.emit == 2 ? d.arg : -1;
  uint32_t used = 0;
  // The CTAs of the cluster pass the same barriers: what a further step
  // depends on comes from what they sent one another.
  for (int round = 0; round < 2; ++round) {
    Bounds own = {0.f, 0.f, -1, 0};
    if (d.emit == 1)
      own = race_bounds_of<T, kAligned>(c, trow, drow, noise, v0, v1, sh, smem_u32(emit_ring), used);
    if (tid < (int)ranks) {
      const uint32_t to = (uint32_t)tid;
      const float4 f = make_float4(own.lo, own.hi, __int_as_float(own.token), __int_as_float(own.count));
      st_cluster_f32x4(map_to_rank(smem_u32(&sh.bounds[round][rank]), to), f);
      st_cluster_s32(map_to_rank(smem_u32(&sh.again[round][rank]), to),
                     (d.emit != 1 ? 0 : (c.has_draft || c.skip >= 0 ? 2 : 1)) +
                         (*(volatile int*)&sh.abort ? 4 : 0));
    }
    cluster_or_cta_sync(ranks);
    // (every warp the same: a lane looks at a CTA's part)
    const bool in = (uint32_t)lane < ranks;
    const int state = in ? sh.again[round][lane] : 0;
    const Bounds b = in ? sh.bounds[round][lane] : Bounds{0.f, 0.f, -1, 0};
    if (__any_sync(0xffffffffu, state & 4)) flags |= kFlagTimeout;
    const int again = __shfl_sync(0xffffffffu, state, 0) & 3;
    if (again == 0) break;
    // (the bounds are not negative: their bits are in order)
    const float bar = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(b.lo)));
    const bool rival = b.count != 0 && b.hi >= bar;
    const uint32_t who = __ballot_sync(0xffffffffu, rival);
    const uint32_t rivals = __reduce_add_sync(
        0xffffffffu, !rival ? 0u : b.count < 0 ? 2u : (uint32_t)b.count);
    if (rivals == 1 && bar > 0.f) {  // nothing else comes near
      token = __shfl_sync(0xffffffffu, b.token, __ffs(who) - 1);
      break;
    }
    const Bounds mine = sh.bounds[round][rank];
    double s;
    int64_t at;
    race_exact(c, trow, drow, noise, v0, v1, mine.count >= 0, sh, s, at);
    if (tid < (int)ranks) {
      const uint32_t to = (uint32_t)tid;
      st_cluster_f64(map_to_rank(smem_u32(&sh.win[round][rank]), to), s);
      st_cluster_s64(map_to_rank(smem_u32(&sh.win_at[round][rank]), to), at);
    }
    cluster_or_cta_sync(ranks);
    s = sh.win[round][0];
    at = sh.win_at[round][0];
    for (uint32_t k = 1; k < ranks; ++k) better(s, at, sh.win[round][k], sh.win_at[round][k]);
    token = s > 0.0 ? at : -1;
    // nothing left in the residual (p = q up to rounding): the target's own race
    if (s > 0.0 || again == 1) break;
    c.has_draft = false;
    c.skip = -1;
  }
  // After a wait that gave up: the copies on their way end first.
  if (tid == 0 && *(volatile int*)&sh.abort) {
    constexpr uint32_t S = race_stages<T>();
    for (uint32_t k = 0; k < S && k < sh.issued; ++k) {
      const uint32_t n = sh.issued - 1 - k;
      mbar_wait(smem_u32(&sh.full[n % S]), (n / S) & 1u);
    }
  }
  if (rank != 0) return;
  if (token < 0) flags |= kFlagValue;
  const int64_t o = i * (p.K + 1);
  if (tid == 0) {
    p.out_tokens[o + j] = token;
    p.logp[o + j] = token >= 0 ? (float)(log_weight(Elt<T>::load1(trow + token), d.mt, t) -
                                         (double)logf(d.st))
                               : __int_as_float(0x7fc00000);
    p.n_accepted[i] = (int32_t)j;
    p.status[i] = flags;
  }
  for (int64_t k = j + 1 + tid; k <= p.K; k += kRaceThreads) {
    p.out_tokens[o + k] = -1;
    p.logp[o + k] = 0.f;
  }
}

struct VerifyLayout {
  size_t status, part, top, arg, picked, rejected, ticket, total;
};
VerifyLayout verify_layout(int64_t N, int64_t K) {
  VerifyLayout l;
  const size_t n = (size_t)(N < 1 ? 1 : N), rows = n * (size_t)(K + 1);
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at = align_up(at + bytes, 256);
    return p;
  };
  l.status = take(4 * n);
  l.part = take(2 * rows * kMaxSplit * sizeof(float2));
  l.top = take(rows * kMaxSplit * sizeof(float));
  l.arg = take(rows * kMaxSplit * sizeof(int64_t));
  l.picked = take(2 * rows * sizeof(float));
  l.rejected = take(4 * n);
  l.ticket = take(4 * rows);
  l.total = at;
  return l;
}

// Clusters of C emitting CTAs that the device runs at once, asked for once.
template <typename T, bool kAligned>
cudaError_t clusters_at_once(int C, const DeviceInfo& d, int* n) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];
  const bool keep = d.device >= 0 && d.device < kDevices;
  // (the answer + 1; 0: not asked yet)
  const int had = keep ? known[d.device][C].load(std::memory_order_relaxed) : 0;
  if (had > 0) {
    *n = had - 1;
    return cudaSuccess;
  }
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)C;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C);
  cfg.blockDim = dim3(kRaceThreads);
  cfg.dynamicSmemBytes = race_ring<T>();
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(n, verify_emit_kernel<T, kAligned>, &cfg);
  if (e == cudaSuccess && keep) known[d.device][C].store(*n + 1, std::memory_order_relaxed);
  return e;
}

template <typename T, bool kAligned>
cudaError_t launch_emit(VerifyParams p, const VerifyArgs& a, const DeviceInfo& d, cudaStream_t st) {
  cudaError_t e = ensure_dynamic_smem((const void*)verify_emit_kernel<T, kAligned>, (int)race_ring<T>());
  if (e != cudaSuccess) return e;
  // the emitting clusters: as many CTAs each as lets all of them run at once, of
  // at least 8 KiB of logits each (74 clusters of 4 run at once, 36 of 8: 64
  // sequences with 2, 4, 8 CTAs take 70, 59, 69 us, 32 sequences 56, 45, 40)
  int C = 1;
  while (C < kMaxCluster && a.V * (int64_t)sizeof(T) / (2 * C) >= kMinPartBytes) {
    int fit = 0;
    e = clusters_at_once<T, kAligned>(2 * C, d, &fit);
    if (e != cudaSuccess) return e;
    if (a.N > fit) break;
    C *= 2;
  }
  constexpr int EPV = Elt<T>::kPerVec;
  p.chunk = ((a.V + C - 1) / C + EPV - 1) / EPV * EPV;
  return launch_pdl(verify_emit_kernel<T, kAligned>, dim3((unsigned)(a.N * C)), dim3(kRaceThreads),
                    race_ring<T>(), st, (unsigned)C, p,
                    static_cast<const T*>(a.target), static_cast<const T*>(a.draft));
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, const DeviceInfo& d, cudaStream_t st) {
  constexpr int EPV = Elt<T>::kPerVec;
  const VerifyLayout l = verify_layout(a.N, a.K);
  char* ws = static_cast<char*>(a.ws);
  const int64_t row_bytes = a.V * (int64_t)sizeof(T);
  const int kinds = a.draft != nullptr ? 2 : 1;
  // Parts of a row.  A part costs some 3 us of latencies whatever its size, so
  // rows are split in halves until two CTAs per SM are reached (8 KiB at least),
  // further down to 31 KiB until seven are, and down to 96 KiB in any case.  Calls
  // with 1, 2, 4, 8 parts a row: 144 rows of 304 KB 33.0, 28.3, 26.7, 28.3 us; 256
  // of 128 KB 20.5, 19.7, 16.3, 18.2; 1,152 of 64 KB 33.9, 35.3, 42.8, 62.7.
  const int64_t rows = a.N * (a.K + 1) + (kinds == 2 ? a.N * a.K : 0);
  int split = 1, split_log2 = 0;
  while (split < kMaxSplit) {
    const int64_t half = row_bytes / (2 * split), ctas = rows * 2 * split;
    if (!((half >= kMinPartBytes && ctas <= 2 * (int64_t)d.sms) ||
          (half >= 31 * 1024 && ctas <= 7 * (int64_t)d.sms) || half > 48 * 1024))
      break;
    split *= 2;
    ++split_log2;
  }
  if (rows > INT32_MAX / split) return cudaErrorInvalidValue;  // (refused by api.cu)
  VerifyParams p = {};
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
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.status = reinterpret_cast<uint32_t*>(ws + l.status);
  p.part = reinterpret_cast<float2*>(ws + l.part);
  p.top = reinterpret_cast<float*>(ws + l.top);
  p.arg = reinterpret_cast<int64_t*>(ws + l.arg);
  p.picked = reinterpret_cast<float*>(ws + l.picked);
  p.rejected = reinterpret_cast<int32_t*>(ws + l.rejected);
  p.ticket = reinterpret_cast<uint32_t*>(ws + l.ticket);
  p.split = split;
  p.split_log2 = split_log2;
  p.part_elems = ((a.V + split - 1) / split + EPV - 1) / EPV * EPV;
  // Leaving rows out costs a launch and a ticket per part: 279 MB 54-62 us against
  // 66 for all rows, 350 MB 89 against 96; but 74 MB 38 against 34, 175 MB the same.
  p.lazy = a.K > 0 && rows * row_bytes > ((int64_t)192 << 20);
  cudaError_t e;
  if (p.lazy) {
    const int64_t words = a.N * (a.K + 1);
    const int64_t grid = (words + kThreads - 1) / kThreads;
    e = launch_pdl(verify_init_kernel, dim3((unsigned)(grid < d.sms ? grid : d.sms)),
                   dim3(kThreads), 0, st, 1, p.rejected, a.N, p.ticket, a.N * a.K);
    if (e != cudaSuccess) return e;
  }
  const T* target = static_cast<const T*>(a.target);
  const T* draft = static_cast<const T*>(a.draft);
  e = ensure_dynamic_smem((const void*)verify_rows_kernel<T>, (int)kRowRing);
  if (e != cudaSuccess) return e;
  e = launch_pdl(verify_rows_kernel<T>, dim3((unsigned)(rows * split)), dim3(kThreads), kRowRing,
                 st, 1, p, target, draft);
  if (e != cudaSuccess) return e;
  // every row of the arrays that the race reads at a 16-byte boundary
  uintptr_t odd = reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.noise);
  if (a.N > 1) odd |= (uintptr_t)a.nld * 4 | (uintptr_t)a.tls * sizeof(T);
  if (a.K > 0) odd |= (uintptr_t)a.tld * sizeof(T);
  if (draft != nullptr) {
    odd |= reinterpret_cast<uintptr_t>(draft);
    if (a.N > 1) odd |= (uintptr_t)a.dls * sizeof(T);
    if (a.K > 1) odd |= (uintptr_t)a.dld * sizeof(T);
  }
  return odd % 16 == 0 ? launch_emit<T, true>(p, a, d, st) : launch_emit<T, false>(p, a, d, st);
}

}  // namespace

size_t verify_workspace_bytes(int64_t N, int64_t K) { return verify_layout(N, K).total; }

cudaError_t launch_verify(const VerifyArgs& a, const DeviceInfo& d, cudaStream_t st) {
  if (a.N == 0) return cudaMemsetAsync(a.ws, 0, sizeof(WsHeader), st);
  return a.dtype == 0 ? launch_t<float>(a, d, st) : launch_t<uint16_t>(a, d, st);
}

}  // namespace grpo
