// Log-probs of given tokens, entropy and likeliest alternatives of rows of
// logits, and the gradient of the first two.
//
// Forward, with c = log2(e) / T and every thread's running reference r (a maximum, moved
// when a value exceeds it by 8 / c):
//   t_v = (z_v - r) c,  w_v = 2^t_v,  S = sum w_v,  E = sum w_v t_v
// in one pass.  At the end everything is moved to the row's maximum m (S' = S
// 2^d, E' = 2^d (E + d S) with d = (r - m) c) and added in a fixed order:
//   L = ln S,  logp = (z_y - m) / T - L,  entropy = L - ln2 E / S.
// Differences are taken before they are scaled, so no rounding is of the size of
// the logits (rows of lowest values, temperatures near 0); t is held above
// -150, where w is 0, so that -inf adds 0 to E.
//
// Alternatives: each thread also keeps the maximum of every group of vectors it
// reads.  The top-th largest of the maxima of 64 sets of threads is a lower
// bound of the top-th largest logit, which about 1.1 (top 5) to 1.4 (top 32)
// times top logits reach in rows without an order: only the groups whose maximum
// reaches it are read again.
//
// Backward: dz_v = p_v (A + B lg p_v) (+ g / T at the token) with lg p = (z - m) c
// - L log2(e), A = -(g + h H) / T, B = -h ln2 / T.
#include <math.h>

#include "host_ctx.cuh"
#include "ops.cuh"

namespace grpo {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMinTemperature = 1e-6f;  // below it a temperature counts as 0: greedy
constexpr float kLowest = -150.f;         // 2^kLowest is 0 in ex2's range
constexpr float kSlack = 8.f;             // sums may grow to 2^8 of their reference

// Loads that are issued here (the compiler moves others down to where their value is
// wanted, which is at the end of a row's chain).
__device__ __forceinline__ int64_t load_now(const int64_t* p) {
  int64_t x;
  asm volatile("ld.global.nc.s64 %0, [%1];" : "=l"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ float load_now(const float* p) {
  float x;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ float load_now(const uint16_t* p) {
  uint16_t x;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(x) : "l"(p));
  return bf16_bits_to_float(x);
}

// The temperature of sequence i: 1 for greedy ones, NaN for one that is none.
__device__ __forceinline__ float warmth_of(const float* temperature, int64_t i) {
  const float T = temperature != nullptr ? __ldg(temperature + i) : 1.f;
  if (!(T >= 0.f) || isinf(T)) return NAN;
  return T < kMinTemperature ? 1.f : T;
}

// Values in the order of unsigned integers (-0 and +0 are one value), above the
// id's complement: larger keys come first among the alternatives.
__device__ __forceinline__ uint64_t key_of(float x, int64_t v) {
  const uint32_t u = __float_as_uint(x + 0.f);
  const uint32_t o = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return (uint64_t)o << 32 | (uint32_t)~(uint32_t)v;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int64_t key_id(uint64_t k) { return (int64_t)(uint32_t)~(uint32_t)k; }

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

template <typename T>
struct StatsParams {
  const T* logits;
  int64_t N, R, V, seq, row;
  const int64_t* tokens;
  int64_t token_seq, token_row;
  const int32_t* lens;
  const float* temperature;
  int top;
  float* logp;
  float* entropy;
  float* norm;
  int64_t* top_tokens;
  float* top_logp;
  WsHeader* hdr;
  int64_t chunk;  // elements of a row per CTA of its cluster
  int stages;     // of the ring
};

constexpr int kBatch = 4;       // vectors of 16 bytes that a thread takes at once
constexpr int kStageVecs = kBatch * kThreads;
constexpr int kStageBytes = 16 * kStageVecs;
constexpr int kMaxStages = 12;  // of the ring that bulk copies fill (as many as there is room for)
constexpr int kSlots = 8;       // groups of a thread whose maxima are kept, the last for a ragged end
constexpr int kCandidates = 512;
constexpr int kHits = 256;

// Running sums of one thread, two lanes of each packed.
struct Sums {
  float ref = 0.f, lim = -INFINITY;  // lim: a larger value moves the reference
  float top = -INFINITY;
  uint64_t s = 0, e = 0;

  __device__ __forceinline__ void make_room(float largest, float c) {
    if (!(largest > lim)) return;
    if (lim != -INFINITY) {
      const float d = fmaxf((ref - largest) * c, kLowest), f = ex2(d);
      const uint64_t f2 = f2_pack(f, f);
      e = f2_mul(f2, f2_fma(f2_pack(d, d), s, e));
      s = f2_mul(f2, s);
    }
    ref = largest;
    lim = largest + __fdividef(kSlack, c);
  }
  __device__ __forceinline__ void add(uint64_t x, uint64_t nref, uint64_t c) {
    float a, b;
    f2_unpack(f2_mul(f2_add(x, nref), c), a, b);
    a = max_keep_nan(a, kLowest);
    b = max_keep_nan(b, kLowest);
    const uint64_t w = f2_pack(ex2(a), ex2(b));
    s = f2_add(s, w);
    e = f2_fma(w, f2_pack(a, b), e);
  }
};

// The elements of a vector in pairs.  (bf16's low halves by byte permutations: as shifts
// they would go to the pipe that the packed arithmetic fills.)
__device__ __forceinline__ void pairs_of(const uint4& d, uint64_t* x, float) {
  x[0] = f2_pack(__uint_as_float(d.x), __uint_as_float(d.y));
  x[1] = f2_pack(__uint_as_float(d.z), __uint_as_float(d.w));
}
__device__ __forceinline__ void pairs_of(const uint4& d, uint64_t* x, uint16_t) {
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t lo;
    asm("prmt.b32 %0, %1, 0, 0x1044;" : "=r"(lo) : "r"(w[k]));
    x[k] = f2_pack(__uint_as_float(lo), bf16_hi(w[k]));
  }
}

constexpr int kMaxSplit = 8;  // CTAs of a cluster that share a row

struct StatsShared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int abort;  // a bounded wait gave up
  float warp_max[kWarps];
  float2 warp_sum[kWarps];
  float4 part[kMaxSplit];  // of the cluster's CTAs, in the first one: m, S, E, whether it gave up
};
// What the choice of the alternatives keeps in shared memory; `Late` lies over the ring,
// which is free by then.
struct TopShared {
  uint64_t part_key[kMaxSplit][kMaxTop];  // of the cluster's CTAs, in the first one: best keys, sorted
  alignas(16) float quad[64];             // maxima of sets of four threads
  float bound;
  int hits, keys, ties;
};
struct Late {
  uint64_t key[kCandidates];
  int hit[kHits];
};

template <typename T>
struct Part {  // elements [v0, v1) of a row; vectors of 16 bytes in [a, b)
  const T* z;
  int64_t v0, v1, a, b;
  int nvec;
  int groups, per;  // groups of `per` batches of U vectors
  unsigned inverse;  // 2^32 / (per U), rounded up: quotients of what is below 2^32 / (per U)
};

// A logit's own bits, from its float, and back.
__device__ __forceinline__ float bits_of(float x, float) { return x; }
__device__ __forceinline__ uint16_t bits_of(float x, uint16_t) {
  return (uint16_t)(__float_as_uint(x) >> 16);
}
__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(uint16_t x) { return bf16_bits_to_float(x); }

__device__ __forceinline__ uint32_t raw_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t raw_of(uint16_t x) { return x; }
// The float behind x.
__device__ __forceinline__ float next_above(float x) {
  const int b = __float_as_int(x + 0.f);
  return __int_as_float(b >= 0 ? b + 1 : b - 1);
}

// The bound: the top-th largest of the 64 sets' maxima, lower sets first; four threads
// count what is before one.  Between two barriers.
__device__ __forceinline__ void find_bound(TopShared& sh, int top) {
  const int set = threadIdx.x / 4, quarter = threadIdx.x % 4 * 16;
  const float mine = sh.quad[set];
  int before = 0;
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    const float4 x = *reinterpret_cast<const float4*>(&sh.quad[quarter + k]);
    const int at = quarter + k;
    before += (x.x > mine || (x.x == mine && at < set)) + (x.y > mine || (x.y == mine && at + 1 < set)) +
              (x.z > mine || (x.z == mine && at + 2 < set)) +
              (x.w > mine || (x.w == mine && at + 3 < set));
  }
  before += __shfl_xor_sync(0xffffffffu, before, 1);
  before += __shfl_xor_sync(0xffffffffu, before, 2);
  if (before == top - 1) sh.bound = mine;
}

// emit(place, key) for the first `top` of late.key[0 .. have): a key's place is the number
// of keys before it (they are all different, but for zeros, which are none); up to eight
// threads count for one.
template <typename Emit>
__device__ __forceinline__ void emit_places(const Late& late, int have, int top, Emit emit) {
  const int tid = threadIdx.x;
  int team = 8;
  while (team > 1 && have * team > kThreads) team /= 2;
#pragma unroll 1
  for (int k0 = 0; k0 < have; k0 += kThreads / team) {
    const int k = k0 + tid / team;
    const uint64_t mine = k < have ? late.key[k] : 0;
    int place = 0;
#pragma unroll 4
    for (int j = tid % team; j < have; j += team) place += late.key[j] > mine;
    for (int o = 1; o < team; o *= 2) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (tid % team == 0 && mine != 0 && place < top) emit(place, mine);
  }
}

// The best `top` of the part's elements (it has as many): emit(place, key)
// for each, by the thread that found it.  Called by the whole CTA after the stream, with
// the bound known.  slot[g][thread]: maxima of groups.  kept: where the part's vectors still
// lie in shared memory, or 0.
template <typename T, typename Emit>
__device__ __forceinline__ void best_of_part(TopShared& sh, Late& late, const T (*slot)[kThreads],
                                             const Part<T>& p, uint32_t kept, int top, Emit emit) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec, U = kBatch;
  constexpr uint32_t kNan = sizeof(T) == 2 ? 0x7fc07fc0u : 0x7fc00000u;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool listed = false;
  const float bound = sh.bound;
  // Appends one of each lane's chosen at a time: store(place, which), `chosen` a bit each.
  const auto append = [&](uint32_t chosen, int* count, auto store) {
    uint32_t votes;
    while ((votes = __ballot_sync(0xffffffffu, chosen != 0)) != 0) {
      int at = 0;
      if (lane == 0) at = atomicAdd(count, __popc(votes));  // (one addition a warp)
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(votes & ((1u << lane) - 1));
      if (chosen != 0) store(at, __ffs(chosen) - 1);
      chosen &= chosen - 1;
    }
  };
  // with the ties at the bound, or (where they are too many) without them
#pragma unroll 1
  for (int strict = 0; strict < 2 && !listed; ++strict) {
    const float least = strict ? next_above(bound) : bound;
    uint32_t groups = 0;
#pragma unroll
    for (int g = 0; g < kSlots; ++g)
      if (g <= p.groups && value_of(slot[g][tid]) >= least) groups |= 1u << g;
    append(groups, &sh.hits, [&](int at, int g) {
      if (at < kHits) late.hit[at] = g * kThreads + tid;
    });
    __syncthreads();
    const int hits = sh.hits;
    if (hits <= kHits) {
      const unsigned each = (unsigned)p.per * U, items = (unsigned)hits * each;
      const bool divide = each > 4096;  // (items reach kHits each: the product with the inverse is
                                        // exact while items each are below 2^32)
      constexpr int kAhead = 2;
#pragma unroll 1
      for (unsigned first = 0; first < items; first += kAhead * kThreads) {
        uint4 d[kAhead];
        int64_t id[kAhead];  // of the vector's first element
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const unsigned w = first + u * kThreads + tid;
          id[u] = 0;
          d[u] = make_uint4(kNan, kNan, kNan, kNan);  // (never chosen)
          if (w >= items) continue;
          const unsigned q = divide ? w / each : __umulhi(w, p.inverse), rest = w - q * each;
          const int h = late.hit[q], t = h % kThreads, g = h / kThreads;
          const int at = (g * (int)each + (int)rest) * kThreads + t;
          if (g == p.groups) {  // a ragged end's element alone
            if (rest != 0) continue;
            id[u] = t < 32 ? p.v0 + t : p.b + t - 32;
            d[u].x = (sizeof(T) == 2 ? kNan << 16 : 0u) | raw_of(p.z[id[u]]);
          } else if (at < p.nvec) {
            id[u] = p.a + (int64_t)at * EPV;
            d[u] = kept != 0 ? ld_shared_v4(kept + 16 * at) : ld_stream(p.z + id[u]);
          }
        }
#pragma unroll 1
        for (int u = 0; u < kAhead && first + u * kThreads < items; ++u) {
          float x[EPV];
          E::unpack(d[0], x);
          uint32_t chosen = 0;
#pragma unroll
          for (int e = 0; e < EPV; ++e)
            if (x[e] >= least) chosen |= 1u << e;
          append(chosen, &sh.keys, [&](int at, int e) {
            if (at < kCandidates) late.key[at] = key_of(E::extract(d[0], e), id[0] + e);
          });
          d[0] = d[1];
          id[0] = id[1];
        }
      }
    }
    __syncthreads();
    const int have = sh.keys;
    listed = hits <= kHits && have <= kCandidates - (strict ? kMaxTop : 0);
    if (listed && (!strict || have >= top)) break;
    __syncthreads();
    if (!listed) {
      if (tid == 0) sh.hits = sh.keys = 0;
      __syncthreads();
    } else {
      // the first ties in the order of their ids
      for (int64_t at = p.v0; at < p.v1; at += kThreads) {
        const int64_t v = at + tid;
        const bool tie = v < p.v1 && E::load1(p.z + v) == bound;
        const uint32_t votes = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) late.hit[warp] = __popc(votes);
        __syncthreads();
        int before = sh.ties, all = sh.ties;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) before += late.hit[w];
          all += late.hit[w];
        }
        before += __popc(votes & ((1u << lane) - 1));
        if (tie && have + before < top) late.key[have + before] = key_of(bound, v);
        __syncthreads();
        if (tid == 0) sh.ties = all;
        if (have + all >= top) break;
      }
      if (tid == 0) sh.keys = top;
      __syncthreads();
    }
  }
  if (!listed) {
    // rows whose largest elements crowd in few threads' groups: every warp keeps
    // the best 32 of its share, one per lane, best first
    uint64_t mine = 0, last = 0;
    for (int64_t at = p.v0 + warp * 32; at < p.v1; at += kThreads) {
      const int64_t v = at + lane;
      const uint64_t k = v < p.v1 ? key_of(E::load1(p.z + v), v) : 0;
      uint32_t better = __ballot_sync(0xffffffffu, k > last);
      while (better != 0) {
        const int from = __ffs(better) - 1;
        better &= better - 1;
        const uint64_t x = __shfl_sync(0xffffffffu, k, from);
        const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
        if (x > mine) mine = lane > 0 && x > up ? up : x;
        last = __shfl_sync(0xffffffffu, mine, top - 1);
      }
    }
    late.key[tid] = mine;
    if (tid == 0) sh.keys = kThreads;
    __syncthreads();
  }
  emit_places(late, sh.keys, top, emit);
}

// Sorts a warp's keys, whose lanes first rise and then fall (or the other way): largest
// first, or last.  (K. Batcher's merge.)
template <typename K>
__device__ __forceinline__ K exchanged(K key, int o, bool first) {
  const K other = __shfl_xor_sync(0xffffffffu, key, o);
  return ((threadIdx.x & o) == 0) == first ? max(key, other) : min(key, other);
}
template <typename K>
__device__ __forceinline__ K sort_merged(K key, bool first) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) key = exchanged(key, o, first);
  return key;
}
// In any order before, in the first `count` lanes (the others' are 0).
template <typename K>
__device__ __forceinline__ K sort_keys(K key, bool first, int count = 32) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
    if (size / 2 >= count) break;  // (sorted, the largest first)
#pragma unroll
    for (int o = size / 2; o > 0; o >>= 1)
      key = exchanged(key, o, size == 32 ? first : (threadIdx.x & size) == 0);
  }
  return key;
}

// The best `top` of the cluster's lists, each sorted and filled up with zeros: one warp merges
// them two by two, a lane a place.  (Of a list that falls and one that rises, the larger one at
// each place are the best 32 of both.)
template <typename Emit>
__device__ __forceinline__ void merge_parts(const TopShared& sh, int parts, int top, Emit emit) {
  const int lane = threadIdx.x;
  if (lane >= 32) return;
  static_assert(kMaxSplit == 8 && kMaxTop == 32, "a place per lane, three rounds");
  uint64_t key[kMaxSplit];
#pragma unroll
  for (int k = 0; k < kMaxSplit; ++k)
    key[k] = k < parts ? sh.part_key[k][k % 2 == 0 ? lane : 31 - lane] : 0;
#pragma unroll
  for (int far = 1; far < kMaxSplit; far *= 2) {
    if (far >= parts) break;
#pragma unroll
    for (int k = 0; k < kMaxSplit; k += 2 * far)
      key[k] = sort_merged(max(key[k], key[k + far]), k / (2 * far) % 2 == 0);
  }
  if (key[0] != 0 && lane < top) emit(lane, key[0]);
}

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void write_header(WsHeader* hdr, uint32_t rows) {
  hdr->flags = kFlagIndirect;
  hdr->status_count = rows;
  hdr->status_check = ~rows;
}

// Thread blocks per SM: as many as have room for their ring in shared memory.  Three
// stages on their way in each keep HBM busy while some of the blocks begin or end a row.
template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 4) token_stats_kernel(const StatsParams<T> p) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec, U = kBatch;
  extern __shared__ __align__(128) char s_dyn[];
  // (behind what a part that fits into the ring leaves there)
  Late& late = *reinterpret_cast<Late*>(s_dyn + p.stages * kStageBytes - sizeof(Late));
  T(*slot)[kThreads] = reinterpret_cast<T(*)[kThreads]>(s_dyn + p.stages * kStageBytes);
  __shared__ StatsShared sh;
  __shared__ TopShared top;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t parts = cluster_size(), rank = cluster_ctarank();
  const uint32_t rows = (uint32_t)(p.N * p.R), r32 = cluster_id_x();  // (below 2^26)
  const int64_t r = r32, i = r32 / max((uint32_t)p.R, 1u), j = r - i * p.R;
  const bool writer = rank == 0 && warp == kWarps - 1 && lane == 0;  // of the row's results
  uint32_t* status = reinterpret_cast<uint32_t*>(p.hdr) + 64 + r;
  uint32_t flags = 0;
  if (p.lens != nullptr && r < rows) {
    pdl_wait();
    pdl_trigger();
    const int64_t len = __ldg(p.lens + i);
    if ((len < 0 || len > p.R) && j == 0) flags = kFlagLengthRange;
    if (j >= len) {  // behind the sequence's end
      if (r == 0 && writer) write_header(p.hdr, rows);
      if (writer) {
        p.logp[r] = p.entropy[r] = p.norm[2 * r] = p.norm[2 * r + 1] = 0.f;
        *status = flags;
      }
      if (kTop && rank == 0 && tid < p.top) {
        p.top_tokens[r * p.top + tid] = -1;
        p.top_logp[r * p.top + tid] = 0.f;
      }
      return;
    }
  }
  Part<T> part;
  part.z = p.logits + i * p.seq + j * p.row;
  part.v0 = min(p.V, rank * p.chunk);
  part.v1 = min(p.V, part.v0 + p.chunk);
  const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(part.z + part.v0) & 15u);
  part.a = min(part.v0 + (int64_t)(((16u - off) & 15u) / sizeof(T)), part.v1);
  part.nvec = (int)((part.v1 - part.a) / EPV);
  part.b = part.a + (int64_t)part.nvec * EPV;
  const int batches = (part.nvec + kStageVecs - 1) / kStageVecs;
  // batch b goes through stage b % stages; thread 0 orders the copies
  const int stages = p.stages;
  const uint32_t ring = smem_u32(s_dyn), full = smem_u32(sh.full), empty = smem_u32(sh.empty);
  const char* source = reinterpret_cast<const char*>(part.z + part.a);
  const auto order = [&](int b, int st) {
    const uint32_t bytes = 16u * (uint32_t)min(kStageVecs, part.nvec - b * kStageVecs);
    mbar_arrive_expect_tx(full + 8 * st, bytes);
    bulk_g2s(ring + st * kStageBytes, source + (int64_t)b * kStageBytes, bytes, full + 8 * st);
  };
  if (tid == 0) {
    sh.abort = 0;
    for (int k = 0; k < min(stages, batches); ++k) {
      mbar_init(full + 8 * k, 1);
      mbar_init(empty + 8 * k, kWarps);
    }
    mbar_init_fence();
  }
  // (without lengths nothing of the caller's memory was read this far)
  pdl_wait();
  pdl_trigger();
  if (r == 0 && writer) write_header(p.hdr, rows);
  if (r >= rows) return;
  if (parts > 1) cluster_arrive_relaxed();  // (the first CTA runs before it is written to)
  int ordered = 0;                          // (thread 0's)
  if (tid == 0)
    for (; ordered < min(stages, batches); ++ordered) order(ordered, ordered);
  __syncthreads();
  part.per = (batches + kSlots - 2) / (kSlots - 1);
  part.groups = part.per > 0 ? (batches + part.per - 1) / part.per : 0;
  part.inverse = 0xffffffffu / (unsigned)max(part.per * U, 1) + 1;
  const float Ti = warmth_of(p.temperature, i);
  const float c = kLog2e / Ti;
  // (used behind the stream)
  const int64_t y = writer ? load_now(p.tokens + i * p.token_seq + j * p.token_row) : -1;
  Sums sum;
  const uint64_t c2 = f2_pack(c, c);
  int batch = 0, st = 0, last = 0;  // the batch's stage, and the one before
  uint32_t phase = 0, last_phase = 0;
  for (int g = 0; g < part.groups; ++g) {
    float group_max = -INFINITY;
    for (int q = 0; q < part.per && batch < batches; ++q, ++batch) {
      // (a warp gives up as a whole: what follows wants all its lanes)
      if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * st, phase))) {
        *(volatile int*)&sh.abort = 1;
        batch = batches;
        break;
      }
      const int n = min(kStageVecs, part.nvec - batch * kStageVecs);
      uint4 d[U];
      if (n == kStageVecs) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          d[u] = ld_shared_v4(ring + st * kStageBytes + 16 * (tid + u * kThreads));
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          d[u] = make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
          if (tid + u * kThreads < n)
            d[u] = ld_shared_v4(ring + st * kStageBytes + 16 * (tid + u * kThreads));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * st);
      // the stage of the batch before this one is free once every warp has read it
      if (tid == 0 && batch >= 1 && ordered < batches) {
        if (mbar_wait(empty + 8 * last, last_phase))
          order(ordered++, last);
        else
          *(volatile int*)&sh.abort = 1;  // (nothing more arrives: every wait ends)
      }
      last = st;
      last_phase = phase;
      if (++st == stages) {
        st = 0;
        phase ^= 1;
      }
      const float largest = E::template batch_max<U>(d);
      group_max = fmaxf(group_max, largest);
      sum.make_room(largest, c);
      const uint64_t nref = f2_pack(-sum.ref, -sum.ref);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint64_t x[EPV / 2];
        pairs_of(d[u], x, T());
#pragma unroll
        for (int e = 0; e < EPV / 2; ++e) sum.add(x[e], nref, c2);
      }
    }
    sum.top = fmaxf(sum.top, group_max);
    if (kTop) slot[g][tid] = bits_of(group_max, T());
  }
  const float at_token = y >= 0 && y < p.V ? load_now(part.z + y) : 0.f;
  {  // a ragged end's element
    int64_t v = -1;
    if (tid < part.a - part.v0)
      v = part.v0 + tid;
    else if (tid >= 32 && tid - 32 < part.v1 - part.b)
      v = part.b + tid - 32;
    float x = -INFINITY;
    if (v >= 0) {
      x = E::load1(part.z + v);
      sum.make_room(x, c);
      sum.top = fmaxf(sum.top, x);
      sum.add(f2_pack(x, -INFINITY), f2_pack(-sum.ref, -sum.ref), c2);
    }
    if (kTop) slot[part.groups][tid] = v >= 0 ? bits_of(x, T()) : bits_of(NAN, T());
  }
  // the row's maximum, then its sums relative to it
  float m = sum.top;
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sh.warp_max[warp] = m;
  if (kTop) {
    float q = fmaxf(sum.top, __shfl_xor_sync(0xffffffffu, sum.top, 1));
    q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 2));
    if (lane % 4 == 0) top.quad[tid / 4] = q;
    if (tid == 0) top.hits = top.keys = top.ties = 0;
  }
  __syncthreads();
  if (kTop) find_bound(top, p.top);
  m = sh.warp_max[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sh.warp_max[w]);
  float s, e, s1, e1;
  f2_unpack(sum.s, s, s1);
  f2_unpack(sum.e, e, e1);
  s += s1;
  e += e1;
  if (sum.lim != -INFINITY) {
    const float d = fmaxf((sum.ref - m) * c, kLowest), f = ex2(d);
    e = f * fmaf(d, s, e);
    s *= f;
  }
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  if (lane == 0) sh.warp_sum[warp] = make_float2(s, e);
  __syncthreads();
  s = e = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    s += sh.warp_sum[w].x;
    e += sh.warp_sum[w].y;
  }
  const uint32_t kept = part.nvec <= (stages * kStageBytes - (int)sizeof(Late)) / 16 ? ring : 0;
  if (sh.abort != 0) {  // some of the row is missing: no distribution, and the reason
    s = NAN;
    flags |= kFlagTimeout;
    if (tid == 0)  // (what may still be on its way)
      for (int b = max(0, ordered - stages); b < ordered; ++b)
        mbar_wait(full + 8 * (b % stages), b / stages & 1);
  }
  if (parts > 1) {
    __syncwarp();  // (the cluster's barriers want whole warps)
    cluster_wait();
    if (kTop) {
      const int got = sh.abort != 0 ? 0 : p.top;
      const uint32_t to = map_to_rank(smem_u32(&top.part_key[rank][0]), 0);
      if (got > 0)
        best_of_part(top, late, slot, part, kept, p.top,
                     [&](int place, uint64_t key) { st_cluster_u64(to + 8 * place, key); });
      if (tid >= got && tid < kMaxTop) st_cluster_u64(to + 8 * tid, 0);
    }
    if (tid == 0)
      st_cluster_f32x4(map_to_rank(smem_u32(&sh.part[rank]), 0), make_float4(m, s, e, sh.abort != 0 ? 1.f : 0.f));
    __syncwarp();
    cluster_sync();
    if (rank != 0) return;
    // (a lane a part, in every eight; a part of nothing but -inf has sums 0)
    const int k = lane % kMaxSplit;
    const float4 q = sh.part[min(k, (int)parts - 1)];
    m = q.x;
#pragma unroll
    for (int o = kMaxSplit / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float d = fmaxf((q.x - m) * c, kLowest), f = k < (int)parts ? ex2(d) : 0.f;
    s = f * q.y;
    e = f * fmaf(d, q.y, q.z);
#pragma unroll
    for (int o = kMaxSplit / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    if (__any_sync(0xffffffffu, q.w != 0.f)) flags |= kFlagTimeout;
  }
  // (a comparison with NaN is false)
  const bool defined = s > 0.f && s < INFINITY && fabsf(m) < INFINITY && c > 0.f;
  const float L = logf(s);
  if (writer) {
    if (!defined)
      flags |= kFlagValue;
    else if (y < 0 || y >= p.V)
      flags |= kFlagTokenRange;
    p.logp[r] = defined && y >= 0 && y < p.V ? (at_token - m) / Ti - L : NAN;
    p.entropy[r] = defined ? L - kLn2 * (e / s) : NAN;
    p.norm[2 * r] = defined ? m : NAN;
    p.norm[2 * r + 1] = defined ? L : NAN;
    *status = flags;
  }
  if (!kTop) return;
  if (!defined) {
    if (tid < p.top) {
      p.top_tokens[r * p.top + tid] = -1;
      p.top_logp[r * p.top + tid] = NAN;
    }
    return;
  }
  const auto write = [&](int place, uint64_t key) {
    p.top_tokens[r * p.top + place] = key_id(key);
    p.top_logp[r * p.top + place] = (key_value(key) - m) / Ti - L;
  };
  if (parts > 1)
    merge_parts(top, (int)parts, p.top, write);
  else
    best_of_part(top, late, slot, part, kept, p.top, write);
}

// ---------------------------------------------------------------------------
// forward, short rows: a warp per row
// ---------------------------------------------------------------------------

// A warp's best keys so far, one per lane, best first.
struct Best {
  uint64_t mine = 0, last = 0;  // last: the top-th

  // Takes the lanes' x where `wanted`.
  __device__ __forceinline__ void take(bool wanted, float x, int64_t v, int top) {
    const uint64_t k = wanted ? key_of(x, v) : 0;
    uint32_t better = __ballot_sync(0xffffffffu, k > last);
    const int lane = threadIdx.x & 31;
    while (better != 0) {
      const int from = __ffs(better) - 1;
      better &= better - 1;
      const uint64_t y = __shfl_sync(0xffffffffu, k, from);
      const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
      if (y > mine) mine = lane > 0 && y > up ? up : y;
      last = __shfl_sync(0xffffffffu, mine, top - 1);
    }
  }
};

// The top-th largest of 64 values, two a lane: a warp's lower bound of the top-th
// largest element where each is the largest of a set.
// (By repeated maxima, or for more of them sorted: 32,768 rows of 1,000 bf16 with 20 53 us by
// sorting and 58 by maxima, with 5 44 and 42.)
__device__ __forceinline__ float warp_bound(float set0, float set1, int top) {
  const auto ordered = [](float x) { return (uint32_t)(key_of(x, 0) >> 32); };
  uint32_t hi = ordered(fmaxf(set0, set1)), lo = ordered(fminf(set0, set1)), best = 0;
  if (top > 8) {
    best = sort_merged(max(sort_keys(hi, true), sort_keys(lo, false)), true);
    best = __shfl_sync(0xffffffffu, best, top - 1);
  } else {
#pragma unroll 1
    for (int k = 0; k < top; ++k) {
      best = __reduce_max_sync(0xffffffffu, hi);
      if ((threadIdx.x & 31) == __ffs(__ballot_sync(0xffffffffu, hi == best)) - 1) {
        hi = lo;
        lo = 0;  // (below every value)
      }
    }
  }
  return key_value((uint64_t)best << 32);
}

// What token_stats_kernel computes.  A row takes one warp longer than a thread block, but
// 32 of them share an SM, without barriers and with a tenth of the instructions that a row costs
// beside its elements (which kernel where: at the launch).
template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 4) token_stats_short_kernel(const StatsParams<T> p) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec, U = 4;
  const int lane = threadIdx.x & 31;
  const uint32_t rows = (uint32_t)(p.N * p.R), r = blockIdx.x * kWarps + threadIdx.x / 32;
  pdl_wait();
  pdl_trigger();
  if (r == 0 && lane == 0) write_header(p.hdr, rows);
  if (r >= rows) return;
  const int64_t i = r / (uint32_t)p.R, j = r - i * p.R;
  uint32_t* status = reinterpret_cast<uint32_t*>(p.hdr) + 64 + r;
  uint32_t flags = 0;
  float* const norm = p.norm + 2 * (int64_t)r;
  int64_t* const top_tokens = p.top_tokens + (int64_t)r * p.top;
  float* const top_logp = p.top_logp + (int64_t)r * p.top;
  if (p.lens != nullptr) {
    const int64_t len = __ldg(p.lens + i);
    if ((len < 0 || len > p.R) && j == 0) flags = kFlagLengthRange;
    if (j >= len) {  // behind the sequence's end
      if (lane == 0) {
        p.logp[r] = p.entropy[r] = norm[0] = norm[1] = 0.f;
        *status = flags;
      }
      if (kTop && lane < p.top) {
        top_tokens[lane] = -1;
        top_logp[lane] = 0.f;
      }
      return;
    }
  }
  const int64_t y = lane == 0 ? __ldg(p.tokens + i * p.token_seq + j * p.token_row) : -1;
  const T* z = p.logits + i * p.seq + j * p.row;
  const float Ti = warmth_of(p.temperature, i);
  const float c = kLog2e / Ti;
  // (short: 32-bit indexes)
  const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(z) & 15u);
  const int V = (int)p.V, a = min((int)(((16u - off) & 15u) / sizeof(T)), V);
  const int nvec = (V - a) / EPV, b = a + nvec * EPV;
  const uint4* vec = reinterpret_cast<const uint4*>(z + a);
  const auto load = [&](uint4* d, int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      d[u] = make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
      if (k0 + 32 * u < nvec) d[u] = __ldg(vec + k0 + 32 * u);
    }
  };
  const int ragged = lane < 16 ? (lane < a ? lane : -1) : (lane - 16 < V - b ? b + lane - 16 : -1);
  const float end = ragged >= 0 ? E::load1(z + ragged) : -INFINITY;

  Sums sum;
  const uint64_t c2 = f2_pack(c, c);
  float set0 = -INFINITY, set1 = end;
#pragma unroll 1
  for (int k0 = lane; k0 - lane < nvec; k0 += 32 * U) {
    uint4 d[U];
    load(d, k0);
    const float even = E::template batch_max<U / 2>(d), odd = E::template batch_max<U / 2>(d + U / 2);
    set0 = fmaxf(set0, even);
    set1 = fmaxf(set1, odd);
    sum.make_room(fmaxf(even, odd), c);
    const uint64_t nref = f2_pack(-sum.ref, -sum.ref);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint64_t x[EPV / 2];
      pairs_of(d[u], x, T());
#pragma unroll
      for (int e = 0; e < EPV / 2; ++e) sum.add(x[e], nref, c2);
    }
  }
  if (ragged >= 0) {
    sum.make_room(end, c);
    sum.add(f2_pack(end, -INFINITY), f2_pack(-sum.ref, -sum.ref), c2);
  }
  const float at_token = y >= 0 && y < V ? E::load1(z + y) : 0.f;
  float m = fmaxf(set0, set1);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s, e, s1, e1;
  f2_unpack(sum.s, s, s1);
  f2_unpack(sum.e, e, e1);
  s += s1;
  e += e1;
  if (sum.lim != -INFINITY) {
    const float d = fmaxf((sum.ref - m) * c, kLowest), f = ex2(d);
    e = f * fmaf(d, s, e);
    s *= f;
  }
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  // (a comparison with NaN is false)
  const bool defined = s > 0.f && s < INFINITY && fabsf(m) < INFINITY && c > 0.f;
  const float L = logf(s);
  if (lane == 0) {
    if (!defined)
      flags |= kFlagValue;
    else if (y < 0 || y >= V)
      flags |= kFlagTokenRange;
    p.logp[r] = defined && y >= 0 && y < V ? (at_token - m) / Ti - L : NAN;
    p.entropy[r] = defined ? L - kLn2 * (e / s) : NAN;
    norm[0] = defined ? m : NAN;
    norm[1] = defined ? L : NAN;
    *status = flags;
  }
  if (!kTop) return;
  // The candidates as a list that the warp sorts, up to two keys a lane; where there are more
  // (ties, crowds in few sets), by insertion of one after the other (32,768 rows of 1,000 bf16
  // with 20 72 us, 58 as lists; with 5 46 and 42).
  constexpr int kList = 64;
  __shared__ uint64_t lists[kTop ? kWarps : 1][kList];
  uint64_t* const list = lists[kTop ? threadIdx.x / 32 : 0];
  Best best;
  if (defined) {
    const float bound = warp_bound(set0, set1, p.top);
    int count = 0;
    const auto append = [&](uint32_t chosen, auto key) {
      uint32_t votes;
      while ((votes = __ballot_sync(0xffffffffu, chosen != 0)) != 0) {
        const int at = count + __popc(votes & ((1u << lane) - 1));
        if (chosen != 0 && at < kList) list[at] = key(__ffs(chosen) - 1);
        count += __popc(votes);
        chosen &= chosen - 1;
      }
    };
    // each(vector, its first element, whether it is one) where one of the warp's has candidates
    const auto second_look = [&](auto each) {
#pragma unroll 1
      for (int k0 = lane; k0 - lane < nvec; k0 += 32 * U) {
        uint4 d[U];
        load(d, k0);
        if (!__any_sync(0xffffffffu, E::template batch_max<U>(d) >= bound)) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool there = k0 + 32 * u < nvec;
          if (__any_sync(0xffffffffu, there && E::template batch_max<1>(d + u) >= bound))
            each(d[u], a + (k0 + 32 * u) * EPV, there);
        }
      }
    };
    append(ragged >= 0 && end >= bound, [&](int) { return key_of(end, ragged); });
    second_look([&](const uint4& d, int v, bool there) {
      float x[EPV];
      E::unpack(d, x);
      uint32_t chosen = 0;
#pragma unroll
      for (int q = 0; q < EPV; ++q)
        if (there && x[q] >= bound) chosen |= 1u << q;
      append(chosen, [&](int q) { return key_of(E::extract(d, q), v + q); });
    });
    __syncwarp();
    if (count <= kList) {
      best.mine = sort_keys(lane < count ? list[lane] : 0, true, count);
      if (count > 32)
        best.mine = sort_merged(
            max(best.mine, sort_keys(lane + 32 < count ? list[lane + 32] : 0, false)), true);
    } else {
      best.take(ragged >= 0 && end >= bound, end, ragged, p.top);
      second_look([&](const uint4& d, int v, bool there) {
        float x[EPV];
        E::unpack(d, x);
#pragma unroll
        for (int q = 0; q < EPV; ++q) {
          const bool wanted = there && x[q] >= bound;
          if (__any_sync(0xffffffffu, wanted)) best.take(wanted, x[q], v + q, p.top);
        }
      });
    }
  }
  if (lane < p.top) {
    top_tokens[lane] = defined ? key_id(best.mine) : -1;
    top_logp[lane] = defined ? (key_value(best.mine) - m) / Ti - L : NAN;
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

template <typename T>
struct StatsBwdParams {
  const T* logits;
  int64_t N, R, V, seq, row;
  const int64_t* tokens;
  int64_t token_seq, token_row;
  const int32_t* lens;
  const float* temperature;
  const float* norm;
  const float* entropy;
  const float* grad_logp;
  const float* grad_entropy;
  T* dlogits;
  int64_t dseq, drow;
  int64_t chunk, split;  // elements per work item, work items per row
};

// The gradient of one element.
struct RowGrad {
  float m, c, L2, A, B, g;  // g: of the log-prob, divided by T
  __device__ __forceinline__ float at(float x) const {
    const float l = max_keep_nan(fmaf(x - m, c, -L2), kLowest);
    return ex2(l) * fmaf(B, l, A);
  }
  // at the token: g (1 - p) without cancellation
  __device__ __forceinline__ float at_token(float x) const {
    const float l = max_keep_nan(fmaf(x - m, c, -L2), kLowest);
    return ex2(l) * fmaf(B, l, A + g) - g * expm1f(l * kLn2);
  }
};

// Of one vector, two elements of a packed operation each; ey: the token's element, or -1.
template <typename T>
__device__ __forceinline__ uint4 grad_vector(const uint4& d, const RowGrad& q, int ey) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec;
  uint64_t x[EPV / 2];
  pairs_of(d, x, T());
  float o[EPV];
#pragma unroll
  for (int e = 0; e < EPV / 2; ++e) {
    float a, b;
    f2_unpack(f2_fma(f2_add(x[e], f2_pack(-q.m, -q.m)), f2_pack(q.c, q.c), f2_pack(-q.L2, -q.L2)), a, b);
    a = max_keep_nan(a, kLowest);
    b = max_keep_nan(b, kLowest);
    const uint64_t f = f2_fma(f2_pack(q.B, q.B), f2_pack(a, b), f2_pack(q.A, q.A));
    f2_unpack(f2_mul(f2_pack(ex2(a), ex2(b)), f), o[2 * e], o[2 * e + 1]);
  }
  if (ey >= 0) {
    const float zy = E::extract(d, ey);
#pragma unroll
    for (int e = 0; e < EPV; ++e)
      if (e == ey) o[e] = q.at_token(zy);
  }
  return E::pack(o);
}

// The 16 bytes that begin kWords words and `bits` bits into lo and hi.
template <int kWords>
__device__ __forceinline__ uint4 from_two(uint4 lo, uint4 hi, unsigned bits) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  return make_uint4(__funnelshift_r(w[kWords], w[kWords + 1], bits),
                    __funnelshift_r(w[kWords + 1], w[kWords + 2], bits),
                    __funnelshift_r(w[kWords + 2], w[kWords + 3], bits),
                    __funnelshift_r(w[kWords + 3], w[kWords + 4], bits));
}
// `shift`: bytes, a multiple of 2.
__device__ __forceinline__ uint4 from_two(uint4 lo, uint4 hi, unsigned shift) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (shift & 8) {
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  }
  return from_two<0>(make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]), (shift & 2) * 8);
}

// nvec vectors of gradients by kStep threads; z: the first one's logits (kShift: `shift` bytes
// behind a 16-byte boundary), y: the token relative to it.
template <typename T, bool kShift, int kStep>
__device__ __forceinline__ void grad_vectors(const T* z, uint4* out, int nvec, unsigned shift,
                                             const RowGrad& q, int64_t y) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec, U = kShift ? 2 : 4;
  const uint4* zvec = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(z) - shift);
  const int ky = y >= 0 && y < (int64_t)nvec * EPV ? (int)(y / EPV) : -1;
  const int ey = ky >= 0 ? (int)(y % EPV) : -1;
  for (int k0 = threadIdx.x % kStep; k0 < nvec; k0 += kStep * U) {
    uint4 d[U], next[kShift ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kStep;
      if (k >= nvec) break;
      if (kShift) {  // (the neighbour's first is this one's second: through L1)
        d[u] = __ldg(zvec + k);
        next[u] = __ldg(zvec + k + 1);
      } else {
        d[u] = ld_stream(zvec + k);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kStep;
      if (k >= nvec) break;
      if (kShift) d[u] = from_two(d[u], next[u], shift);
      st_stream(out + k, grad_vector<T>(d[u], q, k == ky ? ey : -1));
    }
  }
}

// At most kStagedVecs vectors of gradients by a thread block, of logits at any alignment,
// through shared memory: all copies are on their way at once, and a vector is put together
// from two there.
constexpr int kPieceVecs = 2 * kThreads, kPieces = 4, kStagedVecs = kPieces * kPieceVecs;
template <typename T, int kWords>
__device__ __forceinline__ void grad_of_stage(uint32_t from, uint4* out, int nvec, unsigned bits,
                                              const RowGrad& q, int ky, int ey) {
#pragma unroll 1
  for (int piece = 0; piece * kPieceVecs < nvec; ++piece) {
    // this piece, and the next one's first vector
    if (piece == 0)
      cp_async_wait<kPieces - 2>();
    else if (piece == 1)
      cp_async_wait<kPieces - 3>();
    else
      cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = piece * kPieceVecs + u * kThreads + (int)threadIdx.x;
      if (k >= nvec) break;
      // (rows that agree take nothing of the second, whatever it holds)
      const uint4 d = from_two<kWords>(ld_shared_v4(from + 16 * k), ld_shared_v4(from + 16 * (k + 1)), bits);
      st_stream(out + k, grad_vector<T>(d, q, k == ky ? ey : -1));
    }
  }
  __syncthreads();  // (the stage is free)
}
template <typename T>
__device__ __forceinline__ void grad_staged(uint4* stage, const T* z, uint4* out, int nvec,
                                            unsigned shift, const RowGrad& q, int64_t y) {
  constexpr int EPV = Elt<T>::kPerVec;
  const uint4* zvec = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(z) - shift);
  const int ky = y >= 0 && y < (int64_t)nvec * EPV ? (int)(y / EPV) : -1;
  const int ey = ky >= 0 ? (int)(y % EPV) : -1;
  const int tid = threadIdx.x, in = nvec + (nvec > 0 && shift != 0);
  const uint32_t to = smem_u32(stage);
#pragma unroll
  for (int piece = 0; piece < kPieces; ++piece) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = piece * kPieceVecs + u * kThreads + tid;
      if (k < in) cp_async16(to + 16 * k, zvec + k);
    }
    if (piece == kPieces - 1 && tid == 0 && in > kStagedVecs)
      cp_async16(to + 16 * kStagedVecs, zvec + kStagedVecs);
    cp_async_commit();
  }
  // (a loop for each of the four: none selects words)
  const unsigned bits = shift % 4 * 8;
  if (shift < 4)
    grad_of_stage<T, 0>(to, out, nvec, bits, q, ky, ey);
  else if (shift < 8)
    grad_of_stage<T, 1>(to, out, nvec, bits, q, ky, ey);
  else if (shift < 12)
    grad_of_stage<T, 2>(to, out, nvec, bits, q, ky, ey);
  else
    grad_of_stage<T, 3>(to, out, nvec, bits, q, ky, ey);
}

// HBM-bound: 8,192 rows of 151,936 bf16, half of them scored, 545 us (the copy rate); rows
// whose gradient lies at another alignment 6.6 TB/s (2,000 of 151,935: 183 us, 227 with two
// loads a vector instead of the stage).
// Five thread blocks per SM: 99 us for 1,024 rows, 104 with four; staged six, 4% before five;
// one or two warps per row four, which spill a little (52 bytes a thread): 32,768 rows of 1,000
// 27.3 us, 28.2 with five, which spill more, 33.5 with three, which do not.
// kStep: threads to an item: a block's, or one or two warps'.
// kStaged: through shared memory.
template <typename T, int kStep, bool kStaged>
__global__ void __launch_bounds__(kThreads, kStaged ? 6 : kStep < kThreads ? 4 : 5) token_stats_bwd_kernel(
    const StatsBwdParams<T> p) {
  using E = Elt<T>;
  constexpr int EPV = E::kPerVec, kTeams = kThreads / kStep;
  __shared__ uint4 stage[kStaged ? kStagedVecs + 1 : 1];
  const int tid = threadIdx.x % kStep;
  pdl_wait();
  pdl_trigger();
  const uint32_t items = (uint32_t)(p.N * p.R) * (uint32_t)p.split;  // (below 2^31)
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (uint32_t item = blockIdx.x * kTeams + threadIdx.x / kStep; item < items;
       item += gridDim.x * kTeams) {
    const uint32_t row = item / (uint32_t)p.split, seq = row / (uint32_t)p.R;
    const int64_t r = row, i = seq, j = row - seq * (uint32_t)p.R;
    const int64_t v0 = (item - row * (uint32_t)p.split) * p.chunk, v1 = min(p.V, v0 + p.chunk);
    if (v0 >= v1) continue;
    const T* z = p.logits + i * p.seq + j * p.row;
    T* out = p.dlogits + i * p.dseq + j * p.drow;
    // 16-byte vectors of the output in [a, b); the input lies `shift` bytes behind
    // such a boundary there
    const unsigned phase = (unsigned)(reinterpret_cast<uintptr_t>(out + v0) & 15u);
    int64_t a = min(v0 + (int64_t)(((16u - phase) & 15u) / sizeof(T)), v1);
    int nvec = (int)((v1 - a) / EPV);
    const unsigned shift = (unsigned)(reinterpret_cast<uintptr_t>(z + a) & 15u);
    if (shift != 0 && nvec > 0) {
      // a vector is put together from the two of the input that it lies in: both inside
      // the row
      if (a * (int64_t)sizeof(T) < shift) a += EPV, --nvec;
      if (nvec > 0 && (p.V - a - (int64_t)nvec * EPV) * (int64_t)sizeof(T) < 16 - shift) --nvec;
    }
    const int64_t b = a + (int64_t)nvec * EPV;
    uint4* ovec = reinterpret_cast<uint4*>(out + a);
    // (loaded together: one latency)
    const bool inside = p.lens == nullptr || j < __ldg(p.lens + i);
    const float2 norm = __ldg(reinterpret_cast<const float2*>(p.norm) + r);
    const float Ti = warmth_of(p.temperature, i);
    const float gr = p.grad_logp != nullptr ? __ldg(p.grad_logp + r) : 0.f;
    const float hr = p.grad_entropy != nullptr ? __ldg(p.grad_entropy + r) : 0.f;
    const float Hr = p.grad_entropy != nullptr ? __ldg(p.entropy + r) : 0.f;
    const int64_t yr = p.grad_logp != nullptr ? __ldg(p.tokens + i * p.token_seq + j * p.token_row) : -1;
    const float g = inside ? gr : 0.f, h = inside ? hr : 0.f;
    int64_t edge = -1;
    if (tid < 16 && tid < a - v0)  // (at most 15 on either side)
      edge = v0 + tid;
    else if (tid >= 16 && tid - 16 < v1 - b)
      edge = b + tid - 16;
    if (g == 0.f && h == 0.f) {  // zeros, logits not read
      for (int k = tid; k < nvec; k += kStep) st_stream(ovec + k, zero);
      if (edge >= 0) E::store1(out + edge, 0.f);
      continue;
    }
    RowGrad q;
    q.m = norm.x;
    q.L2 = norm.y * kLog2e;
    q.c = kLog2e / Ti;
    q.g = g / Ti;
    q.A = -(q.g + (h != 0.f ? h / Ti * Hr : 0.f));
    q.B = -h / Ti * kLn2;
    int64_t y = -1;
    if (g != 0.f) {
      y = yr;
      if (y < 0 || y >= p.V) q.A = NAN;
    }
    if constexpr (kStaged) {
      grad_staged(stage, z + a, ovec, nvec, shift, q, y - a);
    } else if (kStep == kThreads || shift == 0) {  // (blocks: shifted rows are staged)
      grad_vectors<T, false, kStep>(z + a, ovec, nvec, 0, q, y - a);
    } else {
      grad_vectors<T, true, kStep>(z + a, ovec, nvec, shift, q, y - a);
    }
    if (edge >= 0) {
      const float x = E::load1(z + edge);
      E::store1(out + edge, edge == y ? q.at_token(x) : q.at(x));
    }
  }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------

template <typename T>
cudaError_t stats_run(const TokenStatsArgs& a, const DeviceInfo& d, cudaStream_t st) {
  StatsParams<T> p;
  p.logits = static_cast<const T*>(a.logits);
  p.N = a.N;
  p.R = a.R;
  p.V = a.V;
  p.seq = a.seq;
  p.row = a.row;
  p.tokens = a.tokens;
  p.token_seq = a.token_seq;
  p.token_row = a.token_row;
  p.lens = a.lens;
  p.temperature = a.temperature;
  p.top = a.top;
  p.logp = a.logp;
  p.entropy = a.entropy;
  p.norm = a.norm;
  p.top_tokens = a.top_tokens;
  p.top_logp = a.top_logp;
  p.hdr = static_cast<WsHeader*>(a.ws);
  const int64_t rows = a.N * a.R;
  // A warp per row where the rows are short and many; by warps and by thread blocks, without
  // alternatives, with 5 and with 20 (bf16, us): 600 rows of 2 KB 2.5 and 4.2, 4.4 and 7.8, 5.6
  // and 8.3; 1,200 of 8 KB 4.0 and 7.7, 7.1 and 14.2, 9.7 and 14.8; 300 of 8 KB 3.8 and 3.2,
  // 6.8 and 5.4, 9.4 and 5.8; 2,400 of 32 KB 18.1 and 21.6, 25.3 and 32.8, 31.2 and 34.3;
  // 4,800 of 64 KB 51 and 61, 93 and 86, 96 and 89; 3,600 of 128 KB 85 and 76.  With 32
  // alternatives, which more of the rows' candidates reach: 1,200 of 8 KB 10.9 and 15.7; 2,400 of
  // 16 KB 28 and 30; 4,000 of 32 KB 62 and 57, 8,000 102 and 108, 16,000 183 and 212.
  // Rows of which a block's sets have a few elements each always (8 rows of 1 KB 2.3 and 2.6,
  // 3.9 and 4.7, 5.2 and 20).
  const int64_t row_bytes = a.V * (int64_t)sizeof(T);
  if (row_bytes <= 1024 || (row_bytes <= (a.top == 0 ? 131072 : 32768) &&
                            rows * 2560 >= row_bytes * d.sms * (a.top > 8 ? 2 : 1))) {
    const dim3 blocks((unsigned)((rows + kWarps - 1) / kWarps + (rows == 0)));
    return a.top == 0
               ? launch_pdl(token_stats_short_kernel<T, false>, blocks, dim3(kThreads), 0, st, 1, p)
               : launch_pdl(token_stats_short_kernel<T, true>, blocks, dim3(kThreads), 0, st, 1, p);
  }
  // whole rows where there are more than SMs for them (296 rows of 304 KB 18.0 us, in halves
  // 18.9); below that as many CTAs as leave two per SM (64 rows 7.3 us in quarters, 12.4
  // whole, 8.7 in eighths; one row 4.5 us in eighths, 11.9 whole) of a batch each, or three
  // where each still has 128 KB (224 rows in halves 15.6 us, whole 17.6; of 128 KB rows 8.0
  // and 7.9, of 64 KB 6.3 and 5.1; 80 rows of 1.2 MB in quarters 23.6, in halves 30.5)
  int split = 1;
  while (split < kMaxSplit) {
    const int64_t part = row_bytes / (2 * split);
    if (part < kStageBytes || 2 * split * rows > (part >= 128 * 1024 ? 3 : 2) * (int64_t)d.sms) break;
    split *= 2;
  }
  constexpr int EPV = Elt<T>::kPerVec;
  p.chunk = ((a.V + split - 1) / split + EPV - 1) / EPV * EPV;
  const dim3 grid((unsigned)(rows < 1 ? split : rows * split));
  // The ring: three stages, with which four CTAs fill an SM's shared memory; more where
  // fewer CTAs come to an SM, up to the whole part and room behind it.
  const int slots = a.top == 0 ? 0 : kSlots * kThreads * (int)sizeof(T);
  const int64_t per_sm = (rows * split + d.sms - 1) / d.sms;
  const int64_t batches = (p.chunk * (int64_t)sizeof(T) + kStageBytes - 1) / kStageBytes;
  p.stages = 3;
  while (p.stages < kMaxStages && p.stages <= batches &&
         per_sm * ((p.stages + 1) * kStageBytes + slots + 4096) <= 224 * 1024)
    ++p.stages;
  const int smem = p.stages * kStageBytes + slots;
  const auto kern = a.top == 0 ? token_stats_kernel<T, false> : token_stats_kernel<T, true>;
  const cudaError_t e =
      ensure_dynamic_smem((const void*)kern, kMaxStages * kStageBytes + kSlots * kThreads * 4);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, dim3(kThreads), smem, st, split, p);
}

template <typename T>
cudaError_t bwd_run(const TokenStatsBwdArgs& a, const DeviceInfo& d, cudaStream_t st) {
  constexpr int EPV = Elt<T>::kPerVec;
  StatsBwdParams<T> p;
  p.logits = static_cast<const T*>(a.logits);
  p.N = a.N;
  p.R = a.R;
  p.V = a.V;
  p.seq = a.seq;
  p.row = a.row;
  p.tokens = a.tokens;
  p.token_seq = a.token_seq;
  p.token_row = a.token_row;
  p.lens = a.lens;
  p.temperature = a.temperature;
  p.norm = a.norm;
  p.entropy = a.entropy;
  p.grad_logp = a.grad_logp;
  p.grad_entropy = a.grad_entropy;
  p.dlogits = static_cast<T*>(a.dlogits);
  p.dseq = a.dseq;
  p.drow = a.drow;
  const int64_t row_bytes = a.V * (int64_t)sizeof(T), rows = a.N * a.R;
  // A warp per row where the rows are short and many, two for somewhat longer ones: 32,768 rows
  // of 1,000 bf16 28 us by warps, 40 by pairs, 97 by thread blocks; 4,001 105, 109 and 140;
  // 2,048 rows of 1,000 3.8, 4.6 and 8.0, of 4,000 9.9, 8.8 and 10.3, of 8,000 16.8, 13.6 and
  // 13.2; 600 rows of 2,000 4.0, 3.2 and 4.1, of 6,000 9.7, 6.5 and 5.2.
  if (row_bytes <= 12288 && rows * 1024 >= row_bytes * d.sms) {
    p.split = 1;
    p.chunk = a.V;
    const bool one = row_bytes <= 4096 && rows * 256 >= row_bytes * d.sms;
    const int64_t teams = one ? kWarps : kWarps / 2;
    const int64_t blocks = (rows + teams - 1) / teams, most = 32 * (int64_t)d.sms;
    return launch_pdl(one ? token_stats_bwd_kernel<T, 32, false> : token_stats_bwd_kernel<T, 64, false>,
                      dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, st, 1, p);
  }
  // parts of a row of 32 KB or more (1,024 rows of 304 KB 99 us, whole rows 107); where
  // that leaves few, down to 8 KB (8 rows 3.2 us in 32 parts each, 6.3 in 4), but no more than
  // the SMs hold at once (1,024 rows of 64 KB 25 us whole, 40 in 8 parts)
  p.split = row_split(row_bytes, nullptr, 8);
  while (rows * p.split < 4 * (int64_t)d.sms && row_bytes / (2 * p.split) >= 8192) p.split *= 2;
  // Rows whose gradients lie at another alignment go through shared memory in parts that
  // fit there, as large as that (2,000 rows of 151,935 bf16 in 10 parts 183 us, in 16 199).
  const auto differ = [](int64_t x) { return x * (int64_t)sizeof(T) % 16 != 0; };
  const bool staged =
      ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.dlogits)) & 15) != 0 ||
      (a.N > 1 && differ(a.seq - a.dseq)) || (a.R > 1 && differ(a.row - a.drow));
  constexpr int64_t kMost = (int64_t)kStagedVecs * EPV;
  if (staged && p.split * kMost < a.V) p.split = (a.V + kMost - 1) / kMost;
  p.chunk = ((a.V + p.split - 1) / p.split + EPV - 1) / EPV * EPV;
  const int64_t items = rows * p.split;
  int64_t grid = 256 * (int64_t)d.sms;
  if (grid > items) grid = items;
  if (staged)
    return launch_pdl(token_stats_bwd_kernel<T, kThreads, true>, dim3((unsigned)grid),
                      dim3(kThreads), 0, st, 1, p);
  return launch_pdl(token_stats_bwd_kernel<T, kThreads, false>, dim3((unsigned)grid),
                    dim3(kThreads), 0, st, 1, p);
}

}  // namespace

size_t token_stats_workspace_bytes(int64_t N, int64_t R) {
  return align_up(256 + 4 * (size_t)N * (size_t)R, 256);
}

cudaError_t launch_token_stats(const TokenStatsArgs& a, const DeviceInfo& d, cudaStream_t st) {
  return a.dtype == 0 ? stats_run<float>(a, d, st) : stats_run<uint16_t>(a, d, st);
}

cudaError_t launch_token_stats_bwd(const TokenStatsBwdArgs& a, const DeviceInfo& d,
                                   cudaStream_t st) {
  if (a.N * a.R == 0) return cudaSuccess;
  return a.dtype == 0 ? bwd_run<float>(a, d, st) : bwd_run<uint16_t>(a, d, st);
}

}  // namespace grpo
