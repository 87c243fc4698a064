// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   out[i, :] = s * W[id_i, :]
//   backward  dW[v, :] (+)= s * sum over { i : id_i = v } of dout[i, :]
//
// The backward sorts the tokens by id (a stable radix sort, so the tokens of
// one id stay in position order) while it clears dW, sums each id's rows in
// float32 in that order and writes the rows of the ids that occur.  No
// floating-point atomics: the order of every sum is fixed by n and the ids, so
// results are bitwise reproducible.
//
// Both are HBM-bound copies but for the sort, whose kernels wait on latency:
// 81,920 rows of 896 bfloat16 looked up in 31 us (147 MB written, 46 MB of
// distinct rows read); the gradient of 131,072 tokens (half of them padding)
// over 151,936 ids in 140 us, 82 us of it the zeros of the 545 MB result.
#include <type_traits>

#include "host_ctx.cuh"
#include "ops.cuh"

namespace grpo {
namespace {

// ---------------------------------------------------------------------------
// rows of any alignment
// ---------------------------------------------------------------------------

// A warp takes 256 columns of a row at a time, 8 per lane, 32 apart (so that its
// stores meet): the 16-byte pieces that hold them go to shared memory by
// asynchronous copies, several rows ahead, and every lane reads single elements
// of them.
constexpr int kWarpCols = 256;
// bytes of one row's pieces (one more than its columns fill), and of a CTA's
// rings: a warp reads 256 columns of the last row whatever its width
inline int warp_slot(int64_t d, size_t esize) {
  return ((int)(d < kWarpCols ? d : kWarpCols) * (int)esize + 30) / 16 * 16;
}
inline size_t warp_rings(int64_t d, size_t esize, int depth) {
  return (size_t)kWarps * depth * warp_slot(d, esize) + kWarpCols * esize;
}
// The pieces of `width` bytes from p on, by the warp; `off` bytes of them lie
// before p.  Through L1: neighbouring parts share a piece, and the rows of
// frequent ids would queue at their L2 slices (130,000 rows of 130 floats of 2,979
// ids: 20 us, 25 past L1; but 30,000 rows of 2,047 of 60,000 ids 50, 46).
__device__ __forceinline__ void cp_async16_l1(uint32_t smem_dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(src) : "memory");
}
template <typename T>
__device__ __forceinline__ void copy_pieces(uint32_t to, const char* p, int off, int width) {
  constexpr int kPieces = (kWarpCols * (int)sizeof(T) + 16 + 511) / 512;
  const int lane = threadIdx.x & 31, n = off + width - 16 * lane;
  const char* src = p + (16 * lane - off);
#pragma unroll
  for (int q = 0; q < kPieces; ++q)
    if (512 * q < n) cp_async16_l1(to + 16 * lane + 512 * q, src + 512 * q);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

constexpr int kFwdIds = 512;  // rows of a CTA whose ids wait in shared memory
// units (8 columns) a thread has on their way: 128 bytes
template <typename TW>
__host__ __device__ constexpr int fwd_depth() {
  return sizeof(TW) == 4 ? 4 : 8;
}

// the same in rows' parts of 256 columns, of a warp
template <typename TW>
__host__ __device__ constexpr int any_depth() {
  return sizeof(TW) == 4 ? 4 : 8;
}

// Rows of any alignment: a CTA takes a run of rows, its warps every eighth of
// the rows' parts of 256 columns.  65,536 rows of 901 bfloat16 to float32 in 47 us,
// 79 with loads straight into registers.
template <typename TW, typename TO>
__global__ void __launch_bounds__(kThreads) embed_fwd_any_kernel(
    const int64_t* __restrict__ ids, int64_t n, const TW* __restrict__ w, int64_t V, int64_t d,
    int64_t ldw, float scale, TO* __restrict__ out, int64_t ldo, int rows, int slot_bytes) {
  constexpr int kElt = (int)sizeof(TW), kDepth = any_depth<TW>();
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ int32_t s_id[kFwdIds];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const int nrows = (int)min((int64_t)rows, n - row0);
  for (int k = tid; k < nrows; k += kThreads) {
    const int64_t id = __ldg(ids + row0 + k);
    s_id[k] = id >= 0 && id < V ? (int32_t)id : -1;
  }
  __syncthreads();
  struct At {
    int r, c;  // row of the CTA, first column
  };
  const int parts = (int)((d + kWarpCols - 1) / kWarpCols);
  const int dr = kWarps / parts, dc = (kWarps - dr * parts) * kWarpCols;
  auto step = [&](At& a) {
    a.c += dc;
    a.r += dr;
    if (a.c >= parts * kWarpCols) {
      a.c -= parts * kWarpCols;
      ++a.r;
    }
  };
  At get = {warp / parts, warp % parts * kWarpCols}, put = get;
  const uint32_t ring0 = smem_u32(ring) + warp * (kDepth * slot_bytes);
  const uint32_t ring1 = ring0 + kDepth * slot_bytes;
  const int64_t pitch = ldw * kElt;
  const char* base = reinterpret_cast<const char*>(w);
  auto past = [&](int32_t id, int c) {
    return ((uint32_t)reinterpret_cast<uintptr_t>(base) + (uint32_t)id * (uint32_t)pitch + c * kElt) & 15u;
  };
  auto issue = [&](uint32_t to) {
    if (get.r < nrows) {
      const int32_t id = s_id[get.r];
      if (id >= 0)
        copy_pieces<TW>(to, base + id * pitch + get.c * kElt, (int)past(id, get.c),
                        (int)min((int64_t)kWarpCols, d - get.c) * kElt);
    }
    cp_async_commit();
    step(get);
  };
#pragma unroll 1
  for (int k = 0; k < kDepth; ++k) issue(ring0 + k * slot_bytes);
  uint32_t at = ring0;
  while (put.r < nrows) {
    cp_async_wait<kDepth - 1>();
    __syncwarp();
    // (an id outside the table: NaN whatever is there)
    const int32_t id = s_id[put.r];
    const uint32_t from = at + past(id, put.c) + lane * kElt;
    TO* q = out + (row0 + put.r) * ldo + put.c + lane;
    const float f = id < 0 ? __int_as_float(0x7fc00000) : scale;
    // (32 N columns, or up to as many.  Up to 160 columns five loads per lane, above
    // that eight: 130,000 rows of 130 floats 18.9 us, of 33 18.6, with eight 19.9 and
    // 19.5; 65,536 rows of 901 bfloat16, 133 of them in a row's last part, 37.5 and 38.5)
    auto copy = [&](auto cols, int left) {
      constexpr int N = decltype(cols)::value;
      float x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = lds_elt(from + k * (32 * kElt), TW());
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (32 * k < left) Elt<TO>::store1(q + 32 * k, x[k] * f);
    };
    const int64_t cols = d - put.c;
    if (cols >= kWarpCols)
      copy(std::integral_constant<int, 8>(), kWarpCols);
    else if (cols > 160)
      copy(std::integral_constant<int, 8>(), (int)cols - lane);
    else
      copy(std::integral_constant<int, 5>(), (int)cols - lane);
    __syncwarp();
    step(put);
    issue(at);
    at += slot_bytes;
    if (at == ring1) at = ring0;
  }
  cp_async_wait<0>();
}

// 16-byte aligned rows.  A CTA takes a run of rows; their ids are loaded
// first, and then every thread streams its units of 8 columns through a ring
// of its own in shared memory, kDepth asynchronous copies ahead of its stores.
// The ring costs no registers and needs no barrier (a thread reads back what
// it copied itself), so loads and stores of a CTA overlap all the way: 81,920
// rows of 896 bfloat16 in 31 us; with a CTA's loads in registers, its ids, rows
// and stores one after the other, 55 us.
template <typename TW, typename TO, bool kStream>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(
    const int64_t* __restrict__ ids, int64_t n, const TW* __restrict__ w, int64_t V, int64_t ldw,
    float scale, TO* __restrict__ out, int64_t ldo, int rows, int nu) {
  constexpr int kDepth = fwd_depth<TW>();
  constexpr int kUnit = 8 * (int)sizeof(TW);
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ int32_t s_id[kFwdIds];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const int nrows = (int)min((int64_t)rows, n - row0);
  for (int k = tid; k < nrows; k += kThreads) {
    const int64_t id = __ldg(ids + row0 + k);
    s_id[k] = id >= 0 && id < V ? (int32_t)id : -1;
  }
  __syncthreads();
  const int dr = kThreads / nu, dc = kThreads - dr * nu;
  struct At {
    int r, c;
  };
  auto step = [&](At& a) {
    a.c += dc;
    a.r += dr;
    if (a.c >= nu) {
      a.c -= nu;
      ++a.r;
    }
  };
  At get = {tid / nu, tid - tid / nu * nu}, put = get;
  const uint32_t mine = smem_u32(ring) + tid * kUnit;  // slot k: + k * kThreads * kUnit
  auto issue = [&](int slot) {
    if (get.r < nrows) {
      const int32_t id = s_id[get.r];
      if (id >= 0) {
        const char* src = reinterpret_cast<const char*>(w + id * ldw + 8 * get.c);
        const uint32_t dst = mine + slot * (kThreads * kUnit);
#pragma unroll
        for (int b = 0; b < kUnit; b += 16) cp_async16(dst + b, src + b);
      }
    }
    cp_async_commit();
    step(get);
  };
#pragma unroll
  for (int k = 0; k < kDepth; ++k) issue(k);
  int slot = 0;
  while (put.r < nrows) {
    cp_async_wait<kDepth - 1>();
    Vec8<TW> x;
#pragma unroll
    for (int k = 0; k < Vec8<TW>::kWords; ++k)
      x.v[k] = ld_shared_v4(mine + slot * (kThreads * kUnit) + 16 * k);
    if (s_id[put.r] < 0) x.fill(sizeof(TW) == 4 ? 0x7fc00000u : 0x7fc07fc0u);  // NaN
    x.template store<kStream>(out + (row0 + put.r) * ldo + 8 * put.c, scale);
    step(put);
    issue(slot);
    slot = slot + 1 == kDepth ? 0 : slot + 1;
  }
  cp_async_wait<0>();
}

bool rows_aligned16(const void* p, int64_t ld, size_t esize) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t)ld * esize % 16 == 0;
}

template <typename TW, typename TO>
cudaError_t launch_fwd_t(const EmbedFwdArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const bool vec = a.d % 8 == 0 && rows_aligned16(a.weight, a.ldw, sizeof(TW)) &&
                   rows_aligned16(a.out, a.ldo, sizeof(TO));
  const int nu = (int)((a.d + 7) / 8);
  const TW* w = static_cast<const TW*>(a.weight);
  TO* out = static_cast<TO*>(a.out);
  // runs of rows: 24 CTAs per SM one after the other (31.0 us at 81,920 rows of
  // 896 bfloat16; 6 per SM, all at once, 35.8; 48, 33.5), but not below one ring
  // per thread while two CTAs per SM are left (a warp of unaligned rows: two
  // parts of a row, 5,001 rows of 901 floats 6.2 us; eight, 8.0)
  int64_t rows = (a.n + 24 * (int64_t)dev.sms - 1) / (24 * (int64_t)dev.sms);
  const int64_t parts = (a.d + kWarpCols - 1) / kWarpCols;
  const int64_t full = vec ? (kThreads * fwd_depth<TW>() + nu - 1) / nu
                           : (2 * kWarps + parts - 1) / parts;
  const int64_t spread = (a.n + 2 * (int64_t)dev.sms - 1) / (2 * (int64_t)dev.sms);
  if (rows < full) rows = full < spread ? full : spread;
  if (rows > kFwdIds) rows = kFwdIds;
  const unsigned grid = (unsigned)((a.n + rows - 1) / rows);
  if (!vec) {
    const size_t smem = warp_rings(a.d, sizeof(TW), any_depth<TW>());
    const cudaError_t e = ensure_dynamic_smem((const void*)embed_fwd_any_kernel<TW, TO>, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(embed_fwd_any_kernel<TW, TO>, dim3(grid), dim3(kThreads), smem, st, 1, a.ids,
                      a.n, w, a.V, a.d, a.ldw, a.scale, out, a.ldo, (int)rows,
                      warp_slot(a.d, sizeof(TW)));
  }
  // an output larger than half of L2 is not kept there for its reader
  const bool stream = (size_t)a.n * (size_t)a.d * sizeof(TO) > ((size_t)64 << 20);
  auto kern = stream ? embed_fwd_kernel<TW, TO, true> : embed_fwd_kernel<TW, TO, false>;
  const size_t smem = (size_t)fwd_depth<TW>() * kThreads * 8 * sizeof(TW);
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, 1,
                    a.ids, a.n, w, a.V, a.ldw, a.scale, out, a.ldo, (int)rows, nu);
}

// ---------------------------------------------------------------------------
// backward: sort
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;                   // 9-bit digits
constexpr int kBatch = 4 * kSortThreads;        // elements ranked at a time
constexpr int kMaxTiles = 304;                  // CTAs of a sort pass (two per SM)
constexpr int kMaxPasses = 4;
static_assert(kMaxBins == kSortThreads, "one thread per bin");

constexpr int kMinSegEntries = 8;
constexpr int kMaxSegEntries = 32;

struct SortPlan {
  int bits;       // key bits: ids 0 .. V-1 and the key V of ignored tokens
  int passes;     // radix passes, low digit first
  int dbits;      // bits per digit
  int64_t tile;   // elements per CTA, a multiple of kBatch
  int tiles;
  int seg;            // sorted entries summed by one group of threads
  int64_t seg_tiles;  // such groups
};

// Columns per thread of the summing kernel: 8 side by side of 16-byte aligned
// rows (vec); else 8 of a warp's 256, 32 apart, so that a warp's stores meet.
constexpr int kSumCols = 8;
// Threads per row (whole warps where rows are not aligned), and the columns of
// a row of partial sums: whole CTAs of threads.
int row_threads(int64_t d, bool vec) {
  const int64_t units =
      vec ? (d + kSumCols - 1) / kSumCols : (d + kWarpCols - 1) / kWarpCols * 32;
  return (int)(units < kThreads ? units : kThreads);
}
int64_t padded_cols(int64_t d, bool vec) {
  const int64_t cols = kSumCols * (int64_t)row_threads(d, vec);
  return (d + cols - 1) / cols * cols;
}

SortPlan sort_plan(int64_t n, int64_t V, int64_t d) {
  SortPlan s;
  s.bits = 1;
  while (s.bits < 31 && ((int64_t)1 << s.bits) <= V) ++s.bits;
  s.passes = (s.bits + 8) / 9;
  s.dbits = (s.bits + s.passes - 1) / s.passes;
  int64_t per = (n + kMaxTiles - 1) / kMaxTiles;
  s.tile = (per + kBatch - 1) / kBatch * kBatch;
  if (s.tile < kBatch) s.tile = kBatch;
  s.tiles = (int)((n + s.tile - 1) / s.tile);
  // few tokens: shorter groups, so that there are enough of them (about 512
  // threads on each SM); 4 entries where 8 leave fewer than 64 (777 tokens
  // of 130 columns 11.6 us, 12.8 with 8; 42,115 of 64 columns 32.3, 30.5 with 8)
  s.seg = kMaxSegEntries;
  while (s.seg > kMinSegEntries &&
         (n + s.seg - 1) / s.seg * (padded_cols(d, true) / 8) < kPlanSms * 512)
    s.seg /= 2;
  if (s.seg == kMinSegEntries && (n + 7) / 8 * (padded_cols(d, true) / 8) < kPlanSms * 64) s.seg /= 2;
  s.seg_tiles = (n + s.seg - 1) / s.seg;
  return s;
}

struct BwdLayout {
  size_t key[2], pos[2], hist[kMaxPasses], bad, list, part, total;
};

// header | keys and positions, twice | histograms | flags | partial sums
BwdLayout bwd_layout(int64_t n, int64_t V, int64_t d) {
  const SortPlan s = sort_plan(n, V, d);
  BwdLayout l;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at = align_up(at + bytes, 256);
    return p;
  };
  for (int k = 0; k < 2; ++k) l.key[k] = take(4 * (size_t)n);
  for (int k = 0; k < 2; ++k) l.pos[k] = take(4 * (size_t)n);
  for (int k = 0; k < kMaxPasses; ++k)
    l.hist[k] = take(k < s.passes ? 4 * (size_t)kMaxBins * s.tiles : 0);
  l.bad = take(4 * (size_t)s.tiles);
  l.list = take(8 * (size_t)(s.seg_tiles + 1));
  const int64_t pv = padded_cols(d, true), ps = padded_cols(d, false);
  l.part = take(2 * (size_t)s.seg_tiles * (size_t)(pv > ps ? pv : ps) * 4);
  l.total = at;
  return l;
}

// The rows of dW that the sort's kernels clear beside their own work.  The
// sort is a chain of small latency-bound steps on few SMs, the clearing a
// stream of stores: each kernel of the chain gets CTAs that write its share
// of the zeros, 6.7 TB/s of them.  Every row is cleared (which ids occur is not
// known yet); the rows that occur are written over by the sums.  12,288 tokens
// of 151,936 ids: 87 us a call, 125 us when the rest was cleared after the sort.
struct Clear {
  char* base;      // dense rows: one run of bytes
  int64_t bytes;   // of this kernel's share
  int64_t rows;    // pitched rows: count, width and pitch in bytes
  int64_t width, pitch;
  unsigned first;  // CTAs below it belong to the sort
};
constexpr int64_t kClearBytes = 32768;  // per CTA

__device__ __forceinline__ void clear_rows(const Clear& c) {
  const int64_t k = blockIdx.x - c.first;
  const int nt = blockDim.x;
  if (c.rows == 0) {
    const int64_t a = k * kClearBytes;
    const int64_t n = min(kClearBytes, c.bytes - a);
    char* p = c.base + a;
    // (base is 16-byte aligned; only the last run has a ragged end)
    for (int64_t i = 16 * (int64_t)threadIdx.x; i + 16 <= n; i += 16 * nt)
      st_stream(p + i, make_uint4(0, 0, 0, 0));
    for (int64_t i = n / 16 * 16 + 2 * (int64_t)threadIdx.x; i < n; i += 2 * nt)
      *reinterpret_cast<uint16_t*>(p + i) = 0;
    return;
  }
  const int64_t per = max((int64_t)1, kClearBytes / c.width);
  const int64_t r1 = min(c.rows, (k + 1) * per);
  const uintptr_t any = reinterpret_cast<uintptr_t>(c.base) | (uintptr_t)c.width | (uintptr_t)c.pitch;
  for (int64_t r = k * per; r < r1; ++r) {
    char* row = c.base + r * c.pitch;
    if (any % 16 == 0)
      for (int64_t i = threadIdx.x; i < c.width / 16; i += nt)
        st_stream(row + 16 * i, make_uint4(0, 0, 0, 0));
    else if (any % 4 == 0)
      for (int64_t i = threadIdx.x; i < c.width / 4; i += nt) reinterpret_cast<uint32_t*>(row)[i] = 0;
    else
      for (int64_t i = threadIdx.x; i < c.width / 2; i += nt) reinterpret_cast<uint16_t*>(row)[i] = 0;
  }
}

// Key of an id: ignored tokens sort behind every id.
__device__ __forceinline__ int32_t key_of(int64_t id, int64_t V, int64_t pad_id, int* outside) {
  const bool in = id >= 0 && id < V;
  *outside |= !in && !(pad_id >= 0 && id == pad_id);
  return !in || id == pad_id ? (int32_t)V : (int32_t)id;
}

// First pass over the ids: 32-bit keys, the histogram of each tile's first
// digit, and what the later kernels add to is cleared.
__global__ void __launch_bounds__(kSortThreads) embed_keys_kernel(
    const int64_t* __restrict__ ids, int64_t n, int64_t V, int64_t pad_id, int64_t tile, int dbits,
    int32_t* key, int32_t* hist0, int32_t* hist_rest, int64_t n_rest, uint32_t* bad, int32_t* list,
    const Clear clr) {
  __shared__ int32_t h[kMaxBins];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= clr.first) return clear_rows(clr);
  const int tid = threadIdx.x;
  h[tid] = 0;
  __syncthreads();
  const int64_t all = (int64_t)clr.first * kSortThreads;
  const int64_t me = (int64_t)blockIdx.x * kSortThreads + tid;
  for (int64_t k = me; k < n_rest; k += all) hist_rest[k] = 0;
  if (me == 0) list[0] = 0;
  const int64_t a = (int64_t)blockIdx.x * tile, b = min(a + tile, n);
  const uint32_t mask = (1u << dbits) - 1u;
  int outside = 0;
#pragma unroll 4
  for (int64_t i = a + tid; i < b; i += kSortThreads) {
    const int32_t k = key_of(__ldg(ids + i), V, pad_id, &outside);
    key[i] = k;
    atomicAdd(&h[(uint32_t)k & mask], 1);
  }
  const int any = __syncthreads_or(outside);
  hist0[(int64_t)blockIdx.x * kMaxBins + tid] = h[tid];
  if (tid == 0) bad[blockIdx.x] = any ? kFlagTokenRange : 0u;
}

struct SortShared {
  int32_t base[kMaxBins];
  int32_t wh[kSortWarps][kMaxBins];
  int32_t wsum[kSortWarps];
};

// Exclusive prefix over the bins of `total` (one per thread), plus `before`.
__device__ __forceinline__ void bin_bases(SortShared& sh, int32_t total, int32_t before) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t x = total;
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh.wsum[warp] = x;
  __syncthreads();
  int32_t run = x - total + before;
  for (int k = 0; k < warp; ++k) run += sh.wsum[k];
  sh.base[tid] = run;
}

__device__ __forceinline__ void clear_counts(SortShared& sh) {
#pragma unroll
  for (int k = 0; k < kSortWarps; ++k) sh.wh[k][threadIdx.x] = 0;
}
constexpr int kPerThread = kBatch / kSortThreads;

// A thread's R elements of the batch [at, at + R kSortThreads) below b (a warp's
// are contiguous): keys (-1: none) and positions.
template <int R, typename Load>
__device__ __forceinline__ void load_batch(int64_t at, int64_t b, Load load, int32_t* kk, int32_t* pp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = at + warp * (32 * R) + r * 32 + lane;
    kk[r] = -1;
    pp[r] = 0;
    if (i < b) load(i, kk[r], pp[r]);
  }
}

// Ranks a batch's elements among those of their digit in the same warp, in order
// (lanes with the same digit by one vote per bit), and leaves the warps' counts,
// which are clear before.  (The gradient of 42,115 tokens of 64 columns takes 28.1
// us; with the warp's match instruction, which takes its time for every different
// value, 29.3.)
template <int R>
__device__ __forceinline__ void rank_batch(SortShared& sh, const int32_t* kk, int shift,
                                           uint32_t mask, uint32_t* dg, int32_t* rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t same[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    dg[r] = ((uint32_t)kk[r] >> shift) & mask;
    same[r] = __ballot_sync(0xffffffffu, kk[r] >= 0);
  }
  for (uint32_t bit = 1; bit <= mask; bit <<= 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool on = dg[r] & bit;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      same[r] &= on ? m : ~m;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool live = kk[r] >= 0;
    const uint32_t below = same[r] & ((1u << lane) - 1u);
    const int32_t old = live ? sh.wh[warp][dg[r]] : 0;
    __syncwarp();
    if (live && below == 0) sh.wh[warp][dg[r]] = old + __popc(same[r]);
    __syncwarp();
    rank[r] = old + __popc(below);
  }
  __syncthreads();
}
// The warps' counts of this thread's bin to first positions, from `first` on.
__device__ __forceinline__ int32_t place_counts(SortShared& sh, int32_t first) {
#pragma unroll
  for (int k = 0; k < kSortWarps; ++k) {
    const int32_t c = sh.wh[k][threadIdx.x];
    sh.wh[k][threadIdx.x] = first;
    first += c;
  }
  return first;
}
template <int R, typename Emit>
__device__ __forceinline__ void emit_batch(const SortShared& sh, const int32_t* kk, const int32_t* pp,
                                           const uint32_t* dg, const int32_t* rank, Emit emit) {
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (kk[r] >= 0) emit(kk[r], pp[r], sh.wh[threadIdx.x >> 5][dg[r]] + rank[r]);
  __syncthreads();
}

// One stable radix pass.  Each CTA derives its tile's first output position
// of every digit from the tiles' histograms (all digits below it, then the
// same digit in earlier tiles) and scatters its elements in order.  While it
// does, it counts the next pass's digit per destination tile (integer
// atomics: any order gives the same counts).
__global__ void __launch_bounds__(kSortThreads, 3) embed_scatter_kernel(
    const int32_t* key, const int32_t* pos, int64_t n, int64_t tile, int shift, int dbits,
    const int32_t* hist, int32_t* hist_next, int32_t* key_out, int32_t* pos_out,
    const uint32_t* bad, WsHeader* hdr, const Clear clr) {
  __shared__ SortShared sh;
  const int tid = threadIdx.x;
  const int tiles = (int)clr.first;
  const uint32_t mask = (1u << dbits) - 1u;
  if (blockIdx.x < clr.first) clear_counts(sh);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= clr.first) return clear_rows(clr);
  // (the first batch is on its way while the histograms are added)
  const int64_t a = (int64_t)blockIdx.x * tile, b = min(a + tile, n);
  auto load = [&](int64_t i, int32_t& k, int32_t& p) {
    k = key[i];
    p = pos != nullptr ? pos[i] : (int32_t)i;
  };
  int32_t kk[kPerThread], pp[kPerThread];
  load_batch<kPerThread>(a, b, load, kk, pp);
  const uint32_t tile32 = (uint32_t)tile;  // (n and so tile fit)
  // (16 tiles' counts in flight at a time)
  int32_t before = 0, total = 0;
  for (int t0 = 0; t0 < tiles; t0 += 16) {
    int32_t c[16];
#pragma unroll
    for (int u = 0; u < 16; ++u)
      c[u] = t0 + u < tiles ? hist[(int64_t)(t0 + u) * kMaxBins + tid] : 0;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      before += t0 + u < (int)blockIdx.x ? c[u] : 0;
      total += c[u];
    }
  }
  bin_bases(sh, total, before);
  for (int64_t at = a;;) {
    uint32_t dg[kPerThread];
    int32_t rank[kPerThread];
    rank_batch<kPerThread>(sh, kk, shift, mask, dg, rank);
    sh.base[tid] = place_counts(sh, sh.base[tid]);
    emit_batch<kPerThread>(sh, kk, pp, dg, rank, [&](int32_t k, int32_t p, int32_t to) {
      key_out[to] = k;
      pos_out[to] = p;
      if (hist_next != nullptr)
        atomicAdd(hist_next + (int64_t)((uint32_t)to / tile32) * kMaxBins +
                      (((uint32_t)k >> (shift + dbits)) & mask),
                  1);
    });
    at += kBatch;
    if (at >= b) break;
    clear_counts(sh);
    load_batch<kPerThread>(at, b, load, kk, pp);
  }
  if (bad != nullptr && blockIdx.x == 0) {
    uint32_t f = 0;
    for (int t = tid; t < tiles; t += kSortThreads) f |= bad[t];
    const int any = __syncthreads_or((int)f);
    if (tid == 0) hdr->flags = any ? kFlagTokenRange : 0u;
  }
}

// The whole sort of up to kOneCta tokens by one CTA, R of them per thread: every
// pass ranks all of them and scatters between shared-memory arrays.  4,096 tokens
// of 130 columns take 19.2 us a call, 4,097 by the passes' kernels 22.
constexpr int kOneCta = 4096;
struct OneShared {
  SortShared s;
  int32_t key[2][kOneCta], pos[2][kOneCta];
};
template <int R>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(
    const int64_t* __restrict__ ids, int n, int64_t V, int64_t pad_id, int passes, int dbits,
    int32_t* key_out, int32_t* pos_out, int32_t* list, WsHeader* hdr, const Clear clr) {
  extern __shared__ __align__(16) unsigned char one_raw[];
  OneShared& o = *reinterpret_cast<OneShared*>(one_raw);
  if (blockIdx.x < clr.first) clear_counts(o.s);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= clr.first) return clear_rows(clr);
  const int tid = threadIdx.x;
  const uint32_t mask = (1u << dbits) - 1u;
  int outside = 0;
  int32_t kk[R], pp[R];
  load_batch<R>(
      0, n,
      [&](int64_t i, int32_t& k, int32_t& q) {
        k = key_of(__ldg(ids + i), V, pad_id, &outside);
        q = (int32_t)i;
      },
      kk, pp);
  for (int p = 0; p < passes; ++p) {
    const int shift = p * dbits, to_buf = p & 1;
    uint32_t dg[R];
    int32_t rank[R];
    rank_batch<R>(o.s, kk, shift, mask, dg, rank);
    int32_t total = 0;
#pragma unroll
    for (int k = 0; k < kSortWarps; ++k) total += o.s.wh[k][tid];
    bin_bases(o.s, total, 0);
    place_counts(o.s, o.s.base[tid]);
    const bool last = p + 1 == passes;
    int32_t* ko = last ? key_out : o.key[to_buf];
    int32_t* po = last ? pos_out : o.pos[to_buf];
    emit_batch<R>(o.s, kk, pp, dg, rank, [&](int32_t k, int32_t q, int32_t to) {
      ko[to] = k;
      po[to] = q;
    });
    if (last) break;
    clear_counts(o.s);
    load_batch<R>(
        0, n,
        [&](int64_t i, int32_t& k, int32_t& q) {
          k = ko[i];
          q = po[i];
        },
        kk, pp);
  }
  const int any = __syncthreads_or(outside);
  if (tid == 0) {
    hdr->flags = any ? kFlagTokenRange : 0u;
    list[0] = 0;
  }
}

// ---------------------------------------------------------------------------
// backward: sums of the sorted tokens' rows
// ---------------------------------------------------------------------------

struct SegParams {
  const int32_t* key;
  const int32_t* pos;
  int64_t n, V, d, ldd, ldw, dpad;
  float scale;
  float* part;    // [seg tiles][2][dpad]: an id's rows in a tile that it began before (0), goes on after (1)
  int32_t* list;  // count (8 bytes), then pairs: the tile in which a split id begins, the id
  int seg;          // sorted entries per tile
  int tpr, groups;  // threads per row, rows side by side in a CTA
  int cols;         // columns of one CTA in y
  int slot;         // bytes of a row in a warp's ring (rows that are not aligned)
};

// A thread's 8 columns of a row of dW: contiguous or 32 apart, `left` of the
// row from the first on.
template <typename TW, bool kVec>
__device__ __forceinline__ void write_row(TW* row, int left, bool accumulate, float scale,
                                          const float* acc) {
  constexpr int C = kSumCols, step = 32;
  float x[8];
#pragma unroll
  for (int k = 0; k < C; ++k) x[k] = acc[k] * scale;
  if constexpr (kVec) {
    if (accumulate) {
      Vec8<TW> old;
      old.load(row);
      float o[8];
      old.unpack(o);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] += o[k];
    }
    if (sizeof(TW) == 4 && reinterpret_cast<uintptr_t>(row) % 32 == 0) {
      st_32bytes<false>(row, x);
      return;
    }
#pragma unroll
    for (int k = 0; k < Vec8<TW>::kWords; ++k)
      reinterpret_cast<uint4*>(row)[k] = Elt<TW>::pack(x + k * Elt<TW>::kPerVec);
  } else {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if (k * step >= left) break;
      if (accumulate) {
        if constexpr (sizeof(TW) == 4)
          x[k] += row[k * step];
        else
          x[k] += bf16_bits_to_float(row[k * step]);
      }
      Elt<TW>::store1(row + k * step, x[k]);
    }
  }
}

// Aligned rows that a thread of the summing kernel has on their way, copied
// through a ring of its own in shared memory: 128 bytes of them.
template <typename TD>
__host__ __device__ constexpr int sum_depth() {
  return sizeof(TD) == 4 ? 4 : 8;
}
constexpr int kSumAnyDepth = 6;  // rows of a warp, of any alignment
constexpr int kMaxGroups = 32;

// A group of `tpr` threads takes Q sorted entries (a tile), C columns per
// thread, and writes a row whenever the id changes.  An id that goes on past
// its tile is finished by the group it began in, unless it fills a whole
// further tile: then it is split at the tiles, every tile leaves its partial
// sum, and embed_join_kernel adds them.  Both neighbours decide that from the
// same keys: the id at a tile's first entry a is split iff it began before the
// previous tile (key[a - Q - 1]) or reaches past this one (key[a + Q]).
// HBM-bound at many tokens: 65,536 rows of 896 float32 (235 MB) in 50 us, with
// 8 rows in registers 62 us.  Rows of 901 bfloat16 (65,172 of them): 35 us, 145 with single
// loads into registers.
template <typename TD, typename TW, bool kVec, bool kAcc>
__global__ void __launch_bounds__(kThreads, 4) embed_sum_kernel(const SegParams p,
                                                                const TD* __restrict__ dout,
                                                                TW* dw) {
  extern __shared__ __align__(16) unsigned char sum_ring[];
  __shared__ int32_t s_key[(kMaxGroups + 1) * kMaxSegEntries];
  __shared__ int32_t s_pos[(kMaxGroups + 1) * kMaxSegEntries];
  constexpr int C = kSumCols;
  const int Q = p.seg;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  // keys and positions of the CTA's tiles and of one tile more (for the last
  // one's extension)
  const int64_t base = (int64_t)blockIdx.x * p.groups * Q;
  const int have = (int)min((int64_t)(p.groups + 1) * Q, p.n - base);
  for (int k = tid; k < have; k += kThreads) {
    s_key[k] = p.key[base + k];
    s_pos[k] = p.pos[base + k];
  }
  const int grp = tid / p.tpr, l = tid - grp * p.tpr;
  const int64_t t = (int64_t)blockIdx.x * p.groups + grp;
  const int64_t a = t * Q, b = min(a + Q, p.n);
  const bool live = grp < p.groups && a < p.n;
  const int32_t prev = live && a > 0 ? p.key[a - 1] : -1;
  const int32_t prev2 = live && a > Q ? p.key[a - Q - 1] : -1;
  const int32_t next2 = live && b + Q < p.n ? p.key[b + Q] : -1;
  __syncthreads();
  if (!live) return;
  // first column, and the columns of the CTA from there on
  const int lane = tid & 31, cl = kVec ? 8 * l : l / 32 * kWarpCols + lane;
  const int64_t c0 = (int64_t)blockIdx.y * p.cols + cl;
  const int left = (int)min((int64_t)p.cols, p.d - (int64_t)blockIdx.y * p.cols) - cl;
  if (left + (kVec ? 0 : lane) <= 0) return;  // (a whole warp, where rows are not aligned)
  const int32_t* key = s_key + grp * Q;
  const int32_t* pos = s_pos + grp * Q;
  const int nb = (int)(b - a);  // entries of the tile
  const int32_t first = key[0];
  if (first >= p.V) return;  // ignored tokens from here on
  const int32_t last = key[nb - 1];
  const int32_t next = b < p.n ? key[nb] : -1;
  const bool head = prev == first;
  bool open = head && (prev2 == first || next == first);  // split: this tile's share of it
  const bool goes_on = next == last && last < p.V;
  const bool split = goes_on && (next2 == last || (open && last == first));
  // entries [e0, e1) are this group's: not the ones the tile before finishes,
  // not the ignored ones, and of the next tile those that finish `last`
  int e0 = 0, e1 = nb;
  if (head && !open)
    while (e0 < nb && key[e0] == first) ++e0;
  while (e1 > e0 && key[e1 - 1] >= p.V) --e1;
  if (goes_on && !split)
    while (e1 < nb + Q && a + e1 < p.n && key[e1] == last) ++e1;
  if (e0 >= e1) return;
  // partial sums keep the thread's columns side by side
  float* part = p.part + 2 * t * p.dpad + (int64_t)blockIdx.y * p.cols + C * l;
  float acc[C];
  auto flush_part = [&](int which) {
    float4* q = reinterpret_cast<float4*>(part + which * p.dpad);
#pragma unroll
    for (int c = 0; c < C; c += 4)
      q[c / 4] = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
  };
  int32_t cur = -1;
  auto flush = [&]() {
    if (open)
      flush_part(0);
    else
      write_row<TW, kVec>(dw + cur * p.ldw + c0, left, kAcc, p.scale, acc);
  };
  auto take = [&](int e, const float* v) {
    const int32_t k = key[e];
    if (k != cur) {
      if (cur >= 0) {
        flush();
        open = false;
      }
      cur = k;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = v[c];
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] += v[c];
    }
  };
  if constexpr (kVec) {
    constexpr int kDepth = sum_depth<TD>(), kUnit = 8 * (int)sizeof(TD);
    const uint32_t mine = smem_u32(sum_ring) + tid * kUnit;  // slot k: + k * kThreads * kUnit
    auto issue = [&](int e, int slot) {
      if (e < e1) {
        const char* src = reinterpret_cast<const char*>(dout + (int64_t)pos[e] * p.ldd + c0);
#pragma unroll
        for (int q = 0; q < kUnit; q += 16)
          cp_async16(mine + slot * (kThreads * kUnit) + q, src + q);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kDepth; ++k) issue(e0 + k, k);
    int slot = 0;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      cp_async_wait<kDepth - 1>();
      Vec8<TD> x;
#pragma unroll
      for (int k = 0; k < Vec8<TD>::kWords; ++k)
        x.v[k] = ld_shared_v4(mine + slot * (kThreads * kUnit) + 16 * k);
      float v[8];
      x.unpack(v);
      take(e, v);
      issue(e + kDepth, slot);
      slot = slot + 1 == kDepth ? 0 : slot + 1;
    }
    cp_async_wait<0>();
  } else {
    constexpr int kDepth = kSumAnyDepth, kElt = (int)sizeof(TD);
    const uint32_t ring0 = smem_u32(sum_ring) + tid / 32 * (kDepth * p.slot);
    const uint32_t ring1 = ring0 + kDepth * p.slot;
    const char* col = reinterpret_cast<const char*>(dout + (c0 - lane));  // the warp's first column
    const int width = min(kWarpCols, left + lane) * kElt;
    const int64_t pitch = p.ldd * kElt;
    // bytes of the row's columns behind a 16-byte boundary
    const uint32_t col4 = (uint32_t)reinterpret_cast<uintptr_t>(col), pitch4 = (uint32_t)pitch;
    auto past = [&](int e) { return (col4 + (uint32_t)pos[e] * pitch4) & 15u; };
    auto issue = [&](int e, uint32_t to) {
      if (e < e1) copy_pieces<TD>(to, col + pos[e] * pitch, (int)past(e), width);
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kDepth; ++k) issue(e0 + k, ring0 + k * p.slot);
    uint32_t at = ring0;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      cp_async_wait<kDepth - 1>();
      __syncwarp();
      // (columns behind the row's end: whatever is there, never written)
      const uint32_t from = at + past(e) + lane * kElt;
      float v[C];
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = lds_elt(from + c * (32 * kElt), TD());
      __syncwarp();
      take(e, v);
      issue(e + kDepth, at);
      at += p.slot;
      if (at == ring1) at = ring0;
    }
    cp_async_wait<0>();
  }
  if (split && cur == last) {
    flush_part(open ? 0 : 1);
    if (!open && l == 0 && blockIdx.y == 0)
      reinterpret_cast<int2*>(p.list)[1 + atomicAdd(p.list, 1)] = make_int2((int32_t)t, last);
  } else {
    flush();
  }
}

constexpr int kJoinCols = 128;  // columns of one join item (float4 per lane)
constexpr int kJoinWarps = 16;

// Split ids: the partial sums of their tiles, added per warp over every
// kJoinWarps-th tile and then over the warps, both in order.  A few us as a
// rule; 131,072 tokens of one id (4,096 tiles) take the whole call from 70 us
// (their rows alone) to 143 us.
template <typename TW, bool kVec, bool kAcc>
__global__ void __launch_bounds__(32 * kJoinWarps) embed_join_kernel(const SegParams p, TW* dw) {
  __shared__ float4 s_acc[kJoinWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = p.list[0];
  const int ny = (int)((p.dpad + kJoinCols - 1) / kJoinCols);
  const int64_t items = (int64_t)count * ny;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int2 begin = reinterpret_cast<const int2*>(p.list)[1 + it / ny];
    const int64_t t = begin.x;
    const int32_t v = begin.y;
    const int64_t c = (it % ny) * kJoinCols + 4 * lane;
    // the last tile that begins with the id: the next 32 at once, then by
    // 32-way search (the keys are sorted)
    int64_t last = t + 1, beyond = (p.n + p.seg - 1) / p.seg, stride = 1;
    for (;;) {
      const int64_t k = last + stride * (lane + 1);
      const uint32_t same =
          __ballot_sync(0xffffffffu, k < beyond && p.key[k < beyond ? k * p.seg : 0] == v);
      const int run = __popc(same);
      last += stride * run;
      if (run < 32) beyond = min(beyond, last + stride);
      if (beyond - last <= 1) break;
      stride = max((int64_t)1, (beyond - last) / 32);
    }
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < p.dpad) {
#pragma unroll 8
      for (int64_t k = t + warp; k <= last; k += kJoinWarps) {
        const float4 q = *reinterpret_cast<const float4*>(p.part + (2 * k + (k == t)) * p.dpad + c);
        s.x += q.x;
        s.y += q.y;
        s.z += q.z;
        s.w += q.w;
      }
    }
    __syncthreads();  // the previous item's sums are read
    s_acc[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < p.dpad) {
      for (int k = 1; k < kJoinWarps; ++k) {
        const float4 q = s_acc[k][lane];
        s.x += q.x;
        s.y += q.y;
        s.z += q.z;
        s.w += q.w;
      }
      const float x[4] = {s.x, s.y, s.z, s.w};
      constexpr int C = kSumCols;
      const int64_t cy = c / p.cols;               // the CTA column of embed_sum_kernel
      const int64_t unit = (c - cy * p.cols) / C;  // its thread
      const int o = (int)(c % C);
      const int64_t ncy = min((int64_t)p.cols, p.d - cy * p.cols);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // the partial sums hold each thread's columns side by side
        const int64_t in = kVec ? C * unit + o + k
                                : unit / 32 * kWarpCols + unit % 32 + 32 * (o + k);
        if (in < ncy && unit < p.tpr) {
          TW* q = dw + v * p.ldw + cy * p.cols + in;
          float y = x[k] * p.scale;
          if (kAcc) {
            if constexpr (sizeof(TW) == 4)
              y += *q;
            else
              y += bf16_bits_to_float(*q);
          }
          Elt<TW>::store1(q, y);
        }
      }
    }
  }
}

template <typename TD, typename TW, bool kVec, bool kAcc>
cudaError_t launch_sums(const EmbedBwdArgs& a, SegParams p, const DeviceInfo& dev,
                        cudaStream_t st) {
  const unsigned ny = (unsigned)((p.d + p.cols - 1) / p.cols);
  const int64_t seg_tiles = (p.n + p.seg - 1) / p.seg;
  const int64_t blocks = (seg_tiles + p.groups - 1) / p.groups;
  const size_t ring = kVec ? (size_t)sum_depth<TD>() * kThreads * kSumCols * sizeof(TD)
                           : warp_rings(p.d, sizeof(TD), kSumAnyDepth);
  cudaError_t e = ensure_dynamic_smem((const void*)embed_sum_kernel<TD, TW, kVec, kAcc>, (int)ring);
  if (e != cudaSuccess) return e;
  e = launch_pdl(embed_sum_kernel<TD, TW, kVec, kAcc>, dim3((unsigned)blocks, ny), dim3(kThreads),
                 ring, st, 1, p, static_cast<const TD*>(a.dout), static_cast<TW*>(a.dweight));
  if (e != cudaSuccess || seg_tiles < 2) return e;
  const int64_t items = seg_tiles * ((p.dpad + kJoinCols - 1) / kJoinCols);
  const int64_t grid = items < 4 * (int64_t)dev.sms ? items : 4 * (int64_t)dev.sms;
  return launch_pdl(embed_join_kernel<TW, kVec, kAcc>, dim3((unsigned)grid), dim3(32 * kJoinWarps), 0, st,
                    1, p, static_cast<TW*>(a.dweight));
}

template <typename TD, typename TW>
cudaError_t launch_sums_t(const EmbedBwdArgs& a, const SegParams& p, bool vec,
                          const DeviceInfo& dev, cudaStream_t st) {
  if (vec)
    return a.accumulate ? launch_sums<TD, TW, true, true>(a, p, dev, st)
                        : launch_sums<TD, TW, true, false>(a, p, dev, st);
  return a.accumulate ? launch_sums<TD, TW, false, true>(a, p, dev, st)
                      : launch_sums<TD, TW, false, false>(a, p, dev, st);
}

}  // namespace

cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  if (a.n == 0) return cudaSuccess;
  if (a.wdtype == 0)
    return a.odtype == 0 ? launch_fwd_t<float, float>(a, dev, st) : launch_fwd_t<float, uint16_t>(a, dev, st);
  return a.odtype == 0 ? launch_fwd_t<uint16_t, float>(a, dev, st)
                       : launch_fwd_t<uint16_t, uint16_t>(a, dev, st);
}

size_t embed_workspace_bytes(int64_t n, int64_t V, int64_t d) { return bwd_layout(n, V, d).total; }

cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const SortPlan s = sort_plan(a.n, a.V, a.d);
  const BwdLayout l = bwd_layout(a.n, a.V, a.d);
  char* ws = static_cast<char*>(a.ws);
  auto i32 = [&](size_t off) { return reinterpret_cast<int32_t*>(ws + off); };
  uint32_t* bad = reinterpret_cast<uint32_t*>(ws + l.bad);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  if (a.n == 0) {
    cudaError_t e = cudaMemsetAsync(hdr, 0, sizeof(WsHeader), st);
    if (e != cudaSuccess || a.accumulate) return e;
    const size_t es = a.wdtype == 0 ? 4 : 2;
    return cudaMemset2DAsync(a.dweight, (size_t)a.ldw * es, 0, (size_t)a.d * es, (size_t)a.V, st);
  }
  // the clearing, in equal shares over the sort's kernels
  const size_t we = a.wdtype == 0 ? 4 : 2;
  const bool one = a.n <= kOneCta;
  const int shares = one ? 1 : s.passes + 1;
  const bool dense = a.ldw == a.d && reinterpret_cast<uintptr_t>(a.dweight) % 16 == 0;
  int64_t clear_ctas = 0;
  auto clear_share = [&](int k, unsigned first) {
    Clear c = {};
    c.first = first;
    clear_ctas = 0;
    if (a.accumulate) return c;
    char* base = static_cast<char*>(a.dweight);
    if (dense) {
      const int64_t total = a.V * a.d * (int64_t)we;
      const int64_t runs = (total + kClearBytes - 1) / kClearBytes;
      const int64_t r0 = runs * k / shares, r1 = runs * (k + 1) / shares;
      c.base = base + r0 * kClearBytes;
      c.bytes = (k + 1 == shares ? total : r1 * kClearBytes) - r0 * kClearBytes;
      clear_ctas = r1 - r0;
    } else {
      const int64_t r0 = a.V * k / shares, r1 = a.V * (k + 1) / shares;
      c.base = base + r0 * a.ldw * (int64_t)we;
      c.rows = r1 - r0;
      c.width = a.d * (int64_t)we;
      c.pitch = a.ldw * (int64_t)we;
      const int64_t per = kClearBytes / c.width > 0 ? kClearBytes / c.width : 1;
      clear_ctas = (c.rows + per - 1) / per;
      if (c.rows == 0) c.bytes = 0;
    }
    return c;
  };
  cudaError_t e;
  int out = s.passes & 1;
  if (one) {
    const Clear c = clear_share(0, 1);
    auto kern = a.n <= 2 * kSortThreads   ? embed_sort_kernel<2>
                : a.n <= 4 * kSortThreads ? embed_sort_kernel<4>
                                          : embed_sort_kernel<kOneCta / kSortThreads>;
    e = ensure_dynamic_smem((const void*)kern, (int)sizeof(OneShared));
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)(1 + clear_ctas)), dim3(kSortThreads), sizeof(OneShared), st,
                   1, a.ids, (int)a.n, a.V, a.pad_id, s.passes, s.dbits, i32(l.key[out]),
                   i32(l.pos[out]), i32(l.list), hdr, c);
  } else {
    const int64_t n_rest =
        s.passes > 1 ? (int64_t)(l.hist[s.passes - 1] - l.hist[1]) / 4 + (int64_t)kMaxBins * s.tiles
                     : 0;
    const Clear c = clear_share(0, (unsigned)s.tiles);
    e = launch_pdl(embed_keys_kernel, dim3((unsigned)(s.tiles + clear_ctas)), dim3(kSortThreads), 0,
                   st, 1, a.ids, a.n, a.V, a.pad_id, s.tile, s.dbits, i32(l.key[0]), i32(l.hist[0]),
                   i32(l.hist[1]), n_rest, bad, i32(l.list), c);
    for (int k = 0; k < s.passes && e == cudaSuccess; ++k) {
      const Clear ck = clear_share(k + 1, (unsigned)s.tiles);
      e = launch_pdl(embed_scatter_kernel, dim3((unsigned)(s.tiles + clear_ctas)),
                     dim3(kSortThreads), 0, st, 1, (const int32_t*)i32(l.key[k & 1]),
                     k == 0 ? (const int32_t*)nullptr : (const int32_t*)i32(l.pos[k & 1]), a.n,
                     s.tile, k * s.dbits, s.dbits, (const int32_t*)i32(l.hist[k]),
                     k + 1 < s.passes ? i32(l.hist[k + 1]) : (int32_t*)nullptr,
                     i32(l.key[(k + 1) & 1]), i32(l.pos[(k + 1) & 1]),
                     k == 0 ? (const uint32_t*)bad : (const uint32_t*)nullptr, hdr, ck);
    }
  }
  if (e != cudaSuccess) return e;
  SegParams p = {};
  p.key = i32(l.key[out]);
  p.pos = i32(l.pos[out]);
  p.n = a.n;
  p.V = a.V;
  p.d = a.d;
  p.ldd = a.ldd;
  p.ldw = a.ldw;
  p.scale = a.scale;
  p.part = reinterpret_cast<float*>(ws + l.part);
  p.list = i32(l.list);
  const size_t de = a.ddtype == 0 ? 4 : 2;
  const bool vec = a.d % 8 == 0 && rows_aligned16(a.dout, a.ldd, de) &&
                   rows_aligned16(a.dweight, a.ldw, we);
  p.dpad = padded_cols(a.d, vec);
  p.tpr = row_threads(a.d, vec);
  p.seg = s.seg;
  // rows side by side in a CTA, unless that leaves SMs without one
  const int64_t per = s.seg_tiles / (2 * (int64_t)dev.sms);
  p.groups = kThreads / p.tpr;
  if (p.groups > kMaxGroups) p.groups = kMaxGroups;
  if (p.groups > per) p.groups = per < 1 ? 1 : (int)per;
  p.cols = kSumCols * p.tpr;
  p.slot = warp_slot(a.d, de);
  if (a.ddtype == 0)
    return a.wdtype == 0 ? launch_sums_t<float, float>(a, p, vec, dev, st)
                         : launch_sums_t<float, uint16_t>(a, p, vec, dev, st);
  return a.wdtype == 0 ? launch_sums_t<uint16_t, float>(a, p, vec, dev, st)
                       : launch_sums_t<uint16_t, uint16_t>(a, p, vec, dev, st);
}

}  // namespace grpo
