// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   out[i, :] = s * W[id_i, :]
//   backward  dW[v, :] (+)= s * sum over { i : id_i = v } of dout[i, :]
//
// The backward sorts the tokens by id (a stable radix sort, so the tokens of
// one id stay in position order), sums each id's rows in float32 in that
// order and writes every row of dW once: a sum of tokens' rows, or zeros for
// an id that does not occur.  No floating-point atomics: the order of every
// sum is fixed by n and the ids, so results are bitwise reproducible.
#include "ops.cuh"

namespace grpo {
namespace {

// ---------------------------------------------------------------------------
// element access: 8 columns per thread
// ---------------------------------------------------------------------------

// A thread's 8 columns of a row: contiguous (kVec: 16-byte loads and stores,
// every row 16-byte aligned) or strided by the threads of the row (any
// alignment; neighbouring threads still touch neighbouring elements).
template <typename T, bool kVec>
struct Cols8;

template <>
struct Cols8<uint16_t, true> {
  __device__ static void load(const uint16_t* p, int, int, float* x) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    Elt<uint16_t>::unpack(v, x);
  }
  __device__ static void store(uint16_t* p, int, int, const float* x) {
    *reinterpret_cast<uint4*>(p) = Elt<uint16_t>::pack(x);
  }
  __device__ static void load_rw(const uint16_t* p, int, int, float* x) {
    Elt<uint16_t>::unpack(*reinterpret_cast<const uint4*>(p), x);
  }
};
template <>
struct Cols8<float, true> {
  __device__ static void load(const float* p, int, int, float* x) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    Elt<float>::unpack(a, x);
    Elt<float>::unpack(b, x + 4);
  }
  __device__ static void store(float* p, int, int, const float* x) {
    reinterpret_cast<uint4*>(p)[0] = Elt<float>::pack(x);
    reinterpret_cast<uint4*>(p)[1] = Elt<float>::pack(x + 4);
  }
  __device__ static void load_rw(const float* p, int, int, float* x) {
    Elt<float>::unpack(reinterpret_cast<const uint4*>(p)[0], x);
    Elt<float>::unpack(reinterpret_cast<const uint4*>(p)[1], x + 4);
  }
};
// strided: p points at the thread's first column, `step` apart, `left` columns
// of the row from p on
template <typename T>
struct Cols8<T, false> {
  __device__ static void load(const T* p, int step, int left, float* x) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k * step < left ? Elt<T>::load1(p + k * step) : 0.f;
  }
  __device__ static void load_rw(const T* p, int step, int left, float* x) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = 0.f;
      if (k * step < left) {
        const T v = p[k * step];
        if constexpr (sizeof(T) == 4)
          x[k] = v;
        else
          x[k] = bf16_bits_to_float(v);
      }
    }
  }
  __device__ static void store(T* p, int step, int left, const float* x) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k * step < left) Elt<T>::store1(p + k * step, x[k]);
  }
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

constexpr int kFwdUnroll = 4;  // 8-column units in flight per thread

// One CTA copies `rows` rows; its threads walk the rows' units of 8 columns.
// A strided unit u of a row is columns u, u + nu, ... u + 7 nu.
template <typename TW, typename TO, bool kVec>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(
    const int64_t* __restrict__ ids, int64_t n, const TW* __restrict__ w, int64_t V, int64_t d,
    int64_t ldw, float scale, TO* __restrict__ out, int64_t ldo, int rows, int nu) {
  pdl_wait();
  pdl_trigger();
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const int nrows = (int)min((int64_t)rows, n - row0);
  const int64_t total = (int64_t)nrows * nu;
  for (int64_t base = threadIdx.x; base < total; base += kThreads * kFwdUnroll) {
    float x[kFwdUnroll][8];
    int64_t dst[kFwdUnroll];
    int left[kFwdUnroll];
#pragma unroll
    for (int u = 0; u < kFwdUnroll; ++u) {
      const int64_t k = base + u * kThreads;
      dst[u] = -1;
      if (k < total) {
        const int r = nrows == 1 ? 0 : (int)((uint32_t)k / (uint32_t)nu);
        const int64_t c = k - (int64_t)r * nu;
        const int64_t id = __ldg(ids + row0 + r);
        const int64_t col = kVec ? 8 * c : c;
        left[u] = (int)(d - col);
        dst[u] = (row0 + r) * ldo + col;
        if (id >= 0 && id < V) {
          Cols8<TW, kVec>::load(w + id * ldw + col, nu, left[u], x[u]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[u][e] = __int_as_float(0x7fc00000);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kFwdUnroll; ++u)
      if (dst[u] >= 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] *= scale;
        Cols8<TO, kVec>::store(out + dst[u], nu, left[u], x[u]);
      }
  }
}

bool rows_aligned16(const void* p, int64_t ld, size_t esize) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t)ld * esize % 16 == 0;
}

template <typename TW, typename TO>
cudaError_t launch_fwd_t(const EmbedFwdArgs& a, cudaStream_t st) {
  const bool vec = a.d % 8 == 0 && rows_aligned16(a.weight, a.ldw, sizeof(TW)) &&
                   rows_aligned16(a.out, a.ldo, sizeof(TO));
  const int nu = (int)((a.d + 7) / 8);
  // a CTA's units fill one unrolled step of its threads
  int64_t rows = kThreads * kFwdUnroll / nu;
  if (rows < 1) rows = 1;
  auto kern = vec ? embed_fwd_kernel<TW, TO, true> : embed_fwd_kernel<TW, TO, false>;
  return launch_pdl(kern, dim3((unsigned)((a.n + rows - 1) / rows)), dim3(kThreads), 0, st, 1,
                    a.ids, a.n, static_cast<const TW*>(a.weight), a.V, a.d, a.ldw, a.scale,
                    static_cast<TO*>(a.out), a.ldo, (int)rows, nu);
}

// ---------------------------------------------------------------------------
// backward: sort
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;                   // 9-bit digits
constexpr int kBatch = 4 * kSortThreads;        // elements ranked at a time
constexpr int kPerWarp = kBatch / kSortWarps;   // contiguous elements of one warp
constexpr int kMaxTiles = 304;                  // CTAs of a sort pass (two per SM)
constexpr int kMaxPasses = 4;
static_assert(kMaxBins == kSortThreads, "one thread per bin");

constexpr int kSegEntries = 32;  // sorted entries summed by one group of threads

struct SortPlan {
  int bits;       // key bits: ids 0 .. V-1 and the key V of ignored tokens
  int passes;     // radix passes, low digit first
  int dbits;      // bits per digit
  int64_t tile;   // elements per CTA, a multiple of kBatch
  int tiles;
  int64_t seg_tiles;
};

SortPlan sort_plan(int64_t n, int64_t V) {
  SortPlan s;
  s.bits = 1;
  while (s.bits < 31 && ((int64_t)1 << s.bits) <= V) ++s.bits;
  s.passes = (s.bits + 8) / 9;
  s.dbits = (s.bits + s.passes - 1) / s.passes;
  int64_t per = (n + kMaxTiles - 1) / kMaxTiles;
  s.tile = (per + kBatch - 1) / kBatch * kBatch;
  if (s.tile < kBatch) s.tile = kBatch;
  s.tiles = (int)((n + s.tile - 1) / s.tile);
  s.seg_tiles = (n + kSegEntries - 1) / kSegEntries;
  return s;
}

// Threads per row (8 columns each) of the summing kernel, and the columns of
// its rows of partial sums: whole CTAs of threads.
int row_threads(int64_t d) {
  const int64_t units = (d + 7) / 8;
  return (int)(units < kThreads ? units : kThreads);
}
int64_t padded_cols(int64_t d) {
  const int64_t cols = 8 * (int64_t)row_threads(d);
  return (d + cols - 1) / cols * cols;
}

struct BwdLayout {
  size_t key[2], pos[2], hist[kMaxPasses], bad, present, list, part, total;
  int64_t dpad;
};

// header | keys and positions, twice | histograms | flags | ...
BwdLayout bwd_layout(int64_t n, int64_t V, int64_t d) {
  const SortPlan s = sort_plan(n, V);
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
  l.present = take((size_t)V);
  l.list = take(4 * (size_t)(s.seg_tiles + 1));
  l.dpad = padded_cols(d);
  l.part = take(2 * (size_t)s.seg_tiles * (size_t)l.dpad * 4);
  l.total = at;
  return l;
}

// First pass over the ids: 32-bit keys (ignored tokens sort behind every id),
// the histogram of each tile's first digit, and everything the later kernels
// add to is cleared.
__global__ void __launch_bounds__(kSortThreads) embed_keys_kernel(
    const int64_t* __restrict__ ids, int64_t n, int64_t V, int64_t pad_id, int64_t tile, int dbits,
    int32_t* __restrict__ key, int32_t* __restrict__ hist0, int32_t* __restrict__ hist_rest,
    int64_t n_rest, uint32_t* __restrict__ bad, uint8_t* __restrict__ present, int64_t n_present,
    int32_t* __restrict__ list) {
  __shared__ int32_t h[kMaxBins];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  h[tid] = 0;
  __syncthreads();
  const int64_t all = (int64_t)gridDim.x * kSortThreads;
  const int64_t me = (int64_t)blockIdx.x * kSortThreads + tid;
  for (int64_t k = me; k < n_rest; k += all) hist_rest[k] = 0;
  for (int64_t k = me; k < (n_present + 15) / 16; k += all)
    reinterpret_cast<uint4*>(present)[k] = make_uint4(0, 0, 0, 0);
  if (me == 0) list[0] = 0;
  const int64_t a = (int64_t)blockIdx.x * tile, b = min(a + tile, n);
  const uint32_t mask = (1u << dbits) - 1u;
  int outside = 0;
  for (int64_t i = a + tid; i < b; i += kSortThreads) {
    const int64_t id = __ldg(ids + i);
    const bool in = id >= 0 && id < V;
    const bool skip = !in || id == pad_id;
    outside |= !in && !(pad_id >= 0 && id == pad_id);
    const int32_t k = skip ? (int32_t)V : (int32_t)id;
    key[i] = k;
    atomicAdd(&h[(uint32_t)k & mask], 1);
  }
  const int any = __syncthreads_or(outside);
  hist0[(int64_t)blockIdx.x * kMaxBins + tid] = h[tid];
  if (tid == 0) bad[blockIdx.x] = any ? kFlagTokenRange : 0u;
}

// One stable radix pass.  Each CTA derives its tile's first output position
// of every digit from the tiles' histograms (all digits below it, then the
// same digit in earlier tiles), ranks its elements in order (warp match, then
// a prefix over the warps) and scatters them.  While it does, it counts the
// next pass's digit per destination tile (integer atomics: any order gives
// the same counts).
__global__ void __launch_bounds__(kSortThreads) embed_scatter_kernel(
    const int32_t* key, const int32_t* pos, int64_t n, int64_t tile, int shift, int dbits,
    const int32_t* hist, int32_t* hist_next, int32_t* key_out, int32_t* pos_out,
    const uint32_t* bad, WsHeader* hdr, uint8_t* present, int32_t V) {
  __shared__ int32_t base[kMaxBins];
  __shared__ int32_t wh[kSortWarps][kMaxBins];
  __shared__ int32_t wsum[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = gridDim.x;
  const uint32_t mask = (1u << dbits) - 1u;
  pdl_wait();
  pdl_trigger();
  if (bad != nullptr && blockIdx.x == 0) {
    uint32_t f = 0;
    for (int t = tid; t < tiles; t += kSortThreads) f |= bad[t];
    const int any = __syncthreads_or((int)f);
    if (tid == 0) hdr->flags = any ? kFlagTokenRange : 0u;
  }
  // first output position of digit `tid` in this tile
  int32_t before = 0, total = 0;
#pragma unroll 8
  for (int t = 0; t < tiles; ++t) {
    const int32_t c = hist[(int64_t)t * kMaxBins + tid];
    before += t < (int)blockIdx.x ? c : 0;
    total += c;
  }
  int32_t x = total;
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  int32_t run = x - total + before;
  for (int k = 0; k < warp; ++k) run += wsum[k];
  base[tid] = run;

  const int64_t a = (int64_t)blockIdx.x * tile, b = min(a + tile, n);
  for (int64_t at = a; at < b; at += kBatch) {
#pragma unroll
    for (int k = 0; k < kSortWarps; ++k) wh[k][tid] = 0;
    __syncthreads();
    int32_t kk[kPerWarp / 32], pp[kPerWarp / 32], rank[kPerWarp / 32];
#pragma unroll
    for (int r = 0; r < kPerWarp / 32; ++r) {
      const int64_t i = at + warp * kPerWarp + r * 32 + lane;
      kk[r] = i < b ? key[i] : -1;
      pp[r] = i < b ? (pos != nullptr ? pos[i] : (int32_t)i) : 0;
    }
#pragma unroll
    for (int r = 0; r < kPerWarp / 32; ++r) {
      const bool live = kk[r] >= 0;
      const uint32_t dg = live ? ((uint32_t)kk[r] >> shift) & mask : 0xffffffffu;
      const uint32_t same = __match_any_sync(0xffffffffu, dg);
      const uint32_t below = same & ((1u << lane) - 1u);
      const int32_t old = live ? wh[warp][dg] : 0;
      __syncwarp();
      if (live && below == 0) wh[warp][dg] = old + __popc(same);
      __syncwarp();
      rank[r] = old + __popc(below);
    }
    __syncthreads();
    {
      int32_t first = base[tid];
#pragma unroll
      for (int k = 0; k < kSortWarps; ++k) {
        const int32_t c = wh[k][tid];
        wh[k][tid] = first;
        first += c;
      }
      base[tid] = first;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPerWarp / 32; ++r) {
      if (kk[r] < 0) continue;
      const uint32_t dg = ((uint32_t)kk[r] >> shift) & mask;
      const int32_t to = wh[warp][dg] + rank[r];
      key_out[to] = kk[r];
      pos_out[to] = pp[r];
      if (hist_next != nullptr)
        atomicAdd(hist_next + (int64_t)(to / tile) * kMaxBins +
                      (((uint32_t)kk[r] >> (shift + dbits)) & mask),
                  1);
      if (present != nullptr && kk[r] < V) present[kk[r]] = 1;
    }
    __syncthreads();
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
  const uint8_t* present;
  float* part;    // [seg tiles][2][dpad]: an id's rows in a tile that begins / ends inside the id
  int32_t* list;  // count, then the tiles in which an id begins that ends in a later one
  int64_t seg_blocks;
  int tpr, groups;  // threads per row, rows side by side in a CTA
  int cols;         // columns of one CTA in y (8 per thread of a row)
};

template <typename TW, bool kVec>
__device__ __forceinline__ void write_row(TW* row, int step, int left, bool accumulate,
                                          float scale, const float* acc) {
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = acc[k] * scale;
  if (accumulate) {
    float o[8];
    Cols8<TW, kVec>::load_rw(row, step, left, o);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] += o[k];
  }
  Cols8<TW, kVec>::store(row, step, left, x);
}

constexpr int kSegUnroll = 8;
constexpr int kZeroRows = 16;  // rows of dW one CTA clears

// A group of `tpr` threads sums kSegEntries sorted entries, 8 columns per
// thread, and writes a row whenever the id changes.  Ids that begin before
// or end after the group's entries leave partial sums for
// embed_join_kernel.  CTAs past seg_blocks write the zero rows.
template <typename TD, typename TW, bool kVec, bool kAcc>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const SegParams p,
                                                             const TD* __restrict__ dout,
                                                             TW* __restrict__ dw) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if ((int64_t)blockIdx.x >= p.seg_blocks) {
    const int64_t r0 = ((int64_t)blockIdx.x - p.seg_blocks) * kZeroRows;
    const int nr = (int)min((int64_t)kZeroRows, p.V - r0);
    const int64_t c0 = (int64_t)blockIdx.y * p.cols;
    const int nc = (int)min((int64_t)p.cols, p.d - c0);
    for (int r = 0; r < nr; ++r) {
      if (p.present[r0 + r]) continue;
      TW* row = dw + (r0 + r) * p.ldw + c0;
      if (kVec) {
        for (int k = tid; k < nc * (int)sizeof(TW) / 16; k += kThreads)
          st_stream(reinterpret_cast<char*>(row) + 16 * k, make_uint4(0, 0, 0, 0));
      } else {
        for (int k = tid; k < nc; k += kThreads) row[k] = 0;
      }
    }
    return;
  }
  const int grp = tid / p.tpr, l = tid - grp * p.tpr;
  if (grp >= p.groups) return;
  const int64_t t = (int64_t)blockIdx.x * p.groups + grp;
  const int64_t a = t * kSegEntries, b = min(a + kSegEntries, p.n);
  if (a >= p.n) return;
  int32_t cur = p.key[a];
  if (cur >= p.V) return;  // ignored tokens from here on
  const int64_t c0 = (int64_t)blockIdx.y * p.cols + (kVec ? 8 * l : l);
  const int left = (int)min((int64_t)p.cols, p.d - (int64_t)blockIdx.y * p.cols) - (kVec ? 8 * l : l);
  const int step = p.tpr;
  if (left <= 0) return;
  bool open = a > 0 && p.key[a - 1] == cur;
  // partial sums keep the thread's 8 columns side by side
  float* part = p.part + 2 * t * p.dpad + (int64_t)blockIdx.y * p.cols + 8 * l;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto flush_part = [&](int which) {
    float4* q = reinterpret_cast<float4*>(part + which * p.dpad);
    q[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    q[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  };
  auto flush = [&]() {
    if (open)
      flush_part(0);
    else
      write_row<TW, kVec>(dw + cur * p.ldw + c0, step, left, kAcc, p.scale, acc);
  };
  for (int64_t e = a; e < b && cur < p.V; e += kSegUnroll) {
    int32_t k[kSegUnroll];
    float x[kSegUnroll][8];
#pragma unroll
    for (int u = 0; u < kSegUnroll; ++u) {
      k[u] = e + u < b ? p.key[e + u] : INT32_MAX;
      if (k[u] < p.V)
        Cols8<TD, kVec>::load(dout + (int64_t)p.pos[e + u] * p.ldd + c0, step, left, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kSegUnroll; ++u) {
      if (k[u] == INT32_MAX || cur >= p.V) continue;
      if (k[u] != cur) {
        flush();
        open = false;
        cur = k[u];
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = 0.f;
        if (cur >= p.V) continue;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += x[u][c];
    }
  }
  if (cur >= p.V) return;
  if (b < p.n && p.key[b] == cur) {  // the id goes on in the next tile
    flush_part(open ? 0 : 1);
    if (!open && l == 0 && blockIdx.y == 0) p.list[1 + atomicAdd(p.list, 1)] = (int32_t)t;
  } else {
    flush();
  }
}

constexpr int kJoinCols = 128;  // columns of one join item (float4 per lane)

// Ids that span several tiles: the partial sums of their tiles, added per
// warp over every kWarps-th tile and then over the warps, both in order.
template <typename TW, bool kVec, bool kAcc>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const SegParams p,
                                                              TW* __restrict__ dw) {
  __shared__ float4 s_acc[kWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = p.list[0];
  const int ny = (int)((p.dpad + kJoinCols - 1) / kJoinCols);
  const int64_t items = (int64_t)count * ny;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t t = p.list[1 + it / ny];
    const int64_t c = (it % ny) * kJoinCols + 4 * lane;
    const int64_t next = (t + 1) * kSegEntries;
    const int32_t v = p.key[next];
    // end of the id's entries
    int64_t lo = next + 1, hi = p.n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (p.key[mid] <= v)
        lo = mid + 1;
      else
        hi = mid;
    }
    const int64_t last = (lo - 1) / kSegEntries;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < p.dpad) {
#pragma unroll 4
      for (int64_t k = t + warp; k <= last; k += kWarps) {
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
      for (int k = 1; k < kWarps; ++k) {
        const float4 q = s_acc[k][lane];
        s.x += q.x;
        s.y += q.y;
        s.z += q.z;
        s.w += q.w;
      }
      const float x[4] = {s.x, s.y, s.z, s.w};
      const int64_t cy = c / p.cols;               // the CTA column of embed_sum_kernel
      const int64_t unit = (c - cy * p.cols) / 8;  // its thread
      const int o = (int)(c & 7);
      const int64_t ncy = min((int64_t)p.cols, p.d - cy * p.cols);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // the partial sums hold each thread's 8 columns side by side
        const int64_t in = kVec ? 8 * unit + o + k : unit + (int64_t)(o + k) * p.tpr;
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
  const int64_t seg_tiles = (p.n + kSegEntries - 1) / kSegEntries;
  p.seg_blocks = (seg_tiles + p.groups - 1) / p.groups;
  const int64_t zero_blocks = kAcc ? 0 : (p.V + kZeroRows - 1) / kZeroRows;
  cudaError_t e = launch_pdl(embed_sum_kernel<TD, TW, kVec, kAcc>,
                             dim3((unsigned)(p.seg_blocks + zero_blocks), ny), dim3(kThreads), 0,
                             st, 1, p, static_cast<const TD*>(a.dout), static_cast<TW*>(a.dweight));
  if (e != cudaSuccess || seg_tiles < 2) return e;
  const int64_t items = seg_tiles * ((p.dpad + kJoinCols - 1) / kJoinCols);
  const int64_t grid = items < 4 * (int64_t)dev.sms ? items : 4 * (int64_t)dev.sms;
  return launch_pdl(embed_join_kernel<TW, kVec, kAcc>, dim3((unsigned)grid), dim3(kThreads), 0, st,
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

cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, const DeviceInfo&, cudaStream_t st) {
  if (a.n == 0) return cudaSuccess;
  if (a.wdtype == 0)
    return a.odtype == 0 ? launch_fwd_t<float, float>(a, st) : launch_fwd_t<float, uint16_t>(a, st);
  return a.odtype == 0 ? launch_fwd_t<uint16_t, float>(a, st)
                       : launch_fwd_t<uint16_t, uint16_t>(a, st);
}

size_t embed_workspace_bytes(int64_t n, int64_t V, int64_t d) { return bwd_layout(n, V, d).total; }

cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const SortPlan s = sort_plan(a.n, a.V);
  const BwdLayout l = bwd_layout(a.n, a.V, a.d);
  char* ws = static_cast<char*>(a.ws);
  auto i32 = [&](size_t off) { return reinterpret_cast<int32_t*>(ws + off); };
  uint8_t* present = reinterpret_cast<uint8_t*>(ws + l.present);
  uint32_t* bad = reinterpret_cast<uint32_t*>(ws + l.bad);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  if (a.n == 0) {
    cudaError_t e = cudaMemsetAsync(hdr, 0, sizeof(WsHeader), st);
    if (e != cudaSuccess || a.accumulate) return e;
    const size_t es = a.wdtype == 0 ? 4 : 2;
    return cudaMemset2DAsync(a.dweight, (size_t)a.ldw * es, 0, (size_t)a.d * es, (size_t)a.V, st);
  }
  const int64_t n_rest =
      s.passes > 1 ? (int64_t)(l.hist[s.passes - 1] - l.hist[1]) / 4 + (int64_t)kMaxBins * s.tiles
                   : 0;
  cudaError_t e = launch_pdl(embed_keys_kernel, dim3((unsigned)s.tiles), dim3(kSortThreads), 0, st,
                             1, a.ids, a.n, a.V, a.pad_id, s.tile, s.dbits, i32(l.key[0]),
                             i32(l.hist[0]), i32(l.hist[1]), n_rest, bad, present,
                             a.accumulate ? (int64_t)0 : a.V, i32(l.list));
  for (int k = 0; k < s.passes && e == cudaSuccess; ++k) {
    e = launch_pdl(embed_scatter_kernel, dim3((unsigned)s.tiles), dim3(kSortThreads), 0, st, 1,
                   (const int32_t*)i32(l.key[k & 1]),
                   k == 0 ? (const int32_t*)nullptr : (const int32_t*)i32(l.pos[k & 1]), a.n,
                   s.tile, k * s.dbits, s.dbits, (const int32_t*)i32(l.hist[k]),
                   k + 1 < s.passes ? i32(l.hist[k + 1]) : (int32_t*)nullptr,
                   i32(l.key[(k + 1) & 1]), i32(l.pos[(k + 1) & 1]),
                   k == 0 ? (const uint32_t*)bad : (const uint32_t*)nullptr, hdr,
                   k == 0 && !a.accumulate ? present : (uint8_t*)nullptr, (int32_t)a.V);
  }
  if (e != cudaSuccess) return e;
  SegParams p = {};
  p.key = i32(l.key[s.passes & 1]);
  p.pos = i32(l.pos[s.passes & 1]);
  p.n = a.n;
  p.V = a.V;
  p.d = a.d;
  p.ldd = a.ldd;
  p.ldw = a.ldw;
  p.dpad = l.dpad;
  p.scale = a.scale;
  p.present = present;
  p.part = reinterpret_cast<float*>(ws + l.part);
  p.list = i32(l.list);
  p.tpr = row_threads(a.d);
  p.groups = kThreads / p.tpr;
  p.cols = 8 * p.tpr;
  const size_t de = a.ddtype == 0 ? 4 : 2, we = a.wdtype == 0 ? 4 : 2;
  const bool vec = a.d % 8 == 0 && rows_aligned16(a.dout, a.ldd, de) &&
                   rows_aligned16(a.dweight, a.ldw, we);
  if (a.ddtype == 0)
    return a.wdtype == 0 ? launch_sums_t<float, float>(a, p, vec, dev, st)
                         : launch_sums_t<float, uint16_t>(a, p, vec, dev, st);
  return a.wdtype == 0 ? launch_sums_t<uint16_t, float>(a, p, vec, dev, st)
                       : launch_sums_t<uint16_t, uint16_t>(a, p, vec, dev, st);
}

}  // namespace grpo
