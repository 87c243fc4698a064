// Launchers of the operators around the loss (embedding, gradient clipping,
// draft verification, token statistics, AdamW); defined in embed.cu, gradnorm.cu,
// verify.cu, token_stats.cu and adamw.cu, called by api.cu.  Internal header.
#pragma once

#include "common.cuh"

namespace grpo {

// Asynchronous 16-byte copies global -> shared memory (past L1), by thread.
__device__ __forceinline__ void cp_async16(uint32_t smem_dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// At most N of this thread's groups still on their way.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// max that keeps NaN
__device__ __forceinline__ float max_keep_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The tensor of a table (first[k]: the chunk that tensor k begins with) that a chunk is of.
template <typename Table>
__device__ __forceinline__ int find_tensor(const Table& t, int64_t chunk) {
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

// One element at a shared-memory address, as float.
__device__ __forceinline__ float lds_elt(uint32_t at, uint16_t) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return bf16_bits_to_float(v);
}
__device__ __forceinline__ float lds_elt(uint32_t at, float) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}

template <bool kStream>
__device__ __forceinline__ void st_32bytes(void* p, const float* x) {
  if (kStream)
    asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]),
                 "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  else
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]),
                 "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

// 8 consecutive elements (16-byte aligned) as they are stored, in registers.
template <typename TI>
struct Vec8 {
  static constexpr int kWords = sizeof(TI) / 2;  // of 16 bytes
  uint4 v[kWords];
  __device__ __forceinline__ void load(const TI* p) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) v[k] = reinterpret_cast<const uint4*>(p)[k];
  }
  __device__ __forceinline__ void fill(uint32_t word) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) v[k] = make_uint4(word, word, word, word);
  }
  __device__ __forceinline__ void unpack(float* x) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) Elt<TI>::unpack(v[k], x + k * Elt<TI>::kPerVec);
  }
  // times coef, rounded to TO; kStream: evict-first stores.  8 floats as one
  // store where they are 32-byte aligned: two of 16 bytes by neighbours would
  // each write half of every 32-byte sector (65,172 rows of 896 bfloat16 looked
  // up into float32: 37 us, 55 with two).
  template <bool kStream, typename TO>
  __device__ __forceinline__ void store(TO* q, float coef) const {
    float x[8];
    unpack(x);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] *= coef;
    if (sizeof(TO) == 4 && reinterpret_cast<uintptr_t>(q) % 32 == 0) {
      st_32bytes<kStream>(q, x);
      return;
    }
#pragma unroll
    for (int k = 0; k < (int)sizeof(TO) / 2; ++k) {
      const uint4 w = Elt<TO>::pack(x + k * Elt<TO>::kPerVec);
      if (kStream)
        st_stream(reinterpret_cast<uint4*>(q) + k, w);
      else
        reinterpret_cast<uint4*>(q)[k] = w;
    }
  }
};

// SMs that plans are made for which the workspace's size depends on (its size is
// asked for without a device).
constexpr int kPlanSms = 152;

// ---- embedding lookup and its gradient (embed.cu) ---------------------------

struct EmbedFwdArgs {
  const int64_t* ids;
  int64_t n;
  const void* weight;
  int wdtype;  // 0 f32, 1 bf16
  int64_t V, d, ldw;
  float scale;
  void* out;
  int odtype;
  int64_t ldo;
};
cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, const DeviceInfo& d, cudaStream_t st);

struct EmbedBwdArgs {
  const int64_t* ids;
  int64_t n;
  const void* dout;
  int ddtype;
  int64_t V, d, ldd;
  float scale;
  int64_t pad_id;  // negative: none
  void* dweight;
  int wdtype;
  int64_t ldw;
  bool accumulate;
  void* ws;
};
size_t embed_workspace_bytes(int64_t n, int64_t V, int64_t d);
cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, const DeviceInfo& d, cudaStream_t st);

// ---- gradient norm and clipping (gradnorm.cu) --------------------------------

struct GradTensor {
  const void* data;
  void* out;
  int64_t numel;
  int dt;  // bit 0: data is bf16, bit 1: out is bf16
};
struct ClipArgs {
  const GradTensor* tensors;  // host
  int64_t count;
  int type;  // 0: L2, 1: max |g|
  float max_norm, eps;
  bool norm_only;
  float* stats;  // norm, coefficient
  void* ws;
};
size_t grad_norm_workspace_bytes(int64_t count);
cudaError_t launch_clip(const ClipArgs& a, const DeviceInfo& d, cudaStream_t st);

// ---- verification of drafted tokens (verify.cu) -------------------------------

struct VerifyArgs {
  const void* target;  // [N, K + 1, V], row pitch tld, sequence pitch tls
  const void* draft;   // [N, K, V] or null
  int dtype;
  int64_t N, K, V, tld, tls, dld, dls;
  const int64_t* tokens;  // [N, K]
  const int32_t* lens;    // [N] or null (K each)
  const float* u;         // [N, K]
  const float* noise;     // [N, V], row pitch nld
  int64_t nld;
  const float* temperature;  // [N] or null (1)
  int64_t* out_tokens;       // [N, K + 1]
  int32_t* n_accepted;       // [N]
  float* logp;               // [N, K + 1]
  void* ws;
};
size_t verify_workspace_bytes(int64_t N, int64_t K);
cudaError_t launch_verify(const VerifyArgs& a, const DeviceInfo& d, cudaStream_t st);

// ---- token statistics of logits and their gradient (token_stats.cu) -------------

constexpr int kMaxTop = 32;  // alternatives per row

struct TokenStatsArgs {
  const void* logits;
  int dtype;                           // 0 f32, 1 bf16
  int64_t N, R, V, seq, row;           // rows at i * seq + j * row
  const int64_t* tokens;               // at i * token_seq + j * token_row
  int64_t token_seq, token_row;
  const int32_t* lens;                 // [N] or null (R each)
  const float* temperature;            // [N] or null (1)
  int top;
  float* logp;                         // [N, R]
  float* entropy;                      // [N, R]
  float* norm;                         // [N, R, 2]: largest logit, log of the sum
  int64_t* top_tokens;                 // [N, R, top]
  float* top_logp;
  void* ws;
};
size_t token_stats_workspace_bytes(int64_t N, int64_t R);
cudaError_t launch_token_stats(const TokenStatsArgs& a, const DeviceInfo& d, cudaStream_t st);

struct TokenStatsBwdArgs {
  const void* logits;
  int dtype;
  int64_t N, R, V, seq, row;
  const int64_t* tokens;  // null without grad_logp
  int64_t token_seq, token_row;
  const int32_t* lens;
  const float* temperature;
  const float* norm;
  const float* entropy;       // null without grad_entropy
  const float* grad_logp;     // or null
  const float* grad_entropy;  // or null
  void* dlogits;
  int64_t dseq, drow;
};
cudaError_t launch_token_stats_bwd(const TokenStatsBwdArgs& a, const DeviceInfo& d,
                                   cudaStream_t st);

// ---- AdamW over many tensors (adamw.cu) -------------------------------------------

constexpr int kStateBlock = 256;  // elements that share the scales of 8-bit states

struct AdamwTensor {
  void* param;
  float* master;
  const void* grad;
  void* avg;
  void* sq;
  float* scales;
  int64_t numel;
  int dt;  // bit 0: param is bf16, bit 1: grad is bf16
};
struct AdamwArgs {
  const AdamwTensor* tensors;  // host
  int64_t count;
  bool eight;  // states in 8 bits
  int64_t step;
  const int64_t* step_dev;
  double lr;
  const float* lr_dev;
  double beta1, beta2, eps, decay;
  const float* norm;  // [norm, ...] or null
  double max_norm, norm_eps;
};
cudaError_t launch_adamw(const AdamwArgs& a, const DeviceInfo& d, cudaStream_t st);

}  // namespace grpo
