// The paged 4-bit cache's format (msa_kv4_cache) as the kernels address it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "msa_internal.h"

namespace msa {

constexpr int64_t KV4_MAX_TOKENS = 0x7fff0000;  // of a request
constexpr int KV4_MAX_B = 2048;  // requests of one call: their prefix sums stay in shared memory

struct Kv4View {
  uint8_t* pages;
  int64_t n_pages;
  int32_t page_shift;  // log2 of the tokens of a page
  int32_t Hkv;
  int64_t page_bytes;  // of one KV head
  uint32_t* state;     // [0] error word, [1] arrivals of msa_kv4_slots

  __device__ __forceinline__ int32_t page_tokens() const { return 1 << page_shift; }
  __device__ __forceinline__ int64_t n_slots() const { return n_pages << page_shift; }
};

template <int NG>
struct Kv4Block {  // 16 tokens of one KV head
  static constexpr int BYTES = 2048 + 128 * NG;
  static constexpr int V_CODES = 1024;
  static constexpr int K_SCALES = 2048;
  static constexpr int V_SCALES = 2048 + 64 * NG;
};

__host__ __device__ __forceinline__ constexpr int kv4_v_swizzle(int i) { return 4 * ((i >> 1) & 1); }

constexpr int KV4_PROMPT_MAX_B = 1024;
constexpr int KV4_MAX_CTAS = 160;  // of an attention launch

struct AttendArgs {
  Kv4View c;
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  int64_t q_head, q_row, o_head, o_row;
  const int32_t *table, *kv_lens, *cu_q;
  int64_t table_stride;
  int32_t max_blocks, B, total_q, Hq, group;  // group: query heads of a KV head
  uint32_t group_mul;                         // x / group = (x group_mul) >> (31 + group_shift)
  int32_t group_shift;
  float scale2;                               // softmax scale * log2(e)
  float* lse;
  uint32_t* arrivals;  // [KV4_MAX_CTAS]
  float* partial;      // results of segments over several CTAs
  __device__ __forceinline__ int by_group(int x) const {
    return (int)(((uint64_t)(uint32_t)x * group_mul) >> (31 + group_shift));
  }
  float* heads;        // [KV4_MAX_CTAS][warp][rows][128]: results of segments that began in a warp before
};

// A request's first query row, new tokens and cached tokens, cut to what Q and the table row hold;
// false: something was cut.
__device__ __forceinline__ bool cut_lens(const AttendArgs& a, int32_t q0, int32_t q1, int32_t& n, int32_t& kv) {
  const bool good = q0 >= 0 && q1 >= q0 && q1 <= a.total_q;
  n = good ? q1 - q0 : 0;
  const int32_t most = (int32_t)((int64_t)a.max_blocks << a.c.page_shift);
  const bool fits = kv >= 0 && kv <= most;
  kv = min(max(kv, 0), most);
  return good && fits;
}
__device__ __forceinline__ bool request_lens(const AttendArgs& a, int b, int32_t& q0, int32_t& n, int32_t& kv) {
  q0 = a.cu_q[b];
  const int32_t q1 = a.cu_q[b + 1];
  kv = a.kv_lens[b];
  return cut_lens(a, q0, q1, n, kv);
}

// Many query rows (kv4_prompt.cu), at most KV4_PROMPT_MAX_B requests: two launches; `partial` holds kv4_prompt_partial_bytes().
size_t kv4_prompt_partial_bytes();
cudaError_t launch_kv4_prompt(const AttendArgs& a, int ng, int dev, cudaStream_t st);

inline bool aligned4(std::initializer_list<const void*> pointers) {
  for (const void* p : pointers)
    if (reinterpret_cast<uintptr_t>(p) & 3) return false;
  return true;
}

// Argument checks shared by the calls, and the view the kernels get.
msa_status kv4_view(const msa_kv4_cache* c, Kv4View* v);

}  // namespace msa
