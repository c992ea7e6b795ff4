// The paged 4-bit cache's format (msa_kv4_cache) as the kernels address it.
#pragma once
#include <stdint.h>

#include "msa_internal.h"

namespace msa {

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

// Argument checks shared by the calls, and the view the kernels get.
msa_status kv4_view(const msa_kv4_cache* c, Kv4View* v);

}  // namespace msa
