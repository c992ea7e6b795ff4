// The paged 4-bit cache: block tables and slot maps from request lengths, release, the quantising
// write and the read back.  The format is msa_kv4_cache's.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "kv4.cuh"
#include "msa_internal.h"

namespace msa {

msa_status kv4_view(const msa_kv4_cache* c, Kv4View* v) {
  if (!c || !c->pages || !c->state || c->n_pages < 1 || c->n_pages > 0x7fffffff) return MSA_ERR_INVALID_ARG;
  const size_t bytes = msa_kv4_page_bytes(c->page_tokens, c->group);
  if (!bytes || c->Hkv < 1 || c->Hkv > 1024) return MSA_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(c->pages) | reinterpret_cast<uintptr_t>(c->state)) & 15) return MSA_ERR_ALIGN;
  v->pages = static_cast<uint8_t*>(c->pages);
  v->n_pages = c->n_pages;
  v->page_shift = 0;
  while ((1 << v->page_shift) < c->page_tokens) ++v->page_shift;
  v->Hkv = c->Hkv;
  v->page_bytes = (int64_t)bytes;
  v->state = static_cast<uint32_t*>(c->state);
  return MSA_OK;
}

namespace {

// ---------------------------------------------------------------------------------------
// slot maps
// ---------------------------------------------------------------------------------------
constexpr int SLOT_THREADS = 512;

// Inclusive scans of N values per thread over the block of SLOT_THREADS (every thread calls), and their totals.
// `sums`: [N][SLOT_THREADS / 32].
template <int N>
__device__ __forceinline__ void block_scan(int64_t (&x)[N], int64_t (&total)[N], int64_t* sums) {
  constexpr int WARPS = SLOT_THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] += y;
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < N; ++k) sums[k * WARPS + warp] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    // every warp adds up the warps before it, and all of them
    int64_t s = lane < WARPS ? sums[k * WARPS + lane] : 0, before = lane < warp ? s : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    x[k] += before;
    total[k] = s;
  }
  __syncthreads();  // `sums` is free again
}

// Largest b in [0, n) with cum[b] <= x (cum ascending, cum[0] = 0).
__device__ __forceinline__ int find_last(const int32_t* cum, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (cum[m] <= x) lo = m;
    else hi = m;
  }
  return lo;
}

struct SlotArgs {
  Kv4View c;
  const int32_t *kv_lens, *new_lens, *free_pages, *n_free;
  int32_t *block_table, *kv_out, *n_free_out, *cu_new, *positions;
  int64_t* slots;
  int64_t table_stride, capacity;
  int32_t B, max_blocks, whole;
};

// Every block scans the lengths for itself (B ints, one or a few per thread) and then takes its
// share of the tokens and of the new pages by a search in the two running sums; nothing is passed
// between blocks.  kv_lens_out and n_free_out may be the inputs: they are written by the block
// that arrives last, when every block has read them.  Bound by launch latency for a decode batch (256
// requests: 4.4 us in a graph, 5.2 with a scan for each sum); for prompts by the searches behind the 12 bytes
// written per token (0.73 M tokens of 7 requests: 8.8 us; 10.2 where every block waited for its arrival's answer).
__global__ void __launch_bounds__(SLOT_THREADS) kv4_slots_kernel(const SlotArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* cum_new = sm;                      // [B + 1]
  int32_t* cum_page = cum_new + a.B + 1;      // [B + 1]: pages wanted by the requests before b
  int32_t* kv = cum_page + a.B + 1;           // [B]
  __shared__ int64_t sums[2 * SLOT_THREADS / 32];
  __shared__ int last, bad;
  const int P = a.c.page_shift;
  // the first lengths are asked for together with the count
  int64_t n_free = *a.n_free;
  int32_t next_have = (int)threadIdx.x < a.B ? a.kv_lens[threadIdx.x] : 0;
  int32_t next_new = (int)threadIdx.x < a.B ? a.new_lens[threadIdx.x] : 0;
  if (threadIdx.x == 0) bad = n_free < 0 || n_free > a.c.n_pages;
  n_free = min(max(n_free, (int64_t)0), a.c.n_pages);
  __syncthreads();
  int64_t run_new = 0, run_page = 0;
  for (int b0 = 0; b0 < a.B; b0 += SLOT_THREADS) {
    const int b = b0 + threadIdx.x;
    int64_t n = 0, pages = 0;
    if (b < a.B) {
      const int64_t have = next_have;
      n = next_new;
      if (b + SLOT_THREADS < a.B) next_have = a.kv_lens[b + SLOT_THREADS], next_new = a.new_lens[b + SLOT_THREADS];
      if (have < 0 || n < 0) bad = 1;
      if (n < 0) n = 0;
      kv[b] = (int32_t)have;
      if (have >= 0) {
        const int64_t need = (have + n + (1 << P) - 1) >> P;
        if (need > a.max_blocks) {
          bad = 1;
          pages = -1;
        } else {
          pages = need - ((have + (1 << P) - 1) >> P);
        }
      } else {
        pages = -1;
      }
    }
    // a request that fits no row is marked by the sign of its length and wants no page
    const bool refused = pages < 0;
    int64_t x[2] = {n, refused ? 0 : pages}, all[2];
    block_scan(x, all, sums);
    const int64_t cn = x[0] + run_new, cp = x[1] + run_page;
    if (b < a.B) {
      if (cn > 0x7fffffff || cp > 0x7fffffff) bad = 1;
      cum_new[b + 1] = (int32_t)min(cn, (int64_t)0x7fffffff);
      // a request that passes the map's end wants more pages than there are, and so do all after it
      cum_page[b + 1] = a.whole && cn > a.capacity ? 0x7fffffff : (int32_t)min(cp, (int64_t)0x7fffffff);
      if (refused) kv[b] = kv[b] | (int32_t)0x80000000;
    }
    run_new += all[0];
    run_page += all[1];
  }
  if (threadIdx.x == 0) cum_new[0] = cum_page[0] = 0;
  __syncthreads();
  // this block has read every length: the last block to say so may overwrite them.  One thread asks, and
  // the answer is waited for at the end
  uint32_t before = 0;
  if (gridDim.x > 1 && threadIdx.x == SLOT_THREADS - 1) {
    __threadfence();
    before = atomicAdd(a.c.state + 1, 1u);
  }
  const auto served = [&](int b) { return kv[b] >= 0 && cum_page[b + 1] <= n_free; };

  const int64_t total = min((int64_t)cum_new[a.B], a.capacity);
  if (threadIdx.x == 0 && (cum_new[a.B] > a.capacity || cum_page[a.B] > n_free)) bad = 1;
  const int64_t step = (int64_t)gridDim.x * SLOT_THREADS;
  for (int64_t t = (int64_t)blockIdx.x * SLOT_THREADS + threadIdx.x; t < total; t += step) {
    const int b = find_last(cum_new, a.B, (int32_t)t);
    // (a refused request's length may already be written back: as it was)
    const int32_t have = kv[b] >= 0 ? kv[b] : a.kv_lens[b], pos = (int32_t)((uint32_t)have + (uint32_t)(t - cum_new[b]));
    int64_t slot = -1;
    if (served(b)) {
      const int32_t blk = pos >> P, held = (int32_t)(((int64_t)have + (1 << P) - 1) >> P);
      const int32_t page = blk < held ? a.block_table[b * a.table_stride + blk]
                                      : a.free_pages[n_free - 1 - (cum_page[b] + blk - held)];
      if (page >= 0 && page < a.c.n_pages) slot = ((int64_t)page << P) + (pos & ((1 << P) - 1));
      else bad = 1;
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  const int64_t pages = min((int64_t)cum_page[a.B], n_free);
  for (int64_t k = (int64_t)blockIdx.x * SLOT_THREADS + threadIdx.x; k < pages; k += step) {
    const int b = find_last(cum_page, a.B, (int32_t)k);
    if (!served(b)) continue;
    const int32_t held = (int32_t)(((int64_t)kv[b] + (1 << P) - 1) >> P);
    a.block_table[b * a.table_stride + held + (int32_t)(k - cum_page[b])] = a.free_pages[n_free - 1 - k];
  }
  if (threadIdx.x == SLOT_THREADS - 1) last = before == gridDim.x - 1;
  __syncthreads();
  if (last) {
    int64_t taken = 0;
    for (int b = threadIdx.x; b < a.B; b += SLOT_THREADS) {
      const int32_t n = cum_new[b + 1] - cum_new[b];
      // a refused negative length is handed back as it came
      a.kv_out[b] = kv[b] >= 0 ? kv[b] + (served(b) ? n : 0) : a.kv_lens[b];
      a.cu_new[b + 1] = cum_new[b + 1];
      if (cum_page[b + 1] <= n_free) taken = max(taken, (int64_t)cum_page[b + 1]);
    }
    // the pages handed out are the largest running sum that fits
    for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = taken;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 0; w < SLOT_THREADS / 32; ++w) taken = max(taken, sums[w]);
      a.cu_new[0] = 0;
      *a.n_free_out = (int32_t)(n_free - taken);
      if (gridDim.x > 1) a.c.state[1] = 0;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && bad) atomicOr(a.c.state, DEV_ERR_BOUNDS);
}

struct ReleaseArgs {
  Kv4View c;
  const int32_t* ids;
  int32_t *kv_lens, *block_table, *free_pages, *n_free;
  int64_t table_stride;
  int32_t n, B, max_blocks;
};

// One block: a running sum of the released requests' pages gives each its place on the stack; where an entry named no
// page, the pushed ones then close up.  (Looked over before they are pushed, 65536 entries took 165 us instead of 95:
// a search of the running sum for every entry, twice.)
__global__ void __launch_bounds__(SLOT_THREADS) kv4_release_kernel(const ReleaseArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* ids = sm;            // [n]
  int32_t* cum = ids + a.n;     // [n + 1]: entries of the requests before i
  int32_t* good = cum + a.n + 1;  // [n + 1]: those of them that name a page
  __shared__ int64_t sums[SLOT_THREADS / 32];
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  for (int i = threadIdx.x; i < a.n; i += SLOT_THREADS) ids[i] = a.ids[i];
  __syncthreads();
  int64_t n_free = *a.n_free;
  if (n_free < 0 || n_free > a.c.n_pages) {
    if (threadIdx.x == 0) bad = 1;
    n_free = n_free < 0 ? 0 : a.c.n_pages;
  }
  int64_t run = 0;
  for (int i0 = 0; i0 < a.n; i0 += SLOT_THREADS) {
    const int i = i0 + threadIdx.x;
    int64_t pages = 0;
    if (i < a.n) {
      const int32_t id = ids[i];
      bool ok = id >= 0 && id < a.B;
      if (!ok) bad = 1;
      for (int j = 0; ok && j < i; ++j) ok = ids[j] != id;  // named before: counted there
      if (ok) {
        const int64_t len = a.kv_lens[id];
        pages = len > 0 ? (len + a.c.page_tokens() - 1) >> a.c.page_shift : 0;
        if (len < 0 || pages > a.max_blocks) bad = 1;
        pages = min(pages, (int64_t)a.max_blocks);
      }
    }
    int64_t x[1] = {pages}, all[1];
    block_scan(x, all, sums);
    if (i < a.n) cum[i + 1] = (int32_t)min(x[0] + run, (int64_t)0x7fffffff);
    run += all[0];
  }
  if (threadIdx.x == 0) cum[0] = 0;
  __syncthreads();
  const int64_t room = a.c.n_pages - n_free, total = min(run, (int64_t)0x7fffffff);
  const auto entry_of = [&](int64_t k, int i) { return a.block_table + ids[i] * a.table_stride + (k - cum[i]); };
  const auto names_page = [&](int32_t page) { return page >= 0 && page < a.c.n_pages; };
  int64_t pushed = total;
  if (run <= room) {
    bool broken = false;
    for (int64_t k = threadIdx.x; k < total; k += SLOT_THREADS) {
      int32_t* entry = entry_of(k, find_last(cum, a.n, (int32_t)k));
      const int32_t page = *entry;
      broken |= !names_page(page);
      a.free_pages[n_free + k] = page;  // behind the stack's top until n_free says otherwise
      *entry = -1;
    }
    for (int i = threadIdx.x; i < a.n; i += SLOT_THREADS)
      if (ids[i] >= 0 && ids[i] < a.B) a.kv_lens[ids[i]] = 0;
    if (__syncthreads_or(broken)) {
      if (threadIdx.x == 0) bad = 1;
      pushed = 0;
      for (int64_t k0 = 0; k0 < total; k0 += SLOT_THREADS) {
        const int32_t page = k0 + threadIdx.x < total ? a.free_pages[n_free + k0 + threadIdx.x] : -1;
        int64_t x[1] = {names_page(page)}, all[1];
        block_scan(x, all, sums);  // every page of these is read
        if (names_page(page)) a.free_pages[n_free + pushed + x[0] - 1] = page;
        pushed += all[0];
      }
    }
  } else {
    if (threadIdx.x == 0) bad = 1;
    for (int i = threadIdx.x; i <= a.n; i += SLOT_THREADS) good[i] = 0;
    __syncthreads();
    for (int64_t k = threadIdx.x; k < total; k += SLOT_THREADS) {
      const int i = find_last(cum, a.n, (int32_t)k);
      if (names_page(*entry_of(k, i))) atomicAdd(good + i + 1, 1);
    }
    __syncthreads();
    run = 0;
    for (int i0 = 0; i0 < a.n; i0 += SLOT_THREADS) {
      const int i = i0 + threadIdx.x;
      int64_t x[1] = {i < a.n ? good[i + 1] : 0}, all[1];
      block_scan(x, all, sums);
      if (i < a.n) good[i + 1] = (int32_t)min(x[0] + run, (int64_t)0x7fffffff);
      run += all[0];
    }
    __syncthreads();
    // the requests before the first whose pages the stack has no room for; their entries in order
    const auto released = [&](int i) { return good[i + 1] <= room; };
    pushed = 0;
    for (int64_t k0 = 0; k0 < total; k0 += SLOT_THREADS) {
      const int64_t k = k0 + threadIdx.x;
      const int i = k < total ? find_last(cum, a.n, (int32_t)k) : 0;
      const bool mine = k < total && released(i);
      const int32_t page = mine ? *entry_of(k, i) : -1;
      int64_t x[1] = {names_page(page)}, all[1];
      block_scan(x, all, sums);
      if (names_page(page)) a.free_pages[n_free + pushed + x[0] - 1] = page;
      if (mine) *entry_of(k, i) = -1;
      pushed += all[0];
    }
    for (int i = threadIdx.x; i < a.n; i += SLOT_THREADS)
      if (ids[i] >= 0 && ids[i] < a.B && released(i)) a.kv_lens[ids[i]] = 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    *a.n_free = (int32_t)(n_free + pushed);
    if (bad) atomicOr(a.c.state, DEV_ERR_BOUNDS);
  }
}

// ---------------------------------------------------------------------------------------
// write and read
// ---------------------------------------------------------------------------------------
constexpr int ROW_THREADS = 128;

struct RowArgs {
  Kv4View c;
  __nv_bfloat16 *K, *V;
  int64_t k_head, k_row, v_head, v_row;
  const int64_t* slots;
  int64_t T;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Sixteen channels of a row (lane l of 8: channels 16 l .. 16 l + 15) to sixteen codes in channel
// order, and the group's (step, lo) word.  Smallest and largest value are found together, as the
// smallest of x and of -x in the two halves of a word; a NaN in either is kept.  The product
// (x - lo) * r is rounded to a whole number in one step, by adding 1.5 * 2^23 in the same fused
// operation: a value next to a border falls on its own side, as it would in 64 bits.
template <int NG>
__device__ __forceinline__ uint2 quantise16(const uint4 (&v)[2], uint32_t& scale_word) {
  constexpr uint32_t SIGNS = 0x80008000u;
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  uint32_t lo2 = w[0], hi2 = w[0] ^ SIGNS;
#pragma unroll
  for (int i = 1; i < 8; ++i) lo2 = min2_nan(lo2, w[i]), hi2 = min2_nan(hi2, w[i] ^ SIGNS);
  uint32_t both = min2_nan(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));  // low half lo, high half -hi
#pragma unroll
  for (int o = 4 / NG; o > 0; o >>= 1) both = min2_nan(both, __shfl_xor_sync(0xffffffffu, both, o));
  const float lo = bf_lo(both), range = -bf_hi(both) - lo;
  // range / 15, correctly rounded: a product with the rounded reciprocal and one correction by the
  // exact remainder (Markstein, 1990)
  const float q0 = range * (1.f / 15.f);
  const float q = fmaf(fmaf(-15.f, q0, range), 1.f / 15.f, q0);
  float step = __bfloat162float(__float2bfloat16_rn(q));
  if (step < 0x1p-126f) step = 0.f;
  const float r = step > 0.f ? __frcp_rn(step) : 0.f;
  // a code is the low bits of the sum (no larger than 15: step is within 2^-9 of range / 15, so the
  // largest product is below 15.06); shifted sums added up hold the codes and a constant
  uint2 code = make_uint2(0u - 0x4b400000u * 0x11111111u, 0u - 0x4b400000u * 0x11111111u);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = (e & 1) ? bf_hi(w[e / 2]) : bf_lo(w[e / 2]), y = (e & 1) ? bf_hi(w[4 + e / 2]) : bf_lo(w[4 + e / 2]);
    code.x += __float_as_uint(fmaf(__fsub_rn(x, lo), r, 12582912.f)) << (4 * e);
    code.y += __float_as_uint(fmaf(__fsub_rn(y, lo), r, 12582912.f)) << (4 * e);
  }
  scale_word = (__float_as_uint(step) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
  if (!(range < __int_as_float(0x7f800000))) scale_word = 0x7fc07fc0u, code = make_uint2(0, 0);
  return code;
}

// LANES lanes take one (token, KV head) row of K and of V; the rows of a group are one head's, UNROLL
// neighbouring tokens in flight, neighbouring groups have neighbouring heads.  Their slots, -1 where
// there is nothing to do.
template <int LANES, int UNROLL>
__device__ __forceinline__ void row_item(const RowArgs& a, int64_t& t0, int& h, int64_t (&slot)[UNROLL]) {
  const int64_t item = (int64_t)blockIdx.x * (ROW_THREADS / LANES) + threadIdx.x / LANES;
  const int64_t run = item / a.c.Hkv;
  h = (int)(item - run * a.c.Hkv);
  t0 = run * UNROLL;
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    slot[u] = t0 + u < a.T ? a.slots[t0 + u] : -1;
    if (slot[u] >= a.c.n_slots()) {
      if (threadIdx.x % LANES == 0) atomicOr(a.c.state, DEV_ERR_BOUNDS);
      slot[u] = -1;
    }
  }
}

template <int NG>
__device__ __forceinline__ uint8_t* row_block(const Kv4View& c, int64_t slot, int h) {
  return c.pages + ((slot >> c.page_shift) * c.Hkv + h) * c.page_bytes +
         ((slot & (c.page_tokens() - 1)) >> 4) * Kv4Block<NG>::BYTES;
}

constexpr int APPEND_LANES = 8, APPEND_UNROLL = 2;

// 512 bytes read and 2 (64 + 4 NG) written per row, by 8 lanes of 16 channels: what is worked out once
// a group (its extremes, the step, the reciprocal) costs as much as two rows' codes.  131072 tokens, 4 heads,
// groups of 64: 61 us, 5.7 TB/s (a copy: 6.4), the schedulers issuing 77 % of the time; with 16 lanes of 8
// channels, write and read back took 154 us instead of 133.
template <int NG>
__global__ void __launch_bounds__(ROW_THREADS) kv4_append_kernel(const RowArgs a) {
  using Blk = Kv4Block<NG>;
  constexpr int U = APPEND_UNROLL;
  const int l = threadIdx.x % APPEND_LANES;
  int64_t t0, slot[U];
  int h;
  row_item<APPEND_LANES>(a, t0, h, slot);
  uint4 kx[U][2], vx[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      kx[u][i] = vx[u][i] = make_uint4(0, 0, 0, 0);
      if (slot[u] >= 0) {
        kx[u][i] = *reinterpret_cast<const uint4*>(a.K + h * a.k_head + (t0 + u) * a.k_row + l * 16 + i * 8);
        vx[u][i] = *reinterpret_cast<const uint4*>(a.V + h * a.v_head + (t0 + u) * a.v_row + l * 16 + i * 8);
      }
    }
  const int q = l >> 1, g = 4 * (l & 1) + 2 * (q & 1);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t ks, vs;
    const uint2 kc = quantise16<NG>(kx[u], ks), vc = quantise16<NG>(vx[u], vs);
    // V words hold four channels of two neighbouring quarters of the row (lanes l and l ^ 2): of its
    // four fours a lane keeps two and hands over the two that its partner stores
    const uint32_t other = __shfl_xor_sync(0xffffffffu, (q & 1) ? vc.x : vc.y, 2);
    const uint32_t even = (q & 1) ? other : vc.x, odd = (q & 1) ? vc.y : other;
    if (slot[u] < 0) continue;
    const int i = (int)(slot[u] & 15);
    uint8_t* blk = row_block<NG>(a.c, slot[u], h);
    uint8_t* kp = blk + 64 * i + 32 * (l & 1) + 4 * q;
    *reinterpret_cast<uint32_t*>(kp) = kc.x;
    *reinterpret_cast<uint32_t*>(kp + 16) = kc.y;
    uint8_t* vp = blk + Blk::V_CODES + 64 * i + 4 * (q >> 1);
    *reinterpret_cast<uint32_t*>(vp + 8 * (g ^ kv4_v_swizzle(i))) = __byte_perm(even, odd, 0x5410);
    *reinterpret_cast<uint32_t*>(vp + 8 * ((g + 1) ^ kv4_v_swizzle(i))) = __byte_perm(even, odd, 0x7632);
    if (l % (APPEND_LANES / NG) == 0) {
      const int grp = l / (APPEND_LANES / NG);
      *reinterpret_cast<uint32_t*>(blk + Blk::K_SCALES + 4 * NG * i + 4 * grp) = ks;
      *reinterpret_cast<uint32_t*>(blk + Blk::V_SCALES + 4 * NG * i + 4 * grp) = vs;
    }
  }
}

constexpr int READ_LANES = 16, READ_UNROLL = 4;

__device__ __forceinline__ uint4 dequantise8(uint32_t code, uint32_t scale_word) {
  const float step = bf_lo(scale_word), lo = bf_hi(scale_word);
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)  // 2^23 + code, less 2^23
    x[e] = fmaf(__uint_as_float(((code >> (4 * e)) & 15u) | 0x4b000000u) - 8388608.f, step, lo);
  return make_uint4(bf_pack(x[0], x[1]), bf_pack(x[2], x[3]), bf_pack(x[4], x[5]), bf_pack(x[6], x[7]));
}

// Bound by HBM and, nearly, by issue (78 %): the append's bytes the other way round.  262144 tokens, 4 heads, groups
// of 128: 123 to 129 us, 5.4 TB/s; with one row in flight 147 us.
template <int NG>
__global__ void __launch_bounds__(ROW_THREADS) kv4_read_kernel(const RowArgs a) {
  using Blk = Kv4Block<NG>;
  constexpr int U = READ_UNROLL;
  const int l = threadIdx.x % READ_LANES;
  int64_t t0, slot[U];
  int h;
  row_item<READ_LANES>(a, t0, h, slot);
  const int q = l >> 2, g = 2 * (l & 3) + (q & 1), grp = l / (16 / NG);
  uint32_t kc[U], vw[U], ks[U], vs[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    kc[u] = vw[u] = ks[u] = vs[u] = 0;
    if (slot[u] < 0) continue;
    const int i = (int)(slot[u] & 15);
    const uint8_t* blk = row_block<NG>(a.c, slot[u], h);
    kc[u] = *reinterpret_cast<const uint32_t*>(blk + 64 * i + 16 * (l & 3) + 4 * (l >> 2));
    vw[u] = *reinterpret_cast<const uint32_t*>(blk + Blk::V_CODES + 64 * i + 8 * (g ^ kv4_v_swizzle(i)) + 4 * (q >> 1));
    ks[u] = *reinterpret_cast<const uint32_t*>(blk + Blk::K_SCALES + 4 * NG * i + 4 * grp);
    vs[u] = *reinterpret_cast<const uint32_t*>(blk + Blk::V_SCALES + 4 * NG * i + 4 * grp);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, vw[u], 4);
    const uint32_t vc = (q & 1) ? __byte_perm(other, vw[u], 0x7632) : __byte_perm(vw[u], other, 0x5410);
    if (slot[u] < 0) continue;
    *reinterpret_cast<uint4*>(a.K + h * a.k_head + (t0 + u) * a.k_row + l * 8) = dequantise8(kc[u], ks[u]);
    *reinterpret_cast<uint4*>(a.V + h * a.v_head + (t0 + u) * a.v_row + l * 8) = dequantise8(vc, vs[u]);
  }
}

msa_status row_args(const msa_kv4_cache* cache, const void* K, const void* V, const msa_strides* s,
                    const int64_t* slots, int64_t T, RowArgs* a) {
  const msa_status st = kv4_view(cache, &a->c);
  if (st != MSA_OK) return st;
  if (!s || T < 0) return MSA_ERR_INVALID_ARG;
  if (T == 0) return MSA_OK;
  if (!K || !V || !slots) return MSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) & 15) return MSA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(slots) & 7) return MSA_ERR_ALIGN;
  if (s->k_head % 8 || s->k_row % 8 || s->v_head % 8 || s->v_row % 8) return MSA_ERR_ALIGN;
  if (T > (int64_t(1) << 31) || T * cache->Hkv > (int64_t(1) << 33)) return MSA_ERR_UNSUPPORTED;
  a->K = static_cast<__nv_bfloat16*>(const_cast<void*>(K));
  a->V = static_cast<__nv_bfloat16*>(const_cast<void*>(V));
  a->k_head = s->k_head, a->k_row = s->k_row, a->v_head = s->v_head, a->v_row = s->v_row;
  a->slots = slots;
  a->T = T;
  return MSA_OK;
}

unsigned row_blocks(const RowArgs& a, int lanes, int unroll) {
  const int64_t items = (a.T + unroll - 1) / unroll * a.c.Hkv;
  return (unsigned)((items * lanes + ROW_THREADS - 1) / ROW_THREADS);
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_kv4_page_bytes(int32_t page_tokens, int32_t group) {
  if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1))) return 0;
  if (group != 32 && group != 64 && group != 128) return 0;
  return (size_t)page_tokens * (128 + 8 * (128 / group));
}

msa_status msa_kv4_slots(const msa_kv4_cache* cache, const int32_t* kv_lens, const int32_t* new_lens, int32_t B,
                         int32_t* block_table, int64_t table_stride, int32_t max_blocks, const int32_t* free_pages,
                         const int32_t* n_free, int32_t* kv_lens_out, int32_t* n_free_out, int32_t* cu_new,
                         int64_t* slots, int32_t* positions, int64_t capacity, void* stream) {
  SlotArgs a{};
  const msa_status st = kv4_view(cache, &a.c);
  if (st != MSA_OK) return st;
  if (B < 0 || capacity < 0 || max_blocks < 0) return MSA_ERR_INVALID_ARG;
  if (B > KV4_MAX_B) return MSA_ERR_UNSUPPORTED;
  if (table_stride < max_blocks) return MSA_ERR_SHAPE;
  if (!n_free || !n_free_out || !cu_new || !free_pages) return MSA_ERR_INVALID_ARG;
  if (B && (!kv_lens || !new_lens || !kv_lens_out || (max_blocks && !block_table))) return MSA_ERR_INVALID_ARG;
  if (capacity && (!slots || !positions)) return MSA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slots) & 7) return MSA_ERR_ALIGN;
  if (!aligned4({kv_lens, new_lens, block_table, free_pages, n_free, kv_lens_out, n_free_out, cu_new, positions}))
    return MSA_ERR_ALIGN;
  if (((int64_t)max_blocks << a.c.page_shift) > KV4_MAX_TOKENS) return MSA_ERR_UNSUPPORTED;
  a.kv_lens = kv_lens, a.new_lens = new_lens, a.free_pages = free_pages, a.n_free = n_free;
  a.block_table = block_table, a.kv_out = kv_lens_out, a.n_free_out = n_free_out, a.cu_new = cu_new;
  a.positions = positions, a.slots = slots, a.table_stride = table_stride, a.capacity = capacity;
  a.B = B, a.max_blocks = max_blocks;
  a.whole = cache->flags & MSA_KV4_WHOLE_REQUESTS;
  // one block for a decode batch; more only where there are tokens for them
  const int64_t want = (capacity + 4 * SLOT_THREADS - 1) / (4 * SLOT_THREADS);
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(want, 2 * sm_count()));
  const size_t smem = (3 * (size_t)B + 2) * sizeof(int32_t);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MSA_ERR_CUDA;
  static std::atomic<uint64_t> ready{0};
  if (device_pending(ready, dev)) {
    if (cudaFuncSetAttribute(kv4_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)((3 * KV4_MAX_B + 2) * sizeof(int32_t))) != cudaSuccess)
      return MSA_ERR_CUDA;
    mark_device(ready, dev);
  }
  count_launches(1);
  kv4_slots_kernel<<<grid, SLOT_THREADS, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

msa_status msa_kv4_release(const msa_kv4_cache* cache, const int32_t* ids, int32_t n, int32_t* kv_lens, int32_t B,
                           int32_t* block_table, int64_t table_stride, int32_t max_blocks, int32_t* free_pages,
                           int32_t* n_free, void* stream) {
  ReleaseArgs a{};
  const msa_status st = kv4_view(cache, &a.c);
  if (st != MSA_OK) return st;
  if (n < 0 || B < 0 || max_blocks < 0) return MSA_ERR_INVALID_ARG;
  if (n > KV4_MAX_B) return MSA_ERR_UNSUPPORTED;
  if (table_stride < max_blocks) return MSA_ERR_SHAPE;
  if (n == 0) return MSA_OK;
  if (!ids || !n_free || !free_pages || (B && (!kv_lens || (max_blocks && !block_table)))) return MSA_ERR_INVALID_ARG;
  if (!aligned4({ids, kv_lens, block_table, free_pages, n_free})) return MSA_ERR_ALIGN;
  a.ids = ids, a.kv_lens = kv_lens, a.block_table = block_table, a.free_pages = free_pages, a.n_free = n_free;
  a.table_stride = table_stride, a.n = n, a.B = B, a.max_blocks = max_blocks;
  count_launches(1);
  kv4_release_kernel<<<1, SLOT_THREADS, (3 * (size_t)n + 2) * sizeof(int32_t), static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

msa_status msa_kv4_append(const msa_kv4_cache* cache, const void* K, const void* V, const msa_strides* strides,
                          const int64_t* slots, int64_t T, void* stream) {
  RowArgs a{};
  const msa_status st = row_args(cache, K, V, strides, slots, T, &a);
  if (st != MSA_OK || T == 0) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const unsigned blocks = row_blocks(a, APPEND_LANES, APPEND_UNROLL);
  count_launches(1);
  switch (cache->group) {
    case 128: kv4_append_kernel<1><<<blocks, ROW_THREADS, 0, cs>>>(a); break;
    case 64: kv4_append_kernel<2><<<blocks, ROW_THREADS, 0, cs>>>(a); break;
    default: kv4_append_kernel<4><<<blocks, ROW_THREADS, 0, cs>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

msa_status msa_kv4_read(const msa_kv4_cache* cache, void* K, void* V, const msa_strides* strides,
                        const int64_t* slots, int64_t T, void* stream) {
  RowArgs a{};
  const msa_status st = row_args(cache, K, V, strides, slots, T, &a);
  if (st != MSA_OK || T == 0) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const unsigned blocks = row_blocks(a, READ_LANES, READ_UNROLL);
  count_launches(1);
  switch (cache->group) {
    case 128: kv4_read_kernel<1><<<blocks, ROW_THREADS, 0, cs>>>(a); break;
    case 64: kv4_read_kernel<2><<<blocks, ROW_THREADS, 0, cs>>>(a); break;
    default: kv4_read_kernel<4><<<blocks, ROW_THREADS, 0, cs>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

msa_status msa_kv4_status(const msa_kv4_cache* cache, void* stream) {
  Kv4View v;
  const msa_status st = kv4_view(cache, &v);
  if (st != MSA_OK) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint32_t err = 0;
  if (cudaMemcpyAsync(&err, v.state, 4, cudaMemcpyDeviceToHost, cs) != cudaSuccess) return MSA_ERR_CUDA;
  if (cudaStreamSynchronize(cs) != cudaSuccess) return MSA_ERR_CUDA;
  if (err) {
    if (cudaMemsetAsync(v.state, 0, 4, cs) != cudaSuccess) return MSA_ERR_CUDA;
    if (cudaStreamSynchronize(cs) != cudaSuccess) return MSA_ERR_CUDA;
  }
  if (err & DEV_ERR_TIMEOUT) return MSA_ERR_TIMEOUT;
  if (err & DEV_ERR_BOUNDS) return MSA_ERR_DEVICE_BOUNDS;
  return MSA_OK;
}

}  // extern "C"
