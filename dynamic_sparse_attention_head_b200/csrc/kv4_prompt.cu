// Attention over the paged 4-bit cache for many query rows (prompts over a cached prefix): the tile
// products on tcgen05.
//
// A CTA works on 256 query rows (token * group + head) of one KV head, two streams of 128, against
// tiles of 128 keys that both streams share.  One warp brings a tile's 4-bit blocks in by bulk copies;
// four warps turn them into fp16 operands in 128-byte-swizzled shared memory, the codes entering as
// fp16 subnormals (a mask and one product a pair); two warps issue the products (M = N = 128); two
// warpgroups hold a query row per thread: maximum, exponentials and sums in fp32, O rescaled only
// when the maximum grows by 2^8 or the values' power of two changes.
//
// Scores keep fp32's precision: the operands are exact, as long as the steps of a key's groups lie within 2^4 of
// one another (below, they lose what is under 2^-12 of the largest).  A code less 8 has 3 bits (or is 8, a power of
// two) and a step has 8, so (code - 8) * step fits fp16's 11 bits; what is left, lo + 8 step per group,
// meets the group's sum of the query in 16 more columns, each of the two as a sum of two fp16 parts
// (three of their four products).  A power of two is taken out of each tile's keys and each query row,
// so that fp16's range holds them, and out of single keys where they differ much.  (Keys rounded to fp16 put a
// score off by 3e-4, 30 times what lse may lose.)  Values are lo + code * step rounded to fp16's 11 bits: O is rounded to 8.
//
// Work: the 256-row pairs of a request see more and more keys; pair f and pair (last - f) together see
// nearly the same number, so a request's units (tiles, and one more per pair for its start and end)
// come in equal folds on one line, of which every CTA takes an equal stretch.  A pair cut by a stretch's
// border leaves fp32 rows in the workspace; a second small kernel joins them in a fixed order.
//
// Measured (follow-up prompts of 601 and 316 tokens over 32768 and 10732 cached ones, 28 / 4 heads): 521 us, 630
// TFLOP/s.  (The split below was taken at 538 us.)  A pair of tiles takes 4700 to 6000 cycles.  The tensor pipe needs 2176 of them, the exponentials
// 2048, shared memory about 2550 (147 KB of Q K operands, 64 KB of P V's, 115 KB around the widening); the
// chain through them is what counts: widening 2700 (keys) and 1150 (values), products 1750 under that
// contention, softmax 2440.  Moving the scales' share of the widening to a warp of its own shortened the first
// but not the chain (573 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "kv4.cuh"
#include "msa_internal.h"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int HD = 128;
constexpr int TK = 128;       // keys of a tile
constexpr int PAIR = 256;     // query rows of a CTA's pair of streams
constexpr int PART = HD + 2;  // floats of a partial row: O, maximum, sum
constexpr int THREADS = 512;
constexpr int ATOM = 128 * 128;  // bytes of [128 rows][64 columns] fp16
constexpr int OPERAND = 2 * ATOM;
constexpr int EXTRA = 128 * 32;  // bytes of [128 rows][16 columns] fp16
constexpr int Q_BYTES = OPERAND + EXTRA;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float NEG_INF = -__builtin_huge_valf();
constexpr uint32_t TM_STREAM = 256, TM_OOFF = 128;  // tensor-memory columns: S (then P) and O of a stream
// registers: launched at 128 a thread; control warps 48, softmax 200, dequantising 64 (sum 512 = 4 x 128)
constexpr int REG_CTRL = 48, REG_SOFTMAX = 200, REG_DEQ = 64;
static_assert(REG_CTRL + 2 * REG_SOFTMAX + REG_DEQ <= 512, "register split exceeds the launch allocation");
constexpr int NAN_RING = 4;
// Weights are taken 2^7 above the running maximum's own 1, as far up as fp16 holds them (the maximum may lie 2^8
// above the one in use): P rounds them to 11 bits or, where they are small, to a multiple of 2^-24, so that half a step
// lost is 2^-32 of the largest, while their fp32 sum keeps them all.  Without the factor the keys 17 nats below a sink
// go missing: O of 32768 of them was off by 1.7 % of its norm, at 18 nats by 14 %.
constexpr int W_EXP = 7;
constexpr int DEQ_UNROLL = 2;
// A power of two is taken out of each tile's values, so that the largest lies in [2^-7, 2^-6); fp16 then holds
// 2^-18 of it.  It is the one of the tile before as long as that is no less and at most 2^V_SLACK above what the tile wants
// (a change rescales O), and falls by 2^V_FALL at most, which keeps O in fp32's range.  A key more than 2^V_SPREAD below
// it has a power of its own, at most 2^V_KEY further down, and the weights of such a tile's keys are scaled the other way: a
// token of large values takes no precision from the others, whether or not a row weighs it.
constexpr int V_SLACK = 3, V_FALL = 64, V_SPREAD = 6;
// Keys likewise: steps of a tile's largest key lie in [2^-9, 2^-8), and (code - 8) * step is exact down to steps of
// 2^-17.  A key more than 2^K_SPREAD below the largest has a power of its own, which its scores take back.
constexpr int K_SPREAD = 4;
constexpr int KEY_DOWN = 15;  // the most that a key's own power is below its tile's: half a byte each for K and V

struct PairSeg {
  int32_t b, h, rt;      // request, KV head, pair of row tiles
  int32_t n, kv, q0;     // new tokens, cached tokens, first query row
  int32_t first, count;  // units on the line
  int32_t tiles;         // key tiles its last row sees
};

template <int NG>
struct PromptSmem {
  static constexpr int TILE = TK / 16 * Kv4Block<NG>::BYTES;
  static constexpr int Q = 0;                             // [2 streams] channels, sums
  static constexpr int K = Q + 2 * Q_BYTES;               // [2 slots] channels, lo + 8 step
  static constexpr int V = K + 2 * Q_BYTES;
  static constexpr int RAW = V + OPERAND;                 // [2 slots]
  static constexpr int CONST = RAW + 2 * TILE;            // [K, V, V][128 keys][NG] half2 (step, -8 step; step, lo)
  static constexpr int CTRL = CONST + 3 * TK * NG * 4;
  struct Ctrl {
    uint64_t raw_full[2], raw_empty[2], scale_full[4], k_full[2], k_empty[2], v_full, v_empty;
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_free[2], drain[2];
    union {
      int64_t sums[THREADS / 32];  // until the line is scanned
      uint8_t key_down[4][TK];     // spread tiles: how far a key's own powers of two are down (K low, V high half)
    };
    int32_t nan_from[NAN_RING][4];  // per segment: first key whose value group is NaN
    uint32_t raw_have[2];           // copies made
    uint32_t have[4];               // blocks of 16 keys of a tile that hold keys; bit 8: it is spread
    float k_scale[4];               // power of two taken out of the tile's keys
    int32_t v_exp[4];               // exponent taken out of the values
    int32_t warp_exp[2][4];
    uint32_t tmem;
    int32_t abort, bad;
  };
  static constexpr int CUM = CTRL + (sizeof(Ctrl) + 15) / 16 * 16;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ float fmax3(float a, float b, float c) { return fmaxf(a, fmaxf(b, c)); }

// kind::f16 with fp16 A and B and fp32 accumulation
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// ---- the line of units ----
__device__ __forceinline__ int pairs_of(int32_t n, int32_t group) {
  return (int)(((int64_t)n * group + PAIR - 1) / PAIR);
}
// key tiles that pair rt's last row sees
__device__ __forceinline__ int tiles_of(int32_t n, int32_t kv, int32_t group, int rt) {
  const int64_t last_row = min((int64_t)(rt + 1) * PAIR, (int64_t)n * group) - 1;
  const int seen = kv - n + (int)(last_row / group) + 1;
  return seen <= 0 ? 0 : (seen + TK - 1) / TK;
}
// units of a fold: an upper bound of tiles(f) + tiles(last - f) that does not depend on f (a sum of
// two rounded-down terms is at most the rounded-down sum), and a unit per pair
__device__ __forceinline__ int fold_units(int32_t n, int32_t kv, int32_t group, int rts) {
  const int top = tiles_of(n, kv, group, rts - 1);
  if (rts == 1) return top + 1;
  const int64_t a = (int64_t)(kv - n + TK) * group + PAIR - 1;
  const int64_t sum = (2 * a + (int64_t)(rts - 1) * PAIR) / ((int64_t)TK * group);
  return max((int)max(sum, (int64_t)0), top) + 2;
}

// units of a KV head: whole folds, and the middle pair of an odd number, which is alone
__device__ __forceinline__ int64_t head_units(int32_t n, int32_t kv, int32_t group, int rts) {
  return (int64_t)(rts / 2) * fold_units(n, kv, group, rts) +
         (rts & 1 ? tiles_of(n, kv, group, rts / 2) + 1 : 0);
}

// Running sum of the requests' units into cum [B + 1]; returns the total (above 2^31: too many).
__device__ __forceinline__ int64_t scan_units(const AttendArgs& a, int32_t* cum, int64_t* sums, int* bad) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  if (tid == 0) cum[0] = 0;
  int64_t run = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + tid;
    int64_t x = 0;
    if (b < a.B) {
      int32_t q0, n, kv;
      if (!request_lens(a, b, q0, n, kv)) *bad = 1;
      const int rts = pairs_of(n, a.group);
      if (rts) x = (int64_t)a.c.Hkv * head_units(n, kv, a.group, rts);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int64_t before = run;
    for (int w = 0; w < warp; ++w) before += sums[w];
    if (b < a.B) cum[b + 1] = (int32_t)min(before + x, (int64_t)0x7fffffff);
    for (int w = 0; w < warps; ++w) run += sums[w];
    __syncthreads();
  }
  return run;
}

__device__ __forceinline__ PairSeg locate(const AttendArgs& a, const int32_t* cum, int t) {
  PairSeg s;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (cum[m] <= t) lo = m;
    else hi = m;
  }
  s.b = lo;
  request_lens(a, lo, s.q0, s.n, s.kv);
  const int rts = pairs_of(s.n, a.group), units = fold_units(s.n, s.kv, a.group, rts);
  const int per_head = (int)head_units(s.n, s.kv, a.group, rts);
  s.h = (t - cum[lo]) / per_head;
  const int in_head = t - cum[lo] - s.h * per_head, f = in_head / units, base = t - in_head + f * units;
  const int ta = tiles_of(s.n, s.kv, a.group, f);
  if (f == rts / 2 || t - base <= ta) {  // the middle pair, or a fold's first
    s.rt = f, s.first = base, s.count = ta + 1, s.tiles = ta;
  } else {
    s.rt = rts - 1 - f, s.first = base + ta + 1, s.count = units - ta - 1;
    s.tiles = tiles_of(s.n, s.kv, a.group, s.rt);
  }
  return s;
}

__device__ __forceinline__ int active_ctas(int total, int grid) { return min(grid, max(1, total)); }
__device__ __forceinline__ int line_edge(int total, int active, int i) { return (int)((int64_t)total * i / active); }
__device__ __forceinline__ int line_owner(int total, int active, int t) {
  return (int)((((int64_t)t + 1) * active - 1) / total);
}
__device__ __forceinline__ float* pair_part(const AttendArgs& a, int cta, int which) {
  return a.partial + (2 * (int64_t)cta + which) * PAIR * PART;
}

// What a CTA leaves to the second kernel: the pair that began in its stretch and goes on behind it, up to
// CTA `to` (-1: none).
struct JoinInfo {
  int32_t to, h, rt, n, q0, _pad[3];
};
__device__ __forceinline__ JoinInfo* join_info(const AttendArgs& a) {
  return reinterpret_cast<JoinInfo*>(a.partial + (int64_t)KV4_MAX_CTAS * 2 * PAIR * PART);
}

// 32-byte-swizzled operand of 16 columns: rows of 32 bytes, groups of 8 rows 256 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1u << 16;
  d |= (uint64_t)(256u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)6u << 61;
  return d;
}
__device__ __forceinline__ uint32_t sw32_offset(int row, int chunk) {
  return (uint32_t)(row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4));
}

// Eight codes of a word as fp16 lo + code * step, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 widen8(uint32_t w, __half2 step24, __half2 step20, __half2 lo) {
  const uint32_t w8 = w >> 8;
  const uint32_t c[4] = {w & 0x000f000fu, w & 0x00f000f0u, w8 & 0x000f000fu, w8 & 0x00f000f0u};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&c[i]), (i & 1) ? step20 : step24, lo);
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int NG>
__global__ void __launch_bounds__(THREADS, 1) kv4_prompt_kernel(const __grid_constant__ AttendArgs a) {
  using S = PromptSmem<NG>;
  using Blk = Kv4Block<NG>;
  extern __shared__ __align__(1024) uint8_t smem[];
  typename S::Ctrl& ct = *reinterpret_cast<typename S::Ctrl*>(smem + S::CTRL);
  int32_t* cum = reinterpret_cast<int32_t*>(smem + S::CUM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) join_info(a)[blockIdx.x].to = -1;
  if (smem_addr(smem) & 1023u) {  // swizzled tiles need a 1024-byte aligned base
    if (tid == 0) atomicOr(a.c.state, DEV_ERR_BOUNDS);
    return;
  }
  if (tid == 0) {
    ct.abort = ct.bad = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ct.raw_full[i], 1);
      mbar_init(&ct.raw_empty[i], 128);
      mbar_init(&ct.scale_full[i], 1);
      mbar_init(&ct.scale_full[2 + i], 1);
      mbar_init(&ct.k_full[i], 128);
      mbar_init(&ct.k_empty[i], 2);
      mbar_init(&ct.q_full[i], 128);
      mbar_init(&ct.s_full[i], 1);
      mbar_init(&ct.p_full[i], 128);
      mbar_init(&ct.o_full[i], 1);
      mbar_init(&ct.o_free[i], 128);
      mbar_init(&ct.drain[i], 1);
    }
    mbar_init(&ct.v_full, 128);
    mbar_init(&ct.v_empty, 2);
    fence_barrier_init();
  }
  __syncthreads();
  const int64_t run = scan_units(a, cum, ct.sums, &ct.bad);
  if (blockIdx.x == 0 && tid == 0 && (ct.bad || run > 0x7fffffff)) atomicOr(a.c.state, DEV_ERR_BOUNDS);
  if (run > 0x7fffffff) return;  // more units than the line has numbers for
  const int total = (int)run, active = active_ctas(total, gridDim.x);
  if ((int)blockIdx.x >= active || total == 0) return;
  const int t0 = line_edge(total, active, blockIdx.x), t1 = line_edge(total, active, blockIdx.x + 1);
  if (warp == 1) tmem_alloc<512>(&ct.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ct.tmem;
  volatile int* abort = &ct.abort;

  // tiles of a segment that lie in this stretch
  const auto tiles_from = [&](const PairSeg& s) { return max(t0 - s.first - 1, 0); };
  const auto tiles_to = [&](const PairSeg& s) { return min(min(s.first + s.count, t1) - s.first - 1, s.tiles); };
  const auto rows_of = [&](const PairSeg& s, int stream) {
    return (int)min((int64_t)128, (int64_t)s.n * a.group - ((int64_t)s.rt * PAIR + stream * 128));
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_CTRL));
    if (warp == 0) {
      // ---------------------------------------------------------------- the tiles' 4-bit blocks
      const int copy_shift = min(a.c.page_shift, 7), per = TK >> copy_shift;
      uint32_t kt = 0;
      bool ok = true;
      for (int at = t0; at < t1 && ok;) {
        const PairSeg s = locate(a, cum, at);
        const int last_row = (int)(min((int64_t)(s.rt + 1) * PAIR, (int64_t)s.n * a.group) - 1);
        const int seen = s.kv - s.n + last_row / a.group + 1;
        int32_t entry = -1;
        int entry_at = 0;
        bool entry_ok = false;
        const int to = tiles_to(s);
        for (int tile = tiles_from(s); tile < to; ++tile, ++kt) {
          const int first = tile * per, st = kt & 1;
          if (!entry_ok || first - entry_at >= 32) {  // lane l: the table entry of copy entry_at + l
            entry_at = first;
            entry_ok = true;
            const int tok = (first + lane) << copy_shift, blk = tok >> a.c.page_shift;
            entry = blk < a.max_blocks && tok < seen ? a.table[s.b * a.table_stride + blk] : -1;
          }
          const int32_t page = __shfl_sync(0xffffffffu, entry, (first - entry_at + lane) & 31);
          if (kt >= 2 && !mbar_wait(&ct.raw_empty[st], ((kt >> 1) - 1) & 1, abort)) ok = false;
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          const int tok = (first + lane) << copy_shift;
          const bool want = lane < per && tok < seen, good = want && page >= 0 && page < a.c.n_pages;
          if (want && !good) ct.bad = 1;
          const uint32_t bytes = good ? min(1 << copy_shift >> 4, (seen - tok + 15) >> 4) * Blk::BYTES : 0;
          const uint32_t all = __reduce_add_sync(0xffffffffu, bytes), made = __ballot_sync(0xffffffffu, good);
          if (lane == 0) {
            ct.raw_have[st] = made;
            mbar_arrive_expect_tx(&ct.raw_full[st], all);
          }
          __syncwarp();
          if (good)
            bulk_load(smem_addr(smem + S::RAW + st * S::TILE) + (lane << copy_shift >> 4) * Blk::BYTES,
                      a.c.pages + ((int64_t)page * a.c.Hkv + s.h) * a.c.page_bytes +
                          ((tok & (a.c.page_tokens() - 1)) >> 4) * Blk::BYTES,
                      bytes, &ct.raw_full[st]);
        }
        at = min(s.first + s.count, t1);
      }
      // copies in flight land before the CTA goes away
      for (uint32_t i = kt >= 2 ? kt - 2 : 0; i < kt; ++i) {
        int none = 0;
        mbar_wait(&ct.raw_full[i & 1], (i >> 1) & 1, &none);
      }
    } else if ((warp & 1) && lane == 0) {
      // ---------------------------------------------------------------- MMA issuers: warp 1, 3
      // QK(0), then groups [PV(j), QK(j + 1)].  The two streams' groups may mix on the tensor pipe: Q K reads
      // both operands from shared memory (128 bytes a cycle, all there is), P V one, and side by side they
      // share it better than one after the other (538 us against 563 with the groups held apart by a lock).
      const int st = warp >> 1;
      constexpr uint32_t IDESC_QK = idesc_f16_f32(128, 128, 0, 0), IDESC_PV = idesc_f16_f32(128, 128, 0, 1);
      const uint32_t s_col = tmem + TM_STREAM * st;
      uint32_t kt = 0, mine = 0, done = 0;  // tiles of the CTA, tiles and segments of the stream
      bool ok = true;
      const auto qk = [&](uint32_t k) {
        tc_fence_after();
        uint32_t q_addr = smem_addr(smem + S::Q + st * Q_BYTES), k_addr = smem_addr(smem + S::K + (k & 1) * Q_BYTES);
        asm volatile("" : "+r"(q_addr), "+r"(k_addr));
        umma_ss(s_col, smem_desc_sw32(q_addr + OPERAND), smem_desc_sw32(k_addr + OPERAND), IDESC_QK, 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * ATOM + (kk & 3) * 32;
          umma_ss(s_col, smem_desc_sw128(q_addr + off, 16, 1024), smem_desc_sw128(k_addr + off, 16, 1024), IDESC_QK, 1u);
        }
        umma_commit(&ct.s_full[st]);
        umma_commit(&ct.k_empty[k & 1]);
      };
      for (int at = t0; at < t1 && ok;) {
        const PairSeg s = locate(a, cum, at);
        at = min(s.first + s.count, t1);
        const int n = tiles_to(s) - tiles_from(s);
        if (n <= 0) continue;
        if (rows_of(s, st) <= 0) {  // the pair has no rows for this stream: only hand the tiles on
          // (not before the rows of the stream's last pair have left: the widening warps, which what is handed on here
          // lets run ahead, reuse what those rows still read)
          ok = done == 0 || mbar_wait(&ct.o_free[st], (done - 1) & 1, abort);
          for (int j = 0; j < n && ok; ++j, ++kt) {
            ok = mbar_wait(&ct.k_full[kt & 1], (kt >> 1) & 1, abort);
            if (ok) mbar_arrive(&ct.k_empty[kt & 1]);
            ok = ok && mbar_wait(&ct.v_full, kt & 1, abort);
            if (ok) mbar_arrive(&ct.v_empty);
          }
          continue;
        }
        ok = mbar_wait(&ct.q_full[st], done & 1, abort) && mbar_wait(&ct.k_full[kt & 1], (kt >> 1) & 1, abort);
        if (!ok) break;
        qk(kt);
        for (int j = 0; j < n; ++j, ++kt, ++mine) {
          ok = (j > 0 || done == 0 || mbar_wait(&ct.o_free[st], (done - 1) & 1, abort)) &&
               mbar_wait(&ct.v_full, kt & 1, abort) && mbar_wait(&ct.p_full[st], mine & 1, abort) &&
               (j + 1 == n || mbar_wait(&ct.k_full[(kt + 1) & 1], ((kt + 1) >> 1) & 1, abort));
          if (!ok) break;
          tc_fence_after();
          uint32_t v_addr = smem_addr(smem + S::V);
          asm volatile("" : "+r"(v_addr));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(s_col + TM_OOFF, s_col + 8 * kk, smem_desc_sw128(v_addr + kk * 2048, ATOM, 1024), IDESC_PV,
                    (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&ct.v_empty);
          if (j + 1 < n) qk(kt + 1);
        }
        if (!ok) break;
        umma_commit(&ct.o_full[st]);
        ++done;
      }
      // what was issued is done before tensor memory is given back
      umma_commit(&ct.drain[st]);
      int none = 0;
      mbar_wait(&ct.drain[st], 0, &none);
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFTMAX));
    // ------------------------------------------------------------------ softmax: a row per thread
    const int st = (warp - 4) >> 2, t = (warp & 3) * 32 + lane;
    const uint32_t s_own = tmem + ((uint32_t)((warp & 3) * 32) << 16) + TM_STREAM * st, o_own = s_own + TM_OOFF;
    uint32_t kt = 0, mine = 0, done = 0, segs = 0;
    bool ok = true;
    for (int at = t0; at < t1 && ok;) {
      const PairSeg s = locate(a, cum, at);
      at = min(s.first + s.count, t1);
      const int from = tiles_from(s), n = max(tiles_to(s) - from, 0), rows = rows_of(s, st);
      const bool live = t < rows;
      const int row = s.rt * PAIR + st * 128 + t, token = live ? a.by_group(row) : 0;
      const int hd = s.h * a.group + (live ? row - token * a.group : 0);
      const int lim = live ? s.kv - s.n + token + 1 : 0x7fffffff;
      const int ring = segs & (NAN_RING - 1);
      if (n > 0) ++segs;
      float m_used = NEG_INF, l = 0.f;  // base-2 scores are taken off m_used: the maximum less W_EXP
      int v_exp = -119;
      if (n > 0 && rows > 0) {
        // ---- the query row, a power of two taken out, into the swizzled operand ----
        float row_scale;
        {
          const __nv_bfloat16* q = a.Q + (int64_t)hd * a.q_head + (int64_t)(s.q0 + token) * a.q_row;
          uint4 raw[16];
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            raw[i] = live ? *reinterpret_cast<const uint4*>(q + 8 * i) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmax3(top, fabsf(bf_lo(w[k])), fabsf(bf_hi(w[k])));
          }
          const int ex = (int)((__float_as_uint(top) >> 23) & 255), up = max(-100, min(100, 131 - ex));
          const float norm = pow2(up);
          row_scale = a.scale2 * pow2(-up);
          uint8_t* dst = smem + S::Q + st * Q_BYTES + t * 128;
          float qs[NG];
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) qs[gr] = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint4 v = raw[i];
            uint4 x;  // channels in the order of the keys' codes: 0 4 1 5 2 6 3 7
            x.x = half2_bits(bf_lo(v.x) * norm, bf_lo(v.z) * norm);
            x.y = half2_bits(bf_hi(v.x) * norm, bf_hi(v.z) * norm);
            x.z = half2_bits(bf_lo(v.y) * norm, bf_lo(v.w) * norm);
            x.w = half2_bits(bf_hi(v.y) * norm, bf_hi(v.w) * norm);
            *reinterpret_cast<uint4*>(dst + (i >> 3) * ATOM + (((i & 7) ^ (t & 7)) << 4)) = x;
            qs[i * NG / 16] += norm * (((bf_lo(v.x) + bf_hi(v.x)) + (bf_lo(v.y) + bf_hi(v.y))) +
                                       ((bf_lo(v.z) + bf_hi(v.z)) + (bf_lo(v.w) + bf_hi(v.w))));
          }
          // the groups' sums in two parts of 11 bits: columns 3 g (first), 3 g + 1 (second), 3 g + 2 (first)
          float col[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) col[e] = 0.f;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            col[3 * gr] = col[3 * gr + 2] = __half2float(__float2half_rn(qs[gr]));
            col[3 * gr + 1] = qs[gr] - col[3 * gr];
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<uint4*>(smem + S::Q + st * Q_BYTES + OPERAND + sw32_offset(t, e)) =
                make_uint4(half2_bits(col[8 * e], col[8 * e + 1]), half2_bits(col[8 * e + 2], col[8 * e + 3]),
                           half2_bits(col[8 * e + 4], col[8 * e + 5]), half2_bits(col[8 * e + 6], col[8 * e + 7]));
          fence_proxy_async_smem();
          mbar_arrive(&ct.q_full[st]);
        }
        for (int j = 0; j < n; ++j, ++kt, ++mine) {
          ok = __all_sync(0xffffffffu, mbar_wait(&ct.s_full[st], mine & 1, abort) &&
                                           mbar_wait(&ct.scale_full[kt & 3], (kt >> 2) & 1, abort));
          if (!ok) break;
          const float sc = fmaxf(row_scale * ct.k_scale[kt & 3], 0x1p-126f);  // not 0: it meets -inf below
          const uint32_t have = ct.have[kt & 3];
          const int v_new = ct.v_exp[kt & 3], tok = (from + j) * TK;
          tc_fence_after();
          float sv[128];
          {
            uint32_t rr[4][32];
#pragma unroll
            for (int h = 0; h < 4; ++h) tmem_ld32(s_own + 32 * h, rr[h]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 128; ++c) sv[c] = __uint_as_float(rr[c >> 5][c & 31]);
          }
          if (__any_sync(0xffffffffu, tok + TK > lim) || have != 0xffu) {
            const int open = lim - tok;  // columns this row sees
            if (have >> 8)
#pragma unroll
              for (int c = 0; c < 128; ++c) sv[c] *= pow2(-(int)(ct.key_down[kt & 3][c] & 15u));
#pragma unroll
            for (int c = 0; c < 128; ++c)  // and is on a page
              sv[c] = c < open && ((have >> (c >> 4)) & 1u) ? sv[c] : NEG_INF;
          }
          float m4[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
          for (int c = 0; c < 128; c += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) m4[q] = fmax3(m4[q], sv[c + 2 * q], sv[c + 2 * q + 1]);
          const float top = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
          const float mxs = top == NEG_INF ? NEG_INF : top * sc;
          float alpha = 1.f;
          bool resc = v_new != v_exp;
          if (mxs - m_used > 8.f + W_EXP) {  // also true on the first score (a difference: exact next to the border)
            const float m_new = mxs - (float)W_EXP;
            alpha = m_used == NEG_INF ? 0.f : ex2(m_used - m_new);
            m_used = m_new;
            resc = true;
          }
          if (j > 0 && __any_sync(0xffffffffu, resc)) {  // S complete: so is the P V before it
            // exponents lie within [-119, 110], and a fall is at most V_FALL: two steps of a power of two
            const int d = v_exp - v_new;
            const float f = alpha * pow2(max(d / 2, -120)) * pow2(max(d - d / 2, -120));
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t oo[16];
              tmem_ld16(o_own + 16 * c, oo);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) oo[e] = __float_as_uint(__uint_as_float(oo[e]) * f);
              tmem_st16(o_own + 16 * c, oo);
            }
          }
          v_exp = v_new;
          const float nb = m_used == NEG_INF ? 0.f : -m_used;
          const float2 sc2 = make_float2(sc, sc), nb2 = make_float2(nb, nb);
          float2 rs2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // CAREFUL: scores are rounded first, and a key's weight is scaled by the power of two that its values are
          // up.  The fused product is exact where the maximum is rounded: above 2^24 the difference, half a last
          // place of the maximum, would reach the exponent's range.
          const auto weights = [&](auto careful) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t pk[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float2 s2 = make_float2(sv[32 * h + 2 * c], sv[32 * h + 2 * c + 1]);
                const float2 x = decltype(careful)::value
                                     ? make_float2(__fmul_rn(s2.x, sc) + nb, __fmul_rn(s2.y, sc) + nb)
                                     : __ffma2_rn(s2, sc2, nb2);
                float2 e = make_float2(ex2(x.x), ex2(x.y));
                rs2[c & 1] = __fadd2_rn(rs2[c & 1], e);
                if (decltype(careful)::value && (have >> 8)) {
                  e.x *= pow2(-(int)(ct.key_down[kt & 3][32 * h + 2 * c] >> 4));
                  e.y *= pow2(-(int)(ct.key_down[kt & 3][32 * h + 2 * c + 1] >> 4));
                }
                pk[c] = half2_bits(e.x, e.y);  // 11 bits: O is rounded to 8
              }
              tmem_st16(s_own + 16 * h, pk);
            }
          };
          if (__any_sync(0xffffffffu, (have >> 8) || fabsf(nb) > 0x1p24f)) weights(std::true_type{});
          else weights(std::false_type{});
          l = l * alpha + ((rs2[0].x + rs2[1].x) + (rs2[0].y + rs2[1].y));
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&ct.p_full[st]);
        }
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&ct.o_full[st], done & 1, abort));
        if (!ok) break;
        ++done;
        tc_fence_after();
      } else {
        kt += n;
        if (rows <= 0) continue;
      }

      // ---- the row, to O or to the workspace ----
      const bool whole = s.first >= t0 && s.first + s.count <= t1;
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const float f = inv * pow2(v_exp / 2), f2 = pow2(v_exp - v_exp / 2);  // of tiny values their product may underflow
      float* part = pair_part(a, blockIdx.x, s.first >= t0 ? 1 : 0) + (st * 128 + t) * PART;
      __nv_bfloat16* out = a.O + (int64_t)hd * a.o_head + (int64_t)(s.q0 + token) * a.o_row;
      uint32_t nans = 0;  // value groups that are NaN from some key on that this row sees; read before O is given back
      if (n > 0)
#pragma unroll
        for (int c = 0; c < 4; ++c) nans |= (uint32_t)(ct.nan_from[ring][c] < lim) << c;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t oa[32];
        if (n > 0) {
          tmem_ld32(o_own + 32 * c, oa);
          tmem_wait_ld();
          if (c == 3) {
            tc_fence_before();
            mbar_arrive(&ct.o_free[st]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) oa[e] = 0u;
        }
        const bool nan = (nans >> c) & 1u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float y[8];  // channels 8 (4 c + k) ..: columns hold them in the order 0 4 1 5 2 6 3 7
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = __uint_as_float(oa[8 * k + e]) * f * f2;
            y[(e & 1) * 4 + (e >> 1)] = nan ? __int_as_float(0x7fffffff) : x;
          }
          if (live && whole)
            *reinterpret_cast<uint4*>(out + 32 * c + 8 * k) =
                make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
          if (live && !whole) {
#pragma unroll
            for (int e = 0; e < 8; e += 2)
              *reinterpret_cast<float2*>(part + 32 * c + 8 * k + e) = make_float2(y[e], y[e + 1]);
          }
        }
      }
      if (live && whole && a.lse)
        a.lse[(int64_t)hd * a.total_q + s.q0 + token] = l == 0.f ? NEG_INF : (m_used + log2f(l)) * (1.f / LOG2E);
      if (live && !whole) *reinterpret_cast<float2*>(part + HD) = make_float2(m_used, l);
      if (st == 0 && t == 0 && !whole && s.first >= t0)
        join_info(a)[blockIdx.x] = {line_owner(total, active, s.first + s.count - 1), s.h, s.rt, s.n, s.q0, {}};
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_DEQ));
    // ------------------------------------------------------------------ 4 bits to fp16 operands
    const int d = tid - 384, w4 = warp - 12;
    const int g = lane >> 2, c = lane & 3;
    const int row8 = 8 * w4 + ((g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1);  // reads and writes without bank conflicts
    uint32_t* k_const = reinterpret_cast<uint32_t*>(smem + S::CONST);
    const int copy16 = min(a.c.page_shift, 7) - 4;  // log2 of a copy's blocks
    // the four warps stay in step, a wait that gave up in one thread ends all: every thread passes the same barriers
    const auto sync_deq = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    const auto all_deq = [](bool x) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r)
          : "r"((uint32_t)x)
          : "memory");
      return r != 0;
    };

    const auto any_deq = [](uint32_t x) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r)
          : "r"(x)
          : "memory");
      return r != 0;
    };

    // scales of tile kt: the powers of two, and each row's (step, lo) in fp16; then its keys
    int v_exp = -119, v_top = -119;
    const auto keys = [&](const PairSeg& s, int tile, uint32_t kt, int ring) {
      const bool there = mbar_wait(&ct.raw_full[kt & 1], (kt >> 1) & 1, abort);
      const uint8_t* raw = smem + S::RAW + (kt & 1) * S::TILE;
      const int last_row = (int)(min((int64_t)(s.rt + 1) * PAIR, (int64_t)s.n * a.group) - 1);
      const int key = tile * TK + d, seen = s.kv - s.n + last_row / a.group + 1;
      const uint32_t made = ct.raw_have[kt & 1];
      const bool shown = there && key < seen && (made >> (d >> 4 >> copy16) & 1u);
      const uint8_t* blk = raw + (d >> 4) * Blk::BYTES;
      const uint32_t* kp = reinterpret_cast<const uint32_t*>(blk + Blk::K_SCALES + 4 * NG * (d & 15));
      const uint32_t* vp = reinterpret_cast<const uint32_t*>(blk + Blk::V_SCALES + 4 * NG * (d & 15));
      uint32_t kw[NG], vw[NG];
      float smax = 0.f, lmax = 0.f, vmax = 0.f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        kw[gr] = shown ? kp[gr] : 0u;
        vw[gr] = shown ? vp[gr] : 0u;
        if (isnan(bf_lo(vw[gr]))) {  // held back from the product: rows that see it are set at the end
          const int q0 = gr * 4 / NG, q1 = (gr + 1) * 4 / NG;
          for (int q = q0; q < q1; ++q) atomicMin(&ct.nan_from[ring][q], key);
          vw[gr] = 0u;
        }
        smax = fmaxf(smax, bf_lo(kw[gr]));
        lmax = fmaxf(lmax, fabsf(bf_hi(kw[gr])));
        vmax = fmax3(vmax, fabsf(bf_hi(vw[gr])), fabsf(fmaf(15.f, bf_lo(vw[gr]), bf_hi(vw[gr]))));
      }
      // steps come below 2^-8 (2^24 steps fit fp16), lo below 2^14, values below 2^-6: exponents of the
      // powers of two to take out
      const auto exponent = [](float x, int off) { return (int)(__float_as_uint(x) >> 23) - off; };
      const int ko = max(exponent(smax, 118), exponent(lmax, 140)), vo = exponent(vmax, 120);  // of this key
      const int k_top = __reduce_max_sync(0xffffffffu, ko), v_high = __reduce_max_sync(0xffffffffu, vo);
      if (lane == 0) ct.warp_exp[0][w4] = k_top, ct.warp_exp[1][w4] = v_high;
      sync_deq();
      const auto all4 = [](const int32_t* x) { return max(max(x[0], x[1]), max(x[2], x[3])); };
      const int ke = min(max(all4(ct.warp_exp[0]), -119), 110), ve = min(all4(ct.warp_exp[1]), 110);  // of the tile
      v_top = max(v_top, ve);
      if (ve > v_exp || (ve >= -119 && ve < v_exp - V_SLACK)) v_exp = max(ve, v_top - V_FALL);
      // how far this key's own powers are down; zeros (or nearly: -118, -120) have none
      const int k_down = ko >= -117 && ko < ke - K_SPREAD ? min(ke - ko, KEY_DOWN) : 0;
      const int v_down = vo >= -119 && vo < v_exp - V_SPREAD ? min(v_exp - vo, KEY_DOWN) : 0;
      ct.key_down[kt & 3][d] = (uint8_t)(k_down | v_down << 4);
      const float kn = pow2(k_down - ke), vn = pow2(v_down - v_exp);
      uint32_t* v_const = k_const + (1 + (kt & 1)) * TK * NG;
      float mid[NG];
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const float step = bf_lo(kw[gr]) * kn;
        k_const[d * NG + gr] = half2_bits(step * 16777216.f, -8.f * step);
        v_const[d * NG + gr] = half2_bits(bf_lo(vw[gr]) * vn * 16777216.f, bf_hi(vw[gr]) * vn);
        mid[gr] = fmaf(8.f, step, bf_hi(kw[gr]) * kn);
      }
      const bool spread = any_deq(k_down | v_down);  // the scales are written
      if (d == 0) {
        uint32_t have = (uint32_t)spread << 8;
        for (int b = 0; b < TK / 16; ++b)
          have |= (uint32_t)(tile * TK + 16 * b >= seen || (made >> (b >> copy16) & 1u)) << b;
        // the place of the tile before the three last: every row has handed that one's P on
        ct.have[kt & 3] = have;
        ct.k_scale[kt & 3] = pow2(ke);
        ct.v_exp[kt & 3] = v_exp;
        mbar_arrive(&ct.scale_full[kt & 3]);
      }
      if (!there || (kt >= 2 && !mbar_wait(&ct.k_empty[kt & 1], ((kt >> 1) - 1) & 1, abort))) return false;
      uint8_t* dst = smem + S::K + (kt & 1) * Q_BYTES;
      {
        float col[16];  // against the sums' parts: first, first, second
#pragma unroll
        for (int e = 0; e < 16; ++e) col[e] = 0.f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          col[3 * gr] = col[3 * gr + 1] = __half2float(__float2half_rn(mid[gr]));
          col[3 * gr + 2] = mid[gr] - col[3 * gr];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<uint4*>(dst + OPERAND + sw32_offset(d, e)) =
              make_uint4(half2_bits(col[8 * e], col[8 * e + 1]), half2_bits(col[8 * e + 2], col[8 * e + 3]),
                         half2_bits(col[8 * e + 4], col[8 * e + 5]), half2_bits(col[8 * e + 6], col[8 * e + 7]));
      }
#pragma unroll DEQ_UNROLL
      for (int p = 0; p < 4; ++p) {
        const int r = 32 * p + row8;
        const uint4 x = *reinterpret_cast<const uint4*>(raw + (r >> 4) * Blk::BYTES + 64 * (r & 15) + 16 * c);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 k = *reinterpret_cast<const __half2*>(&k_const[r * NG + i * NG / 4]);
          const __half2 st = __low2half2(k);
          *reinterpret_cast<uint4*>(dst + (i >> 1) * ATOM + r * 128 + (((4 * (i & 1) + c) ^ (r & 7)) << 4)) =
              widen8(w[i], st, __hmul2(st, __float2half2_rn(0.0625f)), __high2half2(k));
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&ct.k_full[kt & 1]);
      return true;
    };
    // the codes of a tile's values, taken out of its blocks ahead of their turn (the blocks' place is free then)
    uint4 v_codes[4];
    const auto take_values = [&](uint32_t kt) {
      const uint8_t* raw = smem + S::RAW + (kt & 1) * S::TILE + Blk::V_CODES;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int r = 32 * p + row8;
        v_codes[p] = *reinterpret_cast<const uint4*>(raw + (r >> 4) * Blk::BYTES + 64 * (r & 15) + 16 * c);
      }
      mbar_arrive(&ct.raw_empty[kt & 1]);
    };
    const auto values = [&](uint32_t kt) {
      if (kt >= 1 && !mbar_wait(&ct.v_empty, (kt - 1) & 1, abort)) return false;
      const uint32_t* v_const = k_const + (1 + (kt & 1)) * TK * NG;
      uint8_t* dst = smem + S::V;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int r = 32 * p + row8, u = c ^ (kv4_v_swizzle(r & 15) >> 1);
        const uint4 x = v_codes[p];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 k = *reinterpret_cast<const __half2*>(&v_const[r * NG + i * NG / 4]);
          const __half2 st = __low2half2(k);
          const uint32_t w = i < 2 ? __byte_perm(x.x, x.z, (i & 1) ? 0x7632 : 0x5410)
                                   : __byte_perm(x.y, x.w, (i & 1) ? 0x7632 : 0x5410);
          *reinterpret_cast<uint4*>(dst + (i >> 1) * ATOM + r * 128 + (((4 * (i & 1) + u) ^ (r & 7)) << 4)) =
              widen8(w, st, __hmul2(st, __float2half2_rn(0.0625f)), __high2half2(k));
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&ct.v_full);
      return true;
    };
    uint32_t kt = 0, segs = 0;
    bool ok = true;
    for (int at = t0; at < t1 && ok;) {
      const PairSeg s = locate(a, cum, at);
      at = min(s.first + s.count, t1);
      const int from = tiles_from(s), n = tiles_to(s) - from;
      if (n <= 0) continue;
      const int ring = segs++ & (NAN_RING - 1);
      // The ring's place was last used four segments ago.  Before they came here these warps waited until both streams
      // had handed on a tile of one of the two segments before this one, and a stream does that, with rows or without,
      // only once the rows of its last pair have read their place and given O back.
      if (d < 4) ct.nan_from[ring][d] = 0x7fffffff;
      sync_deq();
      v_exp = v_top = -119;
      // K(0), then K(j + 1), V(j): values have one buffer, free once both streams' P V before are done
      ok = all_deq(keys(s, from, kt, ring));
      if (ok) take_values(kt);
      for (int j = 0; j < n && ok; ++j, ++kt) {
        if (j + 1 < n) ok = all_deq(keys(s, from + j + 1, kt + 1, ring));
        if (ok) ok = all_deq(values(kt));
        if (ok && j + 1 < n) take_values(kt + 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    if (ct.abort) atomicOr(a.c.state, DEV_ERR_TIMEOUT);
    if (ct.bad) atomicOr(a.c.state, DEV_ERR_BOUNDS);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

// Joins the rows of a pair that several CTAs worked on: block (i, j) takes rows 16 j .. of the pair that
// began in CTA i's stretch and went on behind it, a warp a row.  Few rows over a long context are cut over every
// CTA, and a row's partial results are then read one after the other: with 64 rows a block, 98 rows over 32768 tokens (28 / 4
// heads) took 76 us in all instead of 53; where every block has a pair of its own, 64 are 1 % faster.
constexpr int JOIN_THREADS = 512, JOIN_ROWS = 16;

__global__ void __launch_bounds__(JOIN_THREADS) kv4_prompt_join_kernel(const __grid_constant__ AttendArgs a) {
  const int cta = blockIdx.x;
  const JoinInfo s = join_info(a)[cta];
  if (s.to < 0) return;
  const int rows = (int)min((int64_t)PAIR, (int64_t)s.n * a.group - (int64_t)s.rt * PAIR);
  const int lane = threadIdx.x & 31, ch = lane * 4;
  for (int r = blockIdx.y * JOIN_ROWS + threadIdx.x / 32; r < min(rows, (int)(blockIdx.y + 1) * JOIN_ROWS);
       r += JOIN_THREADS / 32) {
    float top = NEG_INF, sum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 4;  // partial rows on their way together
    for (int k0 = cta; k0 <= s.to; k0 += U) {
      float2 st[U], y0[U], y1[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* p = pair_part(a, min(k0 + u, s.to), k0 + u == cta) + r * PART;
        st[u] = *reinterpret_cast<const float2*>(p + HD);
        y0[u] = *reinterpret_cast<const float2*>(p + ch);
        y1[u] = *reinterpret_cast<const float2*>(p + ch + 2);
        if (k0 + u > s.to) st[u] = make_float2(NEG_INF, 0.f), y0[u] = y1[u] = make_float2(0.f, 0.f);
      }
      float up = top;
#pragma unroll
      for (int u = 0; u < U; ++u) up = fmaxf(up, st[u].x);
      const float f0 = top == NEG_INF ? 0.f : ex2(top - up);
      top = up;
      sum *= f0;
      x.x *= f0, x.y *= f0, x.z *= f0, x.w *= f0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = st[u].x == NEG_INF ? 0.f : ex2(st[u].x - top);
        sum = fmaf(st[u].y, f, sum);
        x.x = fmaf(y0[u].x, f, x.x), x.y = fmaf(y0[u].y, f, x.y), x.z = fmaf(y1[u].x, f, x.z), x.w = fmaf(y1[u].y, f, x.w);
      }
    }
    const int row = s.rt * PAIR + r, token = a.by_group(row), hd = s.h * a.group + row - token * a.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint2 w;
    w.x = pack_bf16x2(x.x * inv, x.y * inv);
    w.y = pack_bf16x2(x.z * inv, x.w * inv);
    *reinterpret_cast<uint2*>(a.O + (int64_t)hd * a.o_head + (int64_t)(s.q0 + token) * a.o_row + ch) = w;
    if (lane == 0 && a.lse)
      a.lse[(int64_t)hd * a.total_q + s.q0 + token] = sum == 0.f ? NEG_INF : (top + log2f(sum)) * (1.f / LOG2E);
  }
}

template <int NG>
cudaError_t launch(const AttendArgs& a, int dev, cudaStream_t st) {
  using S = PromptSmem<NG>;
  static_assert(S::CUM + (KV4_PROMPT_MAX_B + 1) * 4 <= 227 * 1024, "shared memory of one CTA");
  static std::atomic<uint64_t> ready{0};
  if (device_pending(ready, dev)) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_prompt_kernel<NG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               S::CUM + (KV4_PROMPT_MAX_B + 1) * 4);
    if (e != cudaSuccess) return e;
    mark_device(ready, dev);
  }
  const int grid = std::min(sm_count(), KV4_MAX_CTAS);
  count_launches(2);
  kv4_prompt_kernel<NG><<<grid, THREADS, S::CUM + (a.B + 1) * 4, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  kv4_prompt_join_kernel<<<dim3(grid, PAIR / JOIN_ROWS), JOIN_THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv4_prompt_partial_bytes() {
  return (size_t)KV4_MAX_CTAS * (2 * PAIR * PART * sizeof(float) + sizeof(JoinInfo));
}

cudaError_t launch_kv4_prompt(const AttendArgs& a, int ng, int dev, cudaStream_t st) {
  return ng == 1 ? launch<1>(a, dev, st) : ng == 2 ? launch<2>(a, dev, st) : launch<4>(a, dev, st);
}

}  // namespace msa
