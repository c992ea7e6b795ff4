// Attention over the paged 4-bit cache (msa_kv4_attend).
//
// With k_j = lo_j + step_j c_j per group of channels, the scores need no dequantised key:
//   s_j = sum_g step_jg (q_g . c_jg) + lo_jg sum(q_g),
// and with p_j the probabilities, o_g = sum_j (p_j step_jg) c_jg + sum_j p_j lo_jg.  The two
// contractions run on the bare codes, exact in fp16: a nibble masked out of a packed word IS a pair of
// fp16 subnormals (value code * 2^-24, or code * 2^-20 for the upper nibble of a byte), so a
// 32-bit word of eight codes becomes four operand registers with one shift and four ANDs, no
// conversion and no subtraction.  The factors 2^24 and 16 are taken out where the scales enter.
//
// One CTA per SM.  The keys of every (request, KV head, tile of query rows) are cut into tiles of 32;
// the tiles of all of them form one line, of which every CTA takes an equal stretch, whatever the
// lengths are.  A warp owns every W-th tile of the CTA's stretch: it fetches a tile (two blocks of
// 16 tokens, K and V codes and scales contiguous) with one or two bulk copies into a ring of its
// own, so no barrier spans warps while keys stream.  Products are S^T = C_K Q^T and
// O^T = C_V^T P^T (mma.sync m16n8k16: the codes are the 16-row operand, 8 query rows per column
// block), each warp with its own running maximum and sums; the warps' results join in shared memory
// at the end of a segment, and the CTAs' through the workspace, in a fixed order, by the CTA that
// arrives last.  mma.sync rather than tcgen05: the operands go from shared memory to registers as
// 4-bit words and are never written back, and at 8 rows a key the products need under half of
// mma.sync's rate at full HBM bandwidth.
//
// Bound by HBM for long contexts: 2 (64 + 4 NG) bytes per key and KV head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "kv4.cuh"
#include "msa_internal.h"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int HD = 128;       // channels
constexpr int TK = 32;        // keys of a tile
constexpr int MAX_CTAS = 160;
constexpr int MAX_ROWS = 16;  // query rows of a tile, most
constexpr int PART = HD + 2;  // floats of a partial row: O, running maximum, sum
constexpr float LOG2E = 1.4426950408889634f;
constexpr float NEG_INF = -__builtin_huge_valf();

struct AttendArgs {
  Kv4View c;
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  int64_t q_head, q_row, o_head, o_row;
  const int32_t *table, *kv_lens, *cu_q;
  int64_t table_stride;
  int32_t max_blocks, B, total_q, Hq, group;  // group: query heads of a KV head
  float scale2;                               // softmax scale * log2(e)
  float* lse;
  uint32_t* arrivals;  // [MAX_CTAS]
  float* partial;      // [MAX_CTAS][2][MAX_ROWS][PART]
};

// One (request, KV head, tile of query rows) and its place on the line of key tiles.
struct Segment {
  int32_t b, h, rt;      // request, KV head, row tile
  int32_t n, kv, q0;     // new tokens, cached tokens, first query row
  int32_t first, count;  // tiles first .. first + count
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 1 / v of a power of two
__device__ __forceinline__ float inv_pow2(float v) { return __uint_as_float(0x7f000000u - __float_as_uint(v)); }

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Query rows of a KV head are numbered token * group + head of the group.
template <int NT>
__device__ __forceinline__ int row_tiles(int32_t n, int32_t group) {
  return (int)(((int64_t)n * group + 8 * NT - 1) / (8 * NT));
}

// The request's new tokens and cached tokens, cut to what Q and the table row hold.
__device__ __forceinline__ bool request_lens(const AttendArgs& a, int b, int32_t& q0, int32_t& n, int32_t& kv) {
  bool ok = true;
  q0 = a.cu_q[b];
  const int32_t q1 = a.cu_q[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.total_q) {
    ok = false;
    n = 0;
  } else {
    n = q1 - q0;
  }
  kv = a.kv_lens[b];
  const int64_t most = (int64_t)a.max_blocks << a.c.page_shift;
  if (kv < 0 || kv > most) {
    ok = false;
    kv = kv < 0 ? 0 : (int32_t)most;
  }
  return ok;
}

template <int NG, int NT, int W, int STAGES>
struct AttendSmem {
  static constexpr int TILE = 2 * Kv4Block<NG>::BYTES;
  static constexpr int ROWS = 8 * NT;
  static constexpr int JOIN = W / 2;  // warps' results side by side
  static constexpr int RING = 0;
  static constexpr int JOIN_AT = W * STAGES * TILE;
  static constexpr int STAT_AT = JOIN_AT + JOIN * ROWS * HD * 4;  // [JOIN][ROWS][2]
  static constexpr int BARS = STAT_AT + JOIN * ROWS * 2 * 4;
  static constexpr int CUM = BARS + W * STAGES * 8 + 64;  // [B + 1]
};

template <int NG, int NT, int W, int STAGES>
__global__ void __launch_bounds__(W * 32, 1) kv4_attend_kernel(const AttendArgs a) {
  using S = AttendSmem<NG, NT, W, STAGES>;
  using Blk = Kv4Block<NG>;
  constexpr int ROWS = 8 * NT;
  constexpr int THREADS = W * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + S::JOIN_AT);
  float* stat = reinterpret_cast<float*>(smem + S::STAT_AT);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BARS);
  int32_t* cum = reinterpret_cast<int32_t*>(smem + S::CUM);
  __shared__ int64_t sums[32];
  __shared__ int abort_flag, bad, arrived_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  if (tid == 0) {
    abort_flag = 0;
    bad = 0;
    cum[0] = 0;
    for (int i = 0; i < W * STAGES; ++i) mbar_init(bars + i, 1);
    fence_barrier_init();
  }
  __syncthreads();

  // ---- the line of tiles: running sum of the requests' tile counts ----
  int64_t run = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + tid;
    int64_t x = 0;
    if (b < a.B) {
      int32_t q0, n, kv;
      if (!request_lens(a, b, q0, n, kv)) bad = 1;
      x = (int64_t)row_tiles<NT>(n, a.group) * a.c.Hkv * max(1, (kv + TK - 1) / TK);
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
    for (int w = 0; w < W; ++w) run += sums[w];
    __syncthreads();
  }
  if (run > 0x7fffffff) {  // more tiles than the line has numbers for
    if (tid == 0) atomicOr(a.c.state, DEV_ERR_BOUNDS);
    return;
  }
  if (blockIdx.x == 0 && tid == 0 && bad) atomicOr(a.c.state, DEV_ERR_BOUNDS);
  // a CTA takes at least a tile per warp where there are that many
  const int total = (int)run;
  const int active = min((int)gridDim.x, max(1, (total + W - 1) / W));
  if ((int)blockIdx.x >= active || total == 0) return;
  const auto edge = [&](int i) { return (int)((int64_t)total * i / active); };
  const int t0 = edge(blockIdx.x), t1 = edge(blockIdx.x + 1);

  const auto locate = [&](int t) {  // the segment that holds tile t
    Segment s;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (cum[m] <= t) lo = m;
      else hi = m;
    }
    s.b = lo;
    request_lens(a, lo, s.q0, s.n, s.kv);
    s.count = max(1, (s.kv + TK - 1) / TK);
    const int i = (t - cum[lo]) / s.count;
    const int rts = row_tiles<NT>(s.n, a.group);
    s.h = i / rts;
    s.rt = i - s.h * rts;
    s.first = cum[lo] + i * s.count;
    return s;
  };
  // keys that the last row of the segment's tile sees (none: <= 0)
  const auto seen_by_last = [&](const Segment& s) {
    const int last_row = min((s.rt + 1) * ROWS, s.n * a.group) - 1;
    return s.kv - s.n + last_row / a.group + 1;
  };

  // ---- this warp's ring: tiles t0 + warp, + W, ... in order, across segments ----
  uint8_t* ring = smem + S::RING + warp * STAGES * S::TILE;
  uint64_t* bar = bars + warp * STAGES;
  Segment ps = locate(t0);
  int p_seen = seen_by_last(ps);
  int pt = t0 + warp;
  int p_stage = 0, in_flight = 0;
  uint32_t holds = 0;  // 2 bits per stage: which blocks of 16 tokens were fetched
  int2 entry = make_int2(-1, -1);
  int entry_at = 0;    // lane l has the table entries of tile entry_at + W l
  bool entry_ok = false;
  const auto fetch = [&]() {
    if (pt >= t1) return;
    while (pt >= ps.first + ps.count) {
      ps = locate(ps.first + ps.count);
      p_seen = seen_by_last(ps);
      entry_ok = false;
    }
    if (!entry_ok || pt - entry_at >= 32 * W) {
      const int my = pt + W * lane;
      entry = make_int2(-1, -1);
      if (my < ps.first + ps.count) {
        const int b0 = ((my - ps.first) * TK) >> a.c.page_shift, b1 = ((my - ps.first) * TK + 16) >> a.c.page_shift;
        const int32_t* row = a.table + ps.b * a.table_stride;
        if (b0 < a.max_blocks) entry.x = row[b0];
        if (b1 < a.max_blocks) entry.y = b1 == b0 ? entry.x : row[b1];
      }
      entry_at = pt;
      entry_ok = true;
    }
    const int from = (pt - entry_at) / W;
    const int32_t page0 = __shfl_sync(0xffffffffu, entry.x, from), page1 = __shfl_sync(0xffffffffu, entry.y, from);
    const int tok = (pt - ps.first) * TK;
    const bool want0 = tok < p_seen, want1 = tok + 16 < p_seen;
    const bool ok0 = want0 && page0 >= 0 && page0 < a.c.n_pages, ok1 = want1 && page1 >= 0 && page1 < a.c.n_pages;
    if (lane == 0) {
      if (want0 != ok0 || want1 != ok1) bad = 1;
      const uint32_t dst = smem_addr(ring + p_stage * S::TILE);
      uint64_t* br = bar + p_stage;
      const int in_page = (tok & (a.c.page_tokens() - 1)) >> 4;
      const uint8_t* s0 = a.c.pages + ((int64_t)page0 * a.c.Hkv + ps.h) * a.c.page_bytes + in_page * Blk::BYTES;
      mbar_arrive_expect_tx(br, ((int)ok0 + (int)ok1) * Blk::BYTES);
      if (ok0 && ok1 && a.c.page_shift > 4) {
        bulk_load(dst, s0, 2 * Blk::BYTES, br);
      } else {
        if (ok0) bulk_load(dst, s0, Blk::BYTES, br);
        if (ok1)
          bulk_load(dst + Blk::BYTES,
                    a.c.page_shift > 4 ? s0 + Blk::BYTES
                                       : a.c.pages + ((int64_t)page1 * a.c.Hkv + ps.h) * a.c.page_bytes,
                    Blk::BYTES, br);
      }
    }
    holds = (holds & ~(3u << (2 * p_stage))) | (((uint32_t)ok0 | (uint32_t)ok1 << 1) << (2 * p_stage));
    p_stage = p_stage + 1 == STAGES ? 0 : p_stage + 1;
    ++in_flight;
    pt += W;
  };
  for (int i = 0; i < STAGES; ++i) fetch();

  int c_stage = 0;
  uint32_t c_parity = 0;
  int tile = t0 + warp;
  const int key_of = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;  // key of operand row g, in 8

  for (int at = t0; at < t1;) {
    const Segment s = locate(at);
    const int s_end = min(s.first + s.count, t1);
    const int seen = min(seen_by_last(s), s.kv);
    const int row0 = s.rt * ROWS, rows = min(ROWS, s.n * a.group - row0);
    const int seen_first = s.kv - s.n + row0 / a.group + 1;

    // ---- queries: operand B of S^T, column g = row, scaled by a power of two into fp16 ----
    uint32_t qf[NT][8][2];
    float qs[NG][NT][2];
    int lim[NT][2];
    float to_score;
    {
      uint4 raw[NT][4];
      float top = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + g;
        const bool live = nt * 8 + g < rows;
        const int tok = live ? r / a.group : 0, hd = live ? r - tok * a.group : 0;
        const __nv_bfloat16* q = a.Q + (int64_t)(s.h * a.group + hd) * a.q_head + (int64_t)(s.q0 + tok) * a.q_row;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          raw[nt][i] = live ? *reinterpret_cast<const uint4*>(q + 32 * i + 8 * c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[nt][i].x, raw[nt][i].y, raw[nt][i].z, raw[nt][i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf_lo(w[k])), fabsf(bf_hi(w[k]))));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rc = row0 + nt * 8 + 2 * c + e;
          lim[nt][e] = nt * 8 + 2 * c + e < rows ? s.kv - s.n + rc / a.group + 1 : s.kv;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // 2^10 over the largest magnitude, rounded down to a power of two: exact but for elements
      // 2^-24 of the largest and below
      const int ex = (int)((__float_as_uint(top) >> 23) & 255);
      const int up = max(-100, min(100, 136 - ex));
      const float norm = __uint_as_float((uint32_t)(127 + up) << 23);
      to_score = a.scale2 * __uint_as_float((uint32_t)(127 - up) << 23) * 16777216.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = raw[nt][i];
          const float x0 = bf_lo(v.x), x1 = bf_hi(v.x), x2 = bf_lo(v.y), x3 = bf_hi(v.y);
          const float x4 = bf_lo(v.z), x5 = bf_hi(v.z), x6 = bf_lo(v.w), x7 = bf_hi(v.w);
          sum[i] = ((x0 + x1) + (x2 + x3)) + ((x4 + x5) + (x6 + x7));
          const float n16 = norm * 0.0625f;
          qf[nt][2 * i][0] = half2_bits(x0 * norm, x4 * norm);
          qf[nt][2 * i][1] = half2_bits(x1 * n16, x5 * n16);
          qf[nt][2 * i + 1][0] = half2_bits(x2 * norm, x6 * norm);
          qf[nt][2 * i + 1][1] = half2_bits(x3 * n16, x7 * n16);
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          float x = 0.f;
#pragma unroll
          for (int i = gr * 4 / NG; i < (gr + 1) * 4 / NG; ++i) x += sum[i];
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          qs[gr][nt][0] = a.scale2 * __shfl_sync(0xffffffffu, x, 8 * c);
          qs[gr][nt][1] = a.scale2 * __shfl_sync(0xffffffffu, x, 8 * c + 4);
        }
      }
    }

    float o[8][NT][4], z[NG][NT][2], m[NT][2], l[NT][2];
    float vtop = 0x1p-100f;  // power of two above every V step so far
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = NEG_INF;
        l[nt][e] = 0.f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) z[gr][nt][e] = 0.f;
      }
    }

    for (; tile < s_end; tile += W) {
      const bool there = mbar_wait(bar + c_stage, c_parity, &abort_flag);
      const uint8_t* kb = ring + c_stage * S::TILE;
      const uint32_t have = there ? (holds >> (2 * c_stage)) & 3u : 0u;
      const int tok = (tile - s.first) * TK;
      if (have) {
        // keys from here on are hidden from every row: behind the last row's, or on no page
        const bool partial = have != 3u || tok + TK > min(seen_first, s.kv);
        float sc[2][NT][4];
        uint32_t vsw[2][2][NG];
        float vmax = 0.f;
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint8_t* blk = kb + mt * Blk::BYTES;
          const uint4 k0 = *reinterpret_cast<const uint4*>(blk + 64 * key_of + 16 * c);
          const uint4 k1 = *reinterpret_cast<const uint4*>(blk + 64 * (key_of + 8) + 16 * c);
          float acc[NG][NT][4];
#pragma unroll
          for (int gr = 0; gr < NG; ++gr)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[gr][nt][e] = 0.f;
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u0 = w0[i] >> 8, u1 = w1[i] >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(acc[i * NG / 4][nt], w0[i] & 0x000f000fu, w1[i] & 0x000f000fu, w0[i] & 0x00f000f0u,
                       w1[i] & 0x00f000f0u, qf[nt][2 * i][0], qf[nt][2 * i][1]);
              mma16816(acc[i * NG / 4][nt], u0 & 0x000f000fu, u1 & 0x000f000fu, u0 & 0x00f000f0u, u1 & 0x00f000f0u,
                       qf[nt][2 * i + 1][0], qf[nt][2 * i + 1][1]);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int key = tok + 16 * mt + 8 * r + key_of;
            const bool shown = key < seen && ((have >> mt) & 1u);
            uint32_t ksw[NG];
            const uint32_t* kp = reinterpret_cast<const uint32_t*>(blk + Blk::K_SCALES + 4 * NG * (key_of + 8 * r));
            const uint32_t* vp = reinterpret_cast<const uint32_t*>(blk + Blk::V_SCALES + 4 * NG * (key_of + 8 * r));
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              ksw[gr] = kp[gr];
              vsw[mt][r][gr] = vp[gr];
              if (partial && !shown) ksw[gr] = 0, vsw[mt][r][gr] = 0;
              vmax = fmaxf(vmax, bf_lo(vsw[mt][r][gr]));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = 0.f;
#pragma unroll
                for (int gr = 0; gr < NG; ++gr)
                  x = fmaf(acc[gr][nt][2 * r + e], bf_lo(ksw[gr]) * to_score, fmaf(bf_hi(ksw[gr]), qs[gr][nt][e], x));
                if (partial && (!shown || key >= lim[nt][e])) x = NEG_INF;
                sc[mt][nt][2 * r + e] = x;
                grow |= x > m[nt][e] + 8.f;
              }
          }
        }
        grow |= vmax > vtop;
        if (__any_sync(0xffffffffu, grow)) {
          // a score 2^8 above the running maximum (or a V step above every one before): the
          // maximum is taken anew and what was summed so far is scaled down
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
          const float vnew = fmaxf(vtop, __uint_as_float((__float_as_uint(vmax) + 0x007fffffu) & 0x7f800000u));
          const float fv = vtop * inv_pow2(vnew);
          vtop = vnew;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][2 + e]), fmaxf(sc[1][nt][e], sc[1][nt][2 + e]));
#pragma unroll
              for (int off = 16; off > 2; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
              const float mn = fmaxf(m[nt][e], x);
              const float f = mn == m[nt][e] ? 1.f : ex2(m[nt][e] - mn);
              m[nt][e] = mn;
              l[nt][e] *= f;
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) z[gr][nt][e] *= f;
#pragma unroll
              for (int t = 0; t < 8; ++t) {
                o[t][nt][e] *= f * fv;
                o[t][nt][2 + e] *= f * fv;
              }
            }
        }
        const float vinv = 128.f * inv_pow2(vtop);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t pf[NG][NT][2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float p[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                p[nt][e] = ex2(sc[mt][nt][2 * r + e] - (m[nt][e] == NEG_INF ? 0.f : m[nt][e]));
                l[nt][e] += p[nt][e];
              }
            const int key = tok + 16 * mt + 8 * r + key_of;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              const float vs = bf_lo(vsw[mt][r][gr]) * vinv, vz = bf_hi(vsw[mt][r][gr]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  // a key hidden from this row alone may hold NaN: no product with it
                  const bool hidden = partial && key >= lim[nt][e];
                  y[e] = hidden ? 0.f : p[nt][e] * vs;
                  z[gr][nt][e] += hidden ? 0.f : p[nt][e] * vz;
                }
                pf[gr][nt][r] = transpose8x8(half2_bits(y[0], y[1]));
              }
            }
          }
          const uint8_t* vb = kb + mt * Blk::BYTES + Blk::V_CODES;
          uint2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // keys 2c, 2c + 1, 2c + 8, 2c + 9 of the operand
            const int key = ((i & 1) ? 4 + (c ^ 1) : c) + 8 * (i >> 1);
            v[i] = *reinterpret_cast<const uint2*>(vb + 64 * key + 8 * (g ^ kv4_v_swizzle(key)));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t sel = (q & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = (q >> 1) ? __byte_perm(v[0].y, v[1].y, sel) : __byte_perm(v[0].x, v[1].x, sel);
            const uint32_t y = (q >> 1) ? __byte_perm(v[2].y, v[3].y, sel) : __byte_perm(v[2].x, v[3].x, sel);
            const uint32_t x8 = x >> 8, y8 = y >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t b0 = pf[q * NG / 4][nt][0], b1 = pf[q * NG / 4][nt][1];
              mma16816(o[2 * q][nt], x & 0x000f000fu, x & 0x00f000f0u, y & 0x000f000fu, y & 0x00f000f0u, b0, b1);
              mma16816(o[2 * q + 1][nt], x8 & 0x000f000fu, x8 & 0x00f000f0u, y8 & 0x000f000fu, y8 & 0x00f000f0u, b0, b1);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      --in_flight;
      if (++c_stage == STAGES) c_stage = 0, c_parity ^= 1;
      fetch();
    }

    // ---- the warp's rows: sums over its lanes, values instead of codes ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) z[gr][nt][e] += __shfl_xor_sync(0xffffffffu, z[gr][nt][e], off);
        }
    const float of = vtop * 131072.f;  // 2^24 / 2^7
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          o[t][nt][e] = fmaf(o[t][nt][e], of, z[(t >> 1) * NG / 4][nt][e]);
          o[t][nt][2 + e] = fmaf(o[t][nt][2 + e], of * 0.0625f, z[(t >> 1) * NG / 4][nt][e]);
        }
    const auto weight = [](float x, float top) { return x == NEG_INF ? 0.f : ex2(x - top); };
    const int slot = warp & (S::JOIN - 1);
    for (int half = 1; half >= 0; --half) {
      if (warp / S::JOIN == half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = nt * 8 + 2 * c + e;
            float* row = join + (slot * ROWS + r) * HD;
            float* st = stat + (slot * ROWS + r) * 2;
            float f = 1.f, f2 = 0.f;
            if (half == 0) {  // the other half's rows are there: add them
              const float m2 = st[0], l2 = st[1], mn = fmaxf(m[nt][e], m2);
              f = weight(m[nt][e], mn);
              f2 = weight(m2, mn);
              m[nt][e] = mn;
              l[nt][e] = l[nt][e] * f + l2 * f2;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float4* d = reinterpret_cast<float4*>(row + 32 * q + 4 * g);
              float4 x = make_float4(o[2 * q][nt][e] * f, o[2 * q][nt][2 + e] * f, o[2 * q + 1][nt][e] * f,
                                     o[2 * q + 1][nt][2 + e] * f);
              if (half == 0) {
                const float4 y = *d;
                x.x = fmaf(y.x, f2, x.x), x.y = fmaf(y.y, f2, x.y), x.z = fmaf(y.z, f2, x.z), x.w = fmaf(y.w, f2, x.w);
              }
              *d = x;
            }
            __syncwarp();  // the row's statistics were read by every lane of it
            if (g == 0) st[0] = m[nt][e], st[1] = l[nt][e];
          }
      }
      __syncthreads();
    }

    // ---- the CTA's rows, to O or to the workspace ----
    const bool whole = s.first >= t0 && s.first + s.count <= t1;
    const auto write_row = [&](int r, int ch, float4 x, float top, float sum) {
      const int rc = row0 + r, token = rc / a.group, hd = s.h * a.group + rc - token * a.group;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      uint2 w;
      w.x = pack_bf16x2(x.x * inv, x.y * inv);
      w.y = pack_bf16x2(x.z * inv, x.w * inv);
      *reinterpret_cast<uint2*>(a.O + (int64_t)hd * a.o_head + (int64_t)(s.q0 + token) * a.o_row + ch) = w;
      if (ch == 0 && a.lse)
        a.lse[(int64_t)hd * a.total_q + s.q0 + token] = sum == 0.f ? NEG_INF : (top + log2f(sum)) * (1.f / LOG2E);
    };
    float* mine = a.partial + (2 * (int64_t)blockIdx.x + (s.first >= t0 ? 1 : 0)) * MAX_ROWS * PART;
    for (int i = tid; i < rows * (HD / 4); i += THREADS) {
      const int r = i / (HD / 4), ch = (i % (HD / 4)) * 4;
      float top = NEG_INF, sum = 0.f;
#pragma unroll
      for (int j = 0; j < S::JOIN; ++j) top = fmaxf(top, stat[(j * ROWS + r) * 2]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < S::JOIN; ++j) {
        const float f = weight(stat[(j * ROWS + r) * 2], top);
        const float4 y = *reinterpret_cast<const float4*>(join + (j * ROWS + r) * HD + ch);
        sum = fmaf(stat[(j * ROWS + r) * 2 + 1], f, sum);
        x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
      }
      if (whole) {
        write_row(r, ch, x, top, sum);
      } else {
        *reinterpret_cast<float4*>(mine + r * HD + ch) = x;
        if (ch == 0) {
          mine[MAX_ROWS * HD + 2 * r] = top;
          mine[MAX_ROWS * HD + 2 * r + 1] = sum;
        }
      }
    }
    if (!whole) {
      const auto owner = [&](int t) { return (int)((((int64_t)t + 1) * active - 1) / total); };
      const int from = owner(s.first), to = owner(s.first + s.count - 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        arrived_last = atomicAdd(a.arrivals + from, 1u) == (uint32_t)(to - from);
        if (arrived_last) a.arrivals[from] = 0;  // ready for the next launch
        __threadfence();
      }
      __syncthreads();
      if (arrived_last) {
        const auto part = [&](int i) { return a.partial + (2 * (int64_t)i + (i == from ? 1 : 0)) * MAX_ROWS * PART; };
        for (int i = tid; i < rows * (HD / 4); i += THREADS) {
          const int r = i / (HD / 4), ch = (i % (HD / 4)) * 4;
          float top = NEG_INF, sum = 0.f;
          for (int k = from; k <= to; ++k) top = fmaxf(top, __ldcg(part(k) + MAX_ROWS * HD + 2 * r));
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = from; k <= to; ++k) {
            const float* p = part(k);
            const float2 st = __ldcg(reinterpret_cast<const float2*>(p + MAX_ROWS * HD + 2 * r));
            const float4 y = __ldcg(reinterpret_cast<const float4*>(p + r * HD + ch));
            const float f = weight(st.x, top);
            sum = fmaf(st.y, f, sum);
            x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
          }
          write_row(r, ch, x, top, sum);
        }
      }
    }
    __syncthreads();  // join and stat are free again
    at = s_end;
  }
  // nothing is in flight here unless a wait gave up: let what was issued land
  for (; in_flight > 0; --in_flight) {
    int none = 0;
    mbar_wait(bar + c_stage, c_parity, &none);
    if (++c_stage == STAGES) c_stage = 0, c_parity ^= 1;
  }
  __syncthreads();
  if (tid == 0) {
    if (abort_flag) atomicOr(a.c.state, DEV_ERR_TIMEOUT);
    if (bad) atomicOr(a.c.state, DEV_ERR_BOUNDS);
  }
}

template <int NG, int NT, int W, int STAGES>
cudaError_t launch(const AttendArgs& a, int dev, cudaStream_t st) {
  using S = AttendSmem<NG, NT, W, STAGES>;
  static_assert(S::CUM + (KV4_MAX_B + 1) * 4 <= 226 * 1024, "shared memory of one CTA");
  static_assert(8 * NT <= MAX_ROWS, "rows of a partial result");
  static std::atomic<uint64_t> ready{0};
  if (device_pending(ready, dev)) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_attend_kernel<NG, NT, W, STAGES>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               S::CUM + (KV4_MAX_B + 1) * 4);
    if (e != cudaSuccess) return e;
    mark_device(ready, dev);
  }
  count_launches(1);
  kv4_attend_kernel<NG, NT, W, STAGES>
      <<<std::min(sm_count(), MAX_CTAS), W * 32, S::CUM + (a.B + 1) * 4, st>>>(a);
  return cudaGetLastError();
}

template <int NG>
cudaError_t launch_rows(const AttendArgs& a, int max_q, int dev, cudaStream_t st) {
  if ((int64_t)max_q * a.group <= 8) return launch<NG, 1, 16, 2>(a, dev, st);
  return launch<NG, 2, 8, 4>(a, dev, st);
}

constexpr size_t ARRIVALS_BYTES = 1024;
static_assert(ARRIVALS_BYTES >= MAX_CTAS * 4, "a counter per CTA");

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_kv4_attend_workspace_bytes(void) {
  return ARRIVALS_BYTES + (size_t)MAX_CTAS * 2 * MAX_ROWS * PART * sizeof(float);
}

msa_status msa_kv4_attend(const msa_kv4_cache* cache, const void* Q, void* O, const msa_strides* strides,
                          int32_t total_q, int32_t Hq, float scale, const int32_t* block_table, int64_t table_stride,
                          int32_t max_blocks, const int32_t* kv_lens, const int32_t* cu_q, int32_t B, int32_t max_q,
                          float* lse, void* ws, size_t ws_bytes, void* stream) {
  AttendArgs a{};
  const msa_status st = kv4_view(cache, &a.c);
  if (st != MSA_OK) return st;
  if (!strides || total_q < 0 || B < 0 || max_q < 0 || max_blocks < 0 || !(scale > 0.f) || scale > 3.4e38f)
    return MSA_ERR_INVALID_ARG;
  if (Hq < 1 || Hq % cache->Hkv) return MSA_ERR_SHAPE;
  if (table_stride < max_blocks) return MSA_ERR_SHAPE;
  if (B > KV4_MAX_B || Hq > 65536) return MSA_ERR_UNSUPPORTED;
  if (((int64_t)max_blocks << a.c.page_shift) > 0x7fffffff) return MSA_ERR_UNSUPPORTED;
  if ((int64_t)total_q * (Hq / cache->Hkv) > 0x7fffffff) return MSA_ERR_UNSUPPORTED;
  if (!ws) return MSA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) % 256) return MSA_ERR_ALIGN;
  if (ws_bytes < msa_kv4_attend_workspace_bytes()) return MSA_ERR_WORKSPACE;
  if (total_q == 0 || B == 0) return MSA_OK;
  if (!Q || !O || !kv_lens || !cu_q || (max_blocks && !block_table)) return MSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(O)) & 15) return MSA_ERR_ALIGN;
  if (strides->q_head % 8 || strides->q_row % 8 || strides->o_head % 8 || strides->o_row % 8) return MSA_ERR_ALIGN;
  a.Q = static_cast<const __nv_bfloat16*>(Q);
  a.O = static_cast<__nv_bfloat16*>(O);
  a.q_head = strides->q_head, a.q_row = strides->q_row, a.o_head = strides->o_head, a.o_row = strides->o_row;
  a.table = block_table, a.kv_lens = kv_lens, a.cu_q = cu_q, a.table_stride = table_stride;
  a.max_blocks = max_blocks, a.B = B, a.total_q = total_q, a.Hq = Hq, a.group = Hq / cache->Hkv;
  a.scale2 = scale * LOG2E;
  a.lse = lse;
  a.arrivals = static_cast<uint32_t*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ARRIVALS_BYTES);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MSA_ERR_CUDA;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (cache->group) {
    case 128: e = launch_rows<1>(a, max_q, dev, cs); break;
    case 64: e = launch_rows<2>(a, max_q, dev, cs); break;
    default: e = launch_rows<4>(a, max_q, dev, cs); break;
  }
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // extern "C"
