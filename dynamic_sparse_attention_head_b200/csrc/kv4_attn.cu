// Attention over the paged 4-bit cache (msa_kv4_attend).
//
// With k_j = lo_j + step_j c_j per group of channels, the scores need no dequantised key:
//   s_j = sum_g step_jg (q_g . c_jg) + lo_jg sum(q_g),
// and with p_j the probabilities, o_g = sum_j (p_j step_jg) c_jg + sum_j p_j lo_jg.  The two
// contractions run on the bare codes, exact in fp16.  For the scores a nibble masked out of a packed
// word IS a pair of fp16 subnormals (value code * 2^-24, or code * 2^-20 for the upper nibble of a
// byte), so a 32-bit word of eight codes becomes four operand registers with one shift and four
// ANDs, no conversion and no subtraction.  The factors 2^24 and 16 are taken out where the scales
// enter.  The values' codes are centred first (code - 8, one more subtraction a pair, and
// lo + 8 step in place of lo): a tensor core cuts its fp32 sums off instead of rounding them, and
// a long sum of codes of one sign drifts by that, against the sum of lo that it all but cancels
// (1M keys: relative error 3.2e-3 with bare codes).
//
// One CTA per SM.  The keys of every (request, KV head, tile of query rows) are cut into tiles, with
// one unit more per such segment for what its start and end cost; the units of all segments form one
// line, of which every warp takes an equal stretch, whatever the lengths are.  A warp fetches its
// tiles (blocks of 16 tokens, K and V codes and scales contiguous) with bulk copies into a ring of
// its own, ahead across segment borders, so no barrier spans warps while keys stream.  Products are
// S^T = C_K Q^T and O^T = C_V^T P^T (mma.sync m16n8k16: the codes are the 16-row operand, 8 query
// rows per column block), each warp with its own running maximum and sums.  A segment inside one
// warp's stretch is written by it; what crosses warps joins in shared memory at the end, what
// crosses CTAs through the workspace, in a fixed order, by the CTA that arrives last.  mma.sync
// rather than tcgen05: the operands go from shared memory to registers as 4-bit words and are never
// written back, and at 8 rows a key the products need about half of mma.sync's rate at full HBM
// bandwidth.
//
// Floor for long contexts: HBM, 2 (64 + 4 NG) bytes per key and KV head.  Measured: 64 requests of up to 16384
// tokens, 32 / 8 heads, groups of 128: 122 to 126 us, 4.5 TB/s (a copy: 6.44); one token over 1048576, 28 / 4 heads,
// groups of 64: 134 to 136 us, the same rate; 4 requests of up to 700 tokens: 12.3 us.  Bound by the issue of 12 warps an SM (57 to
// 60 %, ALU 56 %: 259 instructions per 16 keys, half of them to take the codes apart) and, for 11 % of the
// time, by the start and the joins.
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

constexpr int HD = 128;       // channels
constexpr int MAX_ROWS = 16;  // query rows of a tile, most
constexpr int MAX_WARP_ROWS = 128;  // warps times rows of a CTA, most
constexpr int PART = HD + 2;  // floats of a partial row: O, running maximum, sum
constexpr float LOG2E = 1.4426950408889634f;
constexpr float NEG_INF = -__builtin_huge_valf();

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

// Codes in bits 0-3 (4-7) of both halves as fp16 code - 8 (16 (code - 8)): the code is set into the
// mantissa of 1024, whose step is one, and 1024 + 8 (1024 + 128) is taken off; both are exact.
template <uint32_t MASK, uint32_t BASE>
__device__ __forceinline__ uint32_t centred(uint32_t w, uint32_t k1024) {
  uint32_t v;  // (w & MASK) | k1024 in one instruction
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "n"(MASK), "r"(k1024));
  const uint32_t b = BASE;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t centred_lo(uint32_t w, uint32_t k1024) {
  return centred<0x000f000fu, 0x64086408u>(w, k1024);
}
__device__ __forceinline__ uint32_t centred_hi(uint32_t w, uint32_t k1024) {
  return centred<0x00f000f0u, 0x64806480u>(w, k1024);
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

__device__ __forceinline__ float weight_of(float x, float top) { return x == NEG_INF ? 0.f : ex2(x - top); }

// Adds U partial results (maximum and sum st, four channels y) to (top, sum, x).
template <int U>
__device__ __forceinline__ void add_parts(float& top, float& sum, float4& x, const float2 (&st)[U], const float4 (&y)[U]) {
  float up = top;
#pragma unroll
  for (int u = 0; u < U; ++u) up = fmaxf(up, st[u].x);
  const float f0 = weight_of(top, up);
  top = up;
  sum *= f0;
  x.x *= f0, x.y *= f0, x.z *= f0, x.w *= f0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float f = weight_of(st[u].x, top);
    sum = fmaf(st[u].y, f, sum);
    x.x = fmaf(y[u].x, f, x.x), x.y = fmaf(y[u].y, f, x.y), x.z = fmaf(y[u].z, f, x.z), x.w = fmaf(y[u].w, f, x.w);
  }
}

// units of a segment: its tiles (2^shift keys each), and one for what its start and end cost
__device__ __forceinline__ int units_of(int kv, int shift) {
  return 1 + (int)(((int64_t)kv + (1 << shift) - 1) >> shift);
}

// The segment that holds unit t.  Out of line: a launch of few tiles is bound by fetching its code.
template <int NT>
__device__ __noinline__ Segment segment_at(const AttendArgs& a, const int32_t* cum, int shift, int t) {
  Segment s;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (cum[m] <= t) lo = m;
    else hi = m;
  }
  s.b = lo;
  request_lens(a, lo, s.q0, s.n, s.kv);
  s.count = units_of(s.kv, shift);
  const int i = (t - cum[lo]) / s.count;
  const int rts = row_tiles<NT>(s.n, a.group);
  s.h = rts == 1 ? i : i / rts;
  s.rt = i - s.h * rts;
  s.first = cum[lo] + i * s.count;
  return s;
}

template <int NG, int NT, int TK, int W, int STAGES>
struct AttendSmem {
  static constexpr int TILE = TK / 16 * Kv4Block<NG>::BYTES;
  static constexpr int ROWS = 8 * NT;
  static constexpr int ROW_BYTES = ROWS * HD * 4;
  static constexpr int RING = 0;  // a warp's tail result lies in its ring once its tiles are used up
  static constexpr int STATS = W * STAGES * TILE;                // [W][head, tail][ROWS][2]
  static constexpr int SEGS = STATS + W * 2 * ROWS * 2 * 4;      // [W + 1]: tails; the CTA's head
  static constexpr int BARS = SEGS + (W + 1) * (int)sizeof(Segment);
  static constexpr int CUM = BARS + W * STAGES * 8;              // [B + 1]
  static_assert(STAGES * TILE >= ROW_BYTES, "a tail result fits the ring");
  static_assert(BARS % 8 == 0 && CUM % 4 == 0, "alignment");
};

template <int NG, int NT, int TK, int W, int STAGES>
__global__ void __launch_bounds__(W * 32, 1) kv4_attend_kernel(const __grid_constant__ AttendArgs a) {
  using S = AttendSmem<NG, NT, TK, W, STAGES>;
  using Blk = Kv4Block<NG>;
  constexpr int ROWS = 8 * NT;
  constexpr int THREADS = W * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  float* heads = a.heads + (int64_t)blockIdx.x * W * ROWS * HD;  // [W][ROWS][HD]
  float* stats = reinterpret_cast<float*>(smem + S::STATS);
  Segment* segs = reinterpret_cast<Segment*>(smem + S::SEGS);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BARS);
  int32_t* cum = reinterpret_cast<int32_t*>(smem + S::CUM);
  __shared__ int abort_flag, bad, last_of[2], last_to[2], line_total, line_shift;
  // 1: has a head, 2: the head's segment ends in the stretch, 4: has a tail, 8: the head is in the workspace
  __shared__ uint8_t ends[W];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  if (tid < W * STAGES) mbar_init(bars + tid, 1);
  if (tid == 0) abort_flag = 0;
  fence_barrier_init();

  // ---- the line of units: running sum of the requests' counts, by one warp ----
  // A unit is a tile of TK keys; or 16 keys, where that still leaves every warp less than a tile: short
  // contexts then spread over more warps.
  if (warp == 0) {
    uint32_t cut = 0;
    uint32_t blocks = 0;  // of 16 keys; of a lane at most 2^24, far above what is asked below
    constexpr int U = 4;  // requests of a lane on their way together
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32 * U) {
      int32_t q0[U], q1[U], kv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = min(b0 + 32 * u + lane, a.B - 1);
        q0[u] = a.cu_q[b], q1[u] = a.cu_q[b + 1], kv[u] = a.kv_lens[b];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int32_t n;
        if (!cut_lens(a, q0[u], q1[u], n, kv[u])) cut = 1;
        const uint64_t x = (uint64_t)row_tiles<NT>(n, a.group) * a.c.Hkv * ((kv[u] + 15) >> 4);
        if (b0 + 32 * u + lane < a.B) blocks = (uint32_t)min((uint64_t)blocks + x, (uint64_t)1 << 24);
      }
    }
    blocks = __reduce_add_sync(0xffffffffu, blocks);
    cut = __any_sync(0xffffffffu, cut);
    const int shift = blocks < gridDim.x * W * (TK / 16) ? 4 : (TK == 64 ? 6 : 5);
    uint64_t run = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int32_t q0, n = 0, kv = 0;
      if (b0 + lane < a.B) request_lens(a, b0 + lane, q0, n, kv);
      uint64_t x = (uint64_t)row_tiles<NT>(n, a.group) * a.c.Hkv * (uint32_t)units_of(kv, shift);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      x += run;
      if (b0 + lane < a.B) cum[b0 + lane + 1] = (int32_t)min(x, (uint64_t)0x7fffffff);
      run = __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      cum[0] = 0;
      line_total = run > 0x7fffffff ? -1 : (int)run;  // -1: more units than the line has numbers for
      line_shift = shift;
      bad = 0;
      if (blockIdx.x == 0 && (cut || run > 0x7fffffff)) atomicOr(a.c.state, DEV_ERR_BOUNDS);
    }
  }
  __syncthreads();
  const int total = line_total, unit_shift = line_shift;
  // a CTA takes at least a unit per warp where there are that many
  const int active = min((int)gridDim.x, max(1, (total + W - 1) / W));
  if ((int)blockIdx.x >= active || total <= 0) return;
  // floor(total i / active) and, below, the i whose stretch holds unit t, in 32 bits: a 64-bit quotient takes
  // several hundred cycles, and a short context's launch waits for four of them
  const int each = total / active, rest = total - each * active;
  const auto edge = [&](int i) { return each * i + rest * i / active; };
  const int t0 = edge(blockIdx.x), t1 = edge(blockIdx.x + 1);
  const uint32_t stretch = t1 - t0;  // of a whole GPU's 2^31 units: times W it fits 32 bits
  const int w0 = t0 + (int)(stretch * warp / W), w1 = t0 + (int)(stretch * (warp + 1) / W);

  const auto locate = [&](int t) { return segment_at<NT>(a, cum, unit_shift, t); };
  // keys that the last row of the segment's tile sees (none: <= 0)
  const auto seen_by_last = [&](const Segment& s) {
    const int last_row = min((s.rt + 1) * ROWS, s.n * a.group) - 1;
    return s.kv - s.n + a.by_group(last_row) + 1;
  };

  // ---- this warp's ring: the tiles of its stretch in order, across segments ----
  uint8_t* ring = smem + S::RING + warp * STAGES * S::TILE;
  uint64_t* bar = bars + warp * STAGES;
  // a copy is a page's part of the unit, or the unit: `per` copies a unit, 2^copy_shift tokens each
  const int copy_shift = min(a.c.page_shift, unit_shift), per = 1 << (unit_shift - copy_shift);
  const Segment first_seg = w0 < w1 ? locate(w0) : Segment{};
  if (w0 < w1) {  // its queries, on their way while the first tiles are looked up
    const int r = first_seg.rt * ROWS + lane % ROWS, token = min(a.by_group(r), first_seg.n - 1);
    const int hd = first_seg.h * a.group + r - a.by_group(r) * a.group;
    const __nv_bfloat16* q = a.Q + (int64_t)hd * a.q_head + (int64_t)(first_seg.q0 + token) * a.q_row;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(q + (lane / ROWS) * (HD * ROWS / 32)));
  }
  Segment ps;
  ps.first = w0;
  ps.count = 0;
  int p_seen = 0, p_tile = 0, p_end = 0;  // producer: next tile of its segment, and the first not its own
  int p_stage = 0, in_flight = 0;
  uint32_t holds = 0;  // `per` bits per stage: which copies were made
  int32_t entry = -1;  // lane l: table entry of copy entry_at + l
  int entry_at = 0;
  bool entry_ok = false;
  const auto fetch = [&]() {
    while (p_tile >= p_end) {  // on to the next segment of the stretch
      const int at = ps.first + ps.count;
      if (at >= w1) return;
      ps = at == w0 ? first_seg : locate(at);
      p_seen = seen_by_last(ps);
      // unit 0 of a segment carries no keys; tiles behind the last row's keys are not needed
      p_tile = max(at, w0) - ps.first - 1;
      p_tile = max(p_tile, 0);
      p_end = min(min(ps.first + ps.count, w1) - ps.first - 1, max(units_of(p_seen, unit_shift) - 1, 0));
      entry_ok = false;
    }
    const int first = p_tile * per;
    if (!entry_ok || first - entry_at >= 32) {
      entry_at = first;
      entry_ok = true;
      const int blk = (first + lane) << copy_shift >> a.c.page_shift;
      entry = -1;
      if (blk < a.max_blocks && ((first + lane) << copy_shift) < p_seen) entry = a.table[ps.b * a.table_stride + blk];
    }
    const int32_t page = __shfl_sync(0xffffffffu, entry, (first - entry_at + lane) & 31);
    const int tok = (first + lane) << copy_shift;
    const bool want = lane < per && tok < p_seen, ok = want && page >= 0 && page < a.c.n_pages;
    if (want && !ok) bad = 1;
    const uint32_t bytes = ok ? min(1 << copy_shift >> 4, (p_seen - tok + 15) >> 4) * Blk::BYTES : 0;
    const uint32_t all = __reduce_add_sync(0xffffffffu, bytes), made = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) mbar_arrive_expect_tx(bar + p_stage, all);
    __syncwarp();
    if (ok)
      bulk_load(smem_addr(ring + p_stage * S::TILE) + (lane << copy_shift >> 4) * Blk::BYTES,
                a.c.pages + ((int64_t)page * a.c.Hkv + ps.h) * a.c.page_bytes +
                    ((tok & (a.c.page_tokens() - 1)) >> 4) * Blk::BYTES,
                bytes, bar + p_stage);
    holds = (holds & ~(((1u << per) - 1) << (4 * p_stage))) | made << (4 * p_stage);
    p_stage = p_stage + 1 == STAGES ? 0 : p_stage + 1;
    ++in_flight;
    ++p_tile;
  };
  for (int i = 0; i < STAGES; ++i) fetch();

  int c_stage = 0;
  uint32_t c_parity = 0;
  uint32_t k1024;  // fp16 1024 twice, kept in a register
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));
  const int key_of = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;  // key of operand row g, in 8
  // four channels of row `rc` (token * group + head) of a segment
  const auto write_row = [&](const Segment& s, int rc, int token, int ch, float4 x, float top, float sum) {
    const int hd = s.h * a.group + rc - token * a.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint2 w;
    w.x = pack_bf16x2(x.x * inv, x.y * inv);
    w.y = pack_bf16x2(x.z * inv, x.w * inv);
    *reinterpret_cast<uint2*>(a.O + (int64_t)hd * a.o_head + (int64_t)(s.q0 + token) * a.o_row + ch) = w;
    if (ch == 0 && a.lse)
      a.lse[(int64_t)hd * a.total_q + s.q0 + token] = sum == 0.f ? NEG_INF : (top + log2f(sum)) * (1.f / LOG2E);
  };
  if (lane == 0) ends[warp] = 0;

  for (int at = w0; at < w1;) {
    const Segment s = at == w0 ? first_seg : locate(at);
    const int s_end = min(s.first + s.count, w1);
    const int seen = seen_by_last(s);
    const int row0 = s.rt * ROWS, rows = min(ROWS, s.n * a.group - row0);
    const int seen_first = s.kv - s.n + a.by_group(row0) + 1;

    // ---- queries: operand B of S^T, column g = row, each row scaled by a power of two of its own into
    // fp16 (a row of large or infinite channels leaves its neighbours as they are) ----
    uint32_t qf[NT][8][2];
    float qs[NG][NT][2];
    int lim[NT][2], token_of[NT][2];
    float to_score[NT][2];  // of columns 2c, 2c + 1, as qs
    {
      uint4 raw[NT][4];
      float top[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + g;
        const bool live = nt * 8 + g < rows;
        const int tok = live ? a.by_group(r) : 0, hd = live ? r - tok * a.group : 0;
        const __nv_bfloat16* q = a.Q + (int64_t)(s.h * a.group + hd) * a.q_head + (int64_t)(s.q0 + tok) * a.q_row;
        top[nt] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          raw[nt][i] = live ? *reinterpret_cast<const uint4*>(q + 32 * i + 8 * c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[nt][i].x, raw[nt][i].y, raw[nt][i].z, raw[nt][i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top[nt] = fmaxf(top[nt], fmaxf(fabsf(bf_lo(w[k])), fabsf(bf_hi(w[k]))));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rc = row0 + nt * 8 + 2 * c + e;
          token_of[nt][e] = a.by_group(rc);
          lim[nt][e] = nt * 8 + 2 * c + e < rows ? s.kv - s.n + token_of[nt][e] + 1 : s.kv;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        top[nt] = fmaxf(top[nt], __shfl_xor_sync(0xffffffffu, top[nt], 1));
        top[nt] = fmaxf(top[nt], __shfl_xor_sync(0xffffffffu, top[nt], 2));
        // 2^10 over the row's largest magnitude, rounded down to a power of two: exact but for elements
        // 2^-24 of the largest and below.  Its reciprocal and the 2^24 of the codes come back with the
        // softmax scale, in one product a score.
        const int ex = (int)((__float_as_uint(top[nt]) >> 23) & 255);
        const int up = max(-100, min(100, 136 - ex));
        const float norm = __uint_as_float((uint32_t)(127 + up) << 23), norm24 = __uint_as_float((uint32_t)(103 + up) << 23);
        const float back = a.scale2 * __uint_as_float((uint32_t)(127 - up) << 23) * 16777216.f;
        to_score[nt][0] = __shfl_sync(0xffffffffu, back, 8 * c);
        to_score[nt][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
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
          x *= norm24;
          qs[gr][nt][0] = __shfl_sync(0xffffffffu, x, 8 * c);
          qs[gr][nt][1] = __shfl_sync(0xffffffffu, x, 8 * c + 4);
        }
      }
    }

    // base: the running maximum, 0 before there is one (limit is -inf then: any score starts it;
    // later a score 2^8 above it does)
    float o[8][NT][4], z[NG][NT][2], base[NT][2], limit[NT][2], l[NT][2];
    float vtop = 0x1p-100f;  // power of two above every V step so far
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        base[nt][e] = 0.f;
        limit[nt][e] = NEG_INF;
        l[nt][e] = 0.f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) z[gr][nt][e] = 0.f;
      }
    }

    // 16 MT keys from `tok` on.  PARTIAL: some are hidden, from all rows (behind the last row's) or from some.
    const auto tile_pass = [&](auto partial_tag, auto mt_tag, const uint8_t* kb, int tok) {
      constexpr bool PARTIAL = decltype(partial_tag)::value;
      constexpr int MT = decltype(mt_tag)::value;
      float sc[MT][NT][4];
      uint32_t vsw[MT][2][NG];
      float vmax = 0.f, top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = NEG_INF;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
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
        const uint32_t x0[4] = {k0.x, k0.y, k0.z, k0.w}, x1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u0 = x0[i] >> 8, u1 = x1[i] >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(acc[i * NG / 4][nt], x0[i] & 0x000f000fu, x1[i] & 0x000f000fu, x0[i] & 0x00f000f0u,
                     x1[i] & 0x00f000f0u, qf[nt][2 * i][0], qf[nt][2 * i][1]);
            mma16816(acc[i * NG / 4][nt], u0 & 0x000f000fu, u1 & 0x000f000fu, u0 & 0x00f000f0u, u1 & 0x00f000f0u,
                     qf[nt][2 * i + 1][0], qf[nt][2 * i + 1][1]);
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int key = tok + 16 * mt + 8 * r + key_of;
          const bool shown = !PARTIAL || key < seen;
          uint32_t ksw[NG];
          const uint32_t* kp = reinterpret_cast<const uint32_t*>(blk + Blk::K_SCALES + 4 * NG * (key_of + 8 * r));
          const uint32_t* vp = reinterpret_cast<const uint32_t*>(blk + Blk::V_SCALES + 4 * NG * (key_of + 8 * r));
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            ksw[gr] = shown ? kp[gr] : 0u;
            vsw[mt][r][gr] = shown ? vp[gr] : 0u;
            vmax = fmaxf(vmax, bf_lo(vsw[mt][r][gr]));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = 0.f;
#pragma unroll
              for (int gr = 0; gr < NG; ++gr)
                x = fmaf(acc[gr][nt][2 * r + e], bf_lo(ksw[gr]), gr ? fmaf(bf_hi(ksw[gr]), qs[gr][nt][e], x) : bf_hi(ksw[gr]) * qs[gr][nt][e]);
              x = fmaf(x, to_score[nt][e], -base[nt][e]);
              if (PARTIAL && (!shown || key >= lim[nt][e])) x = NEG_INF;
              sc[mt][nt][2 * r + e] = x;
              top[nt][e] = fmaxf(top[nt][e], x);
            }
        }
      }
      bool grow = vmax > vtop;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) grow |= top[nt][0] > limit[nt][0] || top[nt][1] > limit[nt][1];
      if (__any_sync(0xffffffffu, grow)) {
        // a score 2^8 above the running maximum (or a V step above every one before): the maximum is
        // taken anew and what was summed so far is scaled down
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
        const float vnew = fmaxf(vtop, __uint_as_float((__float_as_uint(vmax) + 0x007fffffu) & 0x7f800000u));
        const float fv = vtop * inv_pow2(vnew);
        vtop = vnew;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[nt][e];
#pragma unroll
            for (int off = 16; off > 2; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
            // x: how far the largest score is above `base`, the running maximum (0 where there is none)
            const bool rises = x > 0.f || (limit[nt][e] == NEG_INF && x > NEG_INF);
            const float f = rises ? (limit[nt][e] == NEG_INF ? 0.f : ex2(-x)) : 1.f;
            if (rises) {
              base[nt][e] += x;
              limit[nt][e] = 8.f;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) sc[mt][nt][e] -= x, sc[mt][nt][2 + e] -= x;
            }
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
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t pf[NG][NT][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float p[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              p[nt][e] = ex2(sc[mt][nt][2 * r + e]);
              l[nt][e] += p[nt][e];
            }
          const int key = tok + 16 * mt + 8 * r + key_of;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            const float step = bf_lo(vsw[mt][r][gr]), vs = step * vinv;
            const float vz = fmaf(8.f, step, bf_hi(vsw[mt][r][gr]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // a key hidden from this row alone may hold NaN: no product with it
                const bool hidden = PARTIAL && key >= lim[nt][e];
                y[e] = hidden ? 0.f : p[nt][e] * vs;  // to fp16: up to 2^15, and 2^-25 lost of small ones
                z[gr][nt][e] = hidden ? z[gr][nt][e] : fmaf(p[nt][e], vz, z[gr][nt][e]);
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
          const uint32_t a00 = centred_lo(x, k1024), a01 = centred_hi(x, k1024), a02 = centred_lo(y, k1024), a03 = centred_hi(y, k1024);
          const uint32_t a10 = centred_lo(x8, k1024), a11 = centred_hi(x8, k1024), a12 = centred_lo(y8, k1024), a13 = centred_hi(y8, k1024);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t b0 = pf[q * NG / 4][nt][0], b1 = pf[q * NG / 4][nt][1];
            mma16816(o[2 * q][nt], a00, a01, a02, a03, b0, b1);
            mma16816(o[2 * q + 1][nt], a10, a11, a12, a13, b0, b1);
          }
        }
      }
    };

    const int tiles = min(s_end - s.first - 1, max(units_of(seen, unit_shift) - 1, 0));
    for (int tile = max(at - s.first - 1, 0); tile < tiles; ++tile) {
      const bool there = mbar_wait(bar + c_stage, c_parity, &abort_flag);
      const uint8_t* kb = ring + c_stage * S::TILE;
      const uint32_t all = (1u << per) - 1, have = there ? (holds >> (4 * c_stage)) & all : 0u;
      const int tok = tile << unit_shift;
      if ((1 << unit_shift) == TK && have == all && tok + TK <= seen_first) {
        tile_pass(std::false_type{}, std::integral_constant<int, TK / 16>{}, kb, tok);
      } else {
#pragma unroll 1
        for (int b = 0; b < 1 << (unit_shift - 4); ++b)
          if ((have >> (16 * b >> copy_shift) & 1u) && tok + 16 * b < seen)
            tile_pass(std::true_type{}, std::integral_constant<int, 1>{}, kb + b * Blk::BYTES, tok + 16 * b);
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
    const float of = vtop * 0.0078125f;  // 1 / 128
    const bool starts = s.first >= w0, stops = s.first + s.count <= w1;
    // a head (it began in a stretch before) or a tail goes into the ring where it is the stretch's last
    // segment and the ring empty; a head before others goes to the workspace
    const bool last = s_end == w1;
    float* mine = last ? reinterpret_cast<float*>(ring) : heads + warp * ROWS * HD;
    float* mine_st = stats + (2 * warp + (starts ? 1 : 0)) * ROWS * 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * c + e;
        const float top = limit[nt][e] == NEG_INF ? NEG_INF : base[nt][e];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float zq = z[q * NG / 4][nt][e];
          const float4 x = make_float4(fmaf(o[2 * q][nt][e], of, zq), fmaf(o[2 * q][nt][2 + e], of * 0.0625f, zq),
                                       fmaf(o[2 * q + 1][nt][e], of, zq),
                                       fmaf(o[2 * q + 1][nt][2 + e], of * 0.0625f, zq));
          if (starts && stops) {
            if (r < rows) write_row(s, row0 + r, token_of[nt][e], 32 * q + 4 * g, x, top, l[nt][e]);
          } else {
            *reinterpret_cast<float4*>(mine + r * HD + 32 * q + 4 * g) = x;
          }
        }
        if (!(starts && stops) && g == 0) mine_st[2 * r] = top, mine_st[2 * r + 1] = l[nt][e];
      }
    if (lane == 0) {
      if (!starts) {
        ends[warp] |= 1 | (stops ? 2 : 0) | (last ? 0 : 8);
        if (w0 == t0) segs[W] = s;
      } else if (!stops) {
        ends[warp] |= 4;
        segs[warp] = s;
      }
    }
    at = s_end;
  }
  // nothing is in flight here unless a wait gave up: let what was issued land
  for (; in_flight > 0; --in_flight) {
    int none = 0;
    mbar_wait(bar + c_stage, c_parity, &none);
    if (++c_stage == STAGES) c_stage = 0, c_parity ^= 1;
  }
  __syncthreads();

  // ---- segments over several warps: a chain is the tail (or the CTA's head) and the heads after it ----
  const auto part = [&](int i, int which) { return a.partial + (2 * (int64_t)i + which) * MAX_ROWS * PART; };
  const auto owner = [&](int t) {
    int i = min((int)__fdividef((float)t * (float)active, (float)total), active - 1);  // or next to it
    while (edge(i) > t) --i;
    while (edge(i + 1) <= t) ++i;
    return i;
  };
  uint32_t crosses = 0;  // bit 0: the CTA's head, bit 1: its tail, in the workspace
  Segment cross_seg[2];
  uint32_t has_head = 0, stops_in = 0, has_tail = 0, in_ws = 0;  // a bit per warp
  {
    const uint32_t e = lane < W ? ends[lane] : 0u;
    has_head = __ballot_sync(0xffffffffu, e & 1);
    stops_in = __ballot_sync(0xffffffffu, e & 2);
    has_tail = __ballot_sync(0xffffffffu, e & 4);
    in_ws = __ballot_sync(0xffffffffu, e & 8);
  }
  int lead = 0;  // the first warp with a stretch
  while (stretch * (lead + 1) / W == 0) ++lead;
#pragma unroll 1
  for (uint32_t starts = has_tail << 1 | (has_head >> lead & 1); starts; starts &= starts - 1) {
    const int first = __ffs(starts) - 2;  // -1: the CTA's head
    const Segment s = segs[first < 0 ? W : first];
    // the heads after it, up to the one whose segment ends (warps without a stretch have none)
    const uint32_t after = has_head & ~((first < 0 ? 1u << lead : 2u << first) - 1), end = after & stops_in;
    const uint32_t members = (end ? after & (end ^ (end - 1)) : after) | (first < 0 ? 0u : 1u << first);
    const bool whole = s.first >= t0 && s.first + s.count <= t1;
    const int which = s.first >= t0 ? 1 : 0, rows = min(ROWS, s.n * a.group - s.rt * ROWS);
#pragma unroll 1
    for (int i = tid; i < rows * (HD / 4); i += THREADS) {
      const int r = i / (HD / 4), ch = (i % (HD / 4)) * 4;
      float top = NEG_INF, sum = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int U = 4;  // results read together
      for (uint32_t left = members; left;) {
        float2 st[U];
        float4 y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int w = left ? __ffs(left) - 1 : max(first, lead);
          const float* src = w != first && (in_ws >> w & 1)
                                 ? heads + w * ROWS * HD
                                 : reinterpret_cast<const float*>(smem + S::RING + w * STAGES * S::TILE);
          st[u] = *reinterpret_cast<const float2*>(stats + (2 * w + (w == first ? 1 : 0)) * ROWS * 2 + 2 * r);
          y[u] = *reinterpret_cast<const float4*>(src + r * HD + ch);  // heads: written by this CTA
          if (!left) st[u] = make_float2(NEG_INF, 0.f), y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          left &= left - 1;
        }
        add_parts(top, sum, x, st, y);
      }
      if (whole) {
        write_row(s, s.rt * ROWS + r, a.by_group(s.rt * ROWS + r), ch, x, top, sum);
      } else {
        float* dst = part(blockIdx.x, which);
        *reinterpret_cast<float4*>(dst + r * HD + ch) = x;
        if (ch == 0) *reinterpret_cast<float2*>(dst + MAX_ROWS * HD + 2 * r) = make_float2(top, sum);
      }
    }
    if (!whole) {
      crosses |= 1u << which;
      cross_seg[which] = s;
    }
  }

  // ---- segments over several CTAs: joined by the one that arrives last ----
  if (crosses) {
    int from = 0, to = 0;  // of thread w's crossing segment
    if (tid < 2 && (crosses >> tid & 1)) {
      const Segment& s = cross_seg[tid];
      from = owner(s.first), to = owner(s.first + s.count - 1);
    }
    __threadfence();
    __syncthreads();
    if (tid < 2) {
      last_of[tid] = -1;
      if (crosses >> tid & 1) {
        const bool last = atomicAdd(a.arrivals + from, 1u) == (uint32_t)(to - from);
        if (last) a.arrivals[from] = 0;  // ready for the next launch
        if (last) last_of[tid] = from, last_to[tid] = to;
        __threadfence();
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < 2 * ROWS * (HD / 4); i += THREADS) {  // the rows of both
      const int which = i / (ROWS * (HD / 4)), r = i / (HD / 4) % ROWS, ch = (i % (HD / 4)) * 4;
      const int from = last_of[which], to = last_to[which];
      if (from < 0) continue;
      const Segment s = cross_seg[which];
      if (r >= s.n * a.group - s.rt * ROWS) continue;
      float top = NEG_INF, sum = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int U = 8;  // partial results on their way together
      for (int k0 = from; k0 <= to; k0 += U) {
        float2 st[U];
        float4 y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float* p = part(min(k0 + u, to), k0 + u == from);
          st[u] = __ldcg(reinterpret_cast<const float2*>(p + MAX_ROWS * HD + 2 * r));
          y[u] = __ldcg(reinterpret_cast<const float4*>(p + r * HD + ch));
          if (k0 + u > to) st[u] = make_float2(NEG_INF, 0.f), y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        add_parts(top, sum, x, st, y);
      }
      write_row(s, s.rt * ROWS + r, a.by_group(s.rt * ROWS + r), ch, x, top, sum);
    }
  }
  if (tid == 0) {
    if (abort_flag) atomicOr(a.c.state, DEV_ERR_TIMEOUT);
    if (bad) atomicOr(a.c.state, DEV_ERR_BOUNDS);
  }
}

template <int NG, int NT, int TK, int W, int STAGES>
cudaError_t launch(const AttendArgs& a, int dev, cudaStream_t st) {
  using S = AttendSmem<NG, NT, TK, W, STAGES>;
  static_assert(S::CUM + (KV4_MAX_B + 1) * 4 <= 226 * 1024 + 512, "shared memory of one CTA");
  static_assert(8 * NT <= MAX_ROWS && W * 8 * NT <= MAX_WARP_ROWS, "rows of the results in the workspace");
  static std::atomic<uint64_t> ready{0};
  if (device_pending(ready, dev)) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_attend_kernel<NG, NT, TK, W, STAGES>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               S::CUM + (KV4_MAX_B + 1) * 4);
    if (e != cudaSuccess) return e;
    mark_device(ready, dev);
  }
  count_launches(1);
  kv4_attend_kernel<NG, NT, TK, W, STAGES>
      <<<std::min(sm_count(), KV4_MAX_CTAS), W * 32, S::CUM + (a.B + 1) * 4, st>>>(a);
  return cudaGetLastError();
}

template <int NG>
cudaError_t launch_rows(const AttendArgs& a, int max_q, int dev, cudaStream_t st) {
  if ((int64_t)max_q * a.group <= 8) return launch<NG, 1, 64, NG == 4 ? 8 : 12, 2>(a, dev, st);
  return launch<NG, 2, 32, 8, 3>(a, dev, st);
}

// Query rows of a KV head, of a request, from which on the tensor-memory kernel is taken.  It walks over 256
// rows at a time at the cost of 128, the kernel here over 16: measured (28 / 4, 32 / 8 and 16 / 16 heads, 1, 8 and 32
// requests of 32K, 8K and 2K tokens) they meet between 60 and 96 rows (8 x 8K tokens, 28 / 4 heads: 65.9 us here, 73.8
// there at 56 rows, 90.4 and 76.2 at 84; 32 / 8 heads: 105 and 115.5 at 64, 147 and 117 at 96).  Where the table's
// rows hold little, a walk ends before that cost counts and the second launch of the other does: at 600 tokens, 32 / 8
// heads, 29.7 and 37.1 us at 128 rows, 59.3 and 60.9 at 512.
constexpr int PROMPT_ROWS = 80, PROMPT_ROWS_SHORT = 512, SHORT_TOKENS = 1024;
constexpr size_t ARRIVALS_BYTES = 1024;
constexpr size_t PARTIAL_BYTES = (size_t)KV4_MAX_CTAS * 2 * MAX_ROWS * PART * sizeof(float);
static_assert(ARRIVALS_BYTES >= KV4_MAX_CTAS * 4, "a counter per CTA");

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_kv4_attend_workspace_bytes(void) {
  return ARRIVALS_BYTES + std::max(PARTIAL_BYTES + (size_t)KV4_MAX_CTAS * MAX_WARP_ROWS * HD * sizeof(float),
                                   kv4_prompt_partial_bytes());
}

msa_status msa_kv4_attend(const msa_kv4_cache* cache, const void* Q, void* O, const msa_strides* strides,
                          int32_t total_q, int32_t Hq, float scale, const int32_t* block_table, int64_t table_stride,
                          int32_t max_blocks, const int32_t* kv_lens, const int32_t* cu_q, int32_t B, int32_t max_q,
                          float* lse, void* ws, size_t ws_bytes, void* stream) {
  AttendArgs a{};
  const msa_status st = kv4_view(cache, &a.c);
  if (st != MSA_OK) return st;
  if (!strides || total_q < 0 || B < 0 || max_q < 0 || max_blocks < 0 || !(scale > 0.f) || !isfinite(scale * LOG2E))
    return MSA_ERR_INVALID_ARG;
  if (Hq < 1 || Hq % cache->Hkv) return MSA_ERR_SHAPE;
  if (table_stride < max_blocks) return MSA_ERR_SHAPE;
  if (B > KV4_MAX_B || Hq > 65536) return MSA_ERR_UNSUPPORTED;
  // tokens are numbered in 32 bits, those of the tiles that a warp looks ahead to among them
  if (((int64_t)max_blocks << a.c.page_shift) > KV4_MAX_TOKENS) return MSA_ERR_UNSUPPORTED;
  if ((int64_t)total_q * (Hq / cache->Hkv) > 0x7fffffff) return MSA_ERR_UNSUPPORTED;
  if (!ws) return MSA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) % 256) return MSA_ERR_ALIGN;
  if (ws_bytes < msa_kv4_attend_workspace_bytes()) return MSA_ERR_WORKSPACE;
  if (total_q == 0 || B == 0) return MSA_OK;
  if (!Q || !O || !kv_lens || !cu_q || (max_blocks && !block_table)) return MSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(O)) & 15) return MSA_ERR_ALIGN;
  if (!aligned4({block_table, kv_lens, cu_q, lse})) return MSA_ERR_ALIGN;
  if (strides->q_head % 8 || strides->q_row % 8 || strides->o_head % 8 || strides->o_row % 8) return MSA_ERR_ALIGN;
  a.Q = static_cast<const __nv_bfloat16*>(Q);
  a.O = static_cast<__nv_bfloat16*>(O);
  a.q_head = strides->q_head, a.q_row = strides->q_row, a.o_head = strides->o_head, a.o_row = strides->o_row;
  a.table = block_table, a.kv_lens = kv_lens, a.cu_q = cu_q, a.table_stride = table_stride;
  a.max_blocks = max_blocks, a.B = B, a.total_q = total_q, a.Hq = Hq, a.group = Hq / cache->Hkv;
  // x / group for 0 <= x < 2^31 as a product and a shift: with l = ceil(log2 group), 2^(31 + l) / group rounded up
  // is off by less than 2^l / 2^(31 + l) of it (Granlund and Montgomery, 1994)
  int l = 0;
  while ((1 << l) < a.group) ++l;
  a.group_mul = (uint32_t)(((1ull << (31 + l)) + a.group - 1) / a.group);
  a.group_shift = l;
  a.scale2 = scale * LOG2E;
  a.lse = lse;
  a.arrivals = static_cast<uint32_t*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ARRIVALS_BYTES);
  a.heads = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ARRIVALS_BYTES + PARTIAL_BYTES);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MSA_ERR_CUDA;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const int prompt_rows = ((int64_t)max_blocks << a.c.page_shift) < SHORT_TOKENS ? PROMPT_ROWS_SHORT : PROMPT_ROWS;
  if ((int64_t)max_q * a.group >= prompt_rows && B <= KV4_PROMPT_MAX_B) e = launch_kv4_prompt(a, 128 / cache->group, dev, cs);
  else switch (cache->group) {
    case 128: e = launch_rows<1>(a, max_q, dev, cs); break;
    case 64: e = launch_rows<2>(a, max_q, dev, cs); break;
    default: e = launch_rows<4>(a, max_q, dev, cs); break;
  }
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // extern "C"
