// Per-head RMS norm of queries and keys with the rotary position embedding, in one pass.
//
// y = x * rsqrt(mean(x^2) + eps) * w over a row's 128 channels, then pairs (a, b) of frequency i
// become (a cos f - b sin f, b cos f + a sin f) * scale with f = position * inv_freq[i].
//
// The angle: positions reach 2^31 and f is wanted modulo one turn, so each inv_freq is held as the
// 64-bit fraction of a turn per position (round(inv_freq / 2 pi * 2^64)) and multiplied by the
// position in wrapping 64-bit integers: the wrap is the reduction, exact, with an error of
// position * 2^-64 turns from the fraction's rounding.  Its top 32 bits go to sincospif.
//
// Sixteen lanes hold one row, 8 channels (16 bytes) each.  They take the cosines of one token once
// and then walk over a run of its heads, four rows in flight, so the 8 sincospif of a lane are
// shared by the run.  Bound by HBM: 512 bytes a row, read and written once.  131072 tokens, 28 + 4 heads,
// three axes: 387 to 397 us, 5.5 TB/s (a copy: 6.44); with the norm before the rotation, partners exchanged as
// fp32, 471 us (issue-bound).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "kernels.h"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int RD = 128;
constexpr int ROPE_THREADS = 128;
constexpr int ROPE_BLOCKS = 4;  // per SM
constexpr int ROPE_GROUPS = ROPE_THREADS / 16;

struct RopeArgs {
  const __nv_bfloat16 *Q, *K;
  __nv_bfloat16 *Qo, *Ko;
  int64_t q_head, q_row, k_head, k_row, qo_head, qo_row, ko_head, ko_row;
  const uint4 *wq, *wk;  // null: no norm
  const int32_t* pos;
  int64_t pos_stride;
  int64_t T;
  int32_t Hq, H;  // query heads; all heads
  int32_t run, n_runs;  // heads per 16-lane group, groups per token
  int32_t dim;
  float eps, scale;
  uint64_t turn[RD / 2];
  uint8_t axis[RD / 2];
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf_lo(v.x), x[1] = bf_hi(v.x), x[2] = bf_lo(v.y), x[3] = bf_hi(v.y);
  x[4] = bf_lo(v.z), x[5] = bf_hi(v.z), x[6] = bf_lo(v.w), x[7] = bf_hi(v.w);
}

// Two fp32 operations at once (neighbouring channels).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Walks over the heads h0 .. h1 of one kind (queries or keys) of one token.  With the norm's weights
// w taken into the cosines, own[e] = w_e cos and other[e] = +-w_partner sin, a row is
// r * (x * own + x_partner * other), r the row's norm: the partner's channels come over as packed words,
// before any arithmetic.
// `ahead`: the first rows, already on their way.
constexpr int U = 4;

__device__ __forceinline__ void rope_load(uint4 (&v)[U], const __nv_bfloat16* src, int64_t src_head, int left) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    v[u] = make_uint4(0, 0, 0, 0);
    if (u < left) v[u] = __ldcs(reinterpret_cast<const uint4*>(src));
    src += src_head;
  }
}

template <bool NORM, bool INTERLEAVED>
__device__ __forceinline__ void rope_heads(const __nv_bfloat16* src, int64_t src_head, __nv_bfloat16* dst,
                                           int64_t dst_head, int heads, bool live, int partner, bool rotated,
                                           float eps, const float2 (&own)[4], const float2 (&other)[4],
                                           uint4 (&ahead)[U]) {
  // the two groups of a warp may have runs of different lengths: the longer one sets the trip count
  const int trips = __reduce_max_sync(0xffffffffu, (unsigned)((max(heads, 0) + U - 1) / U));
  for (int k = 0; k < trips; ++k, heads -= U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = ahead[u];
    src += U * src_head;
    rope_load(ahead, src, src_head, heads - U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      float2 x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = make_float2(bf_lo(w[e]), bf_hi(w[e]));
        // an unrotated channel has no partner: its word is 0, whatever the row holds
        uint32_t pw = INTERLEAVED ? __funnelshift_l(w[e], w[e], 16) : __shfl_sync(0xffffffffu, w[e], partner);
        if (!rotated) pw = 0;
        y[e] = fma2(make_float2(bf_lo(pw), bf_hi(pw)), other[e], mul2(x[e], own[e]));
      }
      if (NORM) {
        float2 s2 = mul2(x[0], x[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = fma2(x[e], x[e], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, 16);
        const float r = rsqrtf(ss * (1.f / RD) + eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], make_float2(r, r));
      }
      if (live && u < heads)
        __stcs(reinterpret_cast<uint4*>(dst),
               make_uint4(bf_pack(y[0].x, y[0].y), bf_pack(y[1].x, y[1].y), bf_pack(y[2].x, y[2].y),
                          bf_pack(y[3].x, y[3].y)));
      dst += dst_head;
    }
  }
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ uint64_t turn[RD / 2];
  __shared__ uint8_t axis[RD / 2];
  if (threadIdx.x < RD / 2) {
    turn[threadIdx.x] = a.turn[threadIdx.x];
    axis[threadIdx.x] = a.axis[threadIdx.x];
  }
  __syncthreads();
  const int l = threadIdx.x & 15, lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * ROPE_GROUPS + (threadIdx.x >> 4);
  // a warp's two groups shuffle together, so a group without a token walks along on the last one
  const bool live = item < a.T * a.n_runs;
  const int64_t it = live ? item : a.T * a.n_runs - 1;
  const int64_t t = it / a.n_runs;
  const int h0 = (int)(it - t * a.n_runs) * a.run;
  const int h1 = min(h0 + a.run, a.H);
  const int lanes = a.dim >> 3, half = lanes >> 1;  // lanes that hold rotated channels
  const bool rotated = l < lanes;
  // every lane shuffles; lanes behind the rotated channels read their own value
  const int partner = INTERLEAVED || !rotated ? lane : (l < half ? lane + half : lane - half);

  // the first rows are asked for before the angles are worked out
  const int k0 = max(h0 - a.Hq, 0), n_q = min(h1, a.Hq) - h0, n_k = h1 - a.Hq - k0;
  const __nv_bfloat16 *q_src = a.Q + h0 * a.q_head + t * a.q_row + l * 8, *k_src = a.K + k0 * a.k_head + t * a.k_row + l * 8;
  uint4 q_ahead[U], k_ahead[U];
  rope_load(q_ahead, q_src, a.q_head, n_q);
  rope_load(k_ahead, k_src, a.k_head, n_k);

  float cs[8], sn[8];  // of this lane's channels; the sine with the sign of its place in the pair
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
  if (rotated) {
    const int i0 = INTERLEAVED ? 4 * l : 8 * (l < half ? l : l - half);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (INTERLEAVED && (e & 1)) {
        cs[e] = cs[e - 1], sn[e] = -sn[e - 1];
        continue;
      }
      const int i = i0 + (INTERLEAVED ? e / 2 : e);
      const int64_t p = a.pos[axis[i] * a.pos_stride + t];
      const uint64_t ph = (uint64_t)p * turn[i];
      sincospif((float)(int32_t)(ph >> 32) * 0x1p-31f, &sn[e], &cs[e]);
      cs[e] *= a.scale;
      sn[e] *= (INTERLEAVED || l < half) ? -a.scale : a.scale;
    }
  }
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const uint4* w = kind ? a.wk : a.wq;
    float2 own[4], other[4];
    float g[8], gp[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = gp[e] = 1.f;
    if (w) {
      unpack8(__ldg(w + l), g);
      float q[8];
      unpack8(__ldg(w + (partner & 15)), q);
#pragma unroll
      for (int e = 0; e < 8; ++e) gp[e] = INTERLEAVED ? g[e ^ 1] : q[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      own[e] = make_float2(g[2 * e] * cs[2 * e], g[2 * e + 1] * cs[2 * e + 1]);
      other[e] = make_float2(gp[2 * e] * sn[2 * e], gp[2 * e + 1] * sn[2 * e + 1]);
    }
    const int n = kind ? n_k : n_q;
    const __nv_bfloat16* src = kind ? k_src : q_src;
    __nv_bfloat16* dst = (kind ? a.Ko + k0 * a.ko_head + t * a.ko_row : a.Qo + h0 * a.qo_head + t * a.qo_row) + l * 8;
    const int64_t sh = kind ? a.k_head : a.q_head, dh = kind ? a.ko_head : a.qo_head;
    uint4(&ahead)[U] = kind ? k_ahead : q_ahead;
    if (w) rope_heads<true, INTERLEAVED>(src, sh, dst, dh, n, live, partner, rotated, a.eps, own, other, ahead);
    else rope_heads<false, INTERLEAVED>(src, sh, dst, dh, n, live, partner, rotated, a.eps, own, other, ahead);
  }
}

// The fraction of a turn per position, in [0, 1), as 64 bits (what rounds up to a turn wraps to 0).  A call does
// this for every frequency, so those of a model are taken in integers: w = m 2^-s, and m / 2 pi has 117 bits, its
// fraction behind the binary point to 2^-128 (in long double a decode step's call took 5.4 us of host time, more
// than its kernel).
uint64_t turn_of(double w) {
  constexpr long double INV = 0.5L / 3.14159265358979323846264338327950288L;
  constexpr uint64_t HI = 0x28be60db9391054aull, LO = 0x7f09d5f47d4d3770ull;  // 2^128 / 2 pi
  uint64_t bits;
  memcpy(&bits, &w, 8);
  const int ex = (int)(bits >> 52 & 2047), s = 1075 - ex;
  if (ex == 0 || s > 127) return 0;  // below 2^-75: no turn in 2^64 positions
  if (s >= 43) {                     // below 2^10
    const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
    const unsigned __int128 p = (unsigned __int128)m * HI + (uint64_t)((unsigned __int128)m * LO >> 64);
    const uint64_t turn = (uint64_t)((p + ((unsigned __int128)1 << (s - 1))) >> s);
    return bits >> 63 ? 0 - turn : turn;
  }
  long double f = (long double)w * INV;
  f -= floorl(f);
  const long double u = floorl(f * 18446744073709551616.0L + 0.5L);
  return u >= 18446744073709551616.0L ? 0 : (uint64_t)u;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_qk_norm_rope(const void* Q, const void* K, const msa_strides* in, void* Qo, void* Ko,
                                       const msa_strides* out, int64_t T, int32_t Hq, int32_t Hkv, const void* wq,
                                       const void* wk, float eps, const msa_rope* rope, const int32_t* positions,
                                       int64_t pos_stride, void* stream) {
  if (!in || !out || !rope || T < 0 || Hq < 0 || Hkv < 0) return MSA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(rope->scale)) return MSA_ERR_INVALID_ARG;
  if (rope->dim < 0 || rope->dim > RD || rope->dim % 16) return MSA_ERR_SHAPE;
  if (rope->n_axes < 1 || rope->n_axes > 4) return MSA_ERR_INVALID_ARG;
  if (T == 0 || Hq + (int64_t)Hkv == 0) return MSA_OK;
  if ((Hq && (!Q || !Qo)) || (Hkv && (!K || !Ko)) || (rope->dim && !positions)) return MSA_ERR_INVALID_ARG;
  if (rope->dim && rope->n_axes > 1 && pos_stride < T && pos_stride != 0) return MSA_ERR_SHAPE;
  // rows are 128 contiguous elements and heads at most 65536; the token count keeps the grid in range
  if (Hq > 65536 || Hkv > 65536 || T > (int64_t(1) << 31)) return MSA_ERR_UNSUPPORTED;
  const auto misaligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
  if (Hq && (misaligned(Q) || misaligned(Qo) || in->q_head % 8 || in->q_row % 8 || out->q_head % 8 || out->q_row % 8))
    return MSA_ERR_ALIGN;
  if (Hkv && (misaligned(K) || misaligned(Ko) || in->k_head % 8 || in->k_row % 8 || out->k_head % 8 || out->k_row % 8))
    return MSA_ERR_ALIGN;
  if (misaligned(wq) || misaligned(wk) || (reinterpret_cast<uintptr_t>(positions) & 3)) return MSA_ERR_ALIGN;

  RopeArgs a{};
  const int n = rope->dim / 2;
  if (rope->n_axes > 1) {
    int64_t sum = 0;
    for (int x = 0; x < rope->n_axes; ++x) {
      if (rope->sections[x] < 0) return MSA_ERR_INVALID_ARG;
      sum += rope->sections[x];
    }
    if (sum != n) return MSA_ERR_SHAPE;
  }
  for (int i = 0, x = 0, end = rope->n_axes > 1 ? rope->sections[0] : n; i < n; ++i) {
    if (!isfinite(rope->inv_freq[i])) return MSA_ERR_INVALID_ARG;
    while (i >= end) end += rope->sections[++x];
    a.axis[i] = (uint8_t)x;
    a.turn[i] = turn_of(rope->inv_freq[i]);
  }
  a.Q = static_cast<const __nv_bfloat16*>(Q), a.K = static_cast<const __nv_bfloat16*>(K);
  a.Qo = static_cast<__nv_bfloat16*>(Qo), a.Ko = static_cast<__nv_bfloat16*>(Ko);
  a.q_head = in->q_head, a.q_row = in->q_row, a.k_head = in->k_head, a.k_row = in->k_row;
  a.qo_head = out->q_head, a.qo_row = out->q_row, a.ko_head = out->k_head, a.ko_row = out->k_row;
  a.wq = static_cast<const uint4*>(wq), a.wk = static_cast<const uint4*>(wk);
  a.pos = positions, a.pos_stride = pos_stride;
  a.T = T, a.Hq = Hq, a.H = Hq + Hkv;
  a.dim = rope->dim;
  a.eps = eps, a.scale = rope->scale;
  // the longest run of heads that still leaves 64 groups for every SM: a run shares its cosines
  a.run = a.H;
  while (a.run > 1 && T * ((a.H + a.run - 1) / a.run) < (int64_t)sm_count() * 64) a.run = (a.run + 1) / 2;
  a.n_runs = (a.H + a.run - 1) / a.run;
  const int64_t blocks = (T * a.n_runs + ROPE_GROUPS - 1) / ROPE_GROUPS;
  if (blocks > 0x7fffffff) return MSA_ERR_UNSUPPORTED;
  count_launches(1);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (rope->interleaved) qk_norm_rope_kernel<true><<<(unsigned)blocks, ROPE_THREADS, 0, cs>>>(a);
  else qk_norm_rope_kernel<false><<<(unsigned)blocks, ROPE_THREADS, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
