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
// shared by the run.  Bound by HBM: 512 bytes a row, read and written once.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "kernels.h"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int RD = 128;
constexpr int ROPE_THREADS = 128;
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
  int32_t dim, interleaved;
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

__global__ void __launch_bounds__(ROPE_THREADS) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ uint64_t turn[RD / 2];
  __shared__ uint8_t axis[RD / 2];
  if (threadIdx.x < RD / 2) {
    turn[threadIdx.x] = a.turn[threadIdx.x];
    axis[threadIdx.x] = a.axis[threadIdx.x];
  }
  __syncthreads();
  const int l = threadIdx.x & 15;
  const int64_t item = (int64_t)blockIdx.x * ROPE_GROUPS + (threadIdx.x >> 4);
  // a warp's two groups shuffle together, so a group without a token walks along on the last one
  const bool live = item < a.T * a.n_runs;
  const int64_t it = live ? item : a.T * a.n_runs - 1;
  const int64_t t = it / a.n_runs;
  const int h0 = (int)(it - t * a.n_runs) * a.run;
  const int h1 = min(h0 + a.run, a.H);
  const int lanes = a.dim >> 3, half = lanes >> 1;  // lanes that hold rotated channels

  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
  if (l < lanes) {
    const int n = a.interleaved ? 4 : 8;
    const int i0 = a.interleaved ? 4 * l : 8 * (l < half ? l : l - half);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e >= n) break;
      const int64_t p = a.pos[axis[i0 + e] * a.pos_stride + t];
      const uint64_t ph = (uint64_t)p * turn[i0 + e];
      sincospif((float)(int32_t)(ph >> 32) * 0x1p-31f, &sn[e], &cs[e]);
      cs[e] *= a.scale;
      sn[e] *= a.scale;
    }
    if (!a.interleaved && l < half) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
    }
  }
  // every lane shuffles; lanes behind the rotated channels take their own value (sine 0)
  const int lane = threadIdx.x & 31;
  const int partner = a.interleaved || l >= lanes ? lane : (l < half ? lane + half : lane - half);

  constexpr int U = 4;
  // groups of one warp may have runs of different lengths: the longer one sets the trip count
  const int trips = __reduce_max_sync(0xffffffffu, (unsigned)((h1 - h0 + U - 1) / U));
  for (int k = 0; k < trips; ++k) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + k * U + u;
      v[u] = make_uint4(0, 0, 0, 0);
      if (h < h1)
        v[u] = *reinterpret_cast<const uint4*>((h < a.Hq ? a.Q + h * a.q_head + t * a.q_row
                                                         : a.K + (h - a.Hq) * a.k_head + t * a.k_row) + l * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + k * U + u;
      const bool is_q = h < a.Hq;
      float x[8];
      unpack8(v[u], x);
      const uint4* w = is_q ? a.wq : a.wk;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, 16);
      if (w) {
        const float r = rsqrtf(ss * (1.f / RD) + a.eps);
        float g[8];
        unpack8(__ldg(w + l), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * g[e];
      }
      float y[8];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = l < lanes ? x[2 * e] * cs[e] - x[2 * e + 1] * sn[e] : x[2 * e];
          y[2 * e + 1] = l < lanes ? x[2 * e + 1] * cs[e] + x[2 * e] * sn[e] : x[2 * e + 1];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = __shfl_sync(0xffffffffu, x[e], partner);
          y[e] = l < lanes ? fmaf(o, sn[e], x[e] * cs[e]) : x[e];
        }
      }
      if (live && h < h1) {
        __nv_bfloat16* d = (is_q ? a.Qo + h * a.qo_head + t * a.qo_row
                                 : a.Ko + (h - a.Hq) * a.ko_head + t * a.ko_row) + l * 8;
        *reinterpret_cast<uint4*>(d) =
            make_uint4(bf_pack(y[0], y[1]), bf_pack(y[2], y[3]), bf_pack(y[4], y[5]), bf_pack(y[6], y[7]));
      }
    }
  }
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
  if (rope->dim && rope->n_axes > 1 && pos_stride < T) return MSA_ERR_SHAPE;
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
    // fraction of a turn per position, in [0, 1), as 64 bits (a value that rounds up to 1 wraps to 0)
    long double f = (long double)rope->inv_freq[i] / (2.0L * 3.14159265358979323846264338327950288L);
    f -= floorl(f);
    const long double u = floorl(f * 18446744073709551616.0L + 0.5L);
    a.turn[i] = u >= 18446744073709551616.0L ? 0 : (uint64_t)u;
  }
  a.Q = static_cast<const __nv_bfloat16*>(Q), a.K = static_cast<const __nv_bfloat16*>(K);
  a.Qo = static_cast<__nv_bfloat16*>(Qo), a.Ko = static_cast<__nv_bfloat16*>(Ko);
  a.q_head = in->q_head, a.q_row = in->q_row, a.k_head = in->k_head, a.k_row = in->k_row;
  a.qo_head = out->q_head, a.qo_row = out->q_row, a.ko_head = out->k_head, a.ko_row = out->k_row;
  a.wq = static_cast<const uint4*>(wq), a.wk = static_cast<const uint4*>(wk);
  a.pos = positions, a.pos_stride = pos_stride;
  a.T = T, a.Hq = Hq, a.H = Hq + Hkv;
  a.dim = rope->dim, a.interleaved = rope->interleaved != 0;
  a.eps = eps, a.scale = rope->scale;
  // the longest run of heads that still leaves 64 groups for every SM: a run shares its cosines
  a.run = a.H;
  while (a.run > 1 && T * ((a.H + a.run - 1) / a.run) < (int64_t)sm_count() * 64) a.run = (a.run + 1) / 2;
  a.n_runs = (a.H + a.run - 1) / a.run;
  const int64_t blocks = (T * a.n_runs + ROPE_GROUPS - 1) / ROPE_GROUPS;
  if (blocks > 0x7fffffff) return MSA_ERR_UNSUPPORTED;
  count_launches(1);
  qk_norm_rope_kernel<<<(unsigned)blocks, ROPE_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
