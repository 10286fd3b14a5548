// spec_kv4_append / spec_kv4_read: new positions' keys and values rounded
// into a 4-bit cache, and the values a range of positions stands for.
//
// Per block of 16 head dims (x bf16, unit a power of two):
//   scale = e4m3(max|x| / (6 unit)), at least 2^-9, at most 448
//   code  = e2m1(x / (scale unit)), nearest, ties to even, at most 6
// so the block's largest element lands on the largest code.  A NaN makes the
// block's scale NaN (the block then reads as NaN); infinities saturate.
//
// Rounding borders are decided exactly although the quotient is taken as
// x * (1 / (scale unit)): x has 8 significant bits and a border (a midpoint of
// two codes times the scale) at most 7, so they are equal or differ by 2^-8
// relative; the product's error (2^-22) is removed by rounding it to 12 bits
// before the conversion, which puts equal ones back on the border and moves
// none across it.
//
// One thread takes two blocks, 32 bytes in and 9 out each, all loads first.  A
// CTA's rows are consecutive positions of a head (the next head's after the
// last), so that the codes and scales it writes are contiguous while each row
// it reads is a whole 128- or 256-byte line.  Streaming: the bound is HBM, with
// instruction issue close behind (82% of its slots, cold caches).  4 x 8192
// positions of 8 heads, D 128 (172 MB): 33 us, 5.2 TB/s, written and 33 us read
// back.  The same rounding in packed arithmetic took the same time.
#include <math.h>

#include "kernels.h"
#include "kv4.cuh"

namespace sv {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppUnroll = 2;  // blocks per thread

// One call's geometry.  A sequence's rows are (head, position) pairs, head
// first; a CTA takes kAppThreads * kAppUnroll consecutive blocks of one
// sequence (blockIdx.x = sequence x chunk), of K or V (blockIdx.y).
struct AppShape {
  int n, Hkv, log_nb;  // 2^log_nb blocks per row
  uint32_t chunks;     // CTAs per sequence
  uint32_t blocks;     // blocks per sequence
  int64_t S;
};
// Where block t of sequence b lies in the [B, n, Hkv, nb] rows and in the
// cache (-1: its position is outside).
__device__ __forceinline__ void place(const AppShape& a, int b, int64_t start, uint32_t t,
                                      int64_t* in, int64_t* out) {
  const uint32_t blk = t & ((1u << a.log_nb) - 1u), r = t >> a.log_nb;
  const uint32_t h = r / (uint32_t)a.n, j = r - h * (uint32_t)a.n;
  *in = ((((int64_t)b * a.n + j) * a.Hkv + h) << a.log_nb) + blk;
  const int64_t pos = start + j;
  *out = pos < 0 || pos >= a.S ? -1
                               : ((((int64_t)b * a.Hkv + h) * a.S + pos) << a.log_nb) + blk;
}

__global__ void __launch_bounds__(kAppThreads)
    kv4_append(const uint4* __restrict__ k, const uint4* __restrict__ v,
               const int32_t* __restrict__ prefix_len, const AppShape a, float k_unit,
               float v_unit, uint8_t* __restrict__ kc, uint8_t* __restrict__ ks,
               uint8_t* __restrict__ vc, uint8_t* __restrict__ vs) {
  const bool is_v = blockIdx.y != 0;
  const int b = (int)(blockIdx.x / a.chunks);
  const uint32_t t0 = (blockIdx.x - b * a.chunks) * (kAppThreads * kAppUnroll) + threadIdx.x;
  const int64_t start = prefix_len[b];
  const uint4* src = is_v ? v : k;
  const float unit = is_v ? v_unit : k_unit;
  const float inv_unit = 1.f / unit;  // exact: a power of two
  uint4 lo[kAppUnroll], hi[kAppUnroll];
  int64_t to[kAppUnroll];
#pragma unroll
  for (int u = 0; u < kAppUnroll; ++u) {
    const uint32_t t = t0 + u * kAppThreads;
    to[u] = -1;
    if (t < a.blocks) {
      int64_t in;
      place(a, b, start, t, &in, &to[u]);
      if (to[u] >= 0) {
        lo[u] = __ldcs(src + 2 * in);
        hi[u] = __ldcs(src + 2 * in + 1);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kAppUnroll; ++u) {
    if (to[u] < 0) continue;
    const uint32_t w[8] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w, hi[u].x, hi[u].y, hi[u].z, hi[u].w};
    uint32_t mx = 0;  // largest magnitude: bf16 magnitudes order like their bits
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = __vmaxu2(mx, w[i] & 0x7fff7fffu);
    mx = max(mx & 0xffffu, mx >> 16);
    const float amax = __uint_as_float(mx << 16);
    uint32_t sb = f32_to_e4m3(__fdiv_rn(amax * inv_unit, 6.f));  // NaN stays NaN
    if (sb == 0) sb = 1;                                         // 2^-9
    const float s = half2_to_f32(e4m3x2_to_half2(sb)).x;
    const float inv = __frcp_rn(s * unit);
    uint32_t code[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(w[4 * i + e]) * inv;
        x[2 * e + 1] = bf16_hi(w[4 * i + e]) * inv;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = __uint_as_float((__float_as_uint(x[e]) + 0x800u) & 0xfffff000u);
      code[i] = f32x8_to_e2m1(x);
    }
    *reinterpret_cast<uint2*>((is_v ? vc : kc) + to[u] * 8) = make_uint2(code[0], code[1]);
    (is_v ? vs : ks)[to[u]] = (uint8_t)sb;
  }
}

__global__ void __launch_bounds__(kAppThreads)
    kv4_read(const uint8_t* __restrict__ kc, const uint8_t* __restrict__ ks,
             const uint8_t* __restrict__ vc, const uint8_t* __restrict__ vs,
             const int32_t* __restrict__ start_pos, const AppShape a, float k_unit, float v_unit,
             uint4* __restrict__ k, uint4* __restrict__ v) {
  const bool is_v = blockIdx.y != 0;
  const int b = (int)(blockIdx.x / a.chunks);
  const uint32_t t0 = (blockIdx.x - b * a.chunks) * (kAppThreads * kAppUnroll) + threadIdx.x;
  const int64_t start = start_pos[b];
  const float unit = is_v ? v_unit : k_unit;
  uint2 code[kAppUnroll];
  uint32_t sb[kAppUnroll];
  int64_t to[kAppUnroll];
#pragma unroll
  for (int u = 0; u < kAppUnroll; ++u) {
    const uint32_t t = t0 + u * kAppThreads;
    to[u] = -1;
    code[u] = make_uint2(0, 0);
    sb[u] = 0;
    if (t < a.blocks) {
      int64_t from;
      place(a, b, start, t, &to[u], &from);
      if (from >= 0) {
        code[u] = *reinterpret_cast<const uint2*>((is_v ? vc : kc) + from * 8);
        sb[u] = (is_v ? vs : ks)[from];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kAppUnroll; ++u) {
    if (to[u] < 0) continue;
    const float s = half2_to_f32(e4m3x2_to_half2(sb[u])).x * unit;
    uint32_t q[4], o[8];
    e2m1x8_to_half2(code[u].x, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = half2_to_f32(q[i]);
      o[i] = pack_bf16x2(f.x * s, f.y * s);  // exact: six significant bits
    }
    e2m1x8_to_half2(code[u].y, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = half2_to_f32(q[i]);
      o[4 + i] = pack_bf16x2(f.x * s, f.y * s);
    }
    uint4* dst = (is_v ? v : k) + 2 * to[u];
    __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
    __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
  }
}

// Checks shared by the two entry points; sets the geometry and *ctas (0: nothing
// to do).
int check_kv4(const void* k, const void* v, const int32_t* at, int B, int n, int Hkv, int D, int S,
              float k_unit, float v_unit, const void* kc, const void* ks, const void* vc,
              const void* vs, AppShape* a, unsigned* ctas) {
  if (B < 0 || n < 0 || Hkv < 1 || S < 0) return SPEC_ERR_SHAPE;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (!kv4_unit_ok(k_unit) || !kv4_unit_ok(v_unit)) return SPEC_ERR_ARG;
  *ctas = 0;
  if (B == 0 || n == 0) return SPEC_OK;
  // a sequence's blocks are counted in 32 bits, the CTAs by the grid's x
  // dimension, everything else in 64 bits
  const double blocks = (double)n * Hkv * (D / kKv4Block);
  if (blocks > 2147480000.0 || (double)B * Hkv * S > 4.0e15) return SPEC_ERR_SHAPE;
  constexpr int kCta = kAppThreads * kAppUnroll;
  const int64_t chunks = ((int64_t)blocks + kCta - 1) / kCta;
  if (chunks * B > 2147483647) return SPEC_ERR_SHAPE;
  if (!k || !v || !at || !kc || !ks || !vc || !vs) return SPEC_ERR_ARG;
  if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)kc | (uintptr_t)vc) % 16 != 0 ||
      ((uintptr_t)ks | (uintptr_t)vs) % 8 != 0 || (uintptr_t)at % 4 != 0)
    return SPEC_ERR_ARG;
  *a = {n, Hkv, D == 128 ? 3 : 2, (uint32_t)chunks, (uint32_t)blocks, S};
  *ctas = (unsigned)(chunks * B);
  return SPEC_OK;
}

}  // namespace

bool kv4_unit_ok(float u) {
  // a power of two in [2^-64, 2^64]: only exponent bits set
  if (!(u >= 5.42101086242752217e-20f && u <= 1.8446744073709551616e19f)) return false;
  union {
    float f;
    uint32_t i;
  } x;
  x.f = u;
  return (x.i & 0x7fffffu) == 0;
}

ScoreScale score_scale(float scale, float unit) {
  int es, ep, eu;
  const float ms = frexpf(scale, &es);           // [1/2, 1)
  const float mp = frexpf(ms * kLog2e, &ep);     // rounded as scale * log2(e) is
  frexpf(unit, &eu);                             // unit = 2^(eu - 1)
  const int e = es + ep + eu - 2;
  return {ldexpf(1.f, e / 2), ldexpf(2.f * mp, e - e / 2)};
}

}  // namespace sv

using namespace sv;

extern "C" int spec_kv4_append(const void* k, const void* v, const int32_t* prefix_len, int B,
                               int n, int Hkv, int D, int S, float k_unit, float v_unit,
                               uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes,
                               uint8_t* v_scales, void* stream) {
  AppShape a;
  unsigned ctas;
  const int rc = check_kv4(k, v, prefix_len, B, n, Hkv, D, S, k_unit, v_unit, k_codes, k_scales,
                           v_codes, v_scales, &a, &ctas);
  if (rc != SPEC_OK || ctas == 0) return rc;
  kv4_append<<<dim3(ctas, 2), kAppThreads, 0, (cudaStream_t)stream>>>(
      (const uint4*)k, (const uint4*)v, prefix_len, a, k_unit, v_unit, k_codes, k_scales, v_codes,
      v_scales);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" int spec_kv4_read(const uint8_t* k_codes, const uint8_t* k_scales,
                             const uint8_t* v_codes, const uint8_t* v_scales, const int32_t* start,
                             int B, int n, int Hkv, int D, int S, float k_unit, float v_unit,
                             void* k, void* v, void* stream) {
  AppShape a;
  unsigned ctas;
  const int rc = check_kv4(k, v, start, B, n, Hkv, D, S, k_unit, v_unit, k_codes, k_scales,
                           v_codes, v_scales, &a, &ctas);
  if (rc != SPEC_OK || ctas == 0) return rc;
  kv4_read<<<dim3(ctas, 2), kAppThreads, 0, (cudaStream_t)stream>>>(
      k_codes, k_scales, v_codes, v_scales, start, a, k_unit, v_unit, (uint4*)k, (uint4*)v);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
