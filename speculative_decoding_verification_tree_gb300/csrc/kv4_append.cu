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
// One thread takes one block: 32 bytes in, 9 out.  Pure streaming, bound by
// HBM; a warp reads four contiguous 256-byte rows (D 128).
#include "kernels.h"
#include "kv4.cuh"

namespace sv {
namespace {

constexpr int kAppThreads = 256;

__global__ void __launch_bounds__(kAppThreads)
    kv4_append(const uint4* __restrict__ k, const uint4* __restrict__ v,
               const int32_t* __restrict__ prefix_len, int64_t blocks, int n, int Hkv, int nb,
               int64_t S, float k_unit, float v_unit, uint8_t* __restrict__ kc,
               uint8_t* __restrict__ ks, uint8_t* __restrict__ vc, uint8_t* __restrict__ vs) {
  const int64_t t = (int64_t)blockIdx.x * kAppThreads + threadIdx.x;
  if (t >= blocks) return;
  const bool is_v = blockIdx.y != 0;
  // block t of the [B, n, Hkv, nb] input
  const uint4* src = (is_v ? v : k) + 2 * t;
  const uint4 a = __ldg(src), c = __ldg(src + 1);
  const int blk = (int)(t % nb);
  int64_t r = t / nb;
  const int h = (int)(r % Hkv);
  r /= Hkv;
  const int j = (int)(r % n);
  const int b = (int)(r / n);
  const int64_t pos = (int64_t)prefix_len[b] + j;
  if (pos < 0 || pos >= S) return;
  const int64_t row = ((int64_t)b * Hkv + h) * S + pos;
  const float unit = is_v ? v_unit : k_unit;
  const float inv_unit = 1.f / unit;  // exact: a power of two

  const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
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
  uint8_t* cp = (is_v ? vc : kc) + (row * nb + blk) * 8;
  *reinterpret_cast<uint2*>(cp) = make_uint2(code[0], code[1]);
  (is_v ? vs : ks)[row * nb + blk] = (uint8_t)sb;
}

__global__ void __launch_bounds__(kAppThreads)
    kv4_read(const uint8_t* __restrict__ kc, const uint8_t* __restrict__ ks,
             const uint8_t* __restrict__ vc, const uint8_t* __restrict__ vs,
             const int32_t* __restrict__ start, int64_t blocks, int n, int Hkv, int nb, int64_t S,
             float k_unit, float v_unit, uint4* __restrict__ k, uint4* __restrict__ v) {
  const int64_t t = (int64_t)blockIdx.x * kAppThreads + threadIdx.x;
  if (t >= blocks) return;
  const bool is_v = blockIdx.y != 0;
  const int blk = (int)(t % nb);
  int64_t r = t / nb;
  const int h = (int)(r % Hkv);
  r /= Hkv;
  const int j = (int)(r % n);
  const int b = (int)(r / n);
  const int64_t pos = (int64_t)start[b] + j;
  uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (pos >= 0 && pos < S) {
    const int64_t row = ((int64_t)b * Hkv + h) * S + pos;
    const uint2 c =
        *reinterpret_cast<const uint2*>((is_v ? vc : kc) + (row * nb + blk) * 8);
    const float s = half2_to_f32(e4m3x2_to_half2((is_v ? vs : ks)[row * nb + blk])).x *
                    (is_v ? v_unit : k_unit);
    uint32_t q[4];
    e2m1x8_to_half2(c.x, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = half2_to_f32(q[i]);
      o[i] = pack_bf16x2(f.x * s, f.y * s);  // exact: six significant bits
    }
    e2m1x8_to_half2(c.y, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = half2_to_f32(q[i]);
      o[4 + i] = pack_bf16x2(f.x * s, f.y * s);
    }
  }
  uint4* dst = (is_v ? v : k) + 2 * t;
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// Checks shared by the two entry points; *grid_x = CTAs for the blocks.
int check_kv4(const void* k, const void* v, const int32_t* at, int B, int n, int Hkv, int D, int S,
              float k_unit, float v_unit, const void* kc, const void* ks, const void* vc,
              const void* vs, int64_t* blocks) {
  if (B < 0 || n < 0 || Hkv < 1 || S < 0) return SPEC_ERR_SHAPE;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (!kv4_unit_ok(k_unit) || !kv4_unit_ok(v_unit)) return SPEC_ERR_ARG;
  *blocks = 0;
  if (B == 0 || n == 0) return SPEC_OK;
  // [B, n, Hkv] rows and [B, Hkv, S] cache rows are counted in 64 bits; the
  // grid's x dimension holds 2^31 - 1 CTAs
  const double rows = (double)B * n * Hkv;
  if (rows * (D / kKv4Block) / kAppThreads > 2147483000.0) return SPEC_ERR_SHAPE;
  if ((double)B * Hkv * S > 4.0e15) return SPEC_ERR_SHAPE;
  if (!k || !v || !at || !kc || !ks || !vc || !vs) return SPEC_ERR_ARG;
  if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)kc | (uintptr_t)vc) % 16 != 0 ||
      ((uintptr_t)ks | (uintptr_t)vs) % 8 != 0 || (uintptr_t)at % 4 != 0)
    return SPEC_ERR_ARG;
  *blocks = (int64_t)B * n * Hkv * (D / kKv4Block);
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

}  // namespace sv

using namespace sv;

extern "C" int spec_kv4_append(const void* k, const void* v, const int32_t* prefix_len, int B,
                               int n, int Hkv, int D, int S, float k_unit, float v_unit,
                               uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes,
                               uint8_t* v_scales, void* stream) {
  int64_t blocks;
  const int rc = check_kv4(k, v, prefix_len, B, n, Hkv, D, S, k_unit, v_unit, k_codes, k_scales,
                           v_codes, v_scales, &blocks);
  if (rc != SPEC_OK || blocks == 0) return rc;
  const dim3 grid((unsigned)((blocks + kAppThreads - 1) / kAppThreads), 2);
  kv4_append<<<grid, kAppThreads, 0, (cudaStream_t)stream>>>(
      (const uint4*)k, (const uint4*)v, prefix_len, blocks, n, Hkv, D / kKv4Block, S, k_unit,
      v_unit, k_codes, k_scales, v_codes, v_scales);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" int spec_kv4_read(const uint8_t* k_codes, const uint8_t* k_scales,
                             const uint8_t* v_codes, const uint8_t* v_scales, const int32_t* start,
                             int B, int n, int Hkv, int D, int S, float k_unit, float v_unit,
                             void* k, void* v, void* stream) {
  int64_t blocks;
  const int rc = check_kv4(k, v, start, B, n, Hkv, D, S, k_unit, v_unit, k_codes, k_scales,
                           v_codes, v_scales, &blocks);
  if (rc != SPEC_OK || blocks == 0) return rc;
  const dim3 grid((unsigned)((blocks + kAppThreads - 1) / kAppThreads), 2);
  kv4_read<<<grid, kAppThreads, 0, (cudaStream_t)stream>>>(
      k_codes, k_scales, v_codes, v_scales, start, blocks, n, Hkv, D / kKv4Block, S, k_unit,
      v_unit, (uint4*)k, (uint4*)v);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
