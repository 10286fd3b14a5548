// spec_kv_weights: the attention weight every cached position received from
// the accepted rows, summed over the query heads of its key/value head.
//
//   out[b, h, s] = in[b, h, s] + sum_{t, g} 2^(scale log2(e) q_tg . k_s - lse_tg),
//
// over the accepted nodes t that see s (s <= P + t: the committed prefix and
// the path up to themselves) and the query heads g of head h.  The rows'
// base-2 normalisers lse come from the attention call, so one pass over the
// keys suffices and no value row is read: the bound is the keys' bytes plus
// eight bytes per position for in and out.
//
// A warp takes 32 keys: m16n8k16 products of the accepted rows (16 at a time,
// fragments of q in shared memory) with the keys as the 8-wide operand, then
// the column sums of the exponentials.  Keys are read straight from global
// memory into operand registers (a 4-bit row's quarter, or the 16-byte chunks
// c, c + 4, ... of a bf16 row, per lane (g, c)); the k index is a permutation of the head dims
// that q shares.  Column 2 c + x of tile t is key 8 t + 4 x + c, so that the
// sums end up in lane = key order.  Every position belongs to one warp and its
// sum has a fixed order: no atomics.
#include "kernels.h"
#include "kv4.cuh"

namespace sv {
namespace {

constexpr int kWtWarps = 8;
constexpr int kWtThreads = kWtWarps * 32;
constexpr int kWtIters = 4;                            // 32-key blocks per warp
constexpr int kWtKeys = kWtWarps * 32 * kWtIters;      // keys per CTA
constexpr int kWtRows = 64;                            // query rows staged at a time

struct WeightParams {
  const uint16_t* q;
  const void* k;
  const uint8_t* ks;
  const float* lse;
  const int32_t *prefix_len, *path_len, *path_nodes;
  int N, Hq, Hkv, S;
  float scale_log2;
  const float* in;
  float* out;
};

template <int D, bool kKv4>
__global__ void __launch_bounds__(kWtThreads, 2) kv_weights(const WeightParams p) {
  constexpr int kSteps = D / 16;
  __shared__ uint4 qf[kWtRows / 16][kSteps][32];  // a0 a2 a1 a3 per lane
  __shared__ float rowf[kWtRows], rowl[kWtRows];
  __shared__ int rowt[kWtRows];
  __shared__ int bad;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, kvh = blockIdx.y;
  const int64_t row0 = ((int64_t)b * p.Hkv + kvh) * p.S;
  int P = p.prefix_len[b];
  P = P < 0 ? 0 : (P > p.S - p.N ? p.S - p.N : P);
  int n = p.path_len[b];
  const int first = blockIdx.x * kWtKeys;
  if (first >= P + p.N) return;
  // an invalid path adds nothing
  if (threadIdx.x == 0) bad = n < 0 || n > p.N;
  __syncthreads();
  if (!bad && p.path_nodes && threadIdx.x < n) {
    const int v = p.path_nodes[(int64_t)b * p.N + threadIdx.x];
    if (v < 0 || v >= p.N) bad = 1;
  }
  __syncthreads();
  if (bad) n = 0;
  const int L = P + n;
  if (first >= L) return;
  const int Gq = p.Hq / p.Hkv;
  const int R = n * Gq;
  const int groups = (R + kWtRows - 1) / kWtRows;
  const float* in = p.in ? p.in + row0 : nullptr;
  float* out = p.out + row0;

  auto stage = [&](int grp) {
    for (int i = warp; i < kWtRows; i += kWtWarps) {
      const int r = grp * kWtRows + i;
      if (i >= ((min(R - grp * kWtRows, kWtRows) + 15) & ~15)) break;
      const bool valid = r < R;
      const int t = valid ? r / Gq : 0;
      const int hq = kvh * Gq + (valid ? r % Gq : 0);
      const int node = valid && p.path_nodes ? p.path_nodes[(int64_t)b * p.N + t] : t;
      const int64_t qrow = ((int64_t)b * p.N + node) * p.Hq + hq;
      uint2 w = make_uint2(0, 0);
      if (valid && lane < D / 4) w = *reinterpret_cast<const uint2*>(p.q + qrow * D + 4 * lane);
      float up = 1.f;
      uint32_t h0 = w.x, h1 = w.y;
      int s, cc;
      if constexpr (kKv4) {
        // scaled by a power of two to [1, 2): exact in fp16 (see kv4_attn.cu)
        const float x0 = bf16_lo(w.x), x1 = bf16_hi(w.x), x2 = bf16_lo(w.y), x3 = bf16_hi(w.y);
        const float mx =
            warp_max(fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3))));
        int e = (int)(__float_as_uint(mx) >> 23) - 127;
        if (mx == 0.f || e == 128) e = 0;
        e = max(-126, min(126, e));
        const float dn = __uint_as_float((uint32_t)(127 - e) << 23);
        up = __uint_as_float((uint32_t)(127 + e) << 23);
        h0 = pack_half2(x0 * dn, x1 * dn);
        h1 = pack_half2(x2 * dn, x3 * dn);
        cc = lane / (D / 16);
        s = lane % (D / 16);
      } else {
        cc = (lane >> 1) & 3;
        s = 2 * (lane >> 3) + (lane & 1);
      }
      if (lane < D / 4) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(&qf[i >> 4][s][4 * (i & 7) + cc]);
        dst[(i & 8) ? 2 : 0] = h0;
        dst[(i & 8) ? 3 : 1] = h1;
      }
      if (lane == 0) {
        float l = valid ? p.lse[qrow] : neg_inf();
        if (l == neg_inf()) l = -neg_inf();  // a row that saw nothing weighs nothing
        rowf[i] = p.scale_log2 * up;
        rowl[i] = l;
        rowt[i] = valid ? P + t : -1;
      }
    }
  };
  if (groups == 1) stage(0);
  __syncthreads();

  for (int it = 0; it < kWtIters; ++it) {
    const int key0 = first + (it * kWtWarps + warp) * 32;
    const bool live = key0 < L && groups > 0;
    // the 32 keys' operand fragments: [tile][k step][b0, b1]
    uint32_t kb[4][kSteps][2];
    if (live) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int key = key0 + 8 * t + 4 * (g & 1) + (g >> 1);
        const bool have = key < L;
        const int64_t kr = row0 + (have ? key : key0);
        if constexpr (kKv4) {
          constexpr int kW = D / 32;
          uint32_t w[kW];
          uint32_t sc = 0;
          const uint8_t* src = (const uint8_t*)p.k + kr * (D / 2) + 4 * kW * c;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            sc = *reinterpret_cast<const uint16_t*>(p.ks + kr * (D / 16) + 2 * c);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            w[0] = v.x; w[1] = v.y;
            sc = p.ks[kr * (D / 16) + c];
          }
          const uint32_t s2 = e4m3x2_to_half2(sc);
#pragma unroll
          for (int x = 0; x < kW; ++x) {
            uint32_t h[4];
            e2m1x8_to_half2(w[x], h);
            const uint32_t s1 = (D == 128 && x >= 2) ? dup_hi(s2) : dup_lo(s2);
            kb[t][2 * x][0] = hmul2(h[0], s1);
            kb[t][2 * x][1] = hmul2(h[1], s1);
            kb[t][2 * x + 1][0] = hmul2(h[2], s1);
            kb[t][2 * x + 1][1] = hmul2(h[3], s1);
          }
        } else {
          const uint4* src = reinterpret_cast<const uint4*>((const uint16_t*)p.k + kr * D) + c;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            const uint4 v = src[4 * x];
            kb[t][2 * x][0] = v.x;
            kb[t][2 * x][1] = v.y;
            kb[t][2 * x + 1][0] = v.z;
            kb[t][2 * x + 1][1] = v.w;
          }
        }
      }
    }
    float col[4][2] = {};
    for (int grp = 0; grp < groups; ++grp) {
      if (groups > 1) {
        __syncthreads();
        stage(grp);
        __syncthreads();
      }
      const int tiles = (min(R - grp * kWtRows, kWtRows) + 15) / 16;
      if (live) {
        for (int mt = 0; mt < tiles; ++mt) {
          float s[4][4] = {};
#pragma unroll
          for (int x = 0; x < kSteps; ++x) {
            const uint4 a = qf[mt][x][lane];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              if constexpr (kKv4)
                mma16816_f16(s[t], a.x, a.z, a.y, a.w, kb[t][x][0], kb[t][x][1]);
              else
                mma16816_bf16(s[t], a.x, a.z, a.y, a.w, kb[t][x][0], kb[t][x][1]);
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int i = mt * 16 + hf * 8 + g;
            const float f = rowf[i], l = rowl[i];
            const int lim = rowt[i];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float w = ex2(fmaf(s[t][2 * hf + x], f, -l));
                col[t][x] += key0 + 8 * t + 4 * x + c <= lim ? w : 0.f;
              }
          }
        }
      }
    }
    if (key0 < L) {
      float mine = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = col[t][x];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          if (g == 2 * t + x) mine = v;
        }
      const int key = key0 + lane;  // 8 t + 4 x + c with g = 2 t + x
      if (key < L) out[key] = (in && key < P ? in[key] : 0.f) + mine;
    }
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int spec_kv_weights(const void* q, const void* k, const uint8_t* k_scales,
                               const float* lse, const int32_t* prefix_len,
                               const int32_t* path_len, const int32_t* path_nodes, int B, int N,
                               int Hq, int Hkv, int D, int S, float scale, float k_unit,
                               const float* weights, float* out, void* stream) {
  if (B < 0 || B > 65535 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hkv > 65535 ||
      Hq % Hkv != 0 || S < N)
    return SPEC_ERR_SHAPE;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !(scale < 3.4e38f) || !kv4_unit_ok(k_unit)) return SPEC_ERR_ARG;
  if (!k_scales && k_unit != 1.f) return SPEC_ERR_ARG;
  if (B == 0) return SPEC_OK;
  if (!q || !k || !lse || !prefix_len || !path_len || !out) return SPEC_ERR_ARG;
  if (((uintptr_t)q | (uintptr_t)k) % 16 != 0 || (uintptr_t)k_scales % 8 != 0 ||
      ((uintptr_t)lse | (uintptr_t)prefix_len | (uintptr_t)path_len | (uintptr_t)path_nodes |
       (uintptr_t)weights | (uintptr_t)out) %
              4 !=
          0)
    return SPEC_ERR_ARG;
  WeightParams p = {};
  p.q = (const uint16_t*)q;
  p.k = k;
  p.ks = k_scales;
  p.lse = lse;
  p.prefix_len = prefix_len;
  p.path_len = path_len;
  p.path_nodes = path_nodes;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.S = S;
  p.scale_log2 = scale * kLog2e * k_unit;
  p.in = weights;
  p.out = out;
  const dim3 grid((unsigned)((S + kWtKeys - 1) / kWtKeys), (unsigned)Hkv, (unsigned)B);
  cudaStream_t st = (cudaStream_t)stream;
  if (k_scales) {
    if (D == 128)
      kv_weights<128, true><<<grid, kWtThreads, 0, st>>>(p);
    else
      kv_weights<64, true><<<grid, kWtThreads, 0, st>>>(p);
  } else {
    if (D == 128)
      kv_weights<128, false><<<grid, kWtThreads, 0, st>>>(p);
    else
      kv_weights<64, false><<<grid, kWtThreads, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
