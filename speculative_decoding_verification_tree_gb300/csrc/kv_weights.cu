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
// A warp takes 32 keys: m16n8k16 products with the keys as the 16-row operand
// and eight accepted rows (fragments of q in shared memory) as the other, then
// the sums of the exponentials over the rows, most of them in registers.  Lane
// (g, c) takes a quarter of key g's 4-bit row, or the 16-byte chunks c, c + 4,
// ... of its bf16 row; the k index is a permutation of the head dims that q
// shares.  bf16 keys go from global memory straight into operand registers
// (8 KB a warp in flight); 4-bit keys are too small for that (2 KB), so each
// warp keeps a ring of cp.async stages.  Every position belongs to one warp and
// its sum has a fixed order: no atomics.
// Work: the 256-key blocks (32 keys a warp) of all (sequence, head) pairs form
// one line, cut into equal pieces, one per resident CTA.
// Bounds and times (32 sequences of 2 to 4 K keys, 32 / 8 heads, D 128, caches
// cold): bf16, one row a head, 208 MB in 37 us = 5.6 TB/s, HBM; 4-bit after a
// 60-node tree, 64 MB in 34 us = 1.9 TB/s (30 us with keys and weights in L2), the
// latency of conversion, product and exponential in one warp's 32 keys (issue
// 47%; a third CTA per SM, or 4-bit keys loaded straight into registers, measured
// slower).
#include <cfloat>
#include <type_traits>

#include "kernels.h"
#include "kv4.cuh"
#include "line.cuh"

namespace sv {
namespace {

constexpr int kWtWarps = 8;
constexpr int kWtThreads = kWtWarps * 32;
constexpr int kWtKeys = kWtWarps * 32;  // keys of a CTA's iteration
constexpr int kWtCtas = 2;              // per SM
constexpr int kWtStages = 5;            // 32-key stages of a warp's ring (4-bit keys)
constexpr int kWtRows = 64;             // query rows staged at a time
constexpr int kWtNodes = 64;            // most accepted nodes (N)

struct WeightParams {
  const uint16_t* q;
  const void* k;
  const uint8_t* ks;
  const float* lse;
  const int32_t *prefix_len, *path_len, *path_nodes;
  int B, N, Hq, Hkv, S;
  ScoreScale scale;  // scale log2(e) k_unit (4-bit keys)
  float factor;      // scale log2(e) (bf16 keys)
  const float* in;
  float* out;
};

__device__ __forceinline__ int wt_prefix(const WeightParams& p, int b) {
  const int P = p.prefix_len[b];
  return P < 0 ? 0 : (P > p.S - p.N ? p.S - p.N : P);
}
// 256-key blocks of sequence b, all heads (an invalid path is found later: it
// may leave the last block empty).
struct WeightBlocks {
  const WeightParams& p;
  __device__ __forceinline__ int64_t operator()(int b) const {
    const int n = p.path_len[b];
    const int L = wt_prefix(p, b) + (n < 0 || n > p.N ? 0 : n);
    return (int64_t)((L + kWtKeys - 1) / kWtKeys) * p.Hkv;
  }
};

template <int D, bool kKv4>
struct WtSmem {
  static constexpr int kCodes = 32 * (D / 2), kStage = kCodes + 32 * (D / 16);
  unsigned char ring[kKv4 ? kWtWarps * kWtStages * kStage : 16];
  uint2 qf[kWtRows / 8][D / 16][32];  // operand registers b0, b1 per lane
  float rowf[kWtRows], rowl[kWtRows];  // scale, and the normaliser negated
  int rowt[kWtRows], nodes[kWtNodes];
  int64_t line[kWtThreads + 1], tmp[kWtWarps];
};

template <int D, bool kKv4>
__global__ void __launch_bounds__(kWtThreads, kWtCtas) kv_weights(const WeightParams p) {
  constexpr int kSteps = D / 16;
  using Sm = WtSmem<D, kKv4>;
  extern __shared__ __align__(16) unsigned char raw_s[];
  Sm& sm = *reinterpret_cast<Sm*>(raw_s);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int Gq = p.Hq / p.Hkv;
  const WeightBlocks blocks = {p};
  scan_line<kWtThreads>(p.B, blocks, sm.line, sm.tmp);
  const int64_t total = sm.line[kWtThreads];
  const int64_t piece = (total + gridDim.x - 1) / gridDim.x;
  int64_t line_at = (int64_t)blockIdx.x * piece;
  const int64_t line_end = min(total, line_at + piece);
  if (line_at >= total) return;
  int64_t seq_start;
  int b = locate<kWtThreads>(p.B, blocks, sm.line, line_at, &seq_start);

  while (line_at < line_end) {
    const int64_t seq_blocks = blocks(b);
    if (seq_blocks == 0) {  // nothing in this sequence
      ++b;
      continue;
    }
    // ---- the piece's share of one head's keys: first .. last
    const int per_head = (int)(seq_blocks / p.Hkv);
    const int kvh = (int)((line_at - seq_start) / per_head);
    const int64_t head_start = seq_start + (int64_t)kvh * per_head;
    const int k0 = (int)(line_at - head_start);
    const int k1 = (int)min((int64_t)per_head, line_end - head_start);
    const int64_t row0 = ((int64_t)b * p.Hkv + kvh) * p.S;
    const int P = wt_prefix(p, b);
    int n = p.path_len[b];
    int node = threadIdx.x;
    if (p.path_nodes && threadIdx.x < p.N) node = p.path_nodes[(int64_t)b * p.N + threadIdx.x];
    if (threadIdx.x < kWtNodes) sm.nodes[threadIdx.x] = node;
    // an invalid path adds nothing
    const bool bad = n < 0 || n > p.N || ((int)threadIdx.x < n && (node < 0 || node >= p.N));
    if (__syncthreads_or(bad)) n = 0;
    const int L = P + n;
    const int R = n * Gq;
    const int groups = (R + kWtRows - 1) / kWtRows;
    const float* in = p.in ? p.in + row0 : nullptr;
    float* out = p.out + row0;
    const int first = k0 * kWtKeys, last = min(L, k1 * kWtKeys);

    // a stage of this warp's ring: 32 keys' codes, then their scales; keys behind
    // the sequence are zeros, not read.  The source pointers run ahead of the
    // loop by kWtStages - 1 blocks.
    constexpr int kChunks = D / 32;  // 16-byte chunks per key
    const uint32_t ring = smem_u32(sm.ring) + (uint32_t)(warp * kWtStages * Sm::kStage);
    const uint32_t lane_dst = ring + (uint32_t)(lane * 16);
    const uint32_t lane_dst_s = ring + (uint32_t)(Sm::kCodes + lane * (D / 16));
    int fill_key = first + warp * 32;
    const uint8_t* codes = (const uint8_t*)p.k + (row0 + fill_key) * (D / 2) + lane * 16;
    const uint8_t* scales = p.ks + (row0 + fill_key + lane) * (D / 16);
    auto fill = [&](uint32_t slot_at) {
      const int left = last - fill_key;
      if (left >= 32) {
#pragma unroll
        for (int r = 0; r < kChunks; ++r)
          cp_async<16>(lane_dst + slot_at + (uint32_t)(r * 512), codes + r * 512);
        cp_async<D / 16>(lane_dst_s + slot_at, scales);
      } else if (left > 0) {
#pragma unroll
        for (int r = 0; r < kChunks; ++r) {
          const bool take = (r * 32 + lane) / kChunks < left;
          cp_async_or_zero<16>(lane_dst + slot_at + (uint32_t)(r * 512),
                               take ? codes + r * 512 : (const uint8_t*)p.k, take);
        }
        cp_async_or_zero<D / 16>(lane_dst_s + slot_at, lane < left ? scales : p.ks, lane < left);
      }
      cp_async_commit();
      fill_key += kWtKeys;
      codes += kWtKeys * (D / 2);
      scales += kWtKeys * (D / 16);
    };
    if constexpr (kKv4) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kWtStages - 1; ++i) fill((uint32_t)(i * Sm::kStage));
    }

    // the accepted rows of q as operand fragments, their scales, normalisers and
    // last visible positions; every warp takes rows warp, warp + 8, ...
    auto stage = [&](int grp) {
      constexpr int kMine = kWtRows / kWtWarps;
      const int rows = (min(R - grp * kWtRows, kWtRows) + 7) & ~7;
      uint2 w[kMine];
      float l[kMine];
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        const int i = warp + kWtWarps * x, r = grp * kWtRows + i;
        w[x] = make_uint2(0, 0);
        l[x] = neg_inf();
        if (i < rows && r < R) {
          const int t = r / Gq;
          const int64_t qrow = ((int64_t)b * p.N + sm.nodes[t]) * p.Hq + kvh * Gq + (r - t * Gq);
          if (lane < D / 4) w[x] = *reinterpret_cast<const uint2*>(p.q + qrow * D + 4 * lane);
          l[x] = p.lse[qrow];
        }
      }
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        const int i = warp + kWtWarps * x, r = grp * kWtRows + i;
        if (i >= rows) break;
        int up = 0;  // the row was scaled by 2^-up
        uint32_t h0 = w[x].x, h1 = w[x].y;
        int s, cc;
        if constexpr (kKv4) {
          // scaled by a power of two to [1, 2): exact in fp16 (see kv4_attn.cu)
          const float x0 = bf16_lo(h0), x1 = bf16_hi(h0), x2 = bf16_lo(h1), x3 = bf16_hi(h1);
          const float mx =
              warp_max(fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3))));
          int e = (int)(__float_as_uint(mx) >> 23) - 127;
          if (mx == 0.f || e == 128) e = 0;
          e = max(-126, min(126, e));
          const float dn = __uint_as_float((uint32_t)(127 - e) << 23);
          up = e;
          h0 = pack_half2(x0 * dn, x1 * dn);
          h1 = pack_half2(x2 * dn, x3 * dn);
          cc = lane / (D / 16);
          s = lane % (D / 16);
        } else {
          cc = (lane >> 1) & 3;
          s = 2 * (lane >> 3) + (lane & 1);
        }
        if (lane < D / 4) sm.qf[i >> 3][s][4 * (i & 7) + cc] = make_uint2(h0, h1);
        if (lane == 0) {
          sm.rowf[i] = kKv4 ? row_factor(p.scale, up) : p.factor;
          // a row that saw nothing weighs nothing, whatever the keys hold
          const bool blind = l[x] == neg_inf();
          sm.rowl[i] = blind ? l[x] : -l[x];
          sm.rowt[i] = r < R && !blind ? P + r / Gq : -1;
        }
      }
    };
    if (groups == 1) stage(0);
    __syncthreads();

    uint32_t slot_at = 0;  // the stage that holds this iteration's keys
    const float* in_p = in + first + warp * 32 + 8 * c + g;   // the key this lane writes
    float* out_p = out + first + warp * 32 + 8 * c + g;
    for (int at = first; at < last; at += kWtKeys, in_p += kWtKeys, out_p += kWtKeys) {
      const int key0 = at + warp * 32;
      const bool live = key0 < L && groups > 0;
      const int key = key0 + 8 * c + g;
      const float before = in && key < P ? *in_p : 0.f;
      // operand fragments: [8 keys][k step][a0 / a1, a2 / a3]
      uint32_t kb[kKv4 ? 2 : 4][kSteps][2];
      const unsigned char *st_keys = nullptr, *st_scales = nullptr;
      if constexpr (kKv4) {
        cp_async_wait<kWtStages - 2>();
        __syncwarp();
        constexpr uint32_t kEnd = (kWtStages - 1) * Sm::kStage;
        fill(slot_at == 0 ? kEnd : slot_at - Sm::kStage);
        const unsigned char* st = sm.ring + warp * kWtStages * Sm::kStage + slot_at;
        slot_at = slot_at == kEnd ? 0 : slot_at + Sm::kStage;
        st_keys = st + g * (D / 2) + 4 * (D / 32) * c;
        st_scales = st + Sm::kCodes + g * (D / 16);
      } else if (live) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int kk = key0 + 8 * t + g;
          const uint4* src = reinterpret_cast<const uint4*>(
                                 (const uint16_t*)p.k + (row0 + (kk < L ? kk : key0)) * D) + c;
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
      float2 col[4] = {};  // keys 8 t + g, summed over this lane's even and odd rows
      for (int grp = 0; grp < groups; ++grp) {
        if (groups > 1) {
          __syncthreads();
          stage(grp);
          __syncthreads();
        }
        const int tiles = (min(R - grp * kWtRows, kWtRows) + 7) / 8;
        if (live) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // sixteen keys at a time
            if constexpr (kKv4) {
              constexpr int kW = D / 32;
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const unsigned char* kr = st_keys + (16 * u + 8 * t) * (D / 2);
                const unsigned char* sr = st_scales + (16 * u + 8 * t) * (D / 16);
                uint32_t w[kW], s2;
                if constexpr (D == 128) {
                  const uint4 v = *reinterpret_cast<const uint4*>(kr);
                  w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
                  s2 = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(sr + 2 * c));
                } else {
                  const uint2 v = *reinterpret_cast<const uint2*>(kr);
                  w[0] = v.x; w[1] = v.y;
                  s2 = e4m3x2_to_half2(sr[c]);
                }
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
              }
            }
            const uint32_t(&ka)[kSteps][2] = kb[kKv4 ? 0 : 2 * u];
            const uint32_t(&kc)[kSteps][2] = kb[kKv4 ? 1 : 2 * u + 1];
            // kTiles row tiles from nt on; even and odd k steps apart, so that
            // two tiles are four independent chains of products
            auto tiles_of = [&](auto count, int nt) {
              constexpr int kTiles = decltype(count)::value;
              float s[kTiles][2][4];
#pragma unroll
              for (int x = 0; x < kSteps; ++x)
#pragma unroll
                for (int y = 0; y < kTiles; ++y) {
                  const uint2 q = sm.qf[nt + y][x][lane];
                  float(&d)[4] = s[y][x & 1];
                  if (kKv4 && x < 2)
                    mma16816_f16_first(d, ka[x][0], kc[x][0], ka[x][1], kc[x][1], q.x, q.y);
                  else if (kKv4)
                    mma16816_f16(d, ka[x][0], kc[x][0], ka[x][1], kc[x][1], q.x, q.y);
                  else if (x < 2)
                    mma16816_bf16_first(d, ka[x][0], kc[x][0], ka[x][1], kc[x][1], q.x, q.y);
                  else
                    mma16816_bf16(d, ka[x][0], kc[x][0], ka[x][1], kc[x][1], q.x, q.y);
                }
#pragma unroll
              for (int y = 0; y < kTiles; ++y) {
                const int i = (nt + y) * 8 + 2 * c;  // this lane's rows i, i + 1
                const float2 f = *reinterpret_cast<const float2*>(&sm.rowf[i]);
                const float2 l = *reinterpret_cast<const float2*>(&sm.rowl[i]);
                const bool whole = key0 + 31 <= P && (nt + y) * 8 + 8 <= R - grp * kWtRows &&
                                   fminf(l.x, l.y) != neg_inf();
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  const float2 e =
                      ffma2(fadd2(make_float2(s[y][0][2 * t], s[y][0][2 * t + 1]),
                                  make_float2(s[y][1][2 * t], s[y][1][2 * t + 1])),
                            f, l);
                  float2 w = make_float2(ex2(e.x), ex2(e.y));
                  if (!whole) {
                    const int2 lim = *reinterpret_cast<const int2*>(&sm.rowt[i]);
                    const int k = key0 + 16 * u + 8 * t + g;
                    if (k > lim.x) w.x = 0.f;
                    if (k > lim.y) w.y = 0.f;
                  }
                  col[2 * u + t] = fadd2(col[2 * u + t], w);
                }
              }
            };
            int nt = 0;
            for (; nt + 1 < tiles; nt += 2) tiles_of(std::integral_constant<int, 2>(), nt);
            if (nt < tiles) tiles_of(std::integral_constant<int, 1>(), nt);
          }
        }
      }
      if (key0 < L) {
        float mine = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float v = col[t].x + col[t].y;
          v += __shfl_xor_sync(0xffffffffu, v, 1);
          v += __shfl_xor_sync(0xffffffffu, v, 2);
          if (c == t) mine = v;
        }
        if (key < L) *out_p = before + mine;
      }
    }
    if constexpr (kKv4) cp_async_wait<0>();
    __syncthreads();  // the next share stages its own rows
    line_at = head_start + k1;
    if (line_at == seq_start + seq_blocks) {
      seq_start = line_at;
      ++b;
    }
  }
}

template <int D, bool kKv4>
cudaError_t launch_weights(const WeightParams& p, int grid, cudaStream_t st) {
  constexpr int smem = (int)sizeof(WtSmem<D, kKv4>);
  static_assert((smem + 1024) * kWtCtas <= 228 * 1024, "the pieces are resident at once");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem((const void*)kv_weights<D, kKv4>, smem, done);
  if (e != cudaSuccess) return e;
  kv_weights<D, kKv4><<<grid, kWtThreads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int spec_kv_weights(const void* q, const void* k, const uint8_t* k_scales,
                               const float* lse, const int32_t* prefix_len,
                               const int32_t* path_len, const int32_t* path_nodes, int B, int N,
                               int Hq, int Hkv, int D, int S, float scale, float k_unit,
                               const float* weights, float* out, void* stream) {
  if (B < 0 || B > 65535 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || S < N ||
      S > SPEC_MAX_POSITIONS || (int64_t)N * (Hq / Hkv) > (1 << 30) ||
      (double)B * Hkv * S > 4.0e15)
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
  p.scale = score_scale(scale, k_unit);
  p.factor = fminf(scale * kLog2e, FLT_MAX);
  p.in = weights;
  p.out = out;
  p.B = B;
  // one CTA per piece; no more pieces than blocks
  const int64_t most = (((int64_t)S + kWtKeys - 1) / kWtKeys) * B * Hkv;
  const int grid = (int)(most < kWtCtas * 152 ? most : kWtCtas * 152);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (k_scales)
    e = D == 128 ? launch_weights<128, true>(p, grid, st) : launch_weights<64, true>(p, grid, st);
  else
    e = D == 128 ? launch_weights<128, false>(p, grid, st) : launch_weights<64, false>(p, grid, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
