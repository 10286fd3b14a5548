// spec_tree_attention_kv4: tree / single-token attention over the 4-bit cache.
//
//   o_i = sum_s p_is v_s / sum_s p_is,   p_is = 2^(f_i (q_i . k_s) - m_i)
//
// over the visible keys s of query row i, in one pass over the cache with a
// running reference m (f_i carries scale log2(e), k_unit and the row's power
// of two, below).  Query rows of one (sequence, key/value head) are its
// (node, head in the group) pairs, node-major.
//
// Numbers.  Cache values are exact in fp16 (kv4.cuh).  A row of q (bf16, eight
// significant bits) is scaled by the power of two that brings its largest
// element to [1, 2) and is then exact in fp16 down to 2^-14 of it (below that
// the error is 2^-25 of the largest).  p is taken against a reference lifted
// by 2^7 and rounded to fp16 for the second product: at most 2^15, and
// eleven bits for every key within 2^-21 of the reference.  Scores, sums
// and outputs are float32.
//
// Kernel kv4_rows (16 query rows a tile, or 8): warp-level m16n8k16 products whose
// operands are converted in registers, so the cache crosses shared memory
// once, as codes.  Each warp owns a ring of 32-key stages filled with cp.async
// and needs no other warp until its keys are done.
//   S = Q K^T: lane (g, c) = (lane / 4, lane % 4) loads the contiguous
//     quarter c of key g's row; the k index of the product is a permutation
//     of the head dims, the same for Q.
//   O = P V: the lane that holds P's columns of four keys loads their dims
//     [D/8 g, D/8 (g + 1)); the codes of a key pair are interleaved by
//     half bytes so that one conversion yields (v_s[d], v_s'[d]).
//   The stage's rows are permuted (and their 16-byte chunks exchanged) so
//     that neither read has bank conflicts.
// Work: the 32-key blocks of all (sequence, head, row tile) units form one
// line, cut into equal pieces, one per CTA, whatever the sequences' lengths; a
// unit cut by a piece border leaves partial (m, l, O) in the workspace, and
// kv4_combine joins them.
#include <cuda_runtime.h>

#include "kernels.h"
#include "kv4.cuh"

namespace sv {
namespace {

constexpr int kKeys = 32;       // keys per stage
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kMaxCtas = 304;   // two per SM
constexpr int kMinBlocks = 8;   // a CTA's smallest piece: one block per warp
constexpr float kLift = 7.f;    // log2 of the factor that lifts P

struct RowsParams {
  const uint16_t* q;
  const uint8_t *kc, *ks, *vc, *vs;
  const int32_t* prefix_len;
  const uint64_t* mask_bits;
  int B, N, Hq, Hkv, S, R, nrt;
  float scale_log2;  // scale * log2(e) * k_unit
  float v_unit;
  uint16_t* out;
  float* lse;    // or null
  float* part;   // [2 * gridDim.x][rows per tile][D + 2]
};

__device__ __forceinline__ int clamped_prefix(const RowsParams& p, int b) {
  const int v = p.prefix_len[b];
  return v < 0 ? 0 : (v > p.S - p.N ? p.S - p.N : v);
}
__device__ __forceinline__ int seq_blocks(const RowsParams& p, int b) {
  return (clamped_prefix(p, b) + p.N + kKeys - 1) / kKeys;
}

// Inclusive scan over the CTA of each thread's value; `tmp` holds one value
// per warp.  Returns the exclusive prefix; *total the sum.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t* tmp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t x = tmp[w];
    if (w < warp) before += x;
    all += x;
  }
  __syncthreads();
  *total = all;
  return before + s - v;
}

// The line of blocks: sequences in order, each with `units` runs (heads x
// row tiles) of seq_blocks.  Every thread sums a contiguous run of sequences.
struct LineScan {
  int64_t mine, total;  // blocks before this thread's sequences; all blocks
  int first, last;      // this thread's sequences
};
__device__ __forceinline__ LineScan scan_line(const RowsParams& p, int units, int64_t* tmp) {
  LineScan r;
  const int per = (p.B + kThreads - 1) / kThreads;
  r.first = min(p.B, (int)threadIdx.x * per);
  r.last = min(p.B, r.first + per);
  int64_t v = 0;
  for (int b = r.first; b < r.last; ++b) v += (int64_t)seq_blocks(p, b) * units;
  r.mine = cta_scan(v, tmp, &r.total);
  return r;
}
__device__ __forceinline__ int64_t piece_blocks(int64_t total, int ctas) {
  const int64_t q = (total + ctas - 1) / ctas;
  return q < kMinBlocks ? kMinBlocks : q;
}

template <int D>
struct Stage {
  static constexpr int kRow = D / 2;             // bytes of codes per key
  static constexpr int kCodes = kKeys * kRow;
  static constexpr int kSRow = D / kKv4Block;    // bytes of scales per key
  static constexpr int kScales = kKeys * kSRow;
  static constexpr int kK = 0, kV = kCodes, kKS = 2 * kCodes, kVS = 2 * kCodes + kScales;
  static constexpr int kBytes = 2 * kCodes + 2 * kScales;
  // where chunk `ch` (16 bytes) of key `key` lies: see the comment at the top
  __device__ __forceinline__ static int at(int key, int ch) {
    if constexpr (D == 128)
      return (key ^ ((key >> 2) & 1)) * kRow + ((ch ^ (key & 2)) << 4);
    else
      return (key ^ ((key >> 1) & 2)) * kRow + (ch << 4);
  }
};

template <int D, int RT>
struct RowsSmem {
  static constexpr int kRing = kWarps * kStages * Stage<D>::kBytes;
  static constexpr int kPitch = D + 16;  // floats per row of the merge buffer
  static constexpr int kMerge = kWarps * RT * kPitch * 4;
  static_assert(kMerge + kWarps * RT * 8 <= kRing, "the merge buffers lie in the ring");
  unsigned char ring[kRing];
  uint32_t qf[(D / 16) * 32 * (RT / 4)];  // A fragments: a0 a2 (a1 a3) per lane and k step
  float rowf[RT];
  uint64_t rowmask[RT];
  unsigned long long vnan[D / kKv4Block];  // drafted keys whose V block is NaN
  int64_t scan[kWarps];
  int64_t seg_start;
  int seg_b;
};

// One 32-key stage of one warp.
template <int D>
__device__ __forceinline__ void fill_stage(const RowsParams& p, uint32_t st, int64_t row0, int key0,
                                           int L, int lane) {
  using G = Stage<D>;
  constexpr int kChunks = G::kRow / 16;
  const uint8_t* kc = p.kc + (row0 + key0) * G::kRow;
  const uint8_t* vc = p.vc + (row0 + key0) * G::kRow;
  const int left = L - key0;
#pragma unroll
  for (int r = 0; r < kChunks; ++r) {
    const int id = r * 32 + lane;
    const int key = id / kChunks, ch = id % kChunks;
    const bool take = key < left;
    const int64_t off = take ? (int64_t)id * 16 : 0;
    const uint32_t dst = st + (uint32_t)G::at(key, ch);
    cp_async<16>(dst + G::kK, kc + off, take);
    cp_async<16>(dst + G::kV, vc + off, take);
  }
  const bool take = lane < left;
  const int64_t off = (row0 + key0 + (take ? lane : 0)) * G::kSRow;
  cp_async<G::kSRow>(st + G::kKS + (uint32_t)(lane * G::kSRow), p.ks + off, take);
  cp_async<G::kSRow>(st + G::kVS + (uint32_t)(lane * G::kSRow), p.vs + off, take);
}

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, 2) kv4_rows(const RowsParams p) {
  using G = Stage<D>;
  using Sm = RowsSmem<D, RT>;
  constexpr int kHalves = RT / 8;     // row halves a lane holds
  constexpr int kNT = D / 8;          // n tiles of O
  constexpr int kW = D / 32;          // code words a lane loads per key of K
  extern __shared__ __align__(16) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  launch_dependents();

  const int units = p.Hkv * p.nrt;
  const LineScan ls = scan_line(p, units, sm.scan);
  const int64_t piece = piece_blocks(ls.total, (int)gridDim.x);
  int64_t at = (int64_t)blockIdx.x * piece;
  const int64_t end = min(ls.total, at + piece);
  if (at >= ls.total) return;
  {  // the sequence that holds block `at`: one thread's run contains it
    int64_t x = ls.mine;
    for (int b = ls.first; b < ls.last; ++b) {
      const int64_t n = (int64_t)seq_blocks(p, b) * units;
      if (at >= x && at < x + n) {
        sm.seg_b = b;
        sm.seg_start = x;
      }
      x += n;
    }
  }
  __syncthreads();
  int b = sm.seg_b;
  int64_t seq_start = sm.seg_start;
  const int Gq = p.Hq / p.Hkv;

  while (at < end) {
    // ---------------------------------------------------- this segment
    const int P = clamped_prefix(p, b), L = P + p.N;
    const int nblk = (L + kKeys - 1) / kKeys;
    const int unit = (int)((at - seq_start) / nblk);
    const int64_t unit_start = seq_start + (int64_t)unit * nblk;
    const int k0 = (int)(at - unit_start);
    const int k1 = (int)min((int64_t)nblk, end - unit_start);
    const int kvh = unit / p.nrt, rt = unit % p.nrt;
    const int64_t row0 = ((int64_t)b * p.Hkv + kvh) * p.S;

    const uint32_t ring = smem_u32(sm.ring) + (uint32_t)(warp * kStages * G::kBytes);
    const unsigned char* ringp = sm.ring + warp * kStages * G::kBytes;
    const int mine = (k1 - k0 - warp + kWarps - 1) / kWarps;  // blocks k0 + warp + 8 i
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < mine)
        fill_stage<D>(p, ring + (uint32_t)(i * G::kBytes), row0, (k0 + warp + kWarps * i) * kKeys,
                      L, lane);
      cp_async_commit();
    }

    // q rows -> fp16 fragments, each scaled by a power of two
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
      const int row = hf * 8 + warp;  // kWarps == 8 rows per half
      const int r = rt * RT + row;
      const bool valid = r < p.R;
      const int node = valid ? r / Gq : 0;
      const int hq = kvh * Gq + (valid ? r % Gq : 0);
      const uint16_t* src = p.q + (((int64_t)b * p.N + node) * p.Hq + hq) * D;
      float x[D / 32];
      if constexpr (D == 128) {
        const uint2 w = valid ? *reinterpret_cast<const uint2*>(src + 4 * lane) : make_uint2(0, 0);
        x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
      } else {
        const uint32_t w = valid ? *reinterpret_cast<const uint32_t*>(src + 2 * lane) : 0u;
        x[0] = bf16_lo(w); x[1] = bf16_hi(w);
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) mx = fmaxf(mx, fabsf(x[i]));
      mx = warp_max(mx);
      int e = (int)(__float_as_uint(mx) >> 23) - 127;
      if (mx == 0.f || e == 128) e = 0;  // a zero row; an infinite one stays as it is
      e = max(-126, min(126, e));
      const float dn = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) x[i] *= dn;
      // dims 4 s .. 4 s + 3 of quarter c: the a0 / a2 pair of k step s
      uint32_t* dst;
      if constexpr (D == 128) {
        dst = sm.qf + ((lane & 7) * 32 + warp * 4 + (lane >> 3)) * (RT / 4) + 2 * hf;
        dst[0] = pack_half2(x[0], x[1]);
        dst[1] = pack_half2(x[2], x[3]);
      } else {
        dst = sm.qf + (((lane & 7) >> 1) * 32 + warp * 4 + (lane >> 3)) * (RT / 4) + 2 * hf;
        dst[lane & 1] = pack_half2(x[0], x[1]);
      }
      if (lane == 0) {
        sm.rowf[row] = p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
        sm.rowmask[row] = valid ? p.mask_bits[(int64_t)b * p.N + node] : 0ull;
      }
    }
    if (threadIdx.x < D / kKv4Block) sm.vnan[threadIdx.x] = 0ull;
    __syncthreads();

    float f[kHalves], m[kHalves], l[kHalves];
    float o[kNT][4];
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
      f[hf] = sm.rowf[hf * 8 + g];
      m[hf] = neg_inf();
      l[hf] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < kNT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    for (int i = 0; i < mine; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      {
        const int nx = i + kStages - 1;
        if (nx < mine)
          fill_stage<D>(p, ring + (uint32_t)((nx % kStages) * G::kBytes), row0,
                        (k0 + warp + kWarps * nx) * kKeys, L, lane);
        cp_async_commit();
      }
      const unsigned char* st = ringp + (i % kStages) * G::kBytes;
      const int key0 = (k0 + warp + kWarps * i) * kKeys;
      const bool tail = key0 + kKeys > P;

      // ------------------------------------------------------ S = Q K^T
      float s[4][4];
      uint32_t kw[4][kW], ksc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
        const int key = 8 * t + 4 * (g & 1) + (g >> 1);
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(st + G::kK + G::at(key, c));
          kw[t][0] = w.x; kw[t][1] = w.y; kw[t][2] = w.z; kw[t][3] = w.w;
          ksc[t] = e4m3x2_to_half2(
              *reinterpret_cast<const uint16_t*>(st + G::kKS + key * G::kSRow + 2 * c));
        } else {
          const uint2 w =
              *reinterpret_cast<const uint2*>(st + G::kK + G::at(key, c >> 1) + 8 * (c & 1));
          kw[t][0] = w.x; kw[t][1] = w.y;
          ksc[t] = e4m3x2_to_half2(st[G::kKS + key * G::kSRow + c]);
        }
      }
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        uint32_t a[2][RT / 4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t* src = sm.qf + ((2 * w + x) * 32 + lane) * (RT / 4);
          if constexpr (RT == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            a[x][0] = v.x; a[x][1] = v.y; a[x][2] = v.z; a[x][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            a[x][0] = v.x; a[x][1] = v.y;
          }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t h[4];
          e2m1x8_to_half2(kw[t][w], h);
          const uint32_t sc = (D == 128 && w >= 2) ? dup_hi(ksc[t]) : dup_lo(ksc[t]);
#pragma unroll
          for (int x = 0; x < 4; ++x) h[x] = hmul2(h[x], sc);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            mma16816_f16(s[t], a[x][0], RT == 16 ? a[x][RT / 4 - 2] : 0u, a[x][1],
                         RT == 16 ? a[x][RT / 4 - 1] : 0u, h[2 * x], h[2 * x + 1]);
        }
      }
      // ------------------------------------- running softmax, base 2
      if (tail) {
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf) {
          const uint64_t mb = sm.rowmask[hf * 8 + g];
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int d = key0 + 8 * t + 4 * x + c - P;
              const bool vis = d < 0 || (d < p.N && ((mb >> (d & 63)) & 1ull));
              if (!vis) s[t][2 * hf + x] = neg_inf();
            }
        }
      }
      float bm[kHalves];
      bool grow = false;
#pragma unroll
      for (int hf = 0; hf < kHalves; ++hf) {
        float v = fmaxf(s[0][2 * hf], s[0][2 * hf + 1]);
#pragma unroll
        for (int t = 1; t < 4; ++t) v = fmax3f(v, s[t][2 * hf], s[t][2 * hf + 1]);
        bm[hf] = v * f[hf];
        grow |= bm[hf] > m[hf] + 8.f;
      }
      // the reference moves only when a row's maximum grows by more than 2^8
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf) {
          float v = fmaxf(bm[hf], __shfl_xor_sync(0xffffffffu, bm[hf], 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          const bool move = v > m[hf] + 8.f;
          const float mn = move ? v : m[hf];
          const float corr = move ? ex2(m[hf] - mn) : 1.f;  // 0 at the first visible key
          m[hf] = mn;
          l[hf] *= corr;
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            o[j][2 * hf] *= corr;
            o[j][2 * hf + 1] *= corr;
          }
        }
      }
      uint32_t pa[4][kHalves];  // P as A fragments: [tile][half]
#pragma unroll
      for (int hf = 0; hf < kHalves; ++hf) {
        const float nm = m[hf] == neg_inf() ? kLift : kLift - m[hf];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float p0 = ex2(fmaf(s[t][2 * hf], f[hf], nm));
          const float p1 = ex2(fmaf(s[t][2 * hf + 1], f[hf], nm));
          l[hf] += p0 + p1;
          pa[t][hf] = pack_half2(p0, p1);
        }
      }
      // ------------------------------------------------------ O += P V
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t vw[4][D / 64];
        uint32_t sb[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = 16 * u + 4 * x + c;
          if constexpr (D == 128) {
            const uint2 w =
                *reinterpret_cast<const uint2*>(st + G::kV + G::at(key, g >> 1) + 8 * (g & 1));
            vw[x][0] = w.x; vw[x][1] = w.y;
            sb[x] = st[G::kVS + key * G::kSRow + g];
          } else {
            vw[x][0] =
                *reinterpret_cast<const uint32_t*>(st + G::kV + G::at(key, g >> 2) + 4 * (g & 3));
            sb[x] = st[G::kVS + key * G::kSRow + (g >> 1)];
          }
        }
        if (tail) {
          // a NaN block of a drafted key must reach the rows that see the
          // key and no others: it is noted and its scale replaced by zero
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int d = key0 + 16 * u + 4 * x + c - P;
            if (d >= 0 && d < p.N && (sb[x] & 0x7fu) == 0x7fu) {
              atomicOr(&sm.vnan[D == 128 ? g : (g >> 1)], 1ull << d);
              sb[x] = 0;
            }
          }
        }
        const uint32_t s01 = e4m3x2_to_half2(sb[0] | (sb[1] << 8));
        const uint32_t s23 = e4m3x2_to_half2(sb[2] | (sb[3] << 8));
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          constexpr uint32_t kLo = 0x0f0f0f0fu, kHi = 0xf0f0f0f0u;
          uint32_t b0[2][4], b1[2][4];  // [even / odd dim][pair of dims]
          e2m1x8_to_half2((vw[0][w] & kLo) | ((vw[1][w] << 4) & kHi), b0[0]);
          e2m1x8_to_half2(((vw[0][w] >> 4) & kLo) | (vw[1][w] & kHi), b0[1]);
          e2m1x8_to_half2((vw[2][w] & kLo) | ((vw[3][w] << 4) & kHi), b1[0]);
          e2m1x8_to_half2(((vw[2][w] >> 4) & kLo) | (vw[3][w] & kHi), b1[1]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int od = 0; od < 2; ++od)
              mma16816_f16(o[8 * w + 2 * x + od], pa[2 * u][0],
                           kHalves == 2 ? pa[2 * u][kHalves - 1] : 0u, pa[2 * u + 1][0],
                           kHalves == 2 ? pa[2 * u + 1][kHalves - 1] : 0u, hmul2(b0[od][x], s01),
                           hmul2(b1[od][x], s23));
        }
      }
    }

    // ------------------------------------------- the warps' parts joined
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with its ring
    float* mbuf = reinterpret_cast<float*>(sm.ring);
    float2* ml = reinterpret_cast<float2*>(sm.ring + Sm::kMerge);  // [warp][row]: m, l
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
      if (c == 0) ml[warp * RT + hf * 8 + g] = make_float2(m[hf], l[hf]);
    }
    // lane (g, c) holds dims [D/4 c, D/4 (c + 1)) of rows g (and g + 8): column
    // even / odd of n tile j is dim D/8 (2 c) + j / D/8 (2 c + 1) + j.  16-byte
    // chunk index XOR c and the pitch spread the stores over the banks.
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
      float4* dst =
          reinterpret_cast<float4*>(mbuf + (int64_t)(warp * RT + hf * 8 + g) * Sm::kPitch);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int j = 0; j < kNT; j += 4) {
          const int chunk = (D / 16) * c + (x * kNT + j) / 4;
          dst[chunk ^ c] = make_float4(o[j][2 * hf + x], o[j + 1][2 * hf + x],
                                       o[j + 2][2 * hf + x], o[j + 3][2 * hf + x]);
        }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == nblk;
    float* part = p.part;
    if (!whole)
      part += ((int64_t)2 * blockIdx.x + (at == (int64_t)blockIdx.x * piece ? 0 : 1)) * RT *
              (D + 2);
    for (int e = threadIdx.x; e < RT * (D / 4); e += kThreads) {
      const int row = e / (D / 4), pc = e % (D / 4);
      const int chunk = pc ^ ((pc / (D / 16)) & 3);
      const int r = rt * RT + row;
      if (r >= p.R) continue;
      float M = neg_inf();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * RT + row].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 pw = ml[w * RT + row];
        // a part whose reference never moved holds zeros, or NaN scores
        const float k = pw.x == neg_inf() ? 1.f : ex2(pw.x - M);
        const float4 v =
            *reinterpret_cast<const float4*>(mbuf + (int64_t)(w * RT + row) * Sm::kPitch + 4 * pc);
        acc.x += v.x * k;
        acc.y += v.y * k;
        acc.z += v.z * k;
        acc.w += v.w * k;
        sum += pw.y * k;
      }
      if (sm.vnan[chunk * 4 / kKv4Block] & sm.rowmask[row])
        acc = make_float4(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff),
                          __int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
      if (whole) {
        const int node = r / Gq, hq = kvh * Gq + r % Gq;
        const int64_t orow = ((int64_t)b * p.N + node) * p.Hq + hq;
        const float inv = sum == 0.f ? 0.f : p.v_unit / sum;
        *reinterpret_cast<uint2*>(p.out + orow * D + 4 * chunk) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (p.lse && chunk == 0) p.lse[orow] = sum == 0.f ? neg_inf() : M + log2f(sum) - kLift;
      } else {
        float* dst = part + (int64_t)row * (D + 2);
        *reinterpret_cast<float2*>(dst + 4 * chunk) = make_float2(acc.x, acc.y);
        *reinterpret_cast<float2*>(dst + 4 * chunk + 2) = make_float2(acc.z, acc.w);
        if (chunk == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(M, sum);
      }
    }
    __syncthreads();
    at = unit_start + k1;
    if (unit + 1 == units && k1 == nblk) {  // the next block belongs to the next sequence
      seq_start += (int64_t)units * nblk;
      ++b;
    }
  }
}

// Joins the parts of a unit that several CTAs worked on.
template <int D, int RT>
__global__ void __launch_bounds__(kThreads) kv4_combine(const RowsParams p, int ctas) {
  __shared__ int64_t tmp[kWarps];
  __shared__ int64_t seq_start_s;
  __shared__ float wgt[kMaxCtas][RT];
  __shared__ float rowM[RT], rowL[RT];
  const int units = p.Hkv * p.nrt;
  const int b = (int)(blockIdx.x / units), unit = (int)(blockIdx.x % units);
  const LineScan ls = scan_line(p, units, tmp);
  if (b >= ls.first && b < ls.last) {
    int64_t x = ls.mine;
    for (int i = ls.first; i < b; ++i) x += (int64_t)seq_blocks(p, i) * units;
    seq_start_s = x;
  }
  __syncthreads();
  const int64_t piece = piece_blocks(ls.total, ctas);
  const int nblk = seq_blocks(p, b);
  const int64_t t0 = seq_start_s + (int64_t)unit * nblk, t1 = t0 + nblk;
  const int c0 = (int)(t0 / piece), c1 = (int)((t1 - 1) / piece);
  grid_dependency_wait();  // before any exit: this grid must not end first
  if (c0 == c1) return;
  const int n = c1 - c0 + 1;
  const int kvh = unit / p.nrt, rt = unit % p.nrt;
  const int Gq = p.Hq / p.Hkv;
  const int first = 2 * c0 + (t0 == (int64_t)c0 * piece ? 0 : 1);
  auto part = [&](int i, int row) {
    const int64_t slot = i == 0 ? first : 2 * (c0 + i);
    return p.part + (slot * RT + row) * (D + 2);
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int row = warp; row < RT; row += kWarps) {
    if (rt * RT + row >= p.R) continue;
    float M = neg_inf(), sum = 0.f;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, part(i, row)[D]);
    M = warp_max(M);
    for (int i = lane; i < n; i += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(part(i, row) + D);
      const float k = ml.x == neg_inf() ? 1.f : ex2(ml.x - M);
      wgt[i][row] = k;
      sum += ml.y * k;
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      rowM[row] = M;
      rowL[row] = sum;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < RT * (D / 2); e += kThreads) {
    const int row = e / (D / 2), x = e % (D / 2);
    const int r = rt * RT + row;
    if (r >= p.R) continue;
    float2 acc = make_float2(0.f, 0.f);
    for (int i = 0; i < n; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(part(i, row) + 2 * x);
      const float k = wgt[i][row];
      acc.x = fmaf(v.x, k, acc.x);
      acc.y = fmaf(v.y, k, acc.y);
    }
    const int node = r / Gq, hq = kvh * Gq + r % Gq;
    const int64_t orow = ((int64_t)b * p.N + node) * p.Hq + hq;
    const float sum = rowL[row];
    const float inv = sum == 0.f ? 0.f : p.v_unit / sum;
    *reinterpret_cast<uint32_t*>(p.out + orow * D + 2 * x) = pack_bf16x2(acc.x * inv, acc.y * inv);
    if (p.lse && x == 0) p.lse[orow] = sum == 0.f ? neg_inf() : rowM[row] + log2f(sum) - kLift;
  }
}

template <int D, int RT>
cudaError_t launch_rows(RowsParams p, cudaStream_t st) {
  constexpr int smem = (int)sizeof(RowsSmem<D, RT>);
  p.nrt = (p.R + RT - 1) / RT;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem((const void*)kv4_rows<D, RT>, smem, done);
  if (e != cudaSuccess) return e;
  // no more CTAs than pieces of the smallest size could fill
  const int64_t most = (int64_t)p.B * p.Hkv * p.nrt * ((p.S + kKeys - 1) / kKeys);
  const int64_t want = (most + kMinBlocks - 1) / kMinBlocks;
  const int ctas = (int)(want < kMaxCtas ? want : kMaxCtas);
  prof_begin(SPEC_PROF_ATTN, st);
  kv4_rows<D, RT><<<ctas, kThreads, smem, st>>>(p);
  prof_end(SPEC_PROF_ATTN, st);
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.Hkv * p.nrt));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_combine<D, RT>, p, ctas);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_tree_attention_kv4_workspace_bytes(int B, int N, int Hq, int Hkv, int D,
                                                          int S) {
  if (B < 0 || B > 65535 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || S < N ||
      (D != 64 && D != 128))
    return 0;
  const size_t bytes = (size_t)2 * kMaxCtas * 16 * (D + 2) * sizeof(float);
  return (bytes + 255) / 256 * 256;
}

extern "C" int spec_tree_attention_kv4(const void* q, const uint8_t* k_codes,
                                       const uint8_t* k_scales, const uint8_t* v_codes,
                                       const uint8_t* v_scales, const int32_t* prefix_len,
                                       const uint64_t* mask_bits, int B, int N, int Hq, int Hkv,
                                       int D, int S, float scale, float k_unit, float v_unit,
                                       void* out, float* lse, void* workspace, size_t ws_bytes,
                                       void* stream) {
  if (B < 0 || B > 65535 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || S < N)
    return SPEC_ERR_SHAPE;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !(scale < 3.4e38f) || !kv4_unit_ok(k_unit) || !kv4_unit_ok(v_unit))
    return SPEC_ERR_ARG;
  if (B == 0) return SPEC_OK;
  if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !prefix_len || !mask_bits || !out)
    return SPEC_ERR_ARG;
  if (((uintptr_t)k_codes | (uintptr_t)v_codes | (uintptr_t)q | (uintptr_t)out) % 16 != 0 ||
      ((uintptr_t)k_scales | (uintptr_t)v_scales | (uintptr_t)mask_bits) % 8 != 0 ||
      ((uintptr_t)prefix_len | (uintptr_t)lse) % 4 != 0)
    return SPEC_ERR_ARG;
  const int64_t R = (int64_t)N * (Hq / Hkv);
  const int64_t tiles = (R + 15) / 16;
  if ((int64_t)B * Hkv * tiles > 2147483647 || (double)B * Hkv * S > 4.0e15) return SPEC_ERR_SHAPE;
  if (!workspace || (uintptr_t)workspace % 256 != 0 ||
      ws_bytes < spec_tree_attention_kv4_workspace_bytes(B, N, Hq, Hkv, D, S))
    return SPEC_ERR_WORKSPACE;
  RowsParams p = {};
  p.q = (const uint16_t*)q;
  p.kc = k_codes;
  p.ks = k_scales;
  p.vc = v_codes;
  p.vs = v_scales;
  p.prefix_len = prefix_len;
  p.mask_bits = mask_bits;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.S = S;
  p.R = (int)R;
  p.scale_log2 = scale * kLog2e * k_unit;
  p.v_unit = v_unit;
  p.out = (uint16_t*)out;
  p.lse = lse;
  p.part = (float*)workspace;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (D == 128)
    e = R <= 8 ? launch_rows<128, 8>(p, st) : launch_rows<128, 16>(p, st);
  else
    e = R <= 8 ? launch_rows<64, 8>(p, st) : launch_rows<64, 16>(p, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
