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
// Kernel kv4_rows (room for 8, 16, 24 or 32 query rows): warp-level m16n8k16 products
// with the cache as the 16-row operand, converted in registers, so that it
// crosses shared memory once, as codes, and eight query rows waste nothing.
// Each warp owns a ring of 32-key stages filled with cp.async and needs no
// other warp until its keys are done.  Lane (g, c) = (lane / 4, lane % 4):
//   S^T = K Q^T: the lane loads quarter c of key g's codes (16 bytes at D 128);
//     the k index of the product is a permutation of the head dims, shared
//     with Q;
//   P^T changes from accumulator to operand layout by movmatrix;
//   O^T = V^T P^T: the lane loads dims [D/8 g, D/8 (g + 1)) of four keys; the
//     codes of two keys are interleaved by half bytes so that one conversion
//     yields (v_s[d], v_s'[d]).
// A conversion is one instruction per two codes, as is the product with the
// block scale; those two are half of what the kernel issues.
// Product row n of eight keys is key 4 (n & 1) + n / 2, and the stage's rows are
// permuted (and their 16-byte chunks exchanged) so that neither read has bank
// conflicts.
// Work: the 32-key blocks of all (sequence, head) units form one line, cut into
// equal pieces, one per warp, whatever the sequences' lengths; a unit cut by a
// piece border leaves partial (m, l, O) in the workspace, and kv4_combine joins
// them.  Warps never wait for one another.
// Short work, where the join's launch and traffic would cost more than idle
// warps, takes kv4_unit instead: a cluster of CTAs per unit, its warps' results
// joined through distributed shared memory (unit_cluster has the rule).
// Bounds and times (D 128, 32 / 8 heads, single tokens, caches cold): 64 sequences
// of 32 K keys, 2.39 GB of cache, 379 us = 6.3 TB/s, HBM; 32 of 2 to 4 K keys, 114
// MB, 32.7 us = 3.5 TB/s, uneven work (256 CTAs, one per sequence and head, on 304
// places, lengths apart by two: 27 us at the copy rate), then issue (55%) and the
// load latency of a unit's first and last blocks; one sequence of 128 K keys 40.5
// us, the join of 2341 pieces; one of 1 K keys 6.4 us, launch and one block's
// latency.
#include <cuda_runtime.h>
#include <stddef.h>

#include "kernels.h"
#include "kv4.cuh"
#include "kv4_attn.h"
#include "line.cuh"

namespace sv {
namespace {

constexpr int kKeys = 32;       // keys per stage
constexpr int kMinBlocks = 6;   // a warp's smallest piece (a join reads every piece's output)
constexpr float kLift = 7.f;    // log2 of the factor that lifts P
constexpr int kSms = 152;
constexpr int kRowsMax = 32;    // query rows up to which these kernels are used
constexpr int kJoinUnroll = 10; // 32-part groups read at once

struct RowsParams : Kv4Attn {
  float* part;       // [2 * warps][R][D]: O of a unit's piece
  float2* part_ml;   // [2 * warps][R]: its reference and sum
  int warps;         // pieces of the line
};

__device__ __forceinline__ int clamped_prefix(const RowsParams& p, int b) {
  const int v = p.prefix_len[b];
  return v < 0 ? 0 : (v > p.S - p.N ? p.S - p.N : v);
}
__device__ __forceinline__ int seq_blocks(const RowsParams& p, int b) {
  return (clamped_prefix(p, b) + p.N + kKeys - 1) / kKeys;
}

// The line of blocks: sequences in order, each with a run of seq_blocks per head.
struct LineBlocks {
  const RowsParams& p;
  __device__ __forceinline__ int64_t operator()(int b) const {
    return (int64_t)seq_blocks(p, b) * p.Hkv;
  }
};
__device__ __forceinline__ int64_t piece_blocks(int64_t total, int warps) {
  const int64_t q = (total + warps - 1) / warps;
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

// Warps per CTA, CTAs per SM and ring stages by the number of row tiles of
// eight, whose outputs take 32 registers each (D 128).  Products for rows that
// are not there cost as much as others: 20 rows in three tiles 58 us, in four 72
// (32 sequences of 2 to 4 K keys), 182 / 226 (16 of 32 K).  Three tiles with ten
// warps, q in shared memory, 72.  At D 128 kv4_rows spills with two tiles (92 bytes
// stored, 152 loaded a thread, at 168 registers) and with four (56 / 64 at 255).
template <int NT>
struct RowsCfg {
  static constexpr int kWarps = NT == 2 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kCtas = NT == 1 ? 2 : 1;  // per SM
  static constexpr int kStages = NT >= 3 ? 4 : 3;
  static constexpr bool kQShared = NT == 4;  // q's fragments in shared memory
  static constexpr int kPieces = kSms * kCtas * kWarps;
};

template <int D, int NT>
struct RowsSmem {
  static constexpr int kWarps = RowsCfg<NT>::kWarps;
  static constexpr int kRing = kWarps * RowsCfg<NT>::kStages * Stage<D>::kBytes;
  unsigned char ring[kRing];
  static constexpr bool kQ = RowsCfg<NT>::kQShared;
  uint2 qf[kQ ? kWarps : 1][kQ ? D / 16 : 1][NT][32];  // q's operand fragments
  unsigned long long vnan[kWarps][D / kKv4Block];  // drafted keys whose V block is NaN
  int64_t before[RowsCfg<NT>::kThreads + 1];
  int64_t tmp[kWarps];
};

// This lane's share of a stage: 16-byte chunks r * 32 + lane of the codes and
// key `lane`'s scales.  The addresses of a full stage differ from the lane's
// bases by constants.
template <int D>
struct LaneFill {
  using G = Stage<D>;
  static constexpr int kChunks = G::kRow / 16;
  uint32_t dst, dst_s;  // within the stage
  int64_t codes, scales;  // byte offsets of this lane within the cache, stage at key 0
  __device__ __forceinline__ LaneFill(int64_t row0, int lane)
      : dst((uint32_t)G::at(lane / kChunks, lane % kChunks)),
        dst_s((uint32_t)(lane * G::kSRow)),
        codes(row0 * G::kRow + lane * 16),
        scales((row0 + lane) * G::kSRow) {}
  __device__ __forceinline__ void issue(const RowsParams& p, uint32_t st, int key0, int L,
                                        int lane) const {
    const int64_t oc = codes + (int64_t)key0 * G::kRow, os = scales + (int64_t)key0 * G::kSRow;
    const uint8_t *kc = p.kc + oc, *vc = p.vc + oc;
    const int left = L - key0;
    if (left >= kKeys) {
#pragma unroll
      for (int r = 0; r < kChunks; ++r) {
        cp_async<16>(st + dst + G::kK + r * 512, kc + r * 512);
        cp_async<16>(st + dst + G::kV + r * 512, vc + r * 512);
      }
      cp_async<G::kSRow>(st + dst_s + G::kKS, p.ks + os);
      cp_async<G::kSRow>(st + dst_s + G::kVS, p.vs + os);
    } else {  // keys behind the sequence are zeros, not read
#pragma unroll
      for (int r = 0; r < kChunks; ++r) {
        const bool take = (r * 32 + lane) / kChunks < left;
        cp_async_or_zero<16>(st + dst + G::kK + r * 512, take ? kc + r * 512 : p.kc, take);
        cp_async_or_zero<16>(st + dst + G::kV + r * 512, take ? vc + r * 512 : p.vc, take);
      }
      const bool take = lane < left;
      cp_async_or_zero<G::kSRow>(st + dst_s + G::kKS, take ? p.ks + os : p.ks, take);
      cp_async_or_zero<G::kSRow>(st + dst_s + G::kVS, take ? p.vs + os : p.vs, take);
    }
  }
};

// One (sequence, head).
struct Unit {
  int b, kvh, P;
  // the lane's row x of row tile nt (opaque, so that what depends on it is
  // computed where it is used and not held over the key loop)
  __device__ __forceinline__ int row(int nt, int x) const {
    int r = nt * 8 + 2 * (int)(threadIdx.x & 3) + x;
    asm volatile("" : "+r"(r));
    return r;
  }
  __device__ __forceinline__ uint64_t mask(const RowsParams& p, int nt, int x) const {
    const int r = row(nt, x);
    return r < p.R ? p.mask_bits[(int64_t)b * p.N + r / (p.Hq / p.Hkv)] : 0ull;
  }
  __device__ __forceinline__ int64_t out_row(const RowsParams& p, int r) const {
    const int Gq = p.Hq / p.Hkv;
    return ((int64_t)b * p.N + r / Gq) * p.Hq + kvh * Gq + r % Gq;
  }
};
// A lane's references, sums (over its own keys) and outputs of a unit's rows.  m
// tile j, rows g and g + 8 of the product are dims D/8 g + 2 j and + 2 j + 1, so the
// lane holds D/8 contiguous dims of its rows: row x in o[j][nt][x] and o[j][nt][2 + x].
template <int D, int NT>
struct Acc {
  float m[NT][2], l[NT][2], o[D / 16][NT][4];
};

// One warp over keys key0, key0 + step, ... (32 each) below kend.
template <int D, int NT>
__device__ __forceinline__ void run_blocks(const RowsParams& p, RowsSmem<D, NT>& sm,
                                           const Unit& t, int key0, int step, int kend,
                                           Acc<D, NT>& a) {
  using G = Stage<D>;
  constexpr int kStages = RowsCfg<NT>::kStages;
  constexpr int kSteps = D / 16;      // k steps of S
  constexpr int kMT = D / 16;         // m tiles of O^T
  constexpr int kW = D / 32;          // code words a lane loads per key of K
  constexpr bool kQReg = !RowsCfg<NT>::kQShared;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int b = t.b, kvh = t.kvh, P = t.P, L = P + p.N;
  const int Gq = p.Hq / p.Hkv;
  const uint32_t ring = smem_u32(sm.ring) + (uint32_t)(warp * kStages * G::kBytes);
  const unsigned char* ringp = sm.ring + warp * kStages * G::kBytes;
  unsigned long long* vnan = sm.vnan[warp];
  const LaneFill<D> fill(((int64_t)b * p.Hkv + kvh) * p.S, lane);
  __syncwarp();  // the tile before is done with the ring
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    const int k = key0 + i * step;
    if (k < kend) fill.issue(p, ring + (uint32_t)(i * G::kBytes), k, L, lane);
    cp_async_commit();
  }
  if (lane < D / kKv4Block) vnan[lane] = 0ull;

  // q rows -> fp16 fragments, each scaled by a power of two: operand
  // registers b0, b1 of k step s are dims 4 s .. 4 s + 3 of quarter c of row g
  float f[NT][2];  // of this lane's rows 8 nt + 2 c + x
  uint2 qr[kSteps][NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    int r = nt * 8 + g;
    asm volatile("" : "+r"(r));  // as in Unit::row
    const bool valid = r < p.R;
    const int node = valid ? r / Gq : 0;
    const int hq = kvh * Gq + (valid ? r % Gq : 0);
    const uint2* src = reinterpret_cast<const uint2*>(
        p.q + (((int64_t)b * p.N + node) * p.Hq + hq) * D + c * (D / 4));
    uint2 w[kSteps];
    float mx = 0.f;
#pragma unroll
    for (int x = 0; x < kSteps; ++x) {
      w[x] = valid ? src[x] : make_uint2(0, 0);
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(bf16_lo(w[x].x)), fabsf(bf16_hi(w[x].x))),
                           fmaxf(fabsf(bf16_lo(w[x].y)), fabsf(bf16_hi(w[x].y)))));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    int e = (int)(__float_as_uint(mx) >> 23) - 127;
    if (mx == 0.f || e == 128) e = 0;  // a zero row; an infinite one stays as it is
    e = max(-126, min(126, e));
    const float dn = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int x = 0; x < kSteps; ++x) {
      const uint2 h = make_uint2(pack_half2(bf16_lo(w[x].x) * dn, bf16_hi(w[x].x) * dn),
                                 pack_half2(bf16_lo(w[x].y) * dn, bf16_hi(w[x].y) * dn));
      if constexpr (kQReg)
        qr[x][nt] = h;
      else
        sm.qf[warp][x][nt][lane] = h;  // read back by this lane alone
    }
    const float fg = row_factor(p.scale, e);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      f[nt][x] = __shfl_sync(0xffffffffu, fg, 4 * (2 * c + x));
      a.m[nt][x] = neg_inf();
      a.l[nt][x] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < kMT; ++j)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) a.o[j][nt][0] = a.o[j][nt][1] = a.o[j][nt][2] = a.o[j][nt][3] = 0.f;
  // what the lane's rows may see of the drafted keys (up to 16 rows: read
  // early, off the path of the last blocks)
  uint64_t masks[NT][2];
  if constexpr (NT <= 2) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      masks[nt][0] = kend > P ? t.mask(p, nt, 0) : 0ull;
      masks[nt][1] = kend > P ? t.mask(p, nt, 1) : 0ull;
    }
  }
  auto row_mask = [&](int nt, int x) -> uint64_t {
    if constexpr (NT <= 2)
      return masks[nt][x];
    else
      return t.mask(p, nt, x);
  };

  int slot = 0;  // stage that holds key0's block
  for (; key0 < kend; key0 += step) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    {
      const int k = key0 + (kStages - 1) * step;
      const int to = slot == 0 ? kStages - 1 : slot - 1;
      if (k < kend) fill.issue(p, ring + (uint32_t)(to * G::kBytes), k, L, lane);
      cp_async_commit();
    }
    const unsigned char* st = ringp + slot * G::kBytes;
    slot = slot == kStages - 1 ? 0 : slot + 1;
    const bool tail = key0 + kKeys > P;

    // ---------------------------------------------------- S^T = K Q^T
    // accumulators [16-key tile][row tile]: keys g, g, g + 8, g + 8 x rows
    // 2 c, 2 c + 1
    float s[2][NT][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t kw[2][kW], ksc[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = 16 * u + 8 * t + 4 * (g & 1) + (g >> 1);
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
        uint32_t h[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          e2m1x8_to_half2(kw[t][w], h[t]);
          const uint32_t sc = (D == 128 && w >= 2) ? dup_hi(ksc[t]) : dup_lo(ksc[t]);
#pragma unroll
          for (int x = 0; x < 4; ++x) h[t][x] = hmul2(h[t][x], sc);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 q = kQReg ? qr[2 * w + x][nt] : sm.qf[warp][2 * w + x][nt][lane];
            if (w == 0 && x == 0)
              mma16816_f16_first(s[u][nt], h[0][0], h[1][0], h[0][1], h[1][1], q.x, q.y);
            else
              mma16816_f16(s[u][nt], h[0][2 * x], h[1][2 * x], h[0][2 * x + 1], h[1][2 * x + 1],
                           q.x, q.y);
          }
      }
    }
    // ------------------------------------------ running softmax, base 2
    if (tail) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint64_t mb = row_mask(nt, x);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int d = key0 + 16 * u + 8 * t + 4 * (g & 1) + (g >> 1) - P;
              const bool vis = d < 0 || (d < p.N && ((mb >> (d & 63)) & 1ull));
              if (!vis) s[u][nt][2 * t + x] = neg_inf();
            }
        }
    }
    float bm[NT][2];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        bm[nt][x] = fmaxf(fmax3f(s[0][nt][x], s[0][nt][2 + x], s[1][nt][x]), s[1][nt][2 + x]) *
                    f[nt][x];
        grow |= bm[nt][x] > a.m[nt][x] + 8.f;
      }
    // the reference moves only when a row's maximum grows by more than 2^8
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = fmaxf(bm[nt][x], __shfl_xor_sync(0xffffffffu, bm[nt][x], 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          const bool move = v > a.m[nt][x] + 8.f;
          const float mn = move ? v : a.m[nt][x];
          const float corr = move ? ex2(a.m[nt][x] - mn) : 1.f;  // 0 at the first visible key
          a.m[nt][x] = mn;
          a.l[nt][x] *= corr;
#pragma unroll
          for (int j = 0; j < kMT; ++j) {
            a.o[j][nt][x] *= corr;
            a.o[j][nt][2 + x] *= corr;
          }
        }
    }
    uint32_t pb[2][NT][2];  // P^T as operand: [16 keys][row tile][b0, b1]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float n0 = a.m[nt][0] == neg_inf() ? kLift : kLift - a.m[nt][0];
      const float n1 = a.m[nt][1] == neg_inf() ? kLift : kLift - a.m[nt][1];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = ex2(fmaf(s[u][nt][2 * t], f[nt][0], n0));
          const float p1 = ex2(fmaf(s[u][nt][2 * t + 1], f[nt][1], n1));
          a.l[nt][0] += p0;
          a.l[nt][1] += p1;
          pb[u][nt][t] = transpose8x8(pack_half2(p0, p1));
        }
    }
    // -------------------------------------------------- O^T += V^T P^T
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
            atomicOr(&vnan[D == 128 ? g : (g >> 1)], 1ull << d);
            sb[x] = 0;
          }
        }
      }
      const uint32_t s01 = e4m3x2_to_half2(sb[0] | (sb[1] << 8));
      const uint32_t s23 = e4m3x2_to_half2(sb[2] | (sb[3] << 8));
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        constexpr uint32_t kLo = 0x0f0f0f0fu, kHi = 0xf0f0f0f0u;
        uint32_t a0[4], a1[4], a2[4], a3[4];  // even / odd dims x keys 0, 1 / 2, 3
        e2m1x8_to_half2((vw[0][w] & kLo) | ((vw[1][w] << 4) & kHi), a0);
        e2m1x8_to_half2(((vw[0][w] >> 4) & kLo) | (vw[1][w] & kHi), a1);
        e2m1x8_to_half2((vw[2][w] & kLo) | ((vw[3][w] << 4) & kHi), a2);
        e2m1x8_to_half2(((vw[2][w] >> 4) & kLo) | (vw[3][w] & kHi), a3);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t y0 = hmul2(a0[x], s01), y1 = hmul2(a1[x], s01);
          const uint32_t y2 = hmul2(a2[x], s23), y3 = hmul2(a3[x], s23);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816_f16(a.o[4 * w + x][nt], y0, y1, y2, y3, pb[u][nt][0], pb[u][nt][1]);
        }
      }
    }
  }

  cp_async_wait<0>();
  __syncwarp();  // every lane's notes of NaN blocks
  // the sums over the eight lanes that share a row
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float v = a.l[nt][x];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      a.l[nt][x] = v + __shfl_xor_sync(0xffffffffu, v, 16);
    }
  const unsigned long long nan_keys = vnan[D == 128 ? g : (g >> 1)];
  if (nan_keys != 0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (nan_keys & row_mask(nt, x)) {
#pragma unroll
          for (int j = 0; j < kMT; ++j)
            a.o[j][nt][x] = a.o[j][nt][2 + x] = __int_as_float(0x7fffffff);
        }
  }
}

// Many or long sequences: pieces of the line, one per warp.
template <int D, int NT>
__global__ void __launch_bounds__(RowsCfg<NT>::kThreads, RowsCfg<NT>::kCtas)
    kv4_rows(const RowsParams p) {
  using Sm = RowsSmem<D, NT>;
  constexpr int kThreads = RowsCfg<NT>::kThreads;
  constexpr int kMT = D / 16;
  extern __shared__ __align__(16) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
  launch_dependents();

  const LineBlocks line = {p};
  scan_line<kThreads>(p.B, line, sm.before, sm.tmp);
  const int64_t total = sm.before[kThreads];
  const int64_t piece = piece_blocks(total, p.warps);
  const int wid = blockIdx.x * RowsCfg<NT>::kWarps + warp;
  int64_t at = (int64_t)wid * piece;
  const int64_t end = min(total, at + piece);
  if (at >= total) return;
  int64_t seq_start;
  int b = locate<kThreads>(p.B, line, sm.before, at, &seq_start);
  bool first = true;  // the segment starts where the piece does

  while (at < end) {
    const int P = clamped_prefix(p, b);
    const int nblk = (P + p.N + kKeys - 1) / kKeys;
    const int kvh = (int)((at - seq_start) / nblk);
    const int64_t unit_start = seq_start + (int64_t)kvh * nblk;
    const int k0 = (int)(at - unit_start);
    const int k1 = (int)min((int64_t)nblk, end - unit_start);
    const Unit t = {b, kvh, P};
    Acc<D, NT> a;
    run_blocks<D, NT>(p, sm, t, k0 * kKeys, kKeys, k1 * kKeys, a);

    const bool whole = k0 == 0 && k1 == nblk;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = t.row(nt, x);
        if (r >= p.R) continue;
        const float sum = a.l[nt][x];
        if (whole) {
          const int64_t orow = t.out_row(p, r);
          const float inv = sum == 0.f ? 0.f : p.v_unit / sum;
          uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + (D / 8) * g);
#pragma unroll
          for (int j = 0; j < kMT; j += 4)
            dst[j / 4] =
                make_uint4(pack_bf16x2(a.o[j][nt][x] * inv, a.o[j][nt][2 + x] * inv),
                           pack_bf16x2(a.o[j + 1][nt][x] * inv, a.o[j + 1][nt][2 + x] * inv),
                           pack_bf16x2(a.o[j + 2][nt][x] * inv, a.o[j + 2][nt][2 + x] * inv),
                           pack_bf16x2(a.o[j + 3][nt][x] * inv, a.o[j + 3][nt][2 + x] * inv));
          if (p.lse && g == 0)
            p.lse[orow] = sum == 0.f ? neg_inf() : a.m[nt][x] + log2f(sum) - kLift;
        } else {
          const int64_t prow = ((int64_t)2 * wid + (first ? 0 : 1)) * p.R + r;
          float4* dst = reinterpret_cast<float4*>(p.part + prow * D + (D / 8) * g);
#pragma unroll
          for (int j = 0; j < kMT; j += 2)
            dst[j / 2] = make_float4(a.o[j][nt][x], a.o[j][nt][2 + x], a.o[j + 1][nt][x],
                                     a.o[j + 1][nt][2 + x]);
          if (g == 0) p.part_ml[prow] = make_float2(a.m[nt][x], sum);
        }
      }
    at = unit_start + k1;
    first = false;
    if (kvh + 1 == p.Hkv && k1 == nblk) {  // the next block belongs to the next sequence
      seq_start += (int64_t)p.Hkv * nblk;
      ++b;
    }
  }
}

// Few or short sequences: one cluster of CTAs per unit (p.warps = its size),
// one launch, no workspace.  The warps' parts are joined in shared memory, then
// the CTAs' over the cluster.
template <int D, int NT>
__global__ void __launch_bounds__(RowsCfg<NT>::kThreads, RowsCfg<NT>::kCtas)
    kv4_unit(const RowsParams p) {
  using Sm = RowsSmem<D, NT>;
  using Cfg = RowsCfg<NT>;
  constexpr int RT = 8 * NT, kWarps = Cfg::kWarps, kThreads = Cfg::kThreads, kMT = D / 16;
  constexpr int kMerge = kWarps * RT * D * 4;  // the warps' outputs
  constexpr int kOwn = kMerge + kWarps * RT * 8;  // their m, l; then this CTA's output, m, l
  static_assert(kOwn + RT * (D * 4 + 8) <= (int)offsetof(Sm, vnan), "joined in the ring (and qf)");
  extern __shared__ __align__(16) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int C = p.warps;
  const int rank = blockIdx.x % C;
  const int unit = blockIdx.x / C;
  Unit t;
  t.kvh = unit % p.Hkv;
  t.b = unit / p.Hkv;
  t.P = clamped_prefix(p, t.b);
  const int nblk = (t.P + p.N + kKeys - 1) / kKeys;
  // blocks rank * kWarps + warp, + C * kWarps, ...
  Acc<D, NT> a;
  run_blocks<D, NT>(p, sm, t, (rank * kWarps + warp) * kKeys, C * kWarps * kKeys, nblk * kKeys, a);

  __syncthreads();  // every warp is done with its ring
  float* mbuf = reinterpret_cast<float*>(sm.ring);
  float2* ml = reinterpret_cast<float2*>(sm.ring + kMerge);  // [warp][row]
  float* own = reinterpret_cast<float*>(sm.ring + kOwn);     // [row][D]
  float2* own_ml = reinterpret_cast<float2*>(own + RT * D);
  const int rows = p.R;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = nt * 8 + 2 * c + x;
      if (row >= rows) continue;
      if (g == 0) ml[warp * RT + row] = make_float2(a.m[nt][x], a.l[nt][x]);
      // 16-byte chunks XOR c spread the stores over the banks
      float4* dst = reinterpret_cast<float4*>(mbuf + (warp * RT + row) * D);
#pragma unroll
      for (int j = 0; j < kMT; j += 2)
        dst[((D / 32) * g + j / 2) ^ c] = make_float4(
            a.o[j][nt][x], a.o[j][nt][2 + x], a.o[j + 1][nt][x], a.o[j + 1][nt][2 + x]);
    }
  __syncthreads();
  auto emit = [&](int row, int chunk, const float4& v, float M, float sum) {
    const int64_t orow = t.out_row(p, row);
    const float inv = sum == 0.f ? 0.f : p.v_unit / sum;
    *reinterpret_cast<uint2*>(p.out + orow * D + 4 * chunk) =
        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    if (p.lse && chunk == 0) p.lse[orow] = sum == 0.f ? neg_inf() : M + log2f(sum) - kLift;
  };
  for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
    const int row = e / (D / 4), pc = e % (D / 4);
    const int chunk = pc ^ ((row >> 1) & 3);
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
      const float4 v = *reinterpret_cast<const float4*>(mbuf + (w * RT + row) * D + 4 * pc);
      acc.x = fmaf(v.x, k, acc.x);
      acc.y = fmaf(v.y, k, acc.y);
      acc.z = fmaf(v.z, k, acc.z);
      acc.w = fmaf(v.w, k, acc.w);
      sum = fmaf(pw.y, k, sum);
    }
    if (C == 1) {
      emit(row, chunk, acc, M, sum);
    } else {
      *reinterpret_cast<float4*>(own + row * D + 4 * chunk) = acc;
      if (chunk == 0) own_ml[row] = make_float2(M, sum);
    }
  }
  if (C == 1) return;
  cluster_sync();
  for (int e = threadIdx.x * C + rank; e < rows * (D / 4); e += kThreads * C) {
    const int row = e / (D / 4), chunk = e % (D / 4);
    const uint32_t ao = smem_u32(own + row * D + 4 * chunk), am = smem_u32(own_ml + row);
    float M = neg_inf(), sum = 0.f;
    for (int i = 0; i < C; ++i) M = fmaxf(M, ld_dsmem_f32(mapa(am, i)));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < C; ++i) {
      const float2 pw = ld_dsmem_v2(mapa(am, i));
      const float4 v = ld_dsmem_v4(mapa(ao, i));
      const float k = pw.x == neg_inf() ? 1.f : ex2(pw.x - M);
      acc.x = fmaf(v.x, k, acc.x);
      acc.y = fmaf(v.y, k, acc.y);
      acc.z = fmaf(v.z, k, acc.z);
      acc.w = fmaf(v.w, k, acc.w);
      sum = fmaf(pw.y, k, sum);
    }
    emit(row, chunk, acc, M, sum);
  }
  cluster_sync();  // no CTA leaves while another reads its parts
}

// Joins the parts of a unit that several warps worked on: a CTA takes `per_cta`
// rows of a unit, kJoinWarps / per_cta warps a row.  The units are all of
// them, or, when there are more units than piece borders, those that hold a
// border, each found from the first border inside it.  The loads it has in flight
// take registers: left alone the compiler keeps 64 of them (8 sequences of 32 K
// keys, 32 rows: 149 us for 141).
template <int D, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinWarps == 8 ? 2 : 1)
    kv4_combine(const RowsParams p, bool by_border, int per_cta) {
  constexpr int kThreads = kJoinWarps * 32;
  __shared__ int64_t before[kThreads + 1], tmp[kJoinWarps];
  __shared__ float acc_s[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const LineBlocks line = {p};
  scan_line<kThreads>(p.B, line, before, tmp);
  grid_dependency_wait();  // before any exit: this grid must not end first
  const int64_t total = before[kThreads];
  const int64_t piece = piece_blocks(total, p.warps);
  Unit t;
  int nblk;
  int64_t t0;  // the unit's first block
  if (by_border) {
    const int64_t pos = (int64_t)(blockIdx.x + 1) * piece;
    if (pos >= total) return;
    int64_t start;
    t.b = locate<kThreads>(p.B, line, before, pos, &start);
    nblk = seq_blocks(p, t.b);
    t.kvh = (int)((pos - start) / nblk);
    t0 = start + (int64_t)t.kvh * nblk;
    if (t0 == pos || t0 < pos - piece) return;  // not inside, or not the first one inside
  } else {
    t.b = (int)(blockIdx.x / p.Hkv);
    t.kvh = (int)(blockIdx.x % p.Hkv);
    nblk = seq_blocks(p, t.b);
    const int per = (p.B + kThreads - 1) / kThreads;
    t0 = before[t.b / per] + (int64_t)t.kvh * nblk;
    for (int i = t.b / per * per; i < t.b; ++i) t0 += line(i);
  }
  const int c0 = (int)(t0 / piece), c1 = (int)((t0 + nblk - 1) / piece);
  if (c0 == c1) return;
  const int n = c1 - c0 + 1;
  const int lead = t0 == (int64_t)c0 * piece ? 0 : 1;
  const int wpr = max(1, kJoinWarps / per_cta);  // more than one: one row per warp group
  const int last = min((int)(blockIdx.y + 1) * per_cta, p.R);
  const int sub = warp % wpr;
  constexpr int kV = D / 32;  // floats per lane
  for (int row = blockIdx.y * per_cta + warp / wpr; row < last || wpr > 1;
       row += kJoinWarps / wpr) {
    auto part = [&](int i) -> int64_t {
      return ((int64_t)2 * (c0 + i) + (i == 0 ? lead : 0)) * p.R + row;
    };
    float M = neg_inf(), sum = 0.f;  // every warp for itself
    float acc[kV] = {};
    if (row < last) {
      float ls[kJoinUnroll], xs[kJoinUnroll];
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u) {  // the first parts' loads in flight together
        const int i = lane + 32 * u;
        const float2 ml = i < n ? p.part_ml[part(i)] : make_float2(neg_inf(), 0.f);
        xs[u] = ml.x;
        ls[u] = ml.y;
        M = fmaxf(M, ml.x);
      }
      for (int i = lane + 32 * kJoinUnroll; i < n; i += 32) M = fmaxf(M, p.part_ml[part(i)].x);
      M = warp_max(M);
      // a part whose reference never moved holds zeros, or NaN scores
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u)
        sum += ls[u] * (xs[u] == neg_inf() ? 1.f : ex2(xs[u] - M));
      for (int i = lane + 32 * kJoinUnroll; i < n; i += 32) {
        const float2 ml = p.part_ml[part(i)];
        sum += ml.y * (ml.x == neg_inf() ? 1.f : ex2(ml.x - M));
      }
      sum = warp_sum(sum);
#pragma unroll 8
      for (int i = sub; i < n; i += wpr) {
        const int64_t pr = part(i);
        const float x = p.part_ml[pr].x;
        const float k = x == neg_inf() ? 1.f : ex2(x - M);
        const float* src = p.part + pr * D + lane * kV;
        if constexpr (kV == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          acc[0] = fmaf(v.x, k, acc[0]);
          acc[1] = fmaf(v.y, k, acc[1]);
          acc[2] = fmaf(v.z, k, acc[2]);
          acc[3] = fmaf(v.w, k, acc[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          acc[0] = fmaf(v.x, k, acc[0]);
          acc[1] = fmaf(v.y, k, acc[1]);
        }
      }
    }
    if (wpr > 1) {
#pragma unroll
      for (int i = 0; i < kV; ++i) acc_s[warp][lane * kV + i] = acc[i];
      __syncthreads();
      if (sub == 0)
        for (int w = 1; w < wpr; ++w)
#pragma unroll
          for (int i = 0; i < kV; ++i) acc[i] += acc_s[warp + w][lane * kV + i];
    }
    if (sub == 0 && row < last) {
      const int64_t orow = t.out_row(p, row);
      const float inv = sum == 0.f ? 0.f : p.v_unit / sum;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D + lane * kV);
#pragma unroll
      for (int i = 0; i < kV; i += 2) dst[i / 2] = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
      if (p.lse && lane == 0) p.lse[orow] = sum == 0.f ? neg_inf() : M + log2f(sum) - kLift;
    }
    if (wpr > 1) break;
  }
}

// Pieces (warps) a call uses: no more than its blocks could fill.
template <int NT>
int rows_warps(int B, int Hkv, int S) {
  const int64_t blocks = (int64_t)B * Hkv * ((S + kKeys - 1) / kKeys);
  const int64_t want = (blocks + kMinBlocks - 1) / kMinBlocks;
  return (int)(want < RowsCfg<NT>::kPieces ? want : RowsCfg<NT>::kPieces);
}
// CTAs per cluster of kv4_unit, or 0 for pieces of the line, by the cache's
// capacity S (the host does not know the lengths).  Units leave
// some of the resident CTAs idle, or the last wave part empty, for as many
// 32-key blocks a warp as the longest unit may have; pieces cost the join's
// launch and partial outputs.  Measured (32 / 8 heads, D 128): units 6.4 us,
// pieces 15.9 us at one sequence of 1 K keys, 9.6 / 17.0 at 8 K, 22.2 / 21.6
// at 32 K, 75.8 / 40.6 at 128 K; 32 sequences of up to 4 K 31.7 / 34.3, 64 of
// them 57.4 / 55.5 (where the rule stays with units), 64 of 32 K 438 / 381.  One
// sequence of 1 K keys in a cache of 32 K or 128 K positions: pieces, 15.7 us.
template <int NT>
int unit_cluster(int64_t units, int S) {
  constexpr int64_t slots = kSms * RowsCfg<NT>::kCtas;
  constexpr double kIdleBlocks = 8;
  int C = 1;
  while (C < 8 && units * C * 2 <= slots) C *= 2;
  const int64_t waves = (units * C + slots - 1) / slots;
  const double idle = 1.0 - (double)(units * C) / (double)(waves * slots);
  const double blocks = (double)S / kKeys / (C * RowsCfg<NT>::kWarps);
  return idle * blocks * waves > kIdleBlocks ? 0 : C;
}

// Bytes of the pieces' partial results: 0 when clusters do without.
template <int NT>
size_t part_bytes(int B, int Hkv, int R, int D, int S) {
  if (unit_cluster<NT>((int64_t)B * Hkv, S) > 0) return 0;
  return (size_t)2 * rows_warps<NT>(B, Hkv, S) * R * (D + 2) * sizeof(float);
}
size_t attn_ws(int B, int Hkv, int R, int D, int S) {
  if (R > kRowsMax) return kv4_tc_ws(B, Hkv, R, D, S);
  if (R <= 8) return part_bytes<1>(B, Hkv, R, D, S);
  if (R <= 16) return part_bytes<2>(B, Hkv, R, D, S);
  if (R <= 24) return part_bytes<3>(B, Hkv, R, D, S);
  return part_bytes<4>(B, Hkv, R, D, S);
}

template <int D, int NT>
cudaError_t launch_rows(const Kv4Attn& a, void* ws, cudaStream_t st) {
  RowsParams p = {};
  (Kv4Attn&)p = a;
  using Cfg = RowsCfg<NT>;
  constexpr int smem = (int)sizeof(RowsSmem<D, NT>);
  static_assert((smem + 1024) * Cfg::kCtas <= 228 * 1024, "the pieces are resident at once");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem((const void*)kv4_rows<D, NT>, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int64_t units = (int64_t)p.B * p.Hkv;
  const int cluster = unit_cluster<NT>(units, p.S);
  if (cluster > 0) {
    static std::atomic<uint64_t> done_unit{0};
    e = allow_smem((const void*)kv4_unit<D, NT>, smem, done_unit);
    if (e != cudaSuccess) return e;
    p.warps = cluster;
    cfg.gridDim = dim3((unsigned)(units * cluster));
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = smem;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    prof_begin(SPEC_PROF_ATTN, st);
    e = cudaLaunchKernelEx(&cfg, kv4_unit<D, NT>, p);
    prof_end(SPEC_PROF_ATTN, st);
    return e;
  }
  p.warps = rows_warps<NT>(p.B, p.Hkv, p.S);
  p.part = (float*)ws;
  p.part_ml = (float2*)(p.part + (size_t)2 * p.warps * p.R * D);
  prof_begin(SPEC_PROF_ATTN, st);
  kv4_rows<D, NT><<<(p.warps + Cfg::kWarps - 1) / Cfg::kWarps, Cfg::kThreads, smem, st>>>(p);
  prof_end(SPEC_PROF_ATTN, st);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.warps == 1) return e;
  const bool by_border = units > p.warps - 1;
  const int64_t joins = by_border ? p.warps - 1 : units;
  const int per_cta = joins * p.R <= 2 * kSms ? 1 : p.R;
  // a row of a long unit has many parts: sixteen warps read them; elsewhere
  // eight warps share the rows (one sequence of 128 K keys 43 -> 41 us, 64 of
  // 32 K 381 us against 390 with sixteen)
  cfg.gridDim = dim3((unsigned)joins, (unsigned)((p.R + per_cta - 1) / per_cta));
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  if (per_cta == 1) {
    cfg.blockDim = dim3(16 * 32);
    return cudaLaunchKernelEx(&cfg, kv4_combine<D, 16>, p, by_border, per_cta);
  }
  cfg.blockDim = dim3(8 * 32);
  return cudaLaunchKernelEx(&cfg, kv4_combine<D, 8>, p, by_border, per_cta);
}

}  // namespace
}  // namespace sv

using namespace sv;

// More than kRowsMax query rows per key/value head go to the tensor-core kernel
// (kv4_attn_tc.cu).  Measured (D 128): 32 sequences of 2 to 4 K keys, 16 rows
// 48 us here and 73 there, 20 rows 58 / 73, 32 rows 75 / 72 us; one of 1 K keys,
// 32 rows 15 / 14 us; 8 sequences of 32 K keys, 32 rows 141 / 165 us, for which
// 32 rows stay here.
extern "C" size_t spec_tree_attention_kv4_workspace_bytes(int B, int N, int Hq, int Hkv, int D,
                                                          int S) {
  if (B < 0 || B > 65535 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || S < N ||
      S > SPEC_MAX_POSITIONS || (D != 64 && D != 128))
    return 0;
  const int64_t R = (int64_t)N * (Hq / Hkv);
  if (B == 0 || R > (1 << 30) || (int64_t)B * Hkv * ((R + 15) / 16) > 2147483647) return 0;
  return (attn_ws(B, Hkv, (int)R, D, S) + 255) / 256 * 256;
}

extern "C" int spec_tree_attention_kv4(const void* q, const uint8_t* k_codes,
                                       const uint8_t* k_scales, const uint8_t* v_codes,
                                       const uint8_t* v_scales, const int32_t* prefix_len,
                                       const uint64_t* mask_bits, int B, int N, int Hq, int Hkv,
                                       int D, int S, float scale, float k_unit, float v_unit,
                                       void* out, float* lse, void* workspace, size_t ws_bytes,
                                       void* stream) {
  if (B < 0 || B > 65535 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || S < N ||
      S > SPEC_MAX_POSITIONS)
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
  if (R > (1 << 30) || (int64_t)B * Hkv * tiles > 2147483647 || (double)B * Hkv * S > 4.0e15)
    return SPEC_ERR_SHAPE;
  const size_t need = attn_ws(B, Hkv, (int)R, D, S);
  if (need > 0 && (!workspace || (uintptr_t)workspace % 256 != 0 || ws_bytes < need))
    return SPEC_ERR_WORKSPACE;
  Kv4Attn p = {};
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
  p.scale = score_scale(scale, k_unit);
  p.v_unit = v_unit;
  p.out = (uint16_t*)out;
  p.lse = lse;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (R > kRowsMax)
    e = launch_kv4_tc(p, D, workspace, st);
  else if (D == 128)
    e = R <= 8 ? launch_rows<128, 1>(p, workspace, st)
               : (R <= 16 ? launch_rows<128, 2>(p, workspace, st)
                          : (R <= 24 ? launch_rows<128, 3>(p, workspace, st)
                                     : launch_rows<128, 4>(p, workspace, st)));
  else
    e = R <= 8 ? launch_rows<64, 1>(p, workspace, st)
               : (R <= 16 ? launch_rows<64, 2>(p, workspace, st)
                          : (R <= 24 ? launch_rows<64, 3>(p, workspace, st)
                                     : launch_rows<64, 4>(p, workspace, st)));
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
