// spec_tree_attention_kv4 for many query rows per key/value head: the
// fifth-generation tensor cores.
//
// The mathematics and the numbers are kv4_attn.cu's (cache values exact in
// fp16, rows of q scaled by powers of two, weights lifted by 2^7 and rounded
// to fp16, everything else float32).  A CTA takes up to 256 query rows of one
// (sequence, key/value head) as two 128-row tiles, or up to 128 as one, and
// 64-key blocks of the cache, or a share of them (splits, when there are
// fewer units than SMs):
//   dequantisers (4 warps): the codes of the next blocks on their way from HBM
//     in registers while block j's become fp16 rows in a ring of swizzled
//     shared-memory stages (K and V as stored: a 64-dim row per 128 bytes);
//   S issuers (two threads), P V issuers (one thread per tile): S = Q K^T with
//     Q read from TMEM, O += P V with P from shared memory;
//   softmax (8 warps, a thread per row): a running base-2 softmax against a
//     reference maximum that moves only when a row's maximum grows by more
//     than 2^8 (then O is rescaled in TMEM); two P buffers per tile.
// With two tiles each has four softmax warps and one S buffer.  With one, two
// groups of four warps take its blocks in turn, each with an S buffer of its
// own, so that one group exponentiates while the other's scores are made; the
// rows' references pass between the groups block by block.
// Bound: the softmax warps and the single S buffer of a tile.  32 sequences of 2
// to 4 K keys, 240 rows (60 nodes, 4 heads a group), D 128: 108 us = 913 TFLOP/s,
// 1.2 TB/s; per 64-key block of a tile about 1930 cycles, of which the products
// take 1250 of the tensor pipe for both tiles.  One tile: 64 rows 73 us, 128 rows
// 73 us (as half of a two-tile CTA 87 and 79 us).
// TMEM (512 columns): Q_t at columns 64 t, S buffers at 128 and 192, O_t at 256
// + 128 t.  Every mbarrier wait is bounded; a CTA that gives up stops waiting,
// still frees its TMEM after waiting, bounded, for its own products, and returns
// NaN rows and normalisers (there is no status word).
#include "kernels.h"
#include "kv4.cuh"
#include "kv4_attn.h"
#include "tc.cuh"

namespace sv {
namespace {

constexpr int kKB = 64;         // keys per block
constexpr int kMT = 128;        // query rows per tile
constexpr int kTcStages = 4;    // even: with one tile an S issuer takes every other block and must
                                // meet every phase of its stages
static_assert(kTcStages % 2 == 0, "see above");
constexpr int kPTile = kMT * kKB * 2;
constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kDeqWarp = kSoftWarps;     // 4 warps
constexpr int kCtlWarp = kSoftWarps + 4; // 4 warps
constexpr int kTcThreads = (kSoftWarps + 8) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kOrderMax = 256;
constexpr float kLift = 7.f;

struct TcParams {
  Kv4Attn a;
  int gx, splits;   // row CTAs per (sequence, head); shares of its blocks
  float* part;      // [unit][split][CTA's rows][D], when splits > 1
  float2* part_ml;  // [unit][split][CTA's rows]
};

template <int kTiles>
struct __align__(8) TcSmem {
  uint64_t kvfull[kTcStages], kvempty[kTcStages];
  uint64_t sfull[2], sfree[2];         // per S buffer
  uint64_t pfull[2][2], pdone[2][2];   // per tile and P buffer
  uint64_t turn[4][2];                 // one tile: per quadrant and group
  uint64_t qready, drain[2][2];
  unsigned long long vnan[8];
  static constexpr int kShared = kTiles == 1 ? kMT : 1;  // rows whose state groups share
  float mref[kShared], rowf[kShared], lsum[2][kShared];
  uint32_t tmem_base;
  uint32_t dead;
  int seq;
};

template <int D, int kTiles>
struct TcCfg {
  static constexpr int kNG = 2 / kTiles;            // softmax groups per tile
  static constexpr int kRowsCta = kTiles * kMT;
  static constexpr int kHalf = kKB * 64 * 2;        // 64 keys x 64 dims
  static constexpr int kKVTile = kKB * D * 2;
  static constexpr int kStage = 2 * kKVTile;
  static constexpr int kOffP = kTcStages * kStage;
  static constexpr int kOffBar = kOffP + kTiles * 2 * kPTile;
  static constexpr int kSmem = kOffBar + (int)sizeof(TcSmem<kTiles>) + 1024;
  // with the 1 KB the system keeps, within the 196 KB step of the L1 split:
  // the next step leaves the loads 28 KB of L1 (two tiles: 117 us for 107)
  static_assert(kSmem + 1024 <= 196 * 1024, "the L1 split");
  // blocks that a dequantiser thread has in registers
  static constexpr int kAhead = kTiles == 1 ? 4 : 3;
  // f16 operands, float32 D; S: M 128, N 64, both K-major; P V: N D, B MN-major
  static constexpr uint32_t kIdescS =
      (1u << 4) | ((uint32_t)(kKB >> 3) << 17) | ((uint32_t)(kMT >> 4) << 24);
  static constexpr uint32_t kIdescPV =
      (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kMT >> 4) << 24);
};

template <class Sm>
__device__ __forceinline__ void await(Sm& sm, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  if (*(volatile uint32_t*)&sm.dead) return;
  if (!mbar_wait_bounded(bar, parity)) *(volatile uint32_t*)&sm.dead = 1;
}

// Loads that stay where they are written (ahead of the waits they overlap).
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld4(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld2(const uint8_t* p) {
  unsigned short v;
  asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

// One thread's part of a block on its way from HBM: D/2 head dims of one key.
template <int D>
struct Raw {
  uint4 k[D / 64], v[D / 64];
  uint32_t ks, vs;
};

template <int D, int kTiles>
__global__ void __launch_bounds__(kTcThreads, 1) kv4_tc(const TcParams prm) {
  using Cfg = TcCfg<D, kTiles>;
  constexpr int kNG = Cfg::kNG, kRowsCta = Cfg::kRowsCta, kAhead = Cfg::kAhead;
  const Kv4Attn& p = prm.a;
  extern __shared__ __align__(1024) unsigned char araw[];
  const uint32_t raw = smem_u32(araw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* bp = araw + (base - raw);
  using Sm = TcSmem<kTiles>;
  Sm& sm = *reinterpret_cast<Sm*>(bp + Cfg::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, R = p.R, S = p.S, N = p.N;
  const int per_seq = prm.gx * prm.splits * p.Hkv;  // CTAs per sequence
  int b = blockIdx.x / per_seq;
  const int rem = blockIdx.x % per_seq;
  launch_dependents();
  if (p.B > 1 && p.B <= kOrderMax) {
    // longest sequences first, ties by index: the grid's tail is short
    int* len_s = reinterpret_cast<int*>(bp + Cfg::kOffP);
    for (int i = threadIdx.x; i < p.B; i += kTcThreads) {
      const int x = p.prefix_len[i];
      len_s[i] = x < 0 ? 0 : (x > S - N ? S - N : x);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.B; i += kTcThreads) {
      const int li = len_s[i];
      int rank = 0;
      for (int j = 0; j < p.B; ++j) {
        const int lj = len_s[j];
        rank += (lj > li || (lj == li && j < i)) ? 1 : 0;
      }
      if (rank == b) sm.seq = i;
    }
    __syncthreads();
    b = sm.seq;
  }
  const int kvh = rem / (prm.gx * prm.splits);
  const int tile = rem / prm.splits % prm.gx, split = rem % prm.splits;
  const int row0 = tile * kRowsCta;
  const int ntile = min(kTiles, (R - row0 + kMT - 1) / kMT);
  int P = p.prefix_len[b];
  P = P < 0 ? 0 : (P > S - N ? S - N : P);
  const int L = P + N;
  const int nall = (L + kKB - 1) / kKB;
  const int share = (nall + prm.splits - 1) / prm.splits;
  const int j0 = min(nall, split * share);
  const int n = min(nall, j0 + share) - j0;  // this CTA's blocks: j0 .. j0 + n - 1

  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcStages; ++s) {
      mbar_init(&sm.kvfull[s], 128);
      mbar_init(&sm.kvempty[s], ntile);  // released by every tile's issuer
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.sfull[t], 1);
      mbar_init(&sm.sfree[t], kMT);
      for (int w = 0; w < 4; ++w) mbar_init(&sm.turn[w][t], 32);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.pfull[t][i], kMT);
        mbar_init(&sm.pdone[t][i], 1);
        mbar_init(&sm.drain[t][i], 1);
      }
    }
    mbar_init(&sm.qready, kTiles * kMT);
    for (int i = 0; i < 8; ++i) sm.vnan[i] = 0ull;
    sm.dead = 0;
    fence_mbar_init();
  }
  if (warp == kCtlWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp >= kCtlWarp) {
    const int t = (warp - kCtlWarp) & 1;
    if (lane == 0) {
      if (warp < kCtlWarp + 2) {
        // ------------------------------------------------------ S issuers
        // Two tiles: tile t's S of every block.  One: blocks t, t + 2, ...
        // (buffer t).  k counts the buffer's uses.
        if (kNG == 2 || t < ntile) {
          await(sm, &sm.qready, 0);
          fence_after();
          const uint32_t tq = tmem + (uint32_t)(kNG == 2 ? 0 : 64 * t);
          const uint32_t ds = tmem + 128u + (uint32_t)(64 * t);
          const uint64_t dk0 = desc_kmajor(base);
          int k = 0;
          for (int j = kNG == 2 ? t : 0; j < n; j += kNG, ++k) {
            const int s = j % kTcStages;
            await(sm, &sm.kvfull[s], (uint32_t)(j / kTcStages) & 1u);
            if (k >= 1) await(sm, &sm.sfree[t], (uint32_t)((k - 1) & 1));
            fence_after();
            const uint64_t dk = dk0 + (uint64_t)((s * Cfg::kStage) >> 4);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t koff = (uint32_t)((i >> 2) * Cfg::kHalf + (i & 3) * 32);
              mma_f16_ts(ds, tq + (uint32_t)(8 * i), dk + (koff >> 4), Cfg::kIdescS,
                         i > 0 ? 1u : 0u);
            }
            mma_commit(&sm.sfull[t]);
          }
          mma_commit(&sm.drain[t][0]);
          mbar_wait_bounded(&sm.drain[t][0], 0);
        }
      } else if (t < ntile) {
        // -------------------------------------------- tile t's P V issuer
        const uint64_t dv0 = desc_mnmajor(base + Cfg::kKVTile, Cfg::kHalf);
        const uint64_t dp0 = desc_kmajor(base + Cfg::kOffP + (uint32_t)(2 * t * kPTile));
        const uint32_t to = tmem + 256u + (uint32_t)(128 * t);
        for (int j = 0; j < n; ++j) {
          const int s = j % kTcStages;
          await(sm, &sm.pfull[t][j & 1], (uint32_t)((j >> 1) & 1));
          fence_after();
          const uint64_t dp = dp0 + (uint64_t)(((j & 1) * kPTile) >> 4);
          const uint64_t dv = dv0 + (uint64_t)((s * Cfg::kStage) >> 4);
#pragma unroll
          for (int k = 0; k < kKB / 16; ++k)
            mma_f16(to, dp + (uint64_t)(k * 2), dv + (uint64_t)(k * 128), Cfg::kIdescPV,
                    (j > 0 || k > 0) ? 1u : 0u);
          mma_commit(&sm.pdone[t][j & 1]);
          // done with the block's K too: S completed before the softmax wrote P
          mma_commit(&sm.kvempty[s]);
        }
        mma_commit(&sm.drain[t][1]);
        mbar_wait_bounded(&sm.drain[t][1], 0);
      }
    }
  } else if (warp >= kDeqWarp) {
    // ------------------------------------------------------ dequantisers
    const int d = threadIdx.x - kDeqWarp * 32;
    const int key = d & 63, part = d >> 6;
    constexpr int kWords = D / 16;  // code words per thread and operand
    const int64_t row = ((int64_t)b * p.Hkv + kvh) * S + (int64_t)j0 * kKB + key;
    const uint8_t* kc = p.kc + row * (D / 2) + part * (D / 4);
    const uint8_t* vc = p.vc + row * (D / 2) + part * (D / 4);
    const uint8_t* ks = p.ks + row * (D / 16) + part * (D / 32);
    const uint8_t* vs = p.vs + row * (D / 16) + part * (D / 32);
    auto load = [&](Raw<D>& r, int j) {
      const bool have = j < n && (j0 + j) * kKB + key < L;
      const int64_t o = (int64_t)j * kKB;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        r.k[i] = have ? ld16(kc + o * (D / 2) + 16 * i)
                      : make_uint4(0, 0, 0, 0);
        r.v[i] = have ? ld16(vc + o * (D / 2) + 16 * i)
                      : make_uint4(0, 0, 0, 0);
      }
      if constexpr (D == 128) {
        r.ks = have ? ld4(ks + o * 8) : 0u;
        r.vs = have ? ld4(vs + o * 8) : 0u;
      } else {
        r.ks = have ? ld2(ks + o * 4) : 0u;
        r.vs = have ? ld2(vs + o * 4) : 0u;
      }
    };
    // this thread's 16-byte chunks within a tile (D 128: the whole row of
    // half `part`; D 64: chunks 4 part ..)
    unsigned char* dst0 = bp + (D == 128 ? part * Cfg::kHalf : 0);
    auto store = [&](unsigned char* tile_p, const uint4 (&w)[D / 64], uint32_t sc) {
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {  // one scale, 16 dims
        const uint32_t two = e4m3x2_to_half2(sc >> (i & ~1) * 8);
        const uint32_t s2 = (i & 1) ? dup_hi(two) : dup_lo(two);
        const uint4& q = w[i / 2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t h[4];
          e2m1x8_to_half2((i & 1) ? (x ? q.w : q.z) : (x ? q.y : q.x), h);
          const int ch = (D == 128 ? 0 : 4 * part) + 2 * i + x;
          *reinterpret_cast<uint4*>(tile_p + swz(key, ch)) =
              make_uint4(hmul2(h[0], s2), hmul2(h[1], s2), hmul2(h[2], s2), hmul2(h[3], s2));
        }
      }
    };
    auto put = [&](Raw<D>& r, int j) {
      const int s = j % kTcStages;
      const int dk = (j0 + j) * kKB + key - P;  // drafted node of this key
      if (dk >= 0 && dk < N) {
        // a NaN block of a drafted value must reach the rows that see it and
        // no others: it is noted and its scale replaced by zero
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          if (((r.vs >> (8 * i)) & 0x7fu) == 0x7fu) {
            atomicOr(&sm.vnan[part * (D / 32) + i], 1ull << dk);
            r.vs &= ~(0xffu << (8 * i));
          }
      }
      await(sm, &sm.kvempty[s], ((uint32_t)(j / kTcStages) & 1u) ^ 1u);
      store(dst0 + s * Cfg::kStage, r.k, r.ks);
      store(dst0 + s * Cfg::kStage + Cfg::kKVTile, r.v, r.vs);
      fence_async_smem();
      mbar_arrive(&sm.kvfull[s]);
    };
    // kAhead blocks on their way: HBM's latency is longer than a block's time
    Raw<D> r[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(r[i], i);
    for (int j = 0; j < n; j += kAhead)
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (j + i < n) put(r[i], j + i);
        load(r[i], j + i + kAhead);
      }
    __syncwarp();
    asm volatile("bar.arrive 3, %0;" ::"n"(kSoftThreads + 128) : "memory");
  } else {
    // ------------------------------------------------------------ softmax
    const int t = kTiles == 2 ? warp >> 2 : 0;   // tile
    const int grp = kTiles == 2 ? 0 : warp >> 2;  // takes blocks grp, grp + kNG, ...
    const int sb = kTiles == 2 ? t : grp;        // S buffer
    const int qd = warp & 3;                  // TMEM lane quadrant of this warp
    const int r = qd * 32 + lane;
    const int gr = row0 + t * kMT + r;
    const bool valid = t < ntile && gr < R;
    const int node = valid ? gr / G : 0;
    const int hq = kvh * G + (valid ? gr % G : 0);
    const uint64_t mb = valid ? (p.mask_bits[(int64_t)b * N + node] &
                                 (N >= 64 ? ~0ull : ((1ull << N) - 1ull)))
                              : 0ull;
    const int64_t orow = ((int64_t)b * N + node) * p.Hq + hq;
    const uint32_t lanes = (uint32_t)(qd * 32) << 16;
    float f = 0.f;  // scores to base-2 exponents
    if (grp == 0) {  // this row of q as fp16 into Q_t's TMEM lane
      const uint4* src = reinterpret_cast<const uint4*>(p.q + orow * D);
      uint32_t w[D / 2];
      uint32_t top = 0;  // largest magnitude: bf16 magnitudes order like their bits
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = valid ? src[i] : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t y = w[4 * i + x] & 0x7fff7fffu;
          // a NaN does not count (the row is NaN whatever its scale)
          top = max(top, (y & 0xffffu) > 0x7f80u ? 0u : (y & 0xffffu));
          top = max(top, (y >> 16) > 0x7f80u ? 0u : (y >> 16));
        }
      }
      int e = (int)(top >> 7) - 127;
      if (top == 0u || e == 128) e = 0;  // a zero row; an infinite one stays as it is
      e = max(-126, min(126, e));
      const float dn = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < D / 2; ++i) w[i] = pack_half2(bf16_lo(w[i]) * dn, bf16_hi(w[i]) * dn);
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = w[32 * h + i];
        tst32(tmem + lanes + (uint32_t)(64 * t + 32 * h), x);
      }
      tst_wait();
      fence_before();
      f = row_factor(p.scale, e);
      if (kNG == 2) {
        sm.rowf[r] = f;
        sm.mref[r] = neg_inf();
      }
      mbar_arrive(&sm.qready);
    }
    if constexpr (kNG == 2) {
      named_sync(1, kMT * kNG);
      f = sm.rowf[r];
    }
    float m = neg_inf(), l = 0.f;  // the reference that this thread's sum is against
    if (t < ntile) {
      const uint32_t tS = tmem + lanes + 128u + (uint32_t)(64 * sb);
      const uint32_t tO = tmem + lanes + 256u + (uint32_t)(128 * t);
      unsigned char* pt0 = bp + Cfg::kOffP + 2 * t * kPTile;
      for (int j = grp; j < n; j += kNG) {
        await(sm, &sm.sfull[sb], (uint32_t)((j / kNG) & 1));
        __syncwarp();
        fence_after();
        float s[64];
        {
          uint32_t ra[32], rb[32];
          tld32(tS, ra);
          tld32(tS + 32u, rb);
          tld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = __uint_as_float(ra[i]);
            s[32 + i] = __uint_as_float(rb[i]);
          }
        }
        fence_before();
        mbar_arrive(&sm.sfree[sb]);  // the S issuer may write the buffer's next block
        const int key0 = (j0 + j) * kKB;
        if (!valid || key0 + kKB > P) {
          const int npre = min(max(P - key0, 0), 64);
          const uint64_t pre = npre >= 64 ? ~0ull : ((1ull << npre) - 1ull);
          const int off = key0 - P;
          const uint64_t dr = off >= 0 ? (off < 64 ? (mb >> off) : 0ull)
                                       : (off > -64 ? (mb << (-off)) : 0ull);
          const uint64_t vis = valid ? (pre | dr) : 0ull;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (!((vis >> i) & 1ull)) s[i] = neg_inf();
        }
        float bm4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) bm4[c] = fmax3f(s[c], s[c + 4], s[c + 8]);
#pragma unroll
        for (int i = 12; i < 60; i += 8)
#pragma unroll
          for (int c = 0; c < 4; ++c) bm4[c] = fmax3f(bm4[c], s[i + c], s[i + 4 + c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) bm4[c] = fmaxf(bm4[c], s[60 + c]);
        const float bm = fmaxf(fmax3f(bm4[0], bm4[1], bm4[2]), bm4[3]) * f;
        float now = m;  // the row's reference after the block before
        if constexpr (kNG == 2) {
          if (j >= 1) {
            await(sm, &sm.turn[qd][grp], (uint32_t)((grp ? (j >> 1) : (j >> 1) - 1) & 1));
            now = *(volatile float*)&sm.mref[r];
          }
        }
        const bool move = bm > now + 8.f;
        const float mnew = move ? bm : now;
        const float corr = (move && now != neg_inf()) ? ex2(now - mnew) : 1.f;
        if constexpr (kNG == 2) {
          if (move) *(volatile float*)&sm.mref[r] = mnew;
          if (j + 1 < n) mbar_arrive(&sm.turn[qd][grp ^ 1]);
          if (mnew != m) l *= ex2(m - mnew);  // m = -inf: l is 0
        } else {
          l *= corr;
        }
        m = mnew;
        const float nm = m == neg_inf() ? kLift : kLift - m;
        uint32_t pk[32];
        const float2 sc2 = make_float2(f, f), nm2 = make_float2(nm, nm);
        float2 ls4[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 e = ffma2(make_float2(s[2 * i], s[2 * i + 1]), sc2, nm2);
          const float p0 = ex2(e.x), p1 = ex2(e.y);
          ls4[i & 1] = fadd2(ls4[i & 1], make_float2(p0, p1));
          pk[i] = pack_half2(p0, p1);
        }
        const float2 lsa = fadd2(ls4[0], ls4[1]);
        l += lsa.x + lsa.y;
        // P buffer j & 1 was read by the P V of block j - 2; a rescale of O_t
        // needs the P V of block j - 1 done too (products complete in order, so
        // after the first wait the second one's parity names block j - 1)
        const bool resc = j > 0 && __any_sync(0xffffffffu, corr != 1.f);
        if (j >= 2) await(sm, &sm.pdone[t][j & 1], (uint32_t)(((j - 2) >> 1) & 1));
        if (resc) await(sm, &sm.pdone[t][(j - 1) & 1], (uint32_t)(((j - 1) >> 1) & 1));
        fence_after();
        if (resc) {
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tld16(tO + (uint32_t)(16 * c), o);
            tld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
            tst16(tO + (uint32_t)(16 * c), o);
          }
          tst_wait();
        }
        unsigned char* pt = pt0 + (j & 1) * kPTile;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(pt + swz(r, c)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_async_smem();
        fence_before();
        mbar_arrive(&sm.pfull[t][j & 1]);
      }
      // O_t / l after the last P V
      await(sm, &sm.drain[t][1], 0);
      fence_after();
    }
    named_sync(3, kSoftThreads + 128);  // every note of a NaN block, every row's last reference
    if (t < ntile) {
      const uint32_t tO = tmem + lanes + 256u + (uint32_t)(128 * t);
      if constexpr (kNG == 2) {
        const float last = *(volatile float*)&sm.mref[r];
        if (last != m) l *= ex2(m - last);
        m = last;
        sm.lsum[grp][r] = l;
        named_sync(1, kMT * kNG);
        l = sm.lsum[0][r] + sm.lsum[1][r];
      }
      // whoever gave up wrote `dead` before the arrival that led here
      bool gave_up = *(volatile uint32_t*)&sm.dead != 0;
#ifdef SV_TEST_GAVE_UP  // a test's build: CTA 0 as if one of its waits had
      gave_up |= blockIdx.x == 0;
#endif
      if (gave_up) l = __int_as_float(0x7fffffff);
      float inv = 1.f;
      float* part = nullptr;
      if (prm.splits == 1) {
        inv = l == 0.f ? 0.f : p.v_unit / l;
        if (valid && p.lse && grp == 0) p.lse[orow] = l == 0.f ? neg_inf() : m + log2f(l) - kLift;
      } else {
        const int64_t unit = ((int64_t)b * p.Hkv + kvh) * prm.gx + tile;
        const int64_t prow = (unit * prm.splits + split) * kRowsCta + t * kMT + r;
        part = prm.part + prow * D;
        if (valid && grp == 0) prm.part_ml[prow] = make_float2(m, l);
      }
      // each group writes its share of the row
#pragma unroll 1
      for (int c = grp * (D / 16 / kNG); c < (grp + 1) * (D / 16 / kNG); ++c) {
        uint32_t o[16];
        __syncwarp();
        if (n > 0) {
          tld16(tO + (uint32_t)(16 * c), o);
          tld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0u;
        }
        if (valid) {
          if (sm.vnan[c] & mb) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = 0x7fffffffu;
          }
          if (part) {
            uint4* dst = reinterpret_cast<uint4*>(part + 16 * c);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              dst[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          } else {
            // a row that saw nothing: no product ever touched it but with zeros
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + 16 * c);
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              y[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
            dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
            dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kCtlWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// Joins the splits: one warp per query row.
template <int D>
__global__ void __launch_bounds__(256) kv4_tc_combine(const TcParams prm, int kRowsCta) {
  const Kv4Attn& p = prm.a;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = blockIdx.x;
  const int tile = (int)(unit % prm.gx);
  const int kvh = (int)(unit / prm.gx % p.Hkv), b = (int)(unit / prm.gx / p.Hkv);
  const int r = blockIdx.y * 8 + warp, gr = tile * kRowsCta + r;
  if (gr >= p.R) return;
  const int64_t prow = unit * prm.splits * kRowsCta + r;
  const float2 ml =
      lane < prm.splits ? prm.part_ml[prow + (int64_t)lane * kRowsCta] : make_float2(neg_inf(), 0.f);
  const float M = warp_max(ml.x);
  // a part that saw nothing (its reference never moved) holds zeros, or NaN
  const float k = ml.x == neg_inf() ? 1.f : ex2(ml.x - M);
  const float sum = warp_sum(ml.y * k);
  constexpr int kV = D / 32;
  float acc[kV] = {};
  for (int i = 0; i < prm.splits; ++i) {
    const float ki = __shfl_sync(0xffffffffu, k, i);
    const float* src = prm.part + (prow + (int64_t)i * kRowsCta) * D + lane * kV;
#pragma unroll
    for (int x = 0; x < kV; ++x) acc[x] = fmaf(src[x], ki, acc[x]);
  }
  const int G = p.Hq / p.Hkv;
  const int64_t orow = ((int64_t)b * p.N + gr / G) * p.Hq + kvh * G + gr % G;
  const float inv = sum == 0.f ? 0.f : p.v_unit / sum;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D + lane * kV);
#pragma unroll
  for (int x = 0; x < kV; x += 2) dst[x / 2] = pack_bf16x2(acc[x] * inv, acc[x + 1] * inv);
  if (p.lse && lane == 0) p.lse[orow] = sum == 0.f ? neg_inf() : M + log2f(sum) - kLift;
}

// Shares of a unit's blocks: the number that fills the SMs best, counted in
// blocks of a unit as long as the cache's capacity S (a CTA's start costs about
// three, the join's launch and traffic about eight; the host does not know the
// lengths).  Measured with this rule and unsplit: 240 rows, one sequence of 128 K
// keys 127 us / 1896 us, of 1 K keys 25.3 / 25.2; five ragged ones of up to 5 K
// keys, 2 heads, D 64 19.1 / 77.4.  Capacity far above the lengths costs empty
// shares: 32 sequences of 2 to 4 K keys, 240 rows, 108 us at S 4160 (unsplit), 352 us
// and 341 MB of partial results at S 131137 (ten shares).
int tc_splits(int64_t units, int S) {
  const int64_t blocks = (S + kKB - 1) / kKB;
  int best = 1;
  int64_t cost = 0;
  for (int s = 1; s <= 32 && s <= blocks; ++s) {
    const int64_t waves = (units * s + 151) / 152;
    const int64_t c = waves * ((blocks + s - 1) / s + 3) + (s > 1 ? 8 : 0);
    if (s == 1 || c < cost) {
      best = s;
      cost = c;
    }
  }
  return best;
}

template <int D, int kTiles>
cudaError_t launch_tc(const Kv4Attn& a, void* ws, cudaStream_t st) {
  using Cfg = TcCfg<D, kTiles>;
  constexpr int kRowsCta = Cfg::kRowsCta;
  TcParams prm;
  prm.a = a;
  prm.gx = (a.R + kRowsCta - 1) / kRowsCta;
  const int64_t units = (int64_t)a.B * a.Hkv * prm.gx;
  prm.splits = tc_splits(units, a.S);
  prm.part = (float*)ws;
  prm.part_ml = (float2*)(prm.part + (size_t)units * prm.splits * kRowsCta * D);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem((const void*)kv4_tc<D, kTiles>, Cfg::kSmem, done);
  if (e != cudaSuccess) return e;
  prof_begin(SPEC_PROF_ATTN, st);
  kv4_tc<D, kTiles><<<(unsigned)(units * prm.splits), kTcThreads, Cfg::kSmem, st>>>(prm);
  prof_end(SPEC_PROF_ATTN, st);
  e = cudaGetLastError();
  if (e != cudaSuccess || prm.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units, (unsigned)(((a.R < kRowsCta ? a.R : kRowsCta) + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_tc_combine<D>, prm, kRowsCta);
}

}  // namespace

size_t kv4_tc_ws(int B, int Hkv, int R, int D, int S) {
  const int rows = R <= kMT ? kMT : 2 * kMT;
  const int64_t units = (int64_t)B * Hkv * ((R + rows - 1) / rows);
  const int splits = tc_splits(units, S);
  return splits == 1 ? 0 : (size_t)units * splits * rows * (D + 2) * sizeof(float);
}

cudaError_t launch_kv4_tc(const Kv4Attn& a, int D, void* ws, cudaStream_t st) {
  if (a.R <= kMT) return D == 128 ? launch_tc<128, 1>(a, ws, st) : launch_tc<64, 1>(a, ws, st);
  return D == 128 ? launch_tc<128, 2>(a, ws, st) : launch_tc<64, 2>(a, ws, st);
}

}  // namespace sv
