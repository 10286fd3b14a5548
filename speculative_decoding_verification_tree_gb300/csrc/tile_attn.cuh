// Attention of tiles of query rows on the fifth-generation tensor cores: the
// kernel behind spec_prompt_attention and spec_tree_attention_shared.
//
// A unit of work is up to 256 query rows of one key/value head -- (token, head in
// the group) pairs, token-major, so that the G query heads that share a key/value
// head are served by one stream of its keys and values -- as two tiles of 128 rows,
// with floor(128 / G) tokens each.  Its keys come in 128-key steps.  Which units and
// steps a CTA takes is a Walk (the two callers differ only there, in the visibility
// of a key and in what happens to a finished row); every warp follows its own copy.
//
//   warp 0      producer: K and V of each step (TMA, 128-byte swizzle) into rings of
//               tiles, Q of each unit as a box of tokens x G heads;
//   warps 1-2   tile t's issuer of S_t = Q_t K^T and O_t += P_t V (tcgen05.mma M 128,
//               float32 in TMEM); the whole warp runs its loop and one elected lane issues
//               (8192 tokens, 32 / 8 heads, D 128, one issuer for both tiles: 537 us when a
//               lone thread runs it, whose operands the compiler cannot know to be
//               uniform, 456 this way);
//   warp 3      every V tile on its way to the products: rows behind the last key
//               become zeros, and in steps that some row does not see in full so do
//               NaN and infinite elements (0 times them would reach rows that do not
//               see them; rows that do see them get them back at the end, times their
//               weight in as far as that is 0 or not);
//   warps 4-11  softmax, a thread per row: S from TMEM, online base-2 softmax against
//               a reference maximum that moves only when a row's maximum grows by
//               more than 2^8 (O is then rescaled in TMEM), P as bf16 pairs into the
//               TMEM columns of S; at a unit's end O / l.
//
// A step's scores come in two halves of 64 keys, each with its own columns and its own
// P: while the softmax works on one half, P V of the other and the next scores of the
// other run.  With whole steps a tile's products and softmax take turns: 418 us for the
// 8192 tokens above instead of 380, although the 64-key products read Q from shared
// memory twice as often.  Also tried there: two softmax threads per row (16 warps, maxima
// exchanged through shared memory: 484 us); four warps of their own for finished rows (no
// gain at any length: registers for the softmax get scarce); registers moved from the
// other warps to the softmax's (no gain: it needs 138).
//
// TMEM (512 columns): S_t's halves at 128 t and 128 t + 64, P_t over the first 32 columns
// of each, O_t at 256 + 128 t.  One issuer per tile keeps the order that this needs:
// S of a half is issued after P V of the same half of the step before, which reads P from
// the same columns, and its commit covers that P V.  A softmax warp that rescales O_t waits
// for the P V of the half before as well.
// Sums, statistics and O are float32.  P is rounded to bf16 for the product, whose
// operands have one type, V's: each weight is off by at most 2^-8 of itself, the row's
// sum is of the unrounded ones.  Outputs are rounded to bf16 once, at the end.  (Against
// 64 bits they differ by 2.2e-3 of their norm, 1.6e-3 of it that last rounding alone.)
// Scores times the scale in base 2 are taken to lie below 2^29 in size: there an FMA
// against the rounded reference is off by up to 2^5 at the row's maximum, which the sums
// bear; float32 tells such scores apart by 32.
//
// Every mbarrier wait is bounded; a CTA that gives up stops waiting, still frees its
// TMEM after waiting, bounded, for its own products and copies, and returns NaN rows
// and normalisers (there is no status word).
#pragma once

#include <cfloat>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tensor_map.h"

namespace sv {
namespace {

constexpr int kRows = 128;       // query rows per tile
constexpr int kKeys = 128;       // keys per step
constexpr int kHalfKeys = kKeys / 2;  // keys of a half step
constexpr int kTaThreads = 384;
constexpr int kTaCtas = 152;     // one per SM
constexpr uint32_t kTaTmemCols = 512;

// kKs and kVs: ring stages of K and of V tiles
template <int D, int kKs, int kVs>
struct TileGeo {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = kKeys * 128;       // 64 dims of 128 rows
  static constexpr int kTile = kHalves * kHalf;   // Q, K or V of 128 rows
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffCtl = kOffRing + (kKs + kVs) * kTile;
  static constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) |
                                      ((uint32_t)(kHalfKeys >> 3) << 17) |
                                      ((uint32_t)(kRows >> 4) << 24);
  // B (V as stored) is MN-major
  static constexpr uint32_t kIdescPV = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                       ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
};

template <int kKs, int kVs>
struct __align__(8) TileCtl {
  uint64_t full[kKs + kVs], empty[kKs + kVs];  // K stages, then V stages
  uint64_t clean[kVs];
  uint64_t qfull[2], qempty[2], sfull[2][2], pfull[2][2], pvdone[2], ofull[2], drain;
  uint32_t tmem_base;
  uint32_t dead;  // a wait gave up
  uint32_t bad;   // a NaN or infinite element of V was taken out
};

template <class Ctl>
__device__ __forceinline__ void await(Ctl& sm, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  if (*(volatile uint32_t*)&sm.dead) return;
  if (!mbar_wait_bounded(bar, parity)) *(volatile uint32_t*)&sm.dead = 1;
}

__device__ __forceinline__ void tma3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                      uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// Rows of 64 bytes, a lane each, written so that four lanes write one row at a time:
// place[i] is the row of lane 4 (lane / 4) + i (its 64 bytes; null: not written).  A
// store then covers 8 rows instead of 16 bytes of each of 32.
__device__ __forceinline__ uint4 pick(bool second, const uint4& a, const uint4& b) {
  return make_uint4(second ? b.x : a.x, second ? b.y : a.y, second ? b.z : a.z,
                    second ? b.w : a.w);
}
__device__ __forceinline__ uint4 swap_lanes(const uint4& v, int mask) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, mask), __shfl_xor_sync(0xffffffffu, v.y, mask),
                    __shfl_xor_sync(0xffffffffu, v.z, mask), __shfl_xor_sync(0xffffffffu, v.w, mask));
}
__device__ __forceinline__ void store_rows(uint4* const (&place)[4], uint4 (&v)[4]) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {  // 2 x 2 blocks across neighbours
    const uint4 got = swap_lanes(pick(odd, v[i + 1], v[i]), 1);
    v[i] = pick(odd, v[i], got);
    v[i + 1] = pick(odd, got, v[i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {     // and across pairs
    const uint4 got = swap_lanes(pick(high, v[i + 2], v[i]), 2);
    v[i] = pick(high, v[i], got);
    v[i + 2] = pick(high, got, v[i + 2]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (place[i]) place[i][lane & 3] = v[i];
}
__device__ __forceinline__ void share_rows(uint4* mine, uint4* (&place)[4]) {
  const uint64_t p = reinterpret_cast<uint64_t>(mine);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    place[i] = reinterpret_cast<uint4*>(__shfl_sync(0xffffffffu, p, (threadIdx.x & 28) + i));
}
// 32 values scaled, as 64 bytes of bf16
__device__ __forceinline__ void pack_row(const float (&o)[32], float mul, uint4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = make_uint4(pack_bf16x2(o[8 * i] * mul, o[8 * i + 1] * mul),
                      pack_bf16x2(o[8 * i + 2] * mul, o[8 * i + 3] * mul),
                      pack_bf16x2(o[8 * i + 4] * mul, o[8 * i + 5] * mul),
                      pack_bf16x2(o[8 * i + 6] * mul, o[8 * i + 7] * mul));
}
// True in one lane of a warp that is whole here.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}
// bit 15 / 31 set where a bf16 half is NaN or infinite
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
// acc + 0 w, bf16 pairs
__device__ __forceinline__ uint32_t times_zero(uint32_t w, uint32_t acc) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(acc));
  return d;
}
// bit 15 / 31 set where a bf16 half is infinite
__device__ __forceinline__ uint32_t infinite2(uint32_t w) {
  const uint32_t x = (w & 0x7fff7fffu) ^ 0x7f807f80u;  // 0: infinite
  return ~((x + 0x7fff7fffu) | x) & 0x80008000u;
}
// Whether a key's weight in a row is 0 (D dims of both, bf16; statistics of the row).
// (One word at a time: this is rare, and the softmax needs the registers.)
template <int D>
__device__ __forceinline__ bool weightless(const uint16_t* q, const uint16_t* k, float scale_log2,
                                           float mref) {
  float s = 0.f;
#pragma unroll 1
  for (int i = 0; i < D; i += 2) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(q + i);
    const uint32_t y = *reinterpret_cast<const uint32_t*>(k + i);
    s = fmaf(bf16_lo(x), bf16_lo(y), s);
    s = fmaf(bf16_hi(x), bf16_hi(y), s);
  }
  return ex2(fmaf(s, scale_log2, mref == neg_inf() ? 0.f : -mref)) == 0.f;
}
// NaN and infinite halves as 0
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  return w & ~((not_finite2(w) >> 15) * 0xffffu);
}

// The Walk of a caller W offers, to whole warps:
//   static setup(prm, shared, scratch), prefetch_maps(prm)   once, before the roles part
//   bool next_unit(), bool next_step(), restart() (the unit's steps from the start)
//   have   tiles of the unit (bits);  act   tiles that take part in the step
//   full   no row of the unit lacks a key of the step
//   load_q / load_k / load_v  the producer's copies
//   keys   keys of the step that exist (the rest of the 128 is not in the sequence)
// and, per softmax thread, a Row (set_row at a unit's start):
//   bool warp_blind(row)          no row of this warp sees anything of the step
//   void hide(row, half, s)       scores of keys 64 half + i that it does not see: -inf
//   bool sees(row, i), const uint16_t *value(i), *key(i)   key i of the step
//   const uint16_t* query(row)    the row's query
//   void finish(...)              what becomes of the row
template <int D, int kKs, int kVs, class W>
__global__ void __launch_bounds__(kTaThreads, 1)
    tile_attn(const __grid_constant__ typename W::Params prm) {
  using Geo = TileGeo<D, kKs, kVs>;
  using Ctl = TileCtl<kKs, kVs>;
  extern __shared__ __align__(1024) unsigned char bp[];  // the swizzle wants 1024 bytes
  const uint32_t base = smem_u32(bp);
  Ctl& sm = *reinterpret_cast<Ctl*>(bp + Geo::kOffCtl);
  typename W::Shared& ws = *reinterpret_cast<typename W::Shared*>(bp + Geo::kOffCtl + sizeof(Ctl));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKs + kVs; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 2);  // given back by both issuers
    }
    for (int s = 0; s < kVs; ++s) mbar_init(&sm.clean[s], 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.qfull[t], 1);
      mbar_init(&sm.qempty[t], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sm.sfull[t][h], 1);
        mbar_init(&sm.pfull[t][h], kRows);
      }
      mbar_init(&sm.pvdone[t], 1);
      mbar_init(&sm.ofull[t], 2);
    }
    mbar_init(&sm.drain, 2);
    sm.dead = sm.bad = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(kTaTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == kTaThreads - 1) W::prefetch_maps(prm);
  W::setup(prm, ws, bp);  // every thread; may use the tiles' space; ends with a barrier
  fence_async_smem();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp < 4) {
    W w(prm, ws);
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      uint32_t n = 0, upar = 0;  // steps; parity of each Q tile's next wait
      uint32_t nk = 0, nv = 0, nq[2] = {0, 0};  // copies begun
      // whether stage s may be filled (once a wait has given up, nothing is copied any
      // more: copies without waits would pile up on a barrier)
      auto slot = [&](int s, uint32_t fill) {
        await(sm, &sm.empty[s], (fill & 1u) ^ 1u);
        if (*(volatile uint32_t*)&sm.dead) return false;
        mbar_expect_tx(&sm.full[s], (uint32_t)Geo::kTile);
        return true;
      };
      while (w.next_unit()) {
        bool first = true;
        while (w.next_step()) {
          if (lane == 0) {
            const int s = (int)(n % kKs);
            if (slot(s, n / kKs)) {
              const uint32_t dst = base + Geo::kOffRing + (uint32_t)(s * Geo::kTile);
#pragma unroll
              for (int h = 0; h < Geo::kHalves; ++h)
                w.load_k(dst + h * Geo::kHalf, 64 * h, &sm.full[s]);
              ++nk;
            }
          }
          if (first) {  // (after the first keys: they need no wait for the unit before)
            first = false;
            if (lane == 0) {
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                if (!((w.have >> t) & 1u)) continue;
                await(sm, &sm.qempty[t], ((upar >> t) & 1u) ^ 1u);
                if (*(volatile uint32_t*)&sm.dead) continue;
                mbar_expect_tx(&sm.qfull[t], w.q_bytes() * Geo::kHalves);
#pragma unroll
                for (int h = 0; h < Geo::kHalves; ++h)
                  w.load_q(t, base + (uint32_t)(t * Geo::kTile + h * Geo::kHalf), 64 * h,
                           &sm.qfull[t]);
                ++nq[t];
              }
            }
            upar ^= w.have;
          }
          if (lane == 0) {
            const int s = (int)(n % kVs);
            if (slot(kKs + s, n / kVs)) {
              const uint32_t dst = base + Geo::kOffRing + (uint32_t)((kKs + s) * Geo::kTile);
#pragma unroll
              for (int h = 0; h < Geo::kHalves; ++h)
                w.load_v(dst + h * Geo::kHalf, 64 * h, &sm.full[kKs + s]);
              ++nv;
            }
          }
          ++n;
          __syncwarp();
        }
      }
      // this CTA's last copy into each stage and each Q tile has landed before it exits
      // (also where an issuer no longer waits for it)
      if (lane == 0) {
        for (uint32_t s = 0; s < (uint32_t)kKs && s < nk; ++s)
          mbar_wait_bounded(&sm.full[s], ((nk - s - 1) / kKs) & 1u);
        for (uint32_t s = 0; s < (uint32_t)kVs && s < nv; ++s)
          mbar_wait_bounded(&sm.full[kKs + s], ((nv - s - 1) / kVs) & 1u);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (nq[t] > 0) mbar_wait_bounded(&sm.qfull[t], (nq[t] - 1) & 1u);
      }
    } else if (warp <= 2) {
      // ------------------------------------------------- tile t's issuer
      // (the whole warp runs this and one elected lane issues: the operands of an
      // issue are then uniform over the warp)
      const int t = warp - 1;
      const uint64_t dring = desc_kmajor(base + Geo::kOffRing);
      const uint64_t dq = desc_kmajor(base + (uint32_t)(t * Geo::kTile));
      const uint64_t dvring = desc_mnmajor(base + Geo::kOffRing + kKs * Geo::kTile, Geo::kHalf);
      const uint32_t tS = tmem + 128u * t, tO = tmem + 256u + 128u * t;
      uint32_t n = 0, qpar = 0, ppar = 0;
      bool pend = false, acc = false, ends = false;
      // O += P V over one half of the keys of the step before
      auto put_pv = [&](int h) {
        await(sm, &sm.pfull[t][h], ppar);
        fence_after();
        const uint64_t dv = dvring + (uint64_t)(((n - 1) % kVs) * Geo::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kHalfKeys / 16; ++k)
            mma_f16_ts(tO, tS + (uint32_t)(64 * h + 8 * k), dv + (uint64_t)((4 * h + k) * 128),
                       Geo::kIdescPV, h > 0 || k > 0 || acc ? 1u : 0u);
          mma_commit(&sm.pvdone[t]);
        }
        __syncwarp();
      };
      // S of one half of the keys of this step
      auto put_s = [&](int h) {
        fence_after();
        const uint64_t dk = dring + (uint64_t)((n % kKs) * Geo::kTile >> 4) +
                            (uint64_t)(h * kHalfKeys * 128 >> 4);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint64_t off = (uint64_t)((i >> 2) * Geo::kHalf + (i & 3) * 32) >> 4;
            mma_f16(tS + 64u * h, dq + off, dk + off, Geo::kIdescS, i > 0 ? 1u : 0u);
          }
          mma_commit(&sm.sfull[t][h]);
        }
        __syncwarp();
      };
      // the V tile of the step before, given back, and a unit that ended with it.  (An
      // issuer whose tile takes no part waits for the tiles all the same: it must not
      // give the next fill of a stage back in place of this one.)
      auto give_v = [&]() {
        if (elect_one()) {
          if (n > 0) mma_commit(&sm.empty[kKs + (n - 1) % kVs]);
          if (ends) {  // every product of the tile's unit is issued
            mma_commit(&sm.ofull[t]);
            // (a plain arrival too: it hands on what this warp saw of the V tiles)
            mbar_arrive(&sm.ofull[t]);
          }
        }
        __syncwarp();
      };
      while (w.next_unit()) {
        const bool have = (w.have >> t) & 1u;
        bool started = false;
        while (w.next_step()) {
          const bool act = (w.act >> t) & 1u;
          auto give_k = [&]() {
            if (elect_one()) mma_commit(&sm.empty[n % kKs]);
            __syncwarp();
          };
          if (!act) {  // its keys are for the other tile only
            await(sm, &sm.full[n % kKs], (n / kKs) & 1u);
            give_k();
          }
          if (n > 0) await(sm, &sm.clean[(n - 1) % kVs], ((n - 1) / kVs) & 1u);
          if (pend) put_pv(0);
          if (act) {
            await(sm, &sm.full[n % kKs], (n / kKs) & 1u);
            // (On a unit's first step this holds up the second half of the product before,
            // and with it the rows of a unit that ended there, until K and Q have landed.)
            if (!started) await(sm, &sm.qfull[t], qpar);
            put_s(0);
          }
          if (pend) {
            put_pv(1);
            ppar ^= 1u;
          }
          give_v();
          if (act) {
            put_s(1);
            give_k();
          }
          pend = act;
          acc = started;
          started |= act;
          ends = false;
          ++n;
        }
        if (have) {
          if (!started) await(sm, &sm.qfull[t], qpar);
          if (elect_one()) mma_commit(&sm.qempty[t]);
          __syncwarp();
          qpar ^= 1u;
        }
        // (A tile without a step in the unit has no end to signal.  Its softmax warps give
        // this warp nothing to wait for there: it could signal the next end as well before
        // they have seen the first, and a wait for a phase that is two behind never ends.)
        ends = started;
      }
      if (n > 0) await(sm, &sm.clean[(n - 1) % kVs], ((n - 1) / kVs) & 1u);
      if (pend) {
        put_pv(0);
        put_pv(1);
      }
      give_v();
      if (elect_one()) mma_commit(&sm.drain);
      __syncwarp();
      mbar_wait_bounded(&sm.drain, 0);
    } else {
      // ----------------------------------------------------------- V tiles
      uint32_t n = 0;
      while (w.next_unit())
        while (w.next_step()) {
          const int s = (int)(n % kVs);
          await(sm, &sm.full[kKs + s], (n / kVs) & 1u);
          if (!w.full) {
            unsigned char* vt = bp + Geo::kOffRing + (kKs + s) * Geo::kTile;
            // x * 0 is NaN where x is not finite, and stays so in a sum
            uint32_t nan[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
            for (int r = lane; r < kKeys; r += 32) {
#pragma unroll
              for (int hf = 0; hf < Geo::kHalves; ++hf) {
                uint4* row = reinterpret_cast<uint4*>(vt + hf * Geo::kHalf + r * 128);
                if (r >= w.keys) {  // behind the last key
#pragma unroll
                  for (int c = 0; c < 8; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
                  continue;
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const uint4 v = row[c ^ (r & 7)];
                  nan[0] = times_zero(v.x, nan[0]);
                  nan[1] = times_zero(v.y, nan[1]);
                  nan[2] = times_zero(v.z, nan[2]);
                  nan[3] = times_zero(v.w, nan[3]);
                }
              }
            }
            if (not_finite2(nan[0]) | not_finite2(nan[1]) | not_finite2(nan[2]) |
                not_finite2(nan[3])) {
              *(volatile uint32_t*)&sm.bad = 1;
#pragma unroll 1
              for (int i = lane; i < kKeys * 32 * Geo::kHalves; i += 32) {
                // (row of 32 words, as this lane has read it)
                const int r = (i & 31) + ((i >> 5) & 3) * 32, word = i >> 7;
                uint32_t* x = reinterpret_cast<uint32_t*>(vt + (word >> 5) * Geo::kHalf + r * 128) +
                              (word & 31);
                *x = finite2(*x);
              }
            }
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.clean[s]);
          ++n;
        }
    }
  } else {
    // --------------------------------------------------------------- softmax
    W w(prm, ws);
    const int t = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + 128u * t;
    const uint32_t tO = tmem + lanes + 256u + 128u * t;
    const float sc = prm.scale_log2;
    uint32_t steps = 0, upar = 0;  // steps of this tile; parity of its next end
    typename W::Row row(prm, r);
    while (w.next_unit()) {
      if (!((w.have >> t) & 1u)) continue;
      w.set_row(row, t);
      float mref = neg_inf(), l = 0.f;
      bool any = false;
      while (w.next_step()) {
        if (!((w.act >> t) & 1u)) continue;
        const bool blind = w.warp_blind(row);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          await(sm, &sm.sfull[t][h], steps & 1u);
          fence_after();
          if (blind) {
            uint32_t z[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0u;
            tst32(tS + 64u * h, z);
          } else {
            float s[kHalfKeys];
            {
              uint32_t a[2][32];
              tld32(tS + 64u * h, a[0]);
              tld32(tS + 64u * h + 32u, a[1]);
              tld_wait();
#pragma unroll
              for (int i = 0; i < kHalfKeys; ++i) s[i] = __uint_as_float(a[i >> 5][i & 31]);
            }
            if (!w.full) w.hide(row, h, s);
            // the scale is positive: the maximum is taken on the raw scores
            float m4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) m4[c] = fmax3f(s[c], s[c + 4], s[c + 8]);
#pragma unroll
            for (int i = 12; i < kHalfKeys - 4; i += 8)
#pragma unroll
              for (int c = 0; c < 4; ++c) m4[c] = fmax3f(m4[c], s[i + c], s[i + 4 + c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) m4[c] = fmaxf(m4[c], s[kHalfKeys - 4 + c]);
            const float bm = fmaxf(fmax3f(m4[0], m4[1], m4[2]), m4[3]) * sc;
            float corr = 1.f;
            // (also at a row's first visible key)
            if (__any_sync(0xffffffffu, bm > mref + 8.f)) {
              const float mnew = bm > mref + 8.f ? bm : mref;
              if (mref != neg_inf()) corr = ex2(mref - mnew);
              mref = mnew;
              // (rows that have seen nothing hold zeros)
              if (__any_sync(0xffffffffu, corr != 1.f)) {
                // the P V of the half step before must be done (that of the one before
                // it is: it was issued before these scores)
                await(sm, &sm.pvdone[t], (h + 1) & 1u);
                fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t o[16];
                  tld16(tO + 16u * c, o);
                  tld_wait();
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                  tst16(tO + 16u * c, o);
                }
              }
            }
            const float nmu = mref == neg_inf() ? 0.f : -mref;
            const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(nmu, nmu);
            float2 ls4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < kHalfKeys / 32; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int j = 32 * c + 2 * i;
                const float2 e = ffma2(make_float2(s[j], s[j + 1]), sc2, nm2);
                const float p0 = ex2(e.x), p1 = ex2(e.y);
                ls4[i & 3] = fadd2(ls4[i & 3], make_float2(p0, p1));
                pk[i] = pack_bf16x2(p0, p1);
              }
              tst16(tS + (uint32_t)(64 * h + 16 * c), pk);
            }
            const float2 lsa = fadd2(fadd2(ls4[0], ls4[1]), fadd2(ls4[2], ls4[3]));
            l = fmaf(l, corr, lsa.x + lsa.y);
          }
          tst_wait();
          fence_before();
          mbar_arrive(&sm.pfull[t][h]);
        }
        any = true;
        ++steps;
      }
      if (any) {
        await(sm, &sm.ofull[t], upar);
        upar ^= 1u;
        fence_after();
      }
      // whoever gave up wrote `dead` before the arrival that led here
      bool gave_up = *(volatile uint32_t*)&sm.dead != 0;
#ifdef SV_TEST_GAVE_UP  // a test's build: CTA 0 as if one of its waits had
      gave_up |= blockIdx.x == 0;
#endif
      if (gave_up) l = __int_as_float(0x7fffffff);
      // (one answer for the warp: the next unit's tiles may be under way)
      const bool bad = __any_sync(0xffffffffu, *(volatile uint32_t*)&sm.bad != 0);
      w.begin_finish(row, t, mref, l);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        if (any) {
          uint32_t x[32];
          tld32(tO + 32u * c, x);
          tld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(x[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (bad) {
          // NaN and infinite values of keys this row sees (0 times infinity is NaN, as in
          // the steps whose values were left as they are)
          W again(w);
          again.restart();
          while (again.next_step()) {
            if (again.full || !((again.act >> t) & 1u)) continue;
            for (int k = 0; k < again.keys; ++k)
              if (again.sees(row, k)) {
                const uint32_t* v = reinterpret_cast<const uint32_t*>(again.value(k) + 32 * c);
                uint32_t inf = 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i) inf |= infinite2(v[i]);
                const float mul =
                    inf && weightless<D>(again.query(row), again.key(k), sc, mref) ? 0.f : 1.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const uint32_t x = v[i], f = not_finite2(x);
                  if (f & 0x8000u) o[2 * i] += bf16_lo(x) * mul;
                  if (f >> 31) o[2 * i + 1] += bf16_hi(x) * mul;
                }
              }
          }
        }
        w.finish(row, t, c, o);
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTaTmemCols)
                 : "memory");
  }
}

// bf16 array [n2, n1, D], strides in bytes (multiples of 16), copied in boxes of 64
// dims x b1 x b2 with the 128-byte swizzle; what lies outside reads as zeros.
bool ta_map(CUtensorMap* map, const void* base, int D, int64_t n1, int64_t n2, int64_t s1,
            int64_t s2, int b1, int b2) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)n1, (cuuint64_t)n2};
  cuuint64_t strides[2] = {(cuuint64_t)s1, (cuuint64_t)s2};
  cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace sv
