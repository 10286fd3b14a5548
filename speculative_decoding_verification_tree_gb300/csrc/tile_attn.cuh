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
//   warp 1      issues S_t = Q_t K^T and O_t += P_t V (tcgen05.mma M 128, float32 in
//               TMEM) for both tiles from one thread: P V of the step before first,
//               then S of this one, tile by tile, so that one tile's products run
//               while the other's softmax does;
//   warps 2-3   every V tile on its way to the products: rows behind the last key
//               become zeros, and in steps that some row does not see in full so do
//               NaN and infinite elements (0 times them would reach rows that do not
//               see them; rows that do see them get them back at the end);
//   warps 4-11  softmax, a thread per row: S from TMEM, online base-2 softmax against
//               a reference maximum that moves only when a row's maximum grows by
//               more than 2^8 (O is then rescaled in TMEM), P as bf16 pairs into the
//               TMEM columns of S; at a unit's end O / l.
//
// TMEM (512 columns): S_t at 128 t, P_t over its first half, O_t at 256 + 128 t.
// One issuing thread keeps the order that this needs: S_t of a step is issued after
// P_t V of the step before, which reads P_t from the same columns, and a commit of S_t
// covers that P V, so a softmax warp that sees S_t may also rescale O_t.
// Sums, statistics and outputs are float32; P is rounded to bf16 for the product and
// the output to bf16 at the end.
//
// Every mbarrier wait is bounded; a CTA that gives up stops waiting, still frees its
// TMEM after waiting, bounded, for its own products and copies, and returns NaN rows
// and normalisers (there is no status word).
#pragma once

#include <cfloat>
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace sv {
namespace {

constexpr int kRows = 128;       // query rows per tile
constexpr int kKeys = 128;       // keys per step
constexpr int kTaThreads = 384;
// Registers per thread after the split: 128 x 72 + 256 x 216 = 384 x 168, what the
// block is launched with.
constexpr int kCtlRegs = 72, kSoftRegs = 216;
static_assert(128 * kCtlRegs + 256 * kSoftRegs <= kTaThreads * 168, "register split");
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
                                      ((uint32_t)(kKeys >> 3) << 17) |
                                      ((uint32_t)(kRows >> 4) << 24);
  // B (V as stored) is MN-major
  static constexpr uint32_t kIdescPV = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                       ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
};

template <int kKs, int kVs>
struct __align__(8) TileCtl {
  uint64_t full[kKs + kVs], empty[kKs + kVs];  // K stages, then V stages
  uint64_t clean[kVs];
  uint64_t qfull[2], qempty[2], sfull[2], pfull[2], ofull[2], drain;
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
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// bit 15 / 31 set where a bf16 half is NaN or infinite
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// The Walk of a caller W offers, to whole warps:
//   static setup(prm, shared, scratch)   once, before the roles part
//   bool next_unit(), bool next_step(), restart() (the unit's steps from the start)
//   have   tiles of the unit (bits);  act   tiles that take part in the step
//   full   no row of the unit lacks a key of the step
//   load_q / load_k / load_v  the producer's copies
//   keys   keys of the step that exist (the rest of the 128 is not in the sequence)
// and, per softmax thread, a Row (set_row at a unit's start):
//   bool warp_blind(row)          no row of this warp sees anything of the step
//   void hide(row, s)             scores of keys the row does not see become -inf
//   bool sees(row, i), const uint16_t* value(i)   key i of the step; its V row
//   void finish(...)              what becomes of the row
template <int D, int kKs, int kVs, class W>
__global__ void __launch_bounds__(kTaThreads, 1)
    tile_attn(const __grid_constant__ typename W::Params prm) {
  using Geo = TileGeo<D, kKs, kVs>;
  using Ctl = TileCtl<kKs, kVs>;
  extern __shared__ __align__(1024) unsigned char araw[];
  const uint32_t raw = smem_u32(araw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* bp = araw + (base - raw);
  Ctl& sm = *reinterpret_cast<Ctl*>(bp + Geo::kOffCtl);
  typename W::Shared& ws = *reinterpret_cast<typename W::Shared*>(bp + Geo::kOffCtl + sizeof(Ctl));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKs + kVs; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < kVs; ++s) mbar_init(&sm.clean[s], 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.qfull[t], 1);
      mbar_init(&sm.qempty[t], 1);
      mbar_init(&sm.sfull[t], 1);
      mbar_init(&sm.pfull[t], kRows);
      mbar_init(&sm.ofull[t], 2);
    }
    mbar_init(&sm.drain, 1);
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
  W::setup(prm, ws, bp);  // every thread; may use the tiles' space; ends with a barrier
  fence_async_smem();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
    W w(prm, ws);
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      uint32_t n = 0, upar = 0;  // steps; parity of each Q tile's next wait
      auto slot = [&](int s, uint32_t fill) {
        await(sm, &sm.empty[s], (fill & 1u) ^ 1u);
        mbar_expect_tx(&sm.full[s], (uint32_t)Geo::kTile);
        return s;
      };
      while (w.next_unit()) {
        bool first = true;
        while (w.next_step()) {
          if (lane == 0) {
            const int s = slot((int)(n % kKs), n / kKs);
            const uint32_t dst = base + Geo::kOffRing + (uint32_t)(s * Geo::kTile);
#pragma unroll
            for (int h = 0; h < Geo::kHalves; ++h)
              w.load_k(dst + h * Geo::kHalf, 64 * h, &sm.full[s]);
          }
          if (first) {  // (after the first keys: they need no wait for the unit before)
            first = false;
            if (lane == 0) {
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                if (!((w.have >> t) & 1u)) continue;
                await(sm, &sm.qempty[t], ((upar >> t) & 1u) ^ 1u);
                mbar_expect_tx(&sm.qfull[t], w.q_bytes() * Geo::kHalves);
#pragma unroll
                for (int h = 0; h < Geo::kHalves; ++h)
                  w.load_q(t, base + (uint32_t)(t * Geo::kTile + h * Geo::kHalf), 64 * h,
                           &sm.qfull[t]);
              }
            }
            upar ^= w.have;
          }
          if (lane == 0) {
            const int s = slot(kKs + (int)(n % kVs), n / kVs);
            const uint32_t dst = base + Geo::kOffRing + (uint32_t)(s * Geo::kTile);
#pragma unroll
            for (int h = 0; h < Geo::kHalves; ++h)
              w.load_v(dst + h * Geo::kHalf, 64 * h, &sm.full[s]);
          }
          ++n;
          __syncwarp();
        }
      }
      // this CTA's last copy into each stage has landed before it exits
      if (lane == 0) {
        for (uint32_t s = 0; s < (uint32_t)kKs && s < n; ++s)
          mbar_wait_bounded(&sm.full[s], ((n - s - 1) / kKs) & 1u);
        for (uint32_t s = 0; s < (uint32_t)kVs && s < n; ++s)
          mbar_wait_bounded(&sm.full[kKs + s], ((n - s - 1) / kVs) & 1u);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ issuer
      const uint64_t dring = desc_kmajor(base + Geo::kOffRing);
      const uint64_t dq0 = desc_kmajor(base);
      const uint64_t dvring = desc_mnmajor(base + Geo::kOffRing + kKs * Geo::kTile, Geo::kHalf);
      uint32_t n = 0, qpar = 0, ppar = 0;
      uint32_t pend = 0, pacc = 0, ends = 0, pv = 0;
      auto put_pv = [&](int t) {  // O_t += P_t V of the step before
        await(sm, &sm.clean[pv % kVs], (pv / kVs) & 1u);
        await(sm, &sm.pfull[t], (ppar >> t) & 1u);
        fence_after();
        const uint64_t dv = dvring + (uint64_t)((pv % kVs) * Geo::kTile >> 4);
        const uint32_t acc = (pacc >> t) & 1u;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_f16_ts(tmem + 256u + 128u * t, tmem + 128u * t + 8u * k, dv + (uint64_t)(k * 128),
                     Geo::kIdescPV, k > 0 ? 1u : acc);
      };
      auto end_tile = [&](int t) {  // every product of the tile's unit is issued
        mma_commit(&sm.ofull[t]);
        // (a plain arrival too: it hands on what this thread saw of the V tiles)
        mbar_arrive(&sm.ofull[t]);
      };
      auto put_s = [&](int t, uint32_t& seen) {
        await(sm, &sm.full[n % kKs], (n / kKs) & 1u);
        if (!((seen >> t) & 1u)) {
          await(sm, &sm.qfull[t], (qpar >> t) & 1u);
          seen |= 1u << t;
        }
        fence_after();
        const uint64_t dk = dring + (uint64_t)((n % kKs) * Geo::kTile >> 4);
        const uint64_t dq = dq0 + (uint64_t)(t * Geo::kTile >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint64_t off = (uint64_t)((i >> 2) * Geo::kHalf + (i & 3) * 32) >> 4;
          mma_f16(tmem + 128u * t, dq + off, dk + off, Geo::kIdescS, i > 0 ? 1u : 0u);
        }
        mma_commit(&sm.sfull[t]);
      };
      while (w.next_unit()) {
        uint32_t started = 0, seen = 0;
        while (w.next_step()) {
          if (lane == 0) {
            uint32_t todo = w.act;
#pragma unroll
            for (int t = 0; t < 2; ++t)
              if (((todo & ~pend) >> t) & 1u) {
                put_s(t, seen);
                todo &= ~(1u << t);
              }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if ((pend >> t) & 1u) put_pv(t);
              if ((ends >> t) & 1u) end_tile(t);
              if ((todo >> t) & 1u) put_s(t, seen);
            }
            if (pend) mma_commit(&sm.empty[kKs + pv % kVs]);
            mma_commit(&sm.empty[n % kKs]);
          }
          ppar ^= pend;
          pend = w.act;
          pacc = started;
          started |= w.act;
          pv = n;
          ends = 0;
          ++n;
          __syncwarp();
        }
        if (lane == 0) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if ((w.have >> t) & 1u) {
              if (!((seen >> t) & 1u)) await(sm, &sm.qfull[t], (qpar >> t) & 1u);
              mma_commit(&sm.qempty[t]);
            }
        }
        qpar ^= w.have;
        ends = w.have;
        __syncwarp();
      }
      if (lane == 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if ((pend >> t) & 1u) put_pv(t);
          if ((ends >> t) & 1u) end_tile(t);
        }
        mma_commit(&sm.drain);
        mbar_wait_bounded(&sm.drain, 0);
      }
    } else {
      // ----------------------------------------------------------- V tiles
      const int tid = (warp - 2) * 32 + lane;
      uint32_t n = 0;
      while (w.next_unit())
        while (w.next_step()) {
          const int s = (int)(n % kVs);
          await(sm, &sm.full[kKs + s], (n / kVs) & 1u);
          if (!w.full) {
            unsigned char* vt = bp + Geo::kOffRing + (kKs + s) * Geo::kTile;
            bool bad = false;
#pragma unroll 1
            for (int r = tid; r < kKeys; r += 64) {
              const bool gone = r >= w.keys;
#pragma unroll 1
              for (int c = 0; c < 8 * Geo::kHalves; ++c) {
                uint4* p = reinterpret_cast<uint4*>(vt + (c >> 3) * Geo::kHalf + swz(r, c & 7));
                if (gone) {
                  *p = make_uint4(0u, 0u, 0u, 0u);
                  continue;
                }
                uint4 v = *p;
                const uint32_t f0 = not_finite2(v.x), f1 = not_finite2(v.y),
                               f2 = not_finite2(v.z), f3 = not_finite2(v.w);
                if (f0 | f1 | f2 | f3) {
                  bad = true;
                  // 0x8000 per half -> 0xffff per half
                  v.x &= ~((f0 >> 15) * 0xffffu);
                  v.y &= ~((f1 >> 15) * 0xffffu);
                  v.z &= ~((f2 >> 15) * 0xffffu);
                  v.w &= ~((f3 >> 15) * 0xffffu);
                  *p = v;
                }
              }
            }
            if (bad) *(volatile uint32_t*)&sm.bad = 1;
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.clean[s]);
          ++n;
        }
    }
  } else {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    W w(prm, ws);
    const int t = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + 128u * t;
    const uint32_t tO = tmem + lanes + 256u + 128u * t;
    const float sc = prm.scale_log2;
    uint32_t spar = 0, upar = 0;
    typename W::Row row(prm, r);
    while (w.next_unit()) {
      if (!((w.have >> t) & 1u)) continue;
      w.set_row(row, t);
      float mref = neg_inf(), l = 0.f;
      bool any = false;
      while (w.next_step()) {
        if (!((w.act >> t) & 1u)) continue;
        await(sm, &sm.sfull[t], spar);
        spar ^= 1u;
        fence_after();
        if (w.warp_blind(row)) {
          uint32_t z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = 0u;
          tst32(tS, z);
          tst32(tS + 32u, z);
        } else {
          uint32_t a[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tld32(tS + 32u * c, a[c]);
          tld_wait();
          float s[kKeys];
#pragma unroll
          for (int i = 0; i < kKeys; ++i) s[i] = __uint_as_float(a[i >> 5][i & 31]);
          if (!w.full) w.hide(row, s);
          // the scale is positive: the maximum is taken on the raw scores
          float m4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) m4[c] = fmax3f(s[c], s[c + 4], s[c + 8]);
#pragma unroll
          for (int i = 12; i < kKeys - 4; i += 8)
#pragma unroll
            for (int c = 0; c < 4; ++c) m4[c] = fmax3f(m4[c], s[i + c], s[i + 4 + c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) m4[c] = fmaxf(m4[c], s[kKeys - 4 + c]);
          const float bm = fmaxf(fmax3f(m4[0], m4[1], m4[2]), m4[3]) * sc;
          const bool move = bm > mref + 8.f;  // (also at the first visible key)
          const float mnew = move ? bm : mref;
          const float corr = (move && mref != neg_inf()) ? ex2(mref - mnew) : 1.f;
          mref = mnew;
          const float nmu = mref == neg_inf() ? 0.f : -mref;
          if (any && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tld16(tO + 16u * c, o);
              tld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
              tst16(tO + 16u * c, o);
            }
          }
          const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(nmu, nmu);
          float2 ls4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < kKeys / 32; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int j = 32 * c + 2 * i;
              const float2 e = ffma2(make_float2(s[j], s[j + 1]), sc2, nm2);
              const float p0 = ex2(e.x), p1 = ex2(e.y);
              ls4[i & 3] = fadd2(ls4[i & 3], make_float2(p0, p1));
              pk[i] = pack_bf16(p0, p1);
            }
            tst16(tS + 16u * c, pk);
          }
          const float2 lsa = fadd2(fadd2(ls4[0], ls4[1]), fadd2(ls4[2], ls4[3]));
          l = fmaf(l, corr, lsa.x + lsa.y);
        }
        any = true;
        tst_wait();
        fence_before();
        mbar_arrive(&sm.pfull[t]);
      }
      await(sm, &sm.ofull[t], upar);
      upar ^= 1u;
      fence_after();
      // whoever gave up wrote `dead` before the arrival that led here
      bool gave_up = *(volatile uint32_t*)&sm.dead != 0;
#ifdef SV_TEST_GAVE_UP  // a test's build: CTA 0 as if one of its waits had
      gave_up |= blockIdx.x == 0;
#endif
      if (gave_up) l = __int_as_float(0x7fffffff);
      const bool bad = *(volatile uint32_t*)&sm.bad != 0;
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
          // NaN and infinite values of keys this row sees (their weight is positive)
          W again(w);
          again.restart();
          while (again.next_step()) {
            if (again.full || !((again.act >> t) & 1u)) continue;
            for (int k = 0; k < again.keys; ++k)
              if (again.sees(row, k)) {
                const uint32_t* v = reinterpret_cast<const uint32_t*>(again.value(k) + 32 * c);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const uint32_t x = v[i], f = not_finite2(x);
                  if (f & 0x8000u) o[2 * i] += bf16_lo(x);
                  if (f >> 31) o[2 * i + 1] += bf16_hi(x);
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

PFN_cuTensorMapEncodeTiled_v12000 ta_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// bf16 array [n2, n1, D], strides in bytes (multiples of 16), copied in boxes of 64
// dims x b1 x b2 with the 128-byte swizzle; what lies outside reads as zeros.
bool ta_map(CUtensorMap* map, const void* base, int D, int64_t n1, int64_t n2, int64_t s1,
            int64_t s2, int b1, int b2) {
  auto fn = ta_encode_fn();
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
