// spec_token_logprobs / spec_token_logprobs_grad: log probabilities of given
// tokens, the rows' entropy and most probable alternatives, and the gradient of
// log probabilities and entropies with respect to the logits.
//
// With k = log2(e) / T, m any logit of the row as reference, d_x = (z_x - m) k,
// S = sum_x 2^d_x and A = sum_x 2^d_x d_x:
//   lse = m k + log2 S                    (base 2)
//   ln p(t) = ln 2 (d_t - log2 S)
//   H = ln 2 (log2 S - A / S)
// so one pass over a row gives all three.  The reference is kept as the logit itself
// and subtracted before the scale: a distance is then off by a relative 2^-23 whatever
// the logits' size, and 0 at the reference.  (z k - m k in one FMA is off by the rounding
// of m k, which for a vocabulary masked with -1e10 is hundreds of powers of two.)  A
// thread's reference is the maximum of its first logits and moves only when a later one
// is above it by more than a factor of 2^10: sums stay far inside float32, and moving is
// rare (a running maximum moves in some lane of a warp at nearly every step).  Bound by
// reading the logits once: 8192 rows of 128256 bf16 logits 313 us, 6.7 TB/s, the measured
// copy rate (303 with the one FMA, which is no choice).
//
// Alternatives: each thread also keeps its largest logit.  The top-th largest of the
// warps' four largest of those (or, for more than 32 alternatives, the smallest of the
// warps' ceil(top / 8)-th largest) is a lower bound of the top-th largest logit of the
// CTA's part, so only threads whose largest reaches it hold candidates.  Their logits are
// read again, from L2, and the few candidates ranked by (value, lower index).  The exact
// top-th of the 256 maxima, by counting, cost more than it saved (224 rows of 128256, 20
// alternatives: 26.8 us; with the smallest of the warps' third largest 28.9, for more is
// read again; now 22.2, of which 16.1 without alternatives).  Parts where the bound leaves
// too few or too many candidates (ties, NaN, masked vocabularies) take an exact radix
// selection instead: 224 such rows of 128256 with 20 alternatives 325 us (13 logits that
// are not -inf, or 2000 side by side), one such row 59; with 128 logits spread out, 16 us.
//
// Few rows are split over the CTAs of a cluster, joined through distributed
// shared memory (one row of 32000 float32 logits, 5 alternatives: 7.9 us; 128: 22).
//
// Gradient: dz_x = (1/T) (sum_j g_j 1[t_j = x] - p_x (sum_j g_j + g_H (ln p_x + H))).
// One read and one write of the row; the given tokens' own terms are put in
// after the dense part, by the CTA that owns their place (their logits are
// read before, so that the gradient may overwrite the logits).  4096 rows of 128256 bf16
// logits 329 us, 95% of the copy rate; 777 odd float32 rows of 50257 inside padded ones
// 50.0 us (their gradient lies at another alignment: logits one by one, gradient in
// 16-byte words).
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = SPEC_MAX_TOP_K;
constexpr int kCandCap = 1024;
constexpr int kAgain = 4;  // groups of flagged threads in flight when they are read again
constexpr int kMaxCluster = 8;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMove = 10.f;    // base-2 distance at which a reference moves
constexpr float kFloor = -200.f; // 2^kFloor is 0: a distance of -inf becomes finite

// A NaN operand gives NaN (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// Order-preserving key: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (isnan(v)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <typename T>
struct Vec;  // a 16-byte group of logits
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  __device__ __forceinline__ static void get(const uint4& r, float (&v)[8]) {
    v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
    v[4] = bf16_lo(r.z); v[5] = bf16_hi(r.z); v[6] = bf16_lo(r.w); v[7] = bf16_hi(r.w);
  }
  __device__ __forceinline__ static uint4 put(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
  __device__ __forceinline__ static void store(uint16_t* p, float v) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    *p = h;
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  __device__ __forceinline__ static void get(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
  }
  __device__ __forceinline__ static uint4 put(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
  __device__ __forceinline__ static void store(float* p, float v) { *p = v; }
};

__device__ __forceinline__ uint4 ldg_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A row's 16-byte groups: `head` logits before the first aligned address, then
// `groups` groups, then the rest.
template <typename T>
struct RowSpan {
  int head, groups, tail;  // tail: first logit behind the groups
  __device__ __forceinline__ RowSpan(const T* row, int V) {
    const int off = (int)(((uintptr_t)row & 15u) / sizeof(T));
    head = min(V, off == 0 ? 0 : (int)(16 / sizeof(T)) - off);
    groups = (V - head) / Vec<T>::kN;
    tail = head + groups * Vec<T>::kN;
  }
  // loose logits: i < loose(V) lies at place(i)
  __device__ __forceinline__ int loose(int V) const { return head + V - tail; }
  __device__ __forceinline__ int place(int i) const { return i < head ? i : tail + i - head; }
};

// A candidate as one number: the larger, the further ahead (value, then lower index).
// 0: none.
using Cand = uint64_t;
__device__ __forceinline__ Cand make_cand(uint32_t key, int idx) {
  return ((uint64_t)key << 32) | (0xFFFFFFFFu - (uint32_t)idx);
}
__device__ __forceinline__ int cand_idx(Cand c) { return (int)(0xFFFFFFFFu - (uint32_t)c); }
__device__ __forceinline__ uint32_t cand_key(Cand c) { return (uint32_t)(c >> 32); }

struct Sums {
  float m, s, a;  // reference (a logit; -inf: none yet), S, A
};
struct LpSmem {
  Sums part[kMaxCluster];  // rank 0: the parts of the row
  float rm[kWarps], rs[kWarps], ra[kWarps];
  float m, s, a;        // this CTA's part
  uint32_t tau[32];
  int nflag, ncand;
  uint16_t flag[kThreads];
  __align__(16) Cand cand[kCandCap];
  Cand best[kMaxTop];   // this CTA's part, best first
  int hist[256];
  int digit, above, base;
};

__device__ __forceinline__ void st_dsmem(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_dsmem64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ Sums join(Sums x, Sums y, float kt) {
  const float m = fmaxf(x.m, y.m);
  if (m == neg_inf()) return {m, x.s + y.s, x.a + y.a};
  // a part without finite logits has s = a = 0 (or NaN); its distance is cut
  // so that 0 times it stays 0
  const float rx = (x.m - m) * kt, ry = (y.m - m) * kt;
  const float dx = fmaxf(rx, kFloor), dy = fmaxf(ry, kFloor);
  const float cx = ex2(rx), cy = ex2(ry);
  return {m, x.s * cx + y.s * cy, (x.a + x.s * dx) * cx + (y.a + y.s * dy) * cy};
}

// The `k` first of this part's logits in the order (value, lower index) by an
// exact radix selection: 8 bits of the key a round, then everything above the
// k-th key and the first ones equal to it.  Every thread calls; `at(i)` is the
// part's i-th logit in index order, n of them, `idx(i)` its place in the row.
// (A CTA whose part holds many equal logits comes here: slow, but exact.)
template <class At, class Idx>
__device__ void select_exact(LpSmem& sm, int n, int k, At at, Idx idx) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t prefix = 0;
  int need = k;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    sm.hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t key = order_key(at(i));
      if (key != 0u && (key & mask) == prefix) atomicAdd(&sm.hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int run = 0, d = 255;
      for (; d > 0; --d) {
        if (run + sm.hist[d] >= need) break;
        run += sm.hist[d];
      }
      sm.digit = d;
      sm.above = run;
    }
    __syncthreads();
    prefix |= (uint32_t)sm.digit << shift;
    need -= sm.above;
    __syncthreads();
  }
  // prefix is the k-th key (0 where there are fewer than k numbers: then every
  // number is above it); `need` entries equal to it belong to the k
  if (tid == 0) {
    sm.ncand = 0;
    sm.base = 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const uint32_t key = order_key(at(i));
    if (key > prefix) sm.cand[atomicAdd(&sm.ncand, 1)] = make_cand(key, idx(i));
  }
  __syncthreads();
  const int above = sm.ncand;
  if (prefix != 0u) {
    for (int i0 = 0; i0 < n; i0 += kThreads) {  // in index order
      const int i = i0 + tid;
      const bool eq = i < n && order_key(at(i)) == prefix;
      const uint32_t bal = __ballot_sync(0xffffffffu, eq);
      if (lane == 0) sm.hist[warp] = __popc(bal);
      __syncthreads();
      int before = sm.base, all = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm.hist[w];
        all += sm.hist[w];
      }
      before += __popc(bal & ((1u << lane) - 1u));
      if (eq && before < need) sm.cand[above + before] = make_cand(prefix, idx(i));
      __syncthreads();
      if (tid == 0) sm.base += all;
      __syncthreads();
      if (sm.base >= need) break;
    }
  }
  __syncthreads();
  if (tid == 0) sm.ncand = above + min(need, prefix != 0u ? sm.base : 0);
  __syncthreads();
}

// One row per cluster.  kEnt: also the entropy.  kTop: also alternatives.
template <typename T, bool kEnt, bool kTop>
__global__ void __launch_bounds__(kThreads, 4)
    token_logprobs(const T* __restrict__ logits, int64_t ld, int R, int V,
                   const int32_t* __restrict__ rows, const int32_t* __restrict__ tokens, int n,
                   int top, float kt, float invT, float move, float* __restrict__ logprob,
                   float* __restrict__ row_lse, float* __restrict__ entropy,
                   int32_t* __restrict__ top_ids, float* __restrict__ top_lp) {
  constexpr int kN = Vec<T>::kN;
  constexpr int kBatch = 8;  // groups in flight per thread
  __shared__ LpSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int64_t out = blockIdx.x / C;
  const int at = rows ? rows[out] : (int)out;
  if (at < 0 || at >= R) {  // no such row (the whole cluster leaves)
    if (rank == 0) {
      for (int j = tid; j < n; j += kThreads) logprob[out * n + j] = 0.f;
      for (int j = tid; j < top; j += kThreads) {
        top_ids[out * top + j] = -1;
        top_lp[out * top + j] = 0.f;
      }
      if (tid == 0) {
        if (row_lse) row_lse[out] = 0.f;
        if (kEnt) entropy[out] = 0.f;
      }
    }
    return;
  }
  const T* row = logits + (int64_t)at * ld;
  const RowSpan<T> span(row, V);
  const uint4* vec = reinterpret_cast<const uint4*>(row + span.head);
  const int per = (span.groups + C - 1) / C;
  const int g0 = min(span.groups, rank * per), g1 = min(span.groups, g0 + per);
  // rank 0 also takes the logits around the groups
  const int loose = rank == 0 ? span.loose(V) : 0;

  // the given token of a thread, on its way while the row is read
  int token = -1;
  float given = 0.f;
  if (rank == 0 && tid < n) {
    token = tokens[out * n + tid];
    if (token >= 0 && token < V) given = ElemIO<T>::get(row, token);
    else token = -1;
  }
  // the reference (0 while there is none: every logit was -inf or NaN) and the logit
  // above which it moves
  float ref = 0.f, limit = neg_inf(), mx = neg_inf();
  float2 s2 = make_float2(0.f, 0.f), a2 = make_float2(0.f, 0.f);
  const float2 kt2 = make_float2(kt, kt);
  auto move_ref = [&](float gm) {
    if (limit != neg_inf()) {
      // (what a far reference leaves is 0, not 0 times an infinite distance)
      const float d = (ref - gm) * kt, c = ex2(d);
      if (kEnt) {
        const float cut = fmaxf(d, kFloor);
        a2.x = (a2.x + s2.x * cut) * c;
        a2.y = (a2.y + s2.y * cut) * c;
      }
      s2.x *= c;
      s2.y *= c;
    }
    ref = gm;
    limit = gm + move;
  };
  auto pair = [&](float z0, float z1) {
    float2 d = fmul2(fadd2(make_float2(z0, z1), make_float2(-ref, -ref)), kt2);
    if (kEnt) {
      d.x = max_nan(d.x, kFloor);
      d.y = max_nan(d.y, kFloor);
    }
    const float2 e = make_float2(ex2(d.x), ex2(d.y));
    s2 = fadd2(s2, e);
    if (kEnt) a2 = ffma2(e, d, a2);
  };
  for (int i = tid; i < loose; i += kThreads) {
    const float z = ElemIO<T>::get(row, span.place(i));
    if (kTop) mx = fmaxf(mx, z);
    if (z > limit) move_ref(z);
    pair(z, neg_inf());
  }
  auto group = [&](const uint4& r) {
    float v[kN];
    Vec<T>::get(r, v);
    float gm;
    if constexpr (kN == 8)
      gm = fmax3f(fmax3f(v[0], v[1], v[2]), fmax3f(v[3], v[4], v[5]), fmaxf(v[6], v[7]));
    else
      gm = fmax3f(fmaxf(v[0], v[1]), v[2], v[3]);
    if (kTop) mx = fmaxf(mx, gm);
    if (gm > limit) move_ref(gm);
#pragma unroll
    for (int i = 0; i < kN; i += 2) pair(v[i], v[i + 1]);
  };
  int g = g0 + tid;
  for (; g + (kBatch - 1) * kThreads < g1; g += kBatch * kThreads) {
    uint4 r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) r[i] = ldg_once(vec + g + i * kThreads);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) group(r[i]);
  }
  for (; g < g1; g += kThreads) group(ldg_once(vec + g));

  Sums t{limit == neg_inf() ? neg_inf() : ref, s2.x + s2.y, a2.x + a2.y};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    t = join(t, Sums{__shfl_xor_sync(0xffffffffu, t.m, o), __shfl_xor_sync(0xffffffffu, t.s, o),
                     __shfl_xor_sync(0xffffffffu, t.a, o)}, kt);
  if (lane == 0) {
    sm.rm[warp] = t.m;
    sm.rs[warp] = t.s;
    sm.ra[warp] = t.a;
  }
  const uint32_t mine = kTop ? order_key(mx) : 0u;
  // how the alternatives' bound is found: the top-th of the warps' `each` largest
  // maxima together (at most 32), or the smallest of the warps' each-th
  const int busy = min(kWarps, (g1 - g0) / 32);
  const bool few = busy > 0 && top <= 32 / busy * busy;
  const int each = busy == 0 ? 0 : (few ? 32 / busy : (top + busy - 1) / busy);
  if constexpr (kTop) {
    // the warps' largest maxima, lanes dropping out one by one (only warps in which
    // every lane has logits; a part without one is selected exactly)
    uint32_t left = mine, rth = 0u;
    if (warp < busy)
      for (int i = 0; i < each; ++i) {
        rth = __reduce_max_sync(0xffffffffu, left);
        const uint32_t who = __ballot_sync(0xffffffffu, left == rth);
        if (lane == __ffs(who) - 1) left = 0u;
        if (few && lane == 0) sm.tau[warp * each + i] = rth;
      }
    if (!few && lane == 0) sm.tau[warp] = warp < busy ? rth : 0xFFFFFFFFu;
    if (tid == 0) sm.nflag = sm.ncand = 0;
  }
  __syncthreads();
  if (tid == 0) {
    Sums all{sm.rm[0], sm.rs[0], sm.ra[0]};
    for (int w = 1; w < kWarps; ++w) all = join(all, Sums{sm.rm[w], sm.rs[w], sm.ra[w]}, kt);
    sm.m = all.m;
    sm.s = all.s;
    sm.a = all.a;
  }
  if constexpr (kTop) {
    uint32_t tau = 0u;
    if (few) {
      const uint32_t e = lane < busy * each ? sm.tau[lane] : 0u;
      int ahead = 0;
#pragma unroll
      for (int o = 0; o < 32; ++o) {
        const uint32_t x = __shfl_sync(0xffffffffu, e, o);
        ahead += x > e || (x == e && o < lane) ? 1 : 0;
      }
      tau = __shfl_sync(0xffffffffu, e, __ffs(__ballot_sync(0xffffffffu, ahead == top - 1)) - 1);
    } else if (each > 0 && each <= 32) {
      tau = sm.tau[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) tau = min(tau, sm.tau[w]);
    }
    constexpr uint32_t kNegInf = 0x007FFFFFu;  // order_key(-inf)
    bool exact = tau <= kNegInf;
    if (!exact) {
      if (mine >= tau) sm.flag[atomicAdd(&sm.nflag, 1)] = (uint16_t)tid;
      for (int i = tid; i < loose; i += kThreads) {
        const int x = span.place(i);
        const uint32_t key = order_key(ElemIO<T>::get(row, x));
        if (key >= tau) {
          const int p = atomicAdd(&sm.ncand, 1);
          if (p < kCandCap) sm.cand[p] = make_cand(key, x);
        }
      }
      __syncthreads();
      const int per_thread = (g1 - g0 + kThreads - 1) / kThreads;
      const int items = sm.nflag * per_thread;
      for (int i0 = tid; i0 < items; i0 += kAgain * kThreads) {
        uint4 raw[kAgain];
        int where[kAgain];
#pragma unroll
        for (int q = 0; q < kAgain; ++q) {
          const int i = i0 + q * kThreads, f = i / per_thread;
          where[q] = i < items ? g0 + sm.flag[f] + (i - f * per_thread) * kThreads : g1;
          if (where[q] < g1) raw[q] = vec[where[q]];
        }
#pragma unroll
        for (int q = 0; q < kAgain; ++q) {
          if (where[q] >= g1) continue;
          float v[kN];
          Vec<T>::get(raw[q], v);
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const uint32_t key = order_key(v[e]);
            if (key >= tau) {
              const int p = atomicAdd(&sm.ncand, 1);
              if (p < kCandCap) sm.cand[p] = make_cand(key, span.head + where[q] * kN + e);
            }
          }
        }
      }
      __syncthreads();
      exact = sm.ncand > kCandCap;
    }
    if (exact) {
      __syncthreads();
      const int inner = (g1 - g0) * kN, lo = rank == 0 ? span.head : 0;
      const int first = span.head + g0 * kN;
      // index order: the loose logits before the groups, the groups, those behind
      auto place = [&](int i) {
        if (i < lo) return i;
        i -= lo;
        return i < inner ? first + i : span.tail + i - inner;
      };
      select_exact(
          sm, inner + loose, min(top, inner + loose),
          [&](int i) { return ElemIO<T>::get(row, place(i)); }, place);
    }
    const int nc = sm.ncand;
    if (tid == 0 && (nc & 1)) sm.cand[nc] = 0;  // (nc = kCandCap is even)
    for (int j = tid; j < top; j += kThreads) sm.best[j] = 0;
    __syncthreads();
    const ulonglong2* two = reinterpret_cast<const ulonglong2*>(sm.cand);
    for (int i = tid; i < nc; i += kThreads) {
      const Cand c = sm.cand[i];
      int r = 0;
#pragma unroll 8
      for (int j = 0; j < (nc + 1) / 2; ++j) {
        const ulonglong2 o = two[j];
        r += (o.x > c) + (o.y > c);
      }
      if (r < top) sm.best[r] = c;
    }
  }
  __syncthreads();

  Sums all{sm.m, sm.s, sm.a};
  if (C > 1) {
    // every part into rank 0's shared memory: its sums, and its list beside the others'
    // (at most kMaxCluster kMaxTop entries: the candidates' own space, which each CTA
    // has finished with when all have arrived)
    cluster_sync();
    if (tid == 0) {
      st_dsmem(mapa(smem_u32(&sm.part[rank].m), 0), __float_as_uint(all.m));
      st_dsmem(mapa(smem_u32(&sm.part[rank].s), 0), __float_as_uint(all.s));
      st_dsmem(mapa(smem_u32(&sm.part[rank].a), 0), __float_as_uint(all.a));
    }
    if (kTop) {
      for (int j = tid; j < top; j += kThreads)
        st_dsmem64(mapa(smem_u32(&sm.cand[rank * top + j]), 0), sm.best[j]);
    }
    cluster_sync();
    if (rank != 0) return;
    all = sm.part[0];
    for (int c = 1; c < C; ++c) all = join(all, sm.part[c], kt);
    if (kTop) {
      // a candidate's place: its own in its list, and in every other list the number
      // ahead of it (binary searches side by side)
      for (int j = tid; j < top; j += kThreads) sm.best[j] = 0;
      __syncthreads();
      int most = 1;
      while (2 * most <= top) most *= 2;
      for (int i = tid; i < C * top; i += kThreads) {
        const Cand c = sm.cand[i];
        if (c == 0) continue;
        int at[kMaxCluster];
#pragma unroll
        for (int l = 0; l < kMaxCluster; ++l) at[l] = 0;
        for (int step = most; step > 0; step >>= 1)
#pragma unroll
          for (int l = 0; l < kMaxCluster; ++l)
            if (l < C && at[l] + step <= top && sm.cand[l * top + at[l] + step - 1] > c)
              at[l] += step;
        int r = 0;
#pragma unroll
        for (int l = 0; l < kMaxCluster; ++l) r += at[l];
        if (r < top) sm.best[r] = c;
      }
      __syncthreads();
    }
  }
  // (a row of nothing but -inf: reference 0, S = 0, lse = -inf)
  const float m = all.m == neg_inf() ? 0.f : all.m;
  const float ls = log2f(all.s), ln = kLn2 * ls;
  // (by 1 / T: z - m may be as large as float32 goes)
  if (tid < n) logprob[out * n + tid] = token >= 0 ? fmaf(given - m, invT, -ln) : 0.f;
  if (kTop) {
    for (int j = tid; j < top; j += kThreads) {
      const Cand c = sm.best[j];
      const bool have = c != 0;
      top_ids[out * top + j] = have ? cand_idx(c) : -1;
      top_lp[out * top + j] =
          have ? fmaf(key_value(cand_key(c)) - m, invT, -ln) : __int_as_float(0x7fffffff);
    }
  }
  if (tid == 0) {
    if (row_lse) row_lse[out] = fmaf(m, kt, ls);
    if (kEnt) entropy[out] = kLn2 * (ls - all.a / all.s);
  }
}

// ------------------------------------------------------------------ gradient
constexpr int kGradGroups = 4;  // 16-byte groups per thread
constexpr int kMaxGiven = SPEC_MAX_CHILDREN + SPEC_MAX_TOP_K;
// From here on half a unit in the last place of a normaliser is 2^-12 or more (a row
// of nothing but finite masks, a very low temperature): the row's own terms are formed
// again instead.
constexpr float kFarLse = 4096.f;

struct GradSmem {
  int id[kMaxGiven];     // the given tokens of the row, -1: none
  float gv[kMaxGiven];   // and their gradients
  float gsum, red[2][kWarps];
};
struct GradRow {         // of a row's dense term
  float kt, invT, G, gh, H;
};
// dense term of a logit with log2 p = d: -(p / T) (G + g_H (ln p + H))
template <bool kEnt>
__device__ __forceinline__ float dense_term(const GradRow& t, float d) {
  if (!kEnt) return ex2(d) * (-t.G * t.invT);
  d = max_nan(d, kFloor);  // p = 0: 0 times a finite logarithm
  return -t.invT * ex2(d) * fmaf(t.gh, fmaf(kLn2, d, t.H), t.G);
}
// The sum of the gradients of given token tid if it is the first of its kind (true).
__device__ __forceinline__ bool given_sum(const GradSmem& sm, int m, float& s) {
  const int tid = threadIdx.x, x = sm.id[tid];
  bool first = true;
  s = 0.f;
  for (int j = 0; j < m && first; ++j)
    if (sm.id[j] == x) {
      first = j >= tid;
      s += sm.gv[j];
    }
  return first;
}

// A whole row by one CTA, from its own largest logit and sum: nothing of it is
// overwritten before they are formed.  (4096 rows of 128256 bf16 logits, all of them
// far: 960 us, 301 where none is; one row 46 us instead of 4.)
template <typename T, bool kEnt>
__device__ __noinline__ void far_row(const T* row, T* dst, int V, int m, const GradRow t,
                                     GradSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float top = neg_inf(), s = 0.f;
#pragma unroll 8
  for (int i = tid; i < V; i += kThreads) top = fmaxf(top, ElemIO<T>::get(row, i));
  top = warp_max(top);
  if (lane == 0) sm.red[0][warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.red[0][w]);
#pragma unroll 8
  for (int i = tid; i < V; i += kThreads) s += ex2((ElemIO<T>::get(row, i) - top) * t.kt);
  s = warp_sum(s);
  if (lane == 0) sm.red[1][warp] = s;
  __syncthreads();
  s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += sm.red[1][w];
  const float ls = log2f(s);
  auto dense = [&](float z) { return dense_term<kEnt>(t, fmaf(z - top, t.kt, -ls)); };
  int put = -1;
  float val = 0.f, g;
  if (tid < m && sm.id[tid] >= 0 && given_sum(sm, m, g)) {
    put = sm.id[tid];
    val = fmaf(g, t.invT, dense(ElemIO<T>::get(row, put)));
  }
  __syncthreads();
  constexpr int kAhead = 8;  // (the stores may be to the logits themselves)
  for (int i0 = tid; i0 < V; i0 += kAhead * kThreads) {
    float z[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j * kThreads < V) z[j] = ElemIO<T>::get(row, i0 + j * kThreads);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j * kThreads < V) Vec<T>::store(dst + i0 + j * kThreads, dense(z[j]));
  }
  __syncthreads();
  if (put >= 0) Vec<T>::store(dst + put, val);
}

// CTA: one chunk of one row (the first one of a row with a far normaliser takes all of
// it).  kEnt: the entropy's gradient too.
template <typename T, bool kEnt>
__global__ void __launch_bounds__(kThreads)
    token_logprobs_grad(const T* logits, int64_t ld, int V, int chunks,
                        const int32_t* __restrict__ tokens, int n,
                        const int32_t* __restrict__ top_ids, int top, float kt, float invT,
                        const float* __restrict__ row_lse, const float* __restrict__ entropy,
                        const float* __restrict__ g_lp, const float* __restrict__ g_top,
                        const float* __restrict__ g_ent, T* grad, int64_t ldg) {
  constexpr int kN = Vec<T>::kN;
  constexpr int kChunk = kThreads * kGradGroups;  // groups per CTA
  __shared__ GradSmem sm;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t r = blockIdx.x / chunks;
  const int c = blockIdx.x % chunks;
  const T* row = logits + r * ld;
  T* dst = grad + r * ldg;
  // groups by the gradient's alignment; the logits are read as 16-byte words
  // where their row lies alike, else one by one
  const RowSpan<T> span(dst, V);
  const bool alike = (((uintptr_t)row ^ (uintptr_t)dst) & 15u) == 0;
  const int g0 = c * kChunk;
  uint4 raw[kGradGroups];
  const uint4* src = reinterpret_cast<const uint4*>(row + span.head);
#pragma unroll
  for (int i = 0; i < kGradGroups; ++i) {
    const int g = g0 + i * kThreads + tid;
    if (g >= span.groups) continue;
    if (alike) {
      raw[i] = src[g];
    } else {
      float v[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) v[e] = ElemIO<T>::get(row, span.head + g * kN + e);
      raw[i] = Vec<T>::put(v);  // the same bits
    }
  }
  const int m = n + top;
  const float lse = row_lse[r];
  const float gh = kEnt ? g_ent[r] : 0.f, H = kEnt ? entropy[r] : 0.f;
  for (int j = tid; j < m; j += kThreads) {
    const int x = j < n ? tokens[r * n + j] : top_ids[r * top + j - n];
    const bool ok = x >= 0 && x < V;
    sm.id[j] = ok ? x : -1;
    sm.gv[j] = ok ? (j < n ? g_lp[r * n + j] : g_top[r * top + j - n]) : 0.f;
  }
  __syncthreads();
  if (tid < 32) {
    float s = 0.f;
    for (int j = lane; j < m; j += 32) s += sm.gv[j];
    s = warp_sum(s);
    if (lane == 0) sm.gsum = s;
  }
  __syncthreads();
  const GradRow t{kt, invT, sm.gsum, gh, H};
  if (fabsf(lse) >= kFarLse) {
    if (c == 0) far_row<T, kEnt>(row, dst, V, m, t, sm);
    return;
  }
  auto dense = [&](float z) { return dense_term<kEnt>(t, fmaf(z, kt, -lse)); };
  // the given tokens inside this chunk: their logits before anything is written
  // (chunk 0 also owns the row's loose logits)
  const int lo = span.head + g0 * kN, hi = span.head + min(span.groups, g0 + kChunk) * kN;
  float val = 0.f;
  int put = -1;
  if (tid < m && sm.id[tid] >= 0) {
    const int x = sm.id[tid];
    const bool here = (x >= lo && x < hi) || (c == 0 && (x < span.head || x >= span.tail));
    float s;
    if (here && given_sum(sm, m, s)) {
      put = x;
      val = fmaf(s, invT, dense(ElemIO<T>::get(row, x)));
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kGradGroups; ++i) {
    const int g = g0 + i * kThreads + tid;
    if (g < span.groups) {
      float v[kN];
      Vec<T>::get(raw[i], v);
#pragma unroll
      for (int e = 0; e < kN; ++e) v[e] = dense(v[e]);
      reinterpret_cast<uint4*>(dst + span.head)[g] = Vec<T>::put(v);
    }
  }
  if (c == 0)
    for (int i = tid; i < span.loose(V); i += kThreads) {
      const int x = span.place(i);
      Vec<T>::store(dst + x, dense(ElemIO<T>::get(row, x)));
    }
  __syncthreads();
  if (put >= 0) Vec<T>::store(dst + put, val);
}

template <typename T, bool kEnt, bool kTop>
cudaError_t launch_lp(const void* logits, int64_t ld, int R, int V, const int32_t* rows, int M,
                      const int32_t* tokens, int n, int top, float kt, float invT, float move,
                      float* logprob, float* row_lse, float* entropy, int32_t* top_ids,
                      float* top_lp, int C, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)M * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs<T, kEnt, kTop>, (const T*)logits, ld, R, V, rows,
                            tokens, n, top, kt, invT, move, logprob, row_lse, entropy, top_ids,
                            top_lp);
}

template <typename T>
cudaError_t launch_lp_t(bool ent, bool with_top, const void* logits, int64_t ld, int R, int V,
                        const int32_t* rows, int M, const int32_t* tokens, int n, int top,
                        float kt, float invT, float move, float* logprob, float* row_lse,
                        float* entropy, int32_t* top_ids, float* top_lp, int C, cudaStream_t st) {
  auto f = ent ? (with_top ? launch_lp<T, true, true> : launch_lp<T, true, false>)
               : (with_top ? launch_lp<T, false, true> : launch_lp<T, false, false>);
  return f(logits, ld, R, V, rows, M, tokens, n, top, kt, invT, move, logprob, row_lse, entropy,
           top_ids, top_lp, C, st);
}

// CTAs per row.  Rows that fill the GPU take one each; fewer are split until about as
// many CTAs run as fit (four on each of 152 SMs), down to parts of 8 KB.
int row_ctas(int M, int V, int el) {
  int C = 1;
  while (C < kMaxCluster && (int64_t)M * C * 2 <= 608 && (int64_t)V * el / (2 * C) >= 8192) C *= 2;
  return C;
}

bool f32_ok(const void* p) { return (uintptr_t)p % 4 == 0; }

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int spec_token_logprobs(const void* logits, int dtype, int64_t ld, int R, int V,
                                   const int32_t* rows, int M, const int32_t* tokens, int n,
                                   int top, float temperature, float* logprob, float* row_lse,
                                   float* entropy, int32_t* top_ids, float* top_logprob,
                                   void* stream) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (R < 0 || M < 0 || V < 1 || V > SPEC_MAX_VOCAB || ld < V || n < 0 || n > SPEC_MAX_CHILDREN ||
      top < 0 || top > SPEC_MAX_TOP_K || top > V)
    return SPEC_ERR_SHAPE;
  if (!rows && M > R) return SPEC_ERR_SHAPE;
  if ((int64_t)M * kMaxCluster >= (int64_t)1 << 31) return SPEC_ERR_SHAPE;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return SPEC_ERR_ARG;
  if (M == 0) return SPEC_OK;
  if ((R > 0 && !logits) || (n > 0 && (!tokens || !logprob)) ||
      (top > 0 && (!top_ids || !top_logprob)))
    return SPEC_ERR_ARG;
  const int el = dtype == SPEC_F32 ? 4 : 2;
  if ((uintptr_t)logits % el != 0 || !f32_ok(rows) || !f32_ok(tokens) || !f32_ok(logprob) ||
      !f32_ok(row_lse) || !f32_ok(entropy) || !f32_ok(top_ids) || !f32_ok(top_logprob))
    return SPEC_ERR_ARG;
  const float kt = fminf(kLog2e / temperature, FLT_MAX), invT = fminf(1.f / temperature, FLT_MAX);
  const int C = row_ctas(M, V, el);
  auto f = dtype == SPEC_F32 ? launch_lp_t<float> : launch_lp_t<uint16_t>;
  const cudaError_t e = f(entropy != nullptr, top > 0, logits, ld, R, V, rows, M, tokens, n, top,
                          kt, invT, kMove / kt, logprob, row_lse, entropy, top_ids, top_logprob,
                          C, (cudaStream_t)stream);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" int spec_token_logprobs_grad(const void* logits, int dtype, int64_t ld, int M, int V,
                                        const int32_t* tokens, int n, const int32_t* top_ids,
                                        int top, float temperature, const float* row_lse,
                                        const float* entropy, const float* g_logprob,
                                        const float* g_top, const float* g_entropy, void* grad,
                                        int64_t ld_grad, void* stream) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (M < 0 || V < 1 || V > SPEC_MAX_VOCAB || ld < V || ld_grad < V || n < 0 ||
      n > SPEC_MAX_CHILDREN || top < 0 || top > SPEC_MAX_TOP_K)
    return SPEC_ERR_SHAPE;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return SPEC_ERR_ARG;
  if ((entropy == nullptr) != (g_entropy == nullptr)) return SPEC_ERR_ARG;
  const int el = dtype == SPEC_F32 ? 4 : 2;
  const int per = kThreads * kGradGroups * (16 / el);
  const int chunks = (V + per - 1) / per;
  if ((int64_t)M * chunks >= (int64_t)1 << 31) return SPEC_ERR_SHAPE;
  if (M == 0) return SPEC_OK;
  if (!logits || !grad || !row_lse || (n > 0 && (!tokens || !g_logprob)) ||
      (top > 0 && (!top_ids || !g_top)))
    return SPEC_ERR_ARG;
  if (((uintptr_t)logits | (uintptr_t)grad) % el != 0 || !f32_ok(tokens) || !f32_ok(top_ids) ||
      !f32_ok(row_lse) || !f32_ok(entropy) || !f32_ok(g_logprob) || !f32_ok(g_top) ||
      !f32_ok(g_entropy))
    return SPEC_ERR_ARG;
  // the gradient may overwrite the logits, row on row, and nothing else of them
  const char *a = (const char*)logits, *b = (const char*)grad;
  const int64_t na = ((int64_t)(M - 1) * ld + V) * el, nb = ((int64_t)(M - 1) * ld_grad + V) * el;
  if (a < b + nb && b < a + na && !(a == b && (ld == ld_grad || M == 1))) return SPEC_ERR_ARG;
  const float kt = fminf(kLog2e / temperature, FLT_MAX), invT = fminf(1.f / temperature, FLT_MAX);
  const unsigned grid = (unsigned)((int64_t)M * chunks);
  cudaStream_t st = (cudaStream_t)stream;
#define SV_GRAD(T, E)                                                                           \
  token_logprobs_grad<T, E><<<grid, kThreads, 0, st>>>(                                         \
      (const T*)logits, ld, V, chunks, tokens, n, top_ids, top, kt, invT, row_lse, entropy,     \
      g_logprob, g_top, g_entropy, (T*)grad, ld_grad)
  if (dtype == SPEC_F32) {
    if (entropy) SV_GRAD(float, true); else SV_GRAD(float, false);
  } else {
    if (entropy) SV_GRAD(uint16_t, true); else SV_GRAD(uint16_t, false);
  }
#undef SV_GRAD
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
