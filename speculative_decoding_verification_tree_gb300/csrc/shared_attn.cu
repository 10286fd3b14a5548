// spec_tree_attention_shared: tree / single-token attention of sequences that share
// a long prefix and have keys of their own behind it (tile_attn.cuh has the kernel).
//
// For sequence b of prefix g, with n = shared_len[g] shared keys, P = prefix_len[b]
// own keys and drafted node i:
//
//   o[b,i,h] = sum_s softmax_s(scale q[b,i,h] . k_s) v_s over the n shared keys, the
//              P own ones and the own keys P + j of every bit j of mask_bits[b, i]
//
// The query rows of all sequences of a prefix are packed into one unit after another
// of up to 256 rows, so a prefix is read once per unit instead of once per sequence.
// A unit's steps are the prefix's 128-key blocks, which all of its rows see, and then
// the own blocks of its sequences one by one, which the rows of the other sequences
// do not see: their P is 0 there.  (A sequence alone would take the same products: a
// tile has 128 rows whether or not they are used; what a step costs is its 64 KB of
// keys and values.)
//
// Work is split by steps, not units: all steps of all units form a line that is cut
// into equal pieces, one per CTA, since a few units of a long prefix are the usual
// case.  A unit that a cut leaves in several pieces is joined by a second kernel from
// float32 outputs and (reference, sum) pairs, both in a fixed order.  A cut unit of at
// most one tile of rows puts them in both tiles, which take its steps in turn: one
// tile's softmax then runs beside the other's products.
//
// Bounds (32 / 8 heads, D 128).  Single tokens of 32 samples behind 32 K keys: 59 us, 30
// of them the bytes at the copy rate.  CTAs whose piece is all shared keys take 2800 cycles
// a step, what 64 KB take at that rate; the rest is the start (3 us: lengths, scans, the
// first loads), own steps, which cost about a sixth more (a V tile of which most rows see
// nothing is checked, one softmax warp of a tile works), and the join.  Trees of 60 nodes
// of 16 samples behind 8 K keys: 124 us = 1.12 PFLOP/s, the products at 53% of the tensor
// pipe, the softmax warps' latency and the join (40 MB of partial results, which cutting
// 128 units into 152 equal pieces of 58 steps leaves; not cut, the longest unit would take
// 73, the mean one 69).
#include "tile_attn.cuh"

namespace sv {
namespace {

constexpr int kMaxPrefixes = SPEC_MAX_PREFIXES;
static_assert(kTaCtas <= 256, "the join's threads find the cut units");
constexpr int kMinSteps = 2;     // steps of a piece, at least

struct SharedHead {  // the unit that begins in a piece and ends in a later one
  int slot;          // -1: there is none
  int tok0, ntok, h, both, last;
  int pad[2];
};
struct SharedPart {  // partial results of the pieces: [piece][slot][tile]
  SharedHead* head;  // [piece]
  float2* ml;        // [..][128]
  float4* o;         // [..][D / 4][128]
};

struct SharedWalk {
  struct Params {
    CUtensorMap q, ks, vs, ko, vo;
    const int32_t *shared_len, *group_start, *prefix_len;
    const uint64_t* mask_bits;
    const uint16_t *q_ptr, *ks_ptr, *ko_ptr, *vs_ptr, *vo_ptr;
    uint16_t* out;
    float* lse;
    SharedPart part;
    int B, N, Hq, Hkv, G, tpt, groups, Sp, S;
    int spu, chunks;  // sequences per unit; units per sequence (one of them is 1)
    float scale_log2;
  };
  struct Shared {
    // unit rows before each prefix, in parts of `chunks` (at most B: 16 bits)
    uint16_t tiles[kMaxPrefixes + 1];
    int firsts[kMaxPrefixes + 1];  // each prefix's first sequence (clamped)
    int slen[kMaxPrefixes];        // and its shared keys (clamped)
    int64_t len, p0, p1;          // steps per piece; this CTA's piece of the line
    int64_t cum;                  // steps (of one head) before the unit that holds p0
    int tile;                     // that unit
  };

  const Params& p;
  const Shared& sh;
  // cursor
  int64_t at, tb;    // line position; position of the unit row's first step
  int tile, turn;
  // the unit row (the same for all heads) and the unit
  int g, b0, nb, tok0, ntok, slen, nsb, nblk;
  int h, j0, j1;
  bool whole, both;  // not cut; cut and in both tiles
  uint32_t have, act;
  // the step
  int j, key0, keys;
  bool full, own;
  int b, jb, nob, P;  // the sequence whose own block it is

  __device__ __forceinline__ static void prefetch_maps(const Params& p) {
    prefetch_map(&p.ks);
    prefetch_map(&p.q);
    prefetch_map(&p.vs);
    prefetch_map(&p.ko);
    prefetch_map(&p.vo);
  }
  __device__ __forceinline__ static int first_of(const Params& p, int g) {
    return min(max(p.group_start[g], 0), p.B);
  }
  __device__ __forceinline__ static int shared_of(const Params& p, int g) {
    return min(max(p.shared_len[g], 0), p.Sp);
  }
  __device__ __forceinline__ static int prefix_of(const Params& p, int b) {
    return min(max(p.prefix_len[b], 0), p.S - p.N);
  }
  __device__ __forceinline__ static int own_blocks(const Params& p, int b) {
    return (prefix_of(p, b) + p.N + kKeys - 1) / kKeys;
  }
  // prefix of unit row i, the row's number there and which part of a sequence it is
  __device__ __forceinline__ static void prefix_of_row(const Params& p, const Shared& sh, int i,
                                                       int& g, int& k, int& part) {
    k = p.chunks > 1 ? i / p.chunks : i;
    part = i - k * p.chunks;
    int lo = 0, hi = p.groups - 1;  // the last prefix with tiles[g] <= k
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sh.tiles[mid] <= k) lo = mid; else hi = mid - 1;
    }
    g = lo;
    k -= sh.tiles[g];
  }
  // Exclusive running sums over the threads of two values at once; tmp: [64].  Ends with
  // a barrier.
  __device__ __forceinline__ static void scan(int64_t& a, int64_t& b, int64_t* tmp,
                                              int64_t& all_a, int64_t& all_b) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kW = kTaThreads / 32;
    int64_t x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += u;
        y += v;
      }
    }
    if (lane == 31) {
      tmp[warp] = x;
      tmp[32 + warp] = y;
    }
    __syncthreads();
    x -= a;
    y -= b;
    all_a = all_b = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < warp) {
        x += tmp[w];
        y += tmp[32 + w];
      }
      all_a += tmp[w];
      all_b += tmp[32 + w];
    }
    a = x;
    b = y;
    __syncthreads();
  }
  __device__ __forceinline__ static int64_t over(int64_t n, int d) {  // n / d
    return n < ((int64_t)1 << 31) ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
  }
  __device__ static void setup(const Params& p, Shared& sh, void* scratch) {
    const int tid = threadIdx.x;
    int64_t* tmp = reinterpret_cast<int64_t*>(scratch);           // [64]
    int64_t* seqs = tmp + 64;      // own steps before sequence tid * ps, [threads + 1]
    static_assert(kMaxPrefixes < kTaThreads, "a thread per prefix");
    launch_dependents();
    if (tid == 0) p.part.head[blockIdx.x].slot = -1;
    // a thread's sequences and its prefix
    const int ps = (p.B + kTaThreads - 1) / kTaThreads;
    int64_t own = 0, rows = 0, all, total;
    if (tid < p.groups) {
      const int lo = first_of(p, tid), hi = first_of(p, tid + 1);
      sh.firsts[tid] = lo;
      if (tid == p.groups - 1) sh.firsts[tid + 1] = hi;
      sh.slen[tid] = shared_of(p, tid);
      rows = hi > lo ? (uint32_t)(hi - lo + p.spu - 1) / (uint32_t)p.spu : 0;
    }
    for (int b = tid * ps; b < min(p.B, (tid + 1) * ps); ++b) own += own_blocks(p, b);
    scan(own, rows, tmp, all, total);
    seqs[tid] = own;
    if (tid == 0) seqs[kTaThreads] = all;
    if (tid <= p.groups) sh.tiles[tid] = (uint16_t)min(rows, (int64_t)65535);
    __syncthreads();
    auto before = [&](int b) {  // own steps before sequence b
      if (ps == 1) return seqs[b];
      int64_t n = seqs[b / ps];
      for (int x = b / ps * ps; x < b; ++x) n += own_blocks(p, x);
      return n;
    };
    auto steps = [&](int i) {  // of unit row i
      int g, k, part;
      prefix_of_row(p, sh, i, g, k, part);
      const int b0 = sh.firsts[g] + k * p.spu, b1 = min(sh.firsts[g + 1], b0 + p.spu);
      return (sh.slen[g] + kKeys - 1) / kKeys + before(b1) - before(b0);
    };
    const int n = (int)min(total, (int64_t)65535) * p.chunks;
    const int per = (n + kTaThreads - 1) / kTaThreads;
    const int first = min(n, tid * per), last = min(n, first + per);
    int64_t mine = 0, none = 0;
    for (int i = first; i < last; ++i) mine += steps(i);
    const int64_t v = mine;
    scan(mine, none, tmp, all, total);
    const int64_t line = all * p.Hkv;
    int64_t len = over(line + gridDim.x - 1, (int)gridDim.x);
    if (len < kMinSteps) len = kMinSteps;
    const int64_t p0 = min(line, len * blockIdx.x), p1 = min(line, p0 + len);
    if (tid == 0) {
      sh.len = len;
      sh.p0 = p0;
      sh.p1 = p1;
    }
    // the thread whose unit rows hold the piece's first step finds it
    const int64_t want = over(p0, p.Hkv);
    if (p0 < line && mine <= want && want < mine + v) {
      int64_t x = mine;
      int i = first;
      for (; i + 1 < last; ++i) {
        const int64_t s = steps(i);
        if (want < x + s) break;
        x += s;
      }
      sh.tile = i;
      sh.cum = x;
    }
    __syncthreads();
  }
  __device__ __forceinline__ SharedWalk(const Params& p_, const Shared& sh_)
      : p(p_), sh(sh_), at(sh_.p0), tb(sh_.cum * p_.Hkv), tile(sh_.tile), turn(0) {
    if (at < sh.p1) load_rows();
  }

  __device__ __forceinline__ void load_rows() {
    const int lane = threadIdx.x & 31;
    int k, part;
    prefix_of_row(p, sh, tile, g, k, part);
    b0 = sh.firsts[g] + k * p.spu;
    nb = min(p.spu, sh.firsts[g + 1] - b0);
    tok0 = b0 * p.N + part * 2 * p.tpt;
    ntok = p.chunks > 1 ? min(2 * p.tpt, p.N - part * 2 * p.tpt) : nb * p.N;
    slen = sh.slen[g];
    nsb = (slen + kKeys - 1) / kKeys;
    int n = 0;
    for (int i = lane; i < nb; i += 32) n += own_blocks(p, b0 + i);
    nblk = nsb + __reduce_add_sync(0xffffffffu, n);
  }
  __device__ __forceinline__ bool next_unit() {
    if (at >= sh.p1) return false;
    if (at >= tb + (int64_t)p.Hkv * nblk) {
      tb += (int64_t)p.Hkv * nblk;
      ++tile;
      load_rows();
    }
    const int64_t off = at - tb;
    h = (int)over(off, nblk);
    j0 = (int)(off - (int64_t)h * nblk);
    j1 = (int)min((int64_t)nblk, j0 + (sh.p1 - at));
    at += j1 - j0;
    whole = j0 == 0 && j1 == nblk;
    both = !whole && ntok <= p.tpt;
    have = both || ntok > p.tpt ? 3u : 1u;
    ++turn;
    if (threadIdx.x == 0 && j0 == 0 && !whole)
      p.part.head[blockIdx.x] = SharedHead{slot(), tok0, ntok, h, both,
                                           (int)((tb + (int64_t)(h + 1) * nblk - 1) / sh.len)};
    restart();
    return true;
  }
  // a cut unit is the first of its piece (slot 0) or the last (slot 1)
  __device__ __forceinline__ int slot() const { return turn == 1 ? 0 : 1; }
  __device__ __forceinline__ void restart() {
    j = j0 - 1;
    b = -1;
  }
  // the sequence that holds own block k of the unit
  __device__ __forceinline__ void seek(int k) {
    const int lane = threadIdx.x & 31;
    for (int i0 = 0;; i0 += 32) {
      const int mine = i0 + lane < nb ? own_blocks(p, b0 + i0 + lane) : 0;
      int s = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, k < s);
      if (m || i0 + 32 >= nb) {
        const int src = m ? __ffs(m) - 1 : 0;
        b = b0 + i0 + src;
        jb = k - __shfl_sync(0xffffffffu, s - mine, src);
        return;
      }
      k -= __shfl_sync(0xffffffffu, s, 31);
    }
  }
  __device__ __forceinline__ bool next_step() {
    if (++j >= j1) return false;
    own = j >= nsb;
    if (!own) {
      key0 = j * kKeys;
      keys = min(kKeys, slen - key0);
      full = keys == kKeys;
      act = both ? 1u << ((j - j0) & 1) : have;
      return true;
    }
    if (b < 0 || ++jb == nob) {  // another sequence
      if (b < 0) {
        seek(j - nsb);
      } else {
        jb = 0;
        ++b;
      }
      P = prefix_of(p, b);
      nob = (P + p.N + kKeys - 1) / kKeys;
    }
    key0 = jb * kKeys;
    keys = min(kKeys, P + p.N - key0);
    full = nb == 1 && key0 + kKeys <= P;
    if (both) {
      act = 1u << ((j - j0) & 1);
    } else {
      const int lo = b * p.N - tok0;  // the sequence's tokens in the unit
      act = (lo < p.tpt ? 1u : 0u) | (lo + p.N > p.tpt ? 2u : 0u);
      act &= have;
    }
    return true;
  }
  __device__ __forceinline__ uint32_t q_bytes() const { return (uint32_t)(p.tpt * p.G * 128); }
  __device__ __forceinline__ void load_q(int t, uint32_t dst, int x, uint64_t* bar) const {
    tma3d(dst, &p.q, x, h * p.G, tok0 + (both ? 0 : t * p.tpt), bar);
  }
  __device__ __forceinline__ void load_k(uint32_t dst, int x, uint64_t* bar) const {
    tma3d(dst, own ? &p.ko : &p.ks, x, key0, (own ? b : g) * p.Hkv + h, bar);
  }
  __device__ __forceinline__ void load_v(uint32_t dst, int x, uint64_t* bar) const {
    tma3d(dst, own ? &p.vo : &p.vs, x, key0, (own ? b : g) * p.Hkv + h, bar);
  }

  struct Row {
    int r, tok, head;  // row of the tile, token in the tile, head in the group
    int token, seq;
    bool valid;
    uint64_t mb;       // drafted keys it sees
    float mul;
    int64_t dst;       // row of the partial results
    uint4* rows[4];    // rows of out that this lane helps to write
    __device__ __forceinline__ Row(const Params& p, int r_)
        : r(r_), tok(r_ / p.G), head(r_ % p.G) {}
  };
  __device__ __forceinline__ void set_row(Row& row, int t) const {
    const int i = (both ? 0 : t * p.tpt) + row.tok;
    row.valid = row.tok < p.tpt && i < ntok;
    row.token = row.valid ? tok0 + i : 0;
    row.seq = row.token / p.N;
    row.mb = row.valid ? p.mask_bits[row.token] & (p.N >= 64 ? ~0ull : (1ull << p.N) - 1ull) : 0ull;
  }
  __device__ __forceinline__ bool warp_blind(const Row& row) const {
    if (!own || full) return false;
    return !__any_sync(0xffffffffu, row.valid && row.seq == b);
  }
  // visibility of the step's keys 32 i .. 32 i + 31
  __device__ __forceinline__ uint32_t word(const Row& row, int i) const {
    const int k0 = key0 + 32 * i;
    const int end = (own ? P : slen) - k0;
    const uint32_t pre = end >= 32 ? ~0u : (end <= 0 ? 0u : (1u << end) - 1u);
    if (!own) return pre;
    if (!row.valid || row.seq != b) return 0u;
    const int off = k0 - P;
    const uint32_t dr = off >= 0 ? (off < 64 ? (uint32_t)(row.mb >> off) : 0u)
                                 : (off > -32 ? (uint32_t)(row.mb << -off) : 0u);
    return pre | dr;
  }
  __device__ __forceinline__ void hide(const Row& row, int half, float (&s)[kHalfKeys]) const {
#pragma unroll
    for (int i = 0; i < kHalfKeys / 32; ++i) {
      const uint32_t w = word(row, 2 * half + i);
#pragma unroll
      for (int e = 0; e < 32; ++e) s[32 * i + e] = (w >> e) & 1u ? s[32 * i + e] : neg_inf();
    }
  }
  __device__ __forceinline__ bool sees(const Row& row, int i) const {
    return row.valid && ((word(row, i >> 5) >> (i & 31)) & 1u);
  }
};

template <int D>
struct SharedWalkD : SharedWalk {
  using SharedWalk::SharedWalk;
  __device__ __forceinline__ int64_t place(int i) const {  // key i of the step
    return own ? (((int64_t)b * p.Hkv + h) * p.S + key0 + i) * D
               : (((int64_t)g * p.Hkv + h) * p.Sp + key0 + i) * D;
  }
  __device__ __forceinline__ const uint16_t* value(int i) const {
    return (own ? p.vo_ptr : p.vs_ptr) + place(i);
  }
  __device__ __forceinline__ const uint16_t* key(int i) const {
    return (own ? p.ko_ptr : p.ks_ptr) + place(i);
  }
  __device__ __forceinline__ const uint16_t* query(const Row& row) const {
    return p.q_ptr + ((int64_t)row.token * p.Hq + h * p.G + row.head) * D;
  }
  __device__ __forceinline__ void begin_finish(Row& row, int t, float mref, float l) const {
    if (!whole) {
      const int64_t s = ((int64_t)blockIdx.x * 2 + slot()) * 2 + t;
      p.part.ml[s * kRows + row.r] = make_float2(mref, l);
      row.dst = s * (D / 4) * kRows + row.r;
      return;
    }
    row.mul = l == 0.f ? 0.f : 1.f / l;
    const int64_t at_ = (int64_t)row.token * p.Hq + h * p.G + row.head;
    share_rows(row.valid ? reinterpret_cast<uint4*>(p.out + at_ * D) : nullptr, row.rows);
    if (row.valid && p.lse) p.lse[at_] = mref + log2f(l);
  }
  __device__ __forceinline__ void finish(Row& row, int, int c, const float (&o)[32]) const {
    if (!whole) {  // 16 bytes of 32 rows side by side
#pragma unroll
      for (int v = 0; v < 8; ++v)
        p.part.o[row.dst + (8 * c + v) * kRows] =
            make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
      return;
    }
    uint4 v[4];
    pack_row(o, row.mul, v);
    store_rows(row.rows, v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row.rows[i]) row.rows[i] += 4;  // the next 32 dims
  }
};

// Joins the pieces of cut units: CTA (cut unit, 8 head dims), thread (share of the pieces,
// tile, row).  All partial results of a row are weighted against one reference, so their
// sums over the shares (and over the tiles that hold the same rows) simply add up.
// Every thread has kAhead pieces' loads in flight, the first before the references are
// exchanged.  With few units of many pieces latency is what it costs, and two shares of
// four loads at a time are quickest (8 units of 19 pieces, D 128: 8.4 us of a kernel,
// 13.2 with one share and a load at a time).  With many units of two or three pieces it
// is the number of threads: one share (128 units, 60-node trees behind 8 K keys: the
// whole call 125 us, 145 with two).
template <int D, int kShares, int kAhead>
__global__ void __launch_bounds__(kShares * 2 * kRows)
    shared_join(SharedPart part, int pieces, int tpt, int G, int Hq, uint16_t* __restrict__ out,
                float* __restrict__ lse) {
  constexpr int kGroups = 2 * kShares;
  __shared__ float top[kGroups][kRows], sum[kGroups][9][kRows];
  __shared__ int cut, before[8];
  const int tid = threadIdx.x, lane = tid & 31;
  const int r = tid % kRows, group = tid / kRows, t = group & 1, share = group >> 1;
  grid_dependency_wait();
  // the blockIdx.x-th piece in which a cut unit begins
  bool have = false;
  if (tid < 256) {  // (a thread per piece)
    have = tid < pieces && part.head[tid].slot >= 0;
    const uint32_t b = __ballot_sync(0xffffffffu, have);
    if (lane == 0) before[tid >> 5] = __popc(b);
    if (tid == 0) cut = -1;
    __syncthreads();
    int n = __popc(b & ((1u << lane) - 1u));
    for (int w = 0; w < tid >> 5; ++w) n += before[w];
    if (have && n == (int)blockIdx.x) cut = tid;
  } else {
    __syncthreads();
  }
  __syncthreads();
  const int c0 = cut;
  if (c0 < 0) return;
  const SharedHead u = part.head[c0];
  auto place = [&](int c) { return ((int64_t)c * 2 + (c == c0 ? u.slot : 0)) * 2 + t; };
  float M = neg_inf();
#pragma unroll 8
  for (int c = c0 + share; c <= u.last; c += kShares) M = fmaxf(M, part.ml[place(c) * kRows + r].x);
  float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float2 ml[kAhead];
  float4 x[kAhead], y[kAhead];
  auto load = [&](int c) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      ml[i] = make_float2(neg_inf(), 0.f);
      x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + kShares * i > u.last) continue;
      const int64_t s = place(c + kShares * i);
      const float4* src = part.o + (s * (D / 4) + 2 * blockIdx.y) * kRows + r;
      ml[i] = part.ml[s * kRows + r];
      x[i] = src[0];
      y[i] = src[kRows];
    }
  };
  load(c0 + share);
  top[group][r] = M;
  __syncthreads();
#pragma unroll
  for (int g = 0; g < kGroups; ++g)
    if (u.both || (g & 1) == t) M = fmaxf(M, top[g][r]);
  const float ref = M == neg_inf() ? 0.f : M;
  for (int c = c0 + share; c <= u.last; c += kShares * kAhead) {
    if (c != c0 + share) load(c);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // (0 for a piece that saw nothing, and for one far below the others: what is
      // infinite there becomes NaN, as it does inside a piece)
      const float w = ex2(ml[i].x - ref);
      l = fmaf(ml[i].y, w, l);
      o[0] = fmaf(x[i].x, w, o[0]); o[1] = fmaf(x[i].y, w, o[1]);
      o[2] = fmaf(x[i].z, w, o[2]); o[3] = fmaf(x[i].w, w, o[3]);
      o[4] = fmaf(y[i].x, w, o[4]); o[5] = fmaf(y[i].y, w, o[5]);
      o[6] = fmaf(y[i].z, w, o[6]); o[7] = fmaf(y[i].w, w, o[7]);
    }
  }
  sum[group][8][r] = l;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[group][i][r] = o[i];
  __syncthreads();
  if (share > 0 || (u.both && t == 1)) return;
  const int tok = r / G, i = (u.both ? 0 : t * tpt) + tok;
  if (tok >= tpt || i >= u.ntok) return;
#pragma unroll
  for (int g = 1; g < kGroups; ++g)
    if (g != t && (u.both || (g & 1) == t)) {
      l += sum[g][8][r];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += sum[g][e][r];
    }
  const int64_t row = (int64_t)(u.tok0 + i) * Hq + u.h * G + r % G;
  const float mul = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint4*>(out + row * D + 8 * blockIdx.y) =
      make_uint4(pack_bf16x2(o[0] * mul, o[1] * mul), pack_bf16x2(o[2] * mul, o[3] * mul),
                 pack_bf16x2(o[4] * mul, o[5] * mul), pack_bf16x2(o[6] * mul, o[7] * mul));
  if (lse && blockIdx.y == 0) lse[row] = M + log2f(l);
}

// Sizes of a call: how rows are packed, and how many pieces the line can have.
struct SharedPlan {
  int G, tpt, spu, chunks, pieces;
  int cuts;  // units that can be cut, at most
  size_t off_ml, off_o, bytes;
};
bool shared_sizes_ok(int B, int N, int Hq, int Hkv, int groups, int Sp, int S) {
  return B >= 0 && B <= 65535 && N >= 1 && N <= 64 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 &&
         Hq / Hkv <= kRows && groups >= 1 && groups <= kMaxPrefixes && Sp >= 0 &&
         Sp <= SPEC_MAX_POSITIONS && S >= N && S <= SPEC_MAX_POSITIONS &&
         (int64_t)B * Hkv < (int64_t)1 << 31 && (int64_t)groups * Hkv < (int64_t)1 << 31;
}
SharedPlan shared_plan(int B, int N, int Hq, int Hkv, int D, int groups, int Sp, int S) {
  SharedPlan s;
  s.G = Hq / Hkv;
  s.tpt = kRows / s.G;
  s.spu = N <= 2 * s.tpt ? 2 * s.tpt / N : 1;
  s.chunks = (N + 2 * s.tpt - 1) / (2 * s.tpt);
  int64_t tiles = s.chunks > 1 ? (int64_t)B * s.chunks : (int64_t)B / s.spu + groups;
  if (tiles > (int64_t)B * s.chunks) tiles = (int64_t)B * s.chunks;
  const int64_t steps = Hkv * (tiles * ((Sp + kKeys - 1) / kKeys) +
                               (int64_t)B * s.chunks * ((S + kKeys - 1) / kKeys));
  const int64_t most = (steps + kMinSteps - 1) / kMinSteps;
  s.pieces = (int)(most < 1 ? 1 : (most < kTaCtas ? most : kTaCtas));
  const int64_t units = tiles * Hkv;
  s.cuts = (int)(units < s.pieces - 1 ? units : s.pieces - 1);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  s.off_ml = up((size_t)s.pieces * sizeof(SharedHead));
  s.off_o = s.off_ml + up((size_t)s.pieces * 4 * kRows * sizeof(float2));
  s.bytes = s.off_o + (size_t)s.pieces * 4 * kRows * D * sizeof(float);
  return s;
}

template <int D>
int launch(const SharedWalk::Params& prm, const SharedPlan& plan, cudaStream_t st) {
  constexpr int kKs = D == 128 ? 2 : 5, kVs = D == 128 ? 3 : 5;
  using Geo = TileGeo<D, kKs, kVs>;
  constexpr size_t smem =
      (size_t)Geo::kOffCtl + sizeof(TileCtl<kKs, kVs>) + sizeof(SharedWalk::Shared);
  static_assert(smem <= 232448, "shared memory of a block");
  auto kernel = tile_attn<D, kKs, kVs, SharedWalkD<D>>;
  static std::atomic<uint64_t> done{0};
  if (allow_smem((const void*)kernel, (int)smem, done) != cudaSuccess) return SPEC_ERR_CUDA;
  kernel<<<plan.pieces, kTaThreads, smem, st>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  if (plan.cuts == 0) return SPEC_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)plan.cuts, D / 8);
  const bool many = plan.pieces >= 4 * plan.cuts;  // pieces of a unit
  cfg.blockDim = dim3((many ? 4 : 2) * kRows);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto join = many ? shared_join<D, 2, 4> : shared_join<D, 1, 2>;
  return cudaLaunchKernelEx(&cfg, join, prm.part, plan.pieces, prm.tpt, prm.G, prm.Hq, prm.out,
                            prm.lse) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_tree_attention_shared_workspace_bytes(int B, int N, int Hq, int Hkv, int D,
                                                             int groups, int Sp, int S) {
  if (!shared_sizes_ok(B, N, Hq, Hkv, groups, Sp, S) || (D != 64 && D != 128) || B == 0) return 0;
  return shared_plan(B, N, Hq, Hkv, D, groups, Sp, S).bytes;
}

extern "C" int spec_tree_attention_shared(
    const void* q, const void* k_prefix, const void* v_prefix, const int32_t* shared_len,
    const int32_t* group_start, const void* k_cache, const void* v_cache, const int32_t* prefix_len,
    const uint64_t* mask_bits, int B, int N, int Hq, int Hkv, int D, int groups, int Sp, int S,
    float scale, void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  if (!shared_sizes_ok(B, N, Hq, Hkv, groups, Sp, S)) return SPEC_ERR_SHAPE;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !(scale < 3.4e38f)) return SPEC_ERR_ARG;
  if (B == 0) return SPEC_OK;
  if (!q || (Sp > 0 && (!k_prefix || !v_prefix)) || !shared_len || !group_start || !k_cache ||
      !v_cache || !prefix_len || !mask_bits || !out)
    return SPEC_ERR_ARG;
  if (((uintptr_t)q | (uintptr_t)k_prefix | (uintptr_t)v_prefix | (uintptr_t)k_cache |
       (uintptr_t)v_cache | (uintptr_t)out) % 16 != 0 ||
      ((uintptr_t)shared_len | (uintptr_t)group_start | (uintptr_t)prefix_len | (uintptr_t)lse) %
              4 != 0 ||
      (uintptr_t)mask_bits % 8 != 0)
    return SPEC_ERR_ARG;
  const SharedPlan plan = shared_plan(B, N, Hq, Hkv, D, groups, Sp, S);
  if (!workspace || (uintptr_t)workspace % 256 != 0 || ws_bytes < plan.bytes)
    return SPEC_ERR_WORKSPACE;
  SharedWalk::Params prm;
  prm.G = plan.G;
  prm.tpt = plan.tpt;
  prm.spu = plan.spu;
  prm.chunks = plan.chunks;
  const int64_t row = (int64_t)D * 2;
  // (without shared keys their maps stand for the caches and are not used)
  const void *ks = Sp > 0 ? k_prefix : k_cache, *vs = Sp > 0 ? v_prefix : v_cache;
  const int64_t sp = Sp > 0 ? Sp : S, np = Sp > 0 ? (int64_t)groups * Hkv : (int64_t)B * Hkv;
  if (!ta_map(&prm.q, q, D, Hq, (int64_t)B * N, row, Hq * row, prm.G, prm.tpt) ||
      !ta_map(&prm.ks, ks, D, sp, np, row, sp * row, kKeys, 1) ||
      !ta_map(&prm.vs, vs, D, sp, np, row, sp * row, kKeys, 1) ||
      !ta_map(&prm.ko, k_cache, D, S, (int64_t)B * Hkv, row, S * row, kKeys, 1) ||
      !ta_map(&prm.vo, v_cache, D, S, (int64_t)B * Hkv, row, S * row, kKeys, 1))
    return SPEC_ERR_CUDA;
  prm.shared_len = shared_len;
  prm.group_start = group_start;
  prm.prefix_len = prefix_len;
  prm.mask_bits = mask_bits;
  prm.q_ptr = (const uint16_t*)q;
  prm.ks_ptr = (const uint16_t*)ks;
  prm.ko_ptr = (const uint16_t*)k_cache;
  prm.vs_ptr = (const uint16_t*)vs;
  prm.vo_ptr = (const uint16_t*)v_cache;
  prm.out = (uint16_t*)out;
  prm.lse = lse;
  char* ws = (char*)workspace;
  prm.part.head = (SharedHead*)ws;
  prm.part.ml = (float2*)(ws + plan.off_ml);
  prm.part.o = (float4*)(ws + plan.off_o);
  prm.B = B;
  prm.N = N;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.groups = groups;
  prm.Sp = Sp;
  prm.S = S;
  prm.scale_log2 = fminf(scale * kLog2e, FLT_MAX);
  cudaStream_t st = (cudaStream_t)stream;
  return D == 128 ? launch<128>(prm, plan, st) : launch<64>(prm, plan, st);
}
