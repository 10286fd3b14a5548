// spec_kv_evict: keep a budget of positions per (sequence, key/value head):
// the most recent ones and, of the others, those of highest accumulated
// attention weight; their rows move together, in order.
//
// Weights are mapped to unsigned keys that order like them (NaN as -inf, -0 as
// +0).  evict_pick, one cluster of CTAs per (sequence, head), reads each weight
// once into shared memory; a thread owns up to 32 consecutive positions, with a
// bit each for kept and undecided.  A radix select over at most four 8-bit
// digits (histograms with a copy per lane residue, summed over the cluster)
// finds the smallest kept key and how many positions holding it are kept (the
// lowest ones); a pass looks at undecided positions only, and there is none
// after the digit whose holders are all kept.  Counts of kept positions, summed
// over lanes, warps and cluster, give each its place; a list in shared memory
// makes the stores of positions and weights contiguous.  Caches too long for a
// cluster's shared memory take evict_select, one CTA that reads the weights from
// memory in every pass.
// The gather: a plane is moved by one thread per word of a kept row when it
// goes to another buffer; in place, a CTA takes a column slice of a (sequence,
// head)'s rows and walks it in chunks, each read whole before it is written.
// That is safe because kept[j] >= j, so a chunk's writes reach no position
// that a later chunk still has to read.
// Bounds and times (pick: latency of its barriers, cluster exchanges and passes;
// gather: HBM): 32 sequences of 2 to 4 K positions, 8 heads, 4-bit rows of D 128,
// half kept (159 MB): 39 us, 13 of them the pick; the gather also pays for the
// other halves of 128-byte lines.  One sequence of 128 K positions, 8 heads, bf16
// rows, 16 K kept (139 MB): 41.5 us, half of them the pick, caches cold; in place
// 62, 36 of them the sweep (33% of DRAM's rate: each CTA's chunks in order, two
// barriers each); the pick of 208 pairs of 45 K weights: 48 us.  (Weights in
// registers, with whole scans in every pass, took 41, 44 and 95: instruction fetch
// of the unrolled code, one CTA per SM.)
#include "kernels.h"
#include "common.cuh"

namespace sv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickMost = 32;     // weights of a thread, at most: a bit each
constexpr int kCopies = 4;        // histogram copies
constexpr int kMaxCluster = 16;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;
constexpr int kSweepUnroll = 4;
constexpr int kSweepMost = 1024;  // threads
constexpr int kMaxPlanes = 9;  // SPEC_EVICT_MAX_PLANES and the weights

// Orders like w, NaN as -inf and -0 as +0 (the sum and the maximum see to that).
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(fmaxf(w + 0.f, neg_inf()));
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ void copy4(float* to, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from)
               : "memory");
}
// The lowest n bits, n clamped to [0, 32].
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}
__device__ __forceinline__ void copy4_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

__global__ void __launch_bounds__(kSelThreads)
    evict_select(const float* __restrict__ weights, const int32_t* __restrict__ length, int Hkv,
                 int S, int budget, int recent, int32_t* __restrict__ kept,
                 int32_t* __restrict__ new_len) {
  launch_dependents();
  __shared__ int hist[256];
  __shared__ int wgt[kSelWarps], weq[kSelWarps];
  __shared__ uint32_t prefix_s;
  __shared__ int want_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t pair = blockIdx.x;
  const int b = (int)(pair / Hkv), h = (int)(pair % Hkv);
  const float* w = weights + pair * S;
  int32_t* kp = kept + pair * budget;
  int len = length[b];
  len = len < 0 ? 0 : (len > S ? S : len);
  const int keep = min(len, budget);
  if (h == 0 && threadIdx.x == 0) new_len[b] = keep;
  if (len <= budget) {
    for (int j = threadIdx.x; j < budget; j += kSelThreads) kp[j] = j < len ? j : -1;
    return;
  }
  const int m = len - recent;         // positions the weights decide about
  const int need = budget - recent;   // of which this many stay
  for (int j = threadIdx.x; j < recent; j += kSelThreads) kp[need + j] = m + j;
  if (need == 0) return;

  // radix select, most significant digit first: after digit d, `prefix` holds
  // the top digits of the need-th largest key
  uint32_t prefix = 0;
  int want = need;  // how many of the keys that share the prefix are kept
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = threadIdx.x; i < m; i += kSelThreads) {
      const uint32_t k = order_key(w[i]);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 255 - 8 l .. 248 - 8 l, largest first
      int cnt[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += cnt[i] = hist[255 - 8 * lane - i];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += u;
      }
      before -= sum;
      if (before < want && want <= before + sum) {
        int left = want - before;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (left > 0 && left <= cnt[i]) {
            prefix_s = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
            want_s = left;
          }
          left -= cnt[i];
        }
      }
    }
    __syncthreads();
    prefix = prefix_s;
    want = want_s;
  }
  // `want` of the positions whose key equals `prefix` are kept, lowest first
  const int run = (m + kSelWarps - 1) / kSelWarps;
  const int lo = min(m, warp * run), hi = min(m, lo + run);
  int gt = 0, eq = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? order_key(w[i]) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < hi && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, i < hi && k == prefix));
  }
  if (lane == 0) {
    wgt[warp] = gt;
    weq[warp] = eq;
  }
  __syncthreads();
  int at = 0, taken = 0;  // kept positions before this warp's run; equal ones among them
  for (int x = 0; x < warp; ++x) {
    const int e = min(weq[x], want - taken);
    at += wgt[x] + e;
    taken += e;
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? order_key(w[i]) : 0u;
    const uint32_t eqm = __ballot_sync(0xffffffffu, i < hi && k == prefix);
    const bool keep_eq = i < hi && k == prefix && taken + __popc(eqm & below) < want;
    const bool on = (i < hi && k > prefix) || keep_eq;
    const uint32_t onm = __ballot_sync(0xffffffffu, on);
    if (on) kp[at + __popc(onm & below)] = i;
    at += __popc(onm);
    taken = min(want, taken + __popc(eqm));
  }
}

// The kept positions of one (sequence, head) and their weights.
// weights_out may be weights: every weight is in shared memory before any is
// written.
__global__ void __launch_bounds__(kPickThreads, 3)
    evict_pick(const float* weights, const int32_t* __restrict__ length, int Hkv, int S,
               int budget, int recent, int64_t S_out, float* weights_out,
               int32_t* __restrict__ kept, int32_t* __restrict__ new_len) {
  launch_dependents();
  extern __shared__ float held[];       // this CTA's weights, then its kept offsets
  __shared__ int hist[2][256];          // this CTA's, by pass parity (read by the cluster)
  __shared__ __align__(16) int copies[256][kCopies];
  __shared__ int total[256];
  // kept for sure | equal to the threshold << 16: of the CTA (read by the cluster), of warps
  __shared__ uint32_t count_s, wcount[kPickWarps];
  __shared__ uint32_t prefix_s;
  __shared__ int want_s;
  __shared__ bool all_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int64_t pair = blockIdx.x / C;
  const int b = (int)(pair / Hkv), h = (int)(pair % Hkv);
  const float* w = weights + pair * S;
  float* wo = weights_out ? weights_out + pair * S_out : nullptr;
  int32_t* kp = kept + pair * budget;
  int len = length[b];
  len = len < 0 ? 0 : (len > S ? S : len);
  if (h == 0 && rank == 0 && threadIdx.x == 0) new_len[b] = min(len, budget);
  if (len <= budget) {  // everything stays
    for (int j = rank * kPickThreads + threadIdx.x; j < budget; j += C * kPickThreads) {
      kp[j] = j < len ? j : -1;
      if (wo && wo != w && j < len) wo[j] = w[j];
    }
    return;  // the whole cluster takes this way
  }
  const int m = len - recent;         // positions the weights decide about
  const int need = budget - recent;   // of which this many stay
  // a thread's run: positions first .. first + steps - 1, laid out an odd number
  // of words apart, so that the lanes' words lie in different banks
  const int steps = (len + C * kPickThreads - 1) / (C * kPickThreads);  // <= kPickMost
  const int stride = steps | 1;
  const int cta0 = rank * kPickThreads * steps;
  const int first = cta0 + threadIdx.x * steps;
  const float* v = held + threadIdx.x * stride;
  {
    int run = warp * 32 + lane / steps, k = lane % steps;  // of the warp's element e
    const int dr = 32 / steps, dk = 32 % steps;
    const int e0 = cta0 + warp * 32 * steps;
    for (int e = lane; e < 32 * steps; e += 32) {
      if (e0 + e < len) copy4(held + run * stride + k, w + e0 + e);
      run += dr;
      k += dk;
      if (k >= steps) k -= steps, ++run;
    }
  }
  copy4_wait();
  __syncwarp();  // a warp holds its lanes' runs
  // bit k: position first + k is kept, or undecided
  uint32_t open = low_bits(min(m - first, steps));
  uint32_t sure = low_bits(min(len - first, steps)) & ~open;

  // radix select, most significant digit first: after digit d, `prefix` holds
  // the top digits of the need-th largest key
  uint32_t prefix = 0, mask = 0;  // mask: its digits so far
  int want = need;  // how many of the keys that share the prefix are kept
  // all holders of the prefix kept: no more digits are needed
  bool all = need == 0;
  for (int pass = 0; pass < 4 && !all; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = threadIdx.x; i < 256 * kCopies; i += kPickThreads) (&copies[0][0])[i] = 0;
    __syncthreads();
    for (uint32_t c = open; c; c &= c - 1) {
      const uint32_t key = order_key(v[__ffs(c) - 1]);
      if ((key & mask) == prefix) {
        atomicAdd(&copies[(key >> shift) & 255u][lane % kCopies], 1);
      } else {
        open ^= c & -c;
        if ((key & mask) > prefix) sure |= c & -c;
      }
    }
    __syncthreads();
    if (threadIdx.x < 256) {
      int sum = 0;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) sum += copies[threadIdx.x][(threadIdx.x + i) % kCopies];
      (C > 1 ? hist[pass & 1] : total)[threadIdx.x] = sum;
    }
    if (C > 1) {
      cluster_sync();
      if (threadIdx.x < 256) {
        const uint32_t at = smem_u32(&hist[pass & 1][threadIdx.x]);
        int part[kMaxCluster];  // the loads in flight together
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          part[r] = r < C ? (int)ld_dsmem_u32(mapa(at, (uint32_t)r)) : 0;
        int sum = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) sum += part[r];
        total[threadIdx.x] = sum;
      }
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 255 - 8 l .. 248 - 8 l, largest first
      int cnt[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += cnt[i] = total[255 - 8 * lane - i];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += u;
      }
      before -= sum;
      if (before < want && want <= before + sum) {
        int left = want - before;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (left > 0 && left <= cnt[i]) {
            prefix_s = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
            want_s = left;
            all_s = left == cnt[i];
          }
          left -= cnt[i];
        }
      }
    }
    __syncthreads();
    prefix = prefix_s;
    want = want_s;
    all = all_s;
    mask |= 255u << shift;
  }
  if (need == 0) prefix = mask = 0xffffffffu;  // above every key: only the recent ones
  // `want` of the positions whose key has the prefix are kept, lowest first
  for (uint32_t c = open; c; c &= c - 1) {
    const uint32_t key = order_key(v[__ffs(c) - 1]) & mask;
    if (key != prefix) {
      open ^= c & -c;
      if (key > prefix) sure |= c & -c;
    }
  }
  const uint32_t mine = __popc(sure) | __popc(open) << 16;  // a CTA's counts fit 16 bits each
  uint32_t upto = mine;  // of the warp's lanes up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) wcount[warp] = upto;
  __syncthreads();
  const uint32_t of_warp = lane < kPickWarps ? wcount[lane] : 0u;
  const uint32_t of_cta = __reduce_add_sync(0xffffffffu, of_warp);
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0u) + upto - mine;
  int at = 0, taken = 0;  // sure ones and equal ones of the CTAs before this one
  if (C > 1) {
    if (threadIdx.x == 0) count_s = of_cta;
    cluster_sync();
    const uint32_t c = lane < rank ? ld_dsmem_u32(mapa(smem_u32(&count_s), (uint32_t)lane)) : 0u;
    at = __reduce_add_sync(0xffffffffu, (int)(c & 0xffffu));
    taken = __reduce_add_sync(0xffffffffu, (int)(c >> 16));
  }
  // the CTA's kept offsets in order, then coalesced stores
  at += min(taken, want);
  const int kept_cta = (int)(of_cta & 0xffffu) + min(taken + (int)(of_cta >> 16), want) -
                       min(taken, want);
  uint16_t* list = reinterpret_cast<uint16_t*>(held + kPickThreads * stride);
  int eq = taken + (int)(before >> 16);  // equal ones before this thread's
  int j = (int)(before & 0xffffu) + min(eq, want) - min(taken, want);
  for (uint32_t c = sure | open; c; c &= c - 1)
    if ((sure & c & -c) || eq++ < want) list[j++] = threadIdx.x * steps + __ffs(c) - 1;
  __syncthreads();
  for (int t = threadIdx.x; t < kept_cta; t += kPickThreads) {
    const int e = list[t];
    kp[at + t] = cta0 + e;
    if (wo) wo[at + t] = held[stride == steps ? e : e + e / steps];
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another reads its counts
}

struct MovePlane {
  const unsigned char* src;
  unsigned char* dst;
  int width;  // bytes of a word: 16, 8, 4 or 1
  int words;  // words per row
};
struct MovePlanes {
  MovePlane p[kMaxPlanes];
};

// A chunk of rows of one (sequence, head) to another buffer.
template <typename W>
__device__ __forceinline__ void gather_rows(const MovePlane& pl, const int32_t* from, int rows,
                                            const unsigned char* src0, unsigned char* dst0) {
  const W* src = reinterpret_cast<const W*>(src0);
  W* dst = reinterpret_cast<W*>(dst0);
  const uint32_t words = (uint32_t)pl.words, total = (uint32_t)rows * words;
  for (uint32_t t0 = threadIdx.x; t0 < total; t0 += kMoveThreads * kMoveUnroll) {
    W v[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const uint32_t t = t0 + u * kMoveThreads;
      if (t < total) {
        const uint32_t r = t / words;
        v[u] = src[(int64_t)from[r] * words + (t - r * words)];
      }
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const uint32_t t = t0 + u * kMoveThreads;
      if (t < total) dst[t] = v[u];
    }
  }
}
// Rows a CTA moves: kMoveUnroll words a thread, and at least one row.
__host__ __device__ constexpr int gather_chunk(int words) {
  const int r = kMoveThreads * kMoveUnroll / words;
  return r < 1 ? 1 : (r > kMoveThreads * 2 ? kMoveThreads * 2 : r);
}
// To another buffer: blockIdx.x = (sequence, head) x chunk, blockIdx.y = plane.
__global__ void __launch_bounds__(kMoveThreads)
    evict_gather(const MovePlanes planes, const int32_t* __restrict__ kept, int64_t pairs,
                 int budget, int64_t S, int64_t S_out) {
  __shared__ int32_t from[kMoveThreads * 2];
  __shared__ int rows_s;
  grid_dependency_wait();
  const MovePlane pl = planes.p[blockIdx.y];
  const int chunk = gather_chunk(pl.words);
  const int chunks = (budget + chunk - 1) / chunk;
  const int64_t pair = blockIdx.x / chunks;
  if (pair >= pairs) return;
  const int j0 = (int)(blockIdx.x % chunks) * chunk;
  const int most = min(chunk, budget - j0);
  if (threadIdx.x == 0) rows_s = 0;
  __syncthreads();
  int mine = 0;
  for (int j = threadIdx.x; j < most; j += kMoveThreads) {
    const int f = kept[pair * budget + j0 + j];
    from[j] = f;
    mine += f >= 0;
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0 && mine) atomicAdd(&rows_s, mine);  // kept rows come first
  __syncthreads();
  const int64_t row = (int64_t)pl.width * pl.words;
  const unsigned char* src = pl.src + pair * S * row;
  unsigned char* dst = pl.dst + (pair * S_out + j0) * row;
  if (pl.width == 16)
    gather_rows<uint4>(pl, from, rows_s, src, dst);
  else if (pl.width == 8)
    gather_rows<uint2>(pl, from, rows_s, src, dst);
  else if (pl.width == 4)
    gather_rows<uint32_t>(pl, from, rows_s, src, dst);
  else
    gather_rows<unsigned char>(pl, from, rows_s, src, dst);
}

// A slice of words w0 .. w0 + nw - 1 of one (sequence, head)'s rows, in place.
template <typename W>
__device__ __forceinline__ void sweep_rows(const MovePlane& pl, const int32_t* __restrict__ kp,
                                           int budget, unsigned char* base0, int w0, int nw) {
  W* base = reinterpret_cast<W*>(base0) + w0;
  // thread t takes word t % nw of rows t / nw, + threads / nw, ... of a chunk
  const int rows = (int)blockDim.x / nw;
  const int tr = threadIdx.x / nw, tw = threadIdx.x % nw;
  W v[2][kSweepUnroll];
  bool move[2][kSweepUnroll];
  auto read = [&](int c, W (&x)[kSweepUnroll], bool (&mv)[kSweepUnroll]) {
#pragma unroll
    for (int u = 0; u < kSweepUnroll; ++u) {
      const int j = (c * kSweepUnroll + u) * rows + tr;
      const int from = tr < rows && j < budget ? kp[j] : -1;
      mv[u] = from >= 0 && from != j;
      if (mv[u]) x[u] = base[(int64_t)from * pl.words + tw];
    }
  };
  auto write = [&](int c, const W (&x)[kSweepUnroll], const bool (&mv)[kSweepUnroll]) {
#pragma unroll
    for (int u = 0; u < kSweepUnroll; ++u)
      if (mv[u]) base[(int64_t)((c * kSweepUnroll + u) * rows + tr) * pl.words + tw] = x[u];
  };
  // chunk c + 1 is read before chunk c is written: its sources lie above every
  // position written until then
  const int chunks = (budget + rows * kSweepUnroll - 1) / (rows * kSweepUnroll);
  read(0, v[0], move[0]);
  for (int c = 0; c < chunks; c += 2) {
    if (c + 1 < chunks) read(c + 1, v[1], move[1]);
    __syncthreads();  // chunk c is read whole
    write(c, v[0], move[0]);
    if (c + 1 >= chunks) break;
    if (c + 2 < chunks) read(c + 2, v[0], move[0]);
    __syncthreads();
    write(c + 1, v[1], move[1]);
  }
}
// In place: blockIdx.x = (sequence, head), blockIdx.y = plane, blockIdx.z = slice of
// at most 32 bytes of the rows.
__global__ void __launch_bounds__(kSweepMost)
    evict_sweep(const MovePlanes planes, const int32_t* __restrict__ kept, int budget, int64_t S) {
  grid_dependency_wait();
  const MovePlane pl = planes.p[blockIdx.y];
  const int per = pl.width == 1 ? 32 : 32 / pl.width;
  const int w0 = blockIdx.z * per;
  const int nw = min(per, pl.words - w0);
  if (nw <= 0) return;
  const int64_t pair = blockIdx.x;
  const int32_t* kp = kept + pair * budget;
  unsigned char* base = pl.dst + pair * S * ((int64_t)pl.width * pl.words);
  if (pl.width == 16)
    sweep_rows<uint4>(pl, kp, budget, base, w0, nw);
  else if (pl.width == 8)
    sweep_rows<uint2>(pl, kp, budget, base, w0, nw);
  else if (pl.width == 4)
    sweep_rows<uint32_t>(pl, kp, budget, base, w0, nw);
  else
    sweep_rows<unsigned char>(pl, kp, budget, base, w0, nw);
}

cudaError_t launch_moves(const MovePlanes& out, int n_out, const MovePlanes& in, int n_in,
                         const int32_t* kept, int64_t pairs, int budget, int S, int S_out,
                         cudaStream_t st) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  if (n_out > 0) {
    int64_t most = 0;
    for (int i = 0; i < n_out; ++i) {
      const int chunk = gather_chunk(out.p[i].words);
      const int64_t c = pairs * ((budget + chunk - 1) / chunk);
      most = most > c ? most : c;
    }
    if (most > 2147483647) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)most, (unsigned)n_out);
    e = cudaLaunchKernelEx(&cfg, evict_gather, out, kept, pairs, budget, (int64_t)S,
                           (int64_t)S_out);
    if (e != cudaSuccess) return e;
  }
  if (n_in > 0) {
    int most = 0;  // slices; rows have at most 65536 bytes
    int64_t ctas = 0;
    for (int i = 0; i < n_in; ++i) {
      const int c = (in.p[i].width * in.p[i].words + 31) / 32;
      most = most > c ? most : c;
      ctas += pairs * c;
    }
    // few CTAs take longer chunks.  The call in place, 1024 / 512 / 256 threads, caches
    // cold: 64 CTAs (4 pairs, 16 K bf16 rows kept) 47 / 60 / 86 us; 128 (8 pairs) 62 /
    // 68 / 95; 256 (16 pairs, 8 K bf16 rows) 58 / 55 / 65; 384 (64 pairs, 8 K 4-bit
    // rows) 65 / 56 / 65; 512 (32 pairs, 4 K bf16 rows) 49 / 47 / 42; 768 (128 pairs, 2
    // K 4-bit rows) 32 / 27 / 25; 1536 (256 pairs) 57 / 47 / 46.  Not the best at 192
    // (32 pairs, 8 K 4-bit rows: 33 / 38 / 51) and 384 of bf16 rows (24 pairs, 8 K
    // rows: 74 / 77 / 63).
    cfg.blockDim = dim3(ctas <= 152 ? kSweepMost : (ctas <= 400 ? kSweepMost / 2 : kMoveThreads));
    cfg.gridDim = dim3((unsigned)pairs, (unsigned)n_in, (unsigned)most);
    e = cudaLaunchKernelEx(&cfg, evict_sweep, in, kept, budget, (int64_t)S);
  }
  return e;
}

// CTAs per cluster of evict_pick for caches of S positions, or 0 (evict_select):
// enough to hold the weights, and more, of at least 2048 weights each (5120 with
// 16, more than the portable size), when there are few (sequence, head) pairs.
// Measured, 8 pairs, 16 K kept of 128 K: 38.5 us in 16 CTAs, 42.9 in 8; 96 K
// 24.4 / 26.3, 64 K 22.9 / 22.6, 32 K 18.8 / 16.5 and 23.7 in 2.
int pick_cluster(int64_t pairs, int S) {
  int C = 1;
  while ((int64_t)C * kPickThreads * kPickMost < S && C < kMaxCluster) C *= 2;
  if ((int64_t)C * kPickThreads * kPickMost < S) return 0;
  while (C < kMaxCluster && pairs * C * 2 <= 152 && S / (2 * C) >= (C < 8 ? 2048 : 5120)) C *= 2;
  return C;
}

// Whether the arrays of a call overlap where they must not: an output with
// another output, or with an input other than the one it replaces in place.
// (A buffer listed twice in place would be moved by two sets of CTAs at once.)
// A buffer that is also an input elsewhere may be moved in place: the weights are
// read, and other buffers written, before planes move; but weights that move in
// place do so first.
struct Range {
  uintptr_t at;
  uint64_t bytes;
  bool meets(const Range& o) const {
    return bytes > 0 && o.bytes > 0 && at < o.at + o.bytes && o.at < at + bytes;
  }
};
bool evict_overlaps(const float* weights, const int32_t* length, int64_t B, int64_t pairs,
                    int64_t S, int budget, int n_planes, const void* const* planes,
                    void* const* planes_out, const int* row_bytes, int64_t S_out,
                    const float* weights_out, const int32_t* kept, const int32_t* new_len) {
  // planes, then the weights; an absent array is empty
  Range in[kMaxPlanes], out[kMaxPlanes];
  for (int i = 0; i < n_planes; ++i) {
    in[i] = {(uintptr_t)planes[i], (uint64_t)(pairs * S) * row_bytes[i]};
    out[i] = {(uintptr_t)planes_out[i], (uint64_t)(pairs * S_out) * row_bytes[i]};
  }
  in[n_planes] = {(uintptr_t)weights, (uint64_t)(pairs * S) * 4};
  out[n_planes] = {(uintptr_t)weights_out, weights_out ? (uint64_t)(pairs * S_out) * 4 : 0};
  const Range small[3] = {{(uintptr_t)kept, (uint64_t)(pairs * budget) * 4},
                          {(uintptr_t)new_len, (uint64_t)B * 4},
                          {(uintptr_t)length, (uint64_t)B * 4}};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if (small[i].meets(small[j])) return true;
  for (int i = 0; i <= n_planes; ++i) {
    for (const Range& s : small)
      if (out[i].meets(s)) return true;
    // kept and new_len are written while planes and weights are read
    if (in[i].meets(small[0]) || in[i].meets(small[1])) return true;
    for (int j = 0; j <= n_planes; ++j) {
      if (j < i && out[i].meets(out[j])) return true;
      const bool itself =
          in[j].at == out[i].at && (i == j || (i < n_planes && in[j].at == in[i].at));
      if (!itself && out[i].meets(in[j])) return true;
    }
  }
  return false;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int spec_kv_evict(const float* weights, const int32_t* length, int B, int Hkv, int S,
                             int budget, int recent, int n_planes, const void* const* planes,
                             void* const* planes_out, const int* row_bytes, int S_out,
                             float* weights_out, int32_t* kept, int32_t* new_len, void* stream) {
  if (B < 0 || Hkv < 1 || S < 0 || S_out < 0 || S > SPEC_MAX_POSITIONS ||
      S_out > SPEC_MAX_POSITIONS || budget < 1 || budget > S_out || recent < 0 ||
      recent > budget || n_planes < 0 || n_planes > SPEC_EVICT_MAX_PLANES)
    return SPEC_ERR_SHAPE;
  // (sequence, head) pairs and the gather's chunks are grid dimensions
  if ((double)B * Hkv * kMaxCluster > 2147483647.0 ||
      (double)B * Hkv * budget > 2147483647.0 * 512)
    return SPEC_ERR_SHAPE;
  if (n_planes > 0 && (!planes || !planes_out || !row_bytes)) return SPEC_ERR_ARG;
  for (int i = 0; i < n_planes; ++i)
    if (row_bytes[i] < 1 || row_bytes[i] > 65536) return SPEC_ERR_SHAPE;
  if (B == 0) return SPEC_OK;
  if (!weights || !length || !kept || !new_len) return SPEC_ERR_ARG;
  if (((uintptr_t)weights | (uintptr_t)length | (uintptr_t)weights_out | (uintptr_t)kept |
       (uintptr_t)new_len) %
          4 !=
      0)
    return SPEC_ERR_ARG;
  for (int i = 0; i < n_planes; ++i) {
    if (!planes[i] || !planes_out[i]) return SPEC_ERR_ARG;
    if (planes[i] == planes_out[i] && S_out != S) return SPEC_ERR_ARG;
  }
  if (weights_out == weights && S_out != S) return SPEC_ERR_ARG;
  const int64_t pairs = (int64_t)B * Hkv;
  if (evict_overlaps(weights, length, B, pairs, S, budget, n_planes, planes, planes_out, row_bytes,
                     S_out, weights_out, kept, new_len))
    return SPEC_ERR_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const int C = pick_cluster(pairs, S);
  cudaError_t e;
  if (C > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * C));
    cfg.blockDim = dim3(kPickThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const int64_t steps = (S + (int64_t)C * kPickThreads - 1) / ((int64_t)C * kPickThreads);
    constexpr int kBytes = kPickThreads * (int)(sizeof(float) + sizeof(uint16_t));  // of a step
    static std::atomic<uint64_t> done{0};
    e = allow_smem((const void*)evict_pick, kBytes * (kPickMost | 1), done);
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
    if (C > 8) {  // more than the portable cluster size
      e = cudaFuncSetAttribute(evict_pick, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return SPEC_ERR_CUDA;
    }
    cfg.dynamicSmemBytes = (size_t)(steps | 1) * kBytes;
    e = cudaLaunchKernelEx(&cfg, evict_pick, weights, length, Hkv, S, budget, recent,
                           (int64_t)S_out, weights_out, kept, new_len);
  } else {
    evict_select<<<(unsigned)pairs, kSelThreads, 0, st>>>(weights, length, Hkv, S, budget, recent,
                                                          kept, new_len);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  // planes to another buffer and in place; the widest word that fits each
  MovePlanes out, in;
  int n_out = 0, n_in = 0;
  for (int i = 0; i <= n_planes; ++i) {
    const bool is_w = i == n_planes;
    if (is_w && (!weights_out || C > 0)) break;  // evict_pick has moved them
    const void* s = is_w ? (const void*)weights : planes[i];
    void* d = is_w ? (void*)weights_out : planes_out[i];
    const int bytes = is_w ? 4 : row_bytes[i];
    const uint64_t al = (uint64_t)(uintptr_t)s | (uint64_t)(uintptr_t)d | (uint64_t)bytes;
    const int width = al % 16 == 0 ? 16 : (al % 8 == 0 ? 8 : (al % 4 == 0 ? 4 : 1));
    const MovePlane pl = {(const unsigned char*)s, (unsigned char*)d, width, bytes / width};
    if (s == d)
      in.p[n_in++] = pl;
    else
      out.p[n_out++] = pl;
  }
  e = launch_moves(out, n_out, in, n_in, kept, pairs, budget, S, S_out, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
