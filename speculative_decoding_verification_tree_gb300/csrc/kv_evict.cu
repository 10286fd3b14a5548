// spec_kv_evict: keep a budget of positions per (sequence, key/value head):
// the most recent ones and, of the others, those of highest accumulated
// attention weight; their rows move together, in order.
//
// evict_select, one CTA per (sequence, head): weights are mapped to unsigned
// keys that order like them (NaN as -inf, -0 as +0), a radix select over four
// 8-bit digits finds the smallest kept key and how many positions holding it
// are kept (the lowest ones), and each warp writes the kept positions of its
// run of the line, in order.
// The gather: a plane is moved by one thread per word of a kept row when it
// goes to another buffer; in place, a CTA takes a column slice of a (sequence,
// head)'s rows and walks it in chunks, each read whole before it is written.
// That is safe because kept[j] >= j, so a chunk's writes reach no position
// that a later chunk still has to read.  The weights are one more plane.
#include "kernels.h"
#include "common.cuh"

namespace sv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kSweepUnroll = 4;
constexpr int kMaxPlanes = 9;  // SPEC_EVICT_MAX_PLANES and the weights

__device__ __forceinline__ uint32_t order_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7fffffffu) > 0x7f800000u) u = 0xff800000u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
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

struct MovePlane {
  const unsigned char* src;
  unsigned char* dst;
  int words;  // words of this launch's width per row
};
struct MovePlanes {
  MovePlane p[kMaxPlanes];
};

// To another buffer: one thread per word of a kept row; blockIdx.y = plane.
template <typename W>
__global__ void __launch_bounds__(kMoveThreads)
    evict_gather(const MovePlanes planes, const int32_t* __restrict__ kept, int64_t rows,
                 int budget, int64_t S, int64_t S_out) {
  grid_dependency_wait();
  const MovePlane pl = planes.p[blockIdx.y];
  const int64_t total = rows * pl.words;
  for (int64_t t = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; t < total;
       t += (int64_t)gridDim.x * kMoveThreads) {
    const int64_t r = t / pl.words;
    const int w = (int)(t - r * pl.words);
    const int from = kept[r];
    if (from < 0) continue;
    const int64_t pair = r / budget;
    const int64_t j = r - pair * budget;
    reinterpret_cast<W*>(pl.dst)[(pair * S_out + j) * pl.words + w] =
        reinterpret_cast<const W*>(pl.src)[(pair * S + from) * pl.words + w];
  }
}

// In place: blockIdx.x = (sequence, head), blockIdx.y = plane, blockIdx.z = slice of
// `width` words of the rows.
template <typename W>
__global__ void __launch_bounds__(kMoveThreads)
    evict_sweep(const MovePlanes planes, const int32_t* __restrict__ kept, int budget, int64_t S,
                int width) {
  grid_dependency_wait();
  const MovePlane pl = planes.p[blockIdx.y];
  const int w0 = blockIdx.z * width;
  const int nw = min(width, pl.words - w0);
  if (nw <= 0) return;
  const int64_t pair = blockIdx.x;
  const int32_t* kp = kept + pair * budget;
  W* base = reinterpret_cast<W*>(pl.dst) + pair * S * pl.words + w0;
  // rows of this chunk: thread t takes word t % nw of rows t / nw, + 256 / nw, ...
  const int rows = kMoveThreads / nw;
  const int tr = threadIdx.x / nw, tw = threadIdx.x % nw;
  for (int j0 = 0; j0 < budget; j0 += rows * kSweepUnroll) {
    W v[kSweepUnroll];
    int from[kSweepUnroll];
#pragma unroll
    for (int u = 0; u < kSweepUnroll; ++u) {
      const int j = j0 + u * rows + tr;
      from[u] = tr < rows && j < budget ? kp[j] : -1;
      if (from[u] == j) from[u] = -1;  // already in place
      if (from[u] >= 0) v[u] = base[(int64_t)from[u] * pl.words + tw];
    }
    __syncthreads();  // the chunk is read before any of it is written
#pragma unroll
    for (int u = 0; u < kSweepUnroll; ++u)
      if (from[u] >= 0) base[(int64_t)(j0 + u * rows + tr) * pl.words + tw] = v[u];
    // the next chunk's sources lie above every position written so far
  }
}

template <typename W>
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
    int most = 0;
    for (int i = 0; i < n_out; ++i) most = most > out.p[i].words ? most : out.p[i].words;
    const int64_t want = (pairs * budget * most + kMoveThreads - 1) / kMoveThreads;
    const int64_t cap = 152 * 64;
    cfg.gridDim = dim3((unsigned)(want < cap ? want : cap), (unsigned)n_out);
    e = cudaLaunchKernelEx(&cfg, evict_gather<W>, out, kept, pairs * budget, budget, (int64_t)S,
                           (int64_t)S_out);
    if (e != cudaSuccess) return e;
  }
  if (n_in > 0) {
    int most = 0;
    for (int i = 0; i < n_in; ++i) most = most > in.p[i].words ? most : in.p[i].words;
    const int width = (int)(32 / sizeof(W));  // a 32-byte sector's words (rows: at most 65536 bytes)
    cfg.gridDim = dim3((unsigned)pairs, (unsigned)n_in, (unsigned)((most + width - 1) / width));
    e = cudaLaunchKernelEx(&cfg, evict_sweep<W>, in, kept, budget, (int64_t)S, width);
  }
  return e;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int spec_kv_evict(const float* weights, const int32_t* length, int B, int Hkv, int S,
                             int budget, int recent, int n_planes, const void* const* planes,
                             void* const* planes_out, const int* row_bytes, int S_out,
                             float* weights_out, int32_t* kept, int32_t* new_len, void* stream) {
  if (B < 0 || Hkv < 1 || S < 0 || S_out < 0 || budget < 1 || budget > S_out || recent < 0 ||
      recent > budget || n_planes < 0 || n_planes > SPEC_EVICT_MAX_PLANES)
    return SPEC_ERR_SHAPE;
  if ((double)B * Hkv > 2147483647.0) return SPEC_ERR_SHAPE;
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
  cudaStream_t st = (cudaStream_t)stream;
  evict_select<<<(unsigned)pairs, kSelThreads, 0, st>>>(weights, length, Hkv, S, budget, recent,
                                                        kept, new_len);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  // planes by word width (16, 4 or 1 bytes), to another buffer or in place
  MovePlanes out[3], in[3];
  int n_out[3] = {0, 0, 0}, n_in[3] = {0, 0, 0};
  const int width[3] = {16, 4, 1};
  for (int i = 0; i <= n_planes; ++i) {
    const bool is_w = i == n_planes;
    if (is_w && !weights_out) break;
    const void* s = is_w ? (const void*)weights : planes[i];
    void* d = is_w ? (void*)weights_out : planes_out[i];
    const int bytes = is_w ? 4 : row_bytes[i];
    const uint64_t al = (uint64_t)(uintptr_t)s | (uint64_t)(uintptr_t)d | (uint64_t)bytes;
    const int c = al % 16 == 0 ? 0 : (al % 4 == 0 ? 1 : 2);
    const MovePlane pl = {(const unsigned char*)s, (unsigned char*)d, bytes / width[c]};
    if (s == d)
      in[c].p[n_in[c]++] = pl;
    else
      out[c].p[n_out[c]++] = pl;
  }
  cudaError_t e = cudaSuccess;
  for (int c = 0; c < 3 && e == cudaSuccess; ++c) {
    if (c == 0)
      e = launch_moves<uint4>(out[c], n_out[c], in[c], n_in[c], kept, pairs, budget, S, S_out, st);
    else if (c == 1)
      e = launch_moves<uint32_t>(out[c], n_out[c], in[c], n_in[c], kept, pairs, budget, S, S_out,
                                 st);
    else
      e = launch_moves<unsigned char>(out[c], n_out[c], in[c], n_in[c], kept, pairs, budget, S,
                                      S_out, st);
  }
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
