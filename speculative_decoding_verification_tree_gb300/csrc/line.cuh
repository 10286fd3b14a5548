// A line of work blocks over sequences of different lengths, cut into equal
// pieces: sequence b owns blocks(b) consecutive blocks, in order.
#pragma once

#include "common.cuh"

namespace sv {

// Thread t sums sequences [t per, (t + 1) per); before[t] = blocks before them,
// before[kThreads] = all blocks.  `before` and `tmp` (one value per warp) lie in
// shared memory; ends with a barrier.
template <int kThreads, class F>
__device__ __forceinline__ void scan_line(int B, F blocks, int64_t* before, int64_t* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (B + kThreads - 1) / kThreads;
  const int first = min(B, (int)threadIdx.x * per), last = min(B, first + per);
  int64_t v = 0;
  for (int b = first; b < last; ++b) v += blocks(b);
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < warp; ++w) base += tmp[w];
  before[threadIdx.x] = base + s - v;
  if (threadIdx.x == kThreads - 1) before[kThreads] = base + s;
  __syncthreads();
}
// The sequence that holds block `at` of the line and its first block (a warp's
// lanes together, any `at` below the total).
template <int kThreads, class F>
__device__ __forceinline__ int locate(int B, F blocks, const int64_t* before, int64_t at,
                                      int64_t* start) {
  const int lane = threadIdx.x & 31;
  const int per = (B + kThreads - 1) / kThreads;
  int n = 0;  // threads whose sequences start at or before `at`
  for (int i = lane; i < kThreads; i += 32) n += before[i] <= at;
  n = __reduce_add_sync(0xffffffffu, n);
  // several threads may start there (sequences without blocks): the last of
  // them that has a sequence; threads behind the last sequence start at the total
  int b = (n - 1) * per;
  int64_t x = before[n - 1];
  for (; per > 1;) {
    const int64_t next = x + blocks(b);
    if (at < next) break;
    x = next;
    ++b;
  }
  *start = x;
  return b;
}

}  // namespace sv
