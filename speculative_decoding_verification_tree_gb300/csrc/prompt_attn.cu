// spec_prompt_attention: causal attention over whole prompts packed one after
// another, with grouped-query heads (tile_attn.cuh has the kernel).
//
//   o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   inside each prompt
//
// A unit is 2 floor(128 / G) consecutive positions of a prompt for one key/value
// head; its steps run from the last visible block of 128 keys down to the first,
// so only the first one or two need a mask.  Units are taken longest first -- by the
// position they end at, over all prompts together -- and dealt to the CTAs in a snake
// (forwards, then backwards), which leaves the CTAs' sums within about one short
// unit of each other without any exchange between them.  Batches of more than
// kLevelMax prompts are taken prompt by prompt (each from its end): there the units of
// many prompts even out, and finding the next longest costs more.  Ordered against not,
// 32 / 8 heads, D 128: 16 prompts of 1 to 4095 tokens 559 us / 607, 32 of 1 to 3000 503 /
// 549, 48 990 / 1002 (of 1 to 200: 45 / 41); 64 1736 / 1672, 128 3261 / 3112, 256 of 1 to
// 1000 1150 / 1062, of 1 to 100 136 / 100.  One of 4000 behind 47 of 200: 177 / 200,
// behind 63: 209 / 192, behind 255 of 100: 254 / 270.
//
// Bound: the tensor pipe and the shared memory that feeds it.  16384 tokens, 32 / 8 heads,
// D 128: 1.44 ms = 1.52 PFLOP/s of visible pairs (88% of cuBLAS's sustained bf16 rate); a
// step of 128 keys and two tiles takes about 3070 cycles, of which the products need 2048
// at the pipe's rate and 2560 at shared memory's (Q and K of S in 64-key halves, V, and the
// copies into the ring).  Prompts of 37 to 4095 tokens: 616 us, 1.24 PFLOP/s: every unit
// adds about 7000 cycles (the first scores, the mask, the last P V and the rows' way out),
// and half of its first step is masked.  1000 tokens: 20 us, 128 units of one CTA each,
// the longest a chain of eight steps.  D 64: the softmax warps, 55 us for prompts of up to
// 2501 tokens at 14 / 2 heads.
#include "tile_attn.cuh"

namespace sv {
namespace {

constexpr int kLevelMax = 48;

struct PromptWalk {
  struct Params {
    CUtensorMap q, k, v;
    const int32_t* seq_start;
    const uint16_t *qptr, *kptr, *vptr;
    uint16_t* out;
    float* lse;
    int64_t q_token, k_token, v_token;  // elements between tokens
    int B, T, Hq, Hkv, G, tpt;  // tpt: tokens per tile
    float scale_log2;
  };
  struct Shared {
    int most;              // units of the longest prompt
    int tiles[kLevelMax];  // units of each prompt, per key/value head
    int starts[kLevelMax + 1];  // (of at most kLevelMax prompts)
  };

  const Params& p;
  const Shared& sh;
  // the place in the order of units
  int turn;           // units this CTA has taken
  int64_t at;         // unit, counted from the cursor
  int level, seq0;    // cursor: level (ordered by length) or first prompt of a chunk
  // the unit
  int a, L, pos0, h, nblk;
  uint32_t have, act;
  // the step
  int j, key0, keys;
  bool full;

  __device__ __forceinline__ static int start_of(const Params& p, int b) {
    return min(max(p.seq_start[b], 0), p.T);
  }
  __device__ __forceinline__ static int tiles_of(const Params& p, int b) {
    const int n = start_of(p, b + 1) - start_of(p, b);
    return n <= 0 ? 0 : (n - 1) / (2 * p.tpt) + 1;
  }
  __device__ __forceinline__ static void prefetch_maps(const Params& p) {
    prefetch_map(&p.k);
    prefetch_map(&p.q);
    prefetch_map(&p.v);
  }
  // n / d for 0 <= n, 0 < d
  __device__ __forceinline__ static int64_t over(int64_t n, int64_t d) {
    return n < ((int64_t)1 << 31) && d < ((int64_t)1 << 31) ? (int64_t)((uint32_t)n / (uint32_t)d)
                                                             : n / d;
  }
  __device__ __forceinline__ static void setup(const Params& p, Shared& sh, void*) {
    if (threadIdx.x == 0) sh.most = 0;
    __syncthreads();
    if (p.B <= kLevelMax)
      for (int b = threadIdx.x; b <= p.B; b += kTaThreads) {
        sh.starts[b] = start_of(p, b);
        if (b == p.B) break;
        const int n = tiles_of(p, b);
        sh.tiles[b] = n;
        atomicMax(&sh.most, n);
      }
    __syncthreads();
  }
  __device__ __forceinline__ PromptWalk(const Params& p_, const Shared& sh_)
      : p(p_), sh(sh_), turn(0), at(0), level(sh_.most - 1), seq0(0) {}

  // takes unit `tile` of prompt b, key/value head `head`
  __device__ __forceinline__ void take(int b, int tile, int head) {
    const bool held = p.B <= kLevelMax;
    a = held ? sh.starts[b] : start_of(p, b);
    L = (held ? sh.starts[b + 1] : start_of(p, b + 1)) - a;
    pos0 = tile * 2 * p.tpt;
    h = head;
    have = pos0 + p.tpt < L ? 3u : 1u;
    restart();
  }
  __device__ __forceinline__ void restart() {
    nblk = (min(L, pos0 + 2 * p.tpt) + kKeys - 1) / kKeys;
    j = nblk;
  }
  __device__ __forceinline__ bool next_unit() {
    const int lane = threadIdx.x & 31;
    // units c, 2 g - 1 - c, 2 g + c, ... of g CTAs
    const int c = blockIdx.x, g = gridDim.x;
    at += turn == 0 ? c : ((turn & 1) ? 2 * g - 1 - 2 * c : 1 + 2 * c);
    ++turn;
    if (p.B <= kLevelMax) {
      // level i: unit i of every prompt that has one; these are the same prompts
      // over a run of levels until a prompt's length lies between
      while (level >= 0) {
        int n = 0, below = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
          const int x = b0 + lane < p.B ? sh.tiles[b0 + lane] : 0;
          n += __popc(__ballot_sync(0xffffffffu, x > level));
          below = max(below, x <= level ? x : 0);
        }
        below = __reduce_max_sync(0xffffffffu, below);
        const int64_t per = (int64_t)n * p.Hkv;
        if (at < per * (level - below + 1)) {
          const int down = (int)over(at, per);
          level -= down;
          at -= per * down;
          int k = (int)at / p.Hkv;  // the k-th prompt that has this level
          for (int b0 = 0; b0 < p.B; b0 += 32) {
            const uint32_t m =
                __ballot_sync(0xffffffffu, b0 + lane < p.B && sh.tiles[b0 + lane] > level);
            if (k < __popc(m)) {
              // the lane whose bit has k set ones below it
              const uint32_t at_k = __ballot_sync(
                  0xffffffffu, ((m >> lane) & 1u) && __popc(m & ((1u << lane) - 1u)) == k);
              take(b0 + __ffs(at_k) - 1, level, (int)at % p.Hkv);
              return true;
            }
            k -= __popc(m);
          }
          return false;
        }
        at -= per * (level - below + 1);
        level = below - 1;
      }
      return false;
    }
    for (; seq0 < p.B; seq0 += 32) {
      const int b = seq0 + lane;
      const int n = b < p.B ? tiles_of(p, b) : 0;
      int64_t s = (int64_t)n * p.Hkv;
      const int64_t own = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, at < s);
      if (m) {
        const int src = __ffs(m) - 1;
        const int in = (int)(at - __shfl_sync(0xffffffffu, s - own, src));
        take(seq0 + src, __shfl_sync(0xffffffffu, n, src) - 1 - in / p.Hkv, in % p.Hkv);
        return true;
      }
      at -= __shfl_sync(0xffffffffu, s, 31);
    }
    return false;
  }
  __device__ __forceinline__ bool next_step() {
    if (--j < 0) return false;
    key0 = j * kKeys;
    keys = min(kKeys, L - key0);
    // tile 0 ends before this block?
    act = (have & 2u) | (key0 < pos0 + p.tpt ? 1u : 0u);
    full = key0 + kKeys - 1 <= pos0;
    return true;
  }
  __device__ __forceinline__ uint32_t q_bytes() const { return (uint32_t)(p.tpt * p.G * 128); }
  __device__ __forceinline__ void load_q(int t, uint32_t dst, int x, uint64_t* bar) const {
    tma3d(dst, &p.q, x, h * p.G, a + pos0 + t * p.tpt, bar);
  }
  __device__ __forceinline__ void load_k(uint32_t dst, int x, uint64_t* bar) const {
    tma3d(dst, &p.k, x, h, a + key0, bar);
  }
  __device__ __forceinline__ void load_v(uint32_t dst, int x, uint64_t* bar) const {
    tma3d(dst, &p.v, x, h, a + key0, bar);
  }

  struct Row {
    int tok, head;   // token in the tile, head in the group
    int pos;         // position in the prompt
    bool valid;
    float mul;
    uint4* dst[4];   // rows of out that this lane helps to write
    __device__ __forceinline__ Row(const Params& p, int r)
        : tok(r / p.G), head(r % p.G) {}
  };
  __device__ __forceinline__ void set_row(Row& row, int t) const {
    row.pos = pos0 + t * p.tpt + row.tok;
    row.valid = row.tok < p.tpt && row.pos < L;
  }
  __device__ __forceinline__ bool warp_blind(const Row&) const { return false; }
  __device__ __forceinline__ void hide(const Row& row, int half, float (&s)[kHalfKeys]) const {
    const int lim = row.pos - key0 - kHalfKeys * half;
#pragma unroll
    for (int i = 0; i < kHalfKeys; ++i) s[i] = i <= lim ? s[i] : neg_inf();
  }
  __device__ __forceinline__ bool sees(const Row& row, int i) const {
    return row.valid && key0 + i <= row.pos;
  }
};

// The head dim is the kernel's: these two know it.
template <int D>
struct PromptWalkD : PromptWalk {
  using PromptWalk::PromptWalk;
  __device__ __forceinline__ const uint16_t* value(int i) const {
    return p.vptr + (int64_t)(a + key0 + i) * p.v_token + (int64_t)h * D;
  }
  __device__ __forceinline__ const uint16_t* key(int i) const {
    return p.kptr + (int64_t)(a + key0 + i) * p.k_token + (int64_t)h * D;
  }
  __device__ __forceinline__ const uint16_t* query(const Row& row) const {
    return p.qptr + (int64_t)(a + row.pos) * p.q_token + (int64_t)(h * p.G + row.head) * D;
  }
  __device__ __forceinline__ void begin_finish(Row& row, int, float mref, float l) const {
    row.mul = l == 0.f ? 0.f : 1.f / l;
    const int64_t at_ = (int64_t)(a + row.pos) * p.Hq + h * p.G + row.head;
    share_rows(row.valid ? reinterpret_cast<uint4*>(p.out + at_ * D) : nullptr, row.dst);
    if (row.valid && p.lse) p.lse[at_] = mref + log2f(l);
  }
  __device__ __forceinline__ void finish(Row& row, int, int, const float (&o)[32]) const {
    uint4 v[4];
    pack_row(o, row.mul, v);
    store_rows(row.dst, v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row.dst[i]) row.dst[i] += 4;  // the next 32 dims
  }
};

template <int D>
int launch(const PromptWalk::Params& prm, cudaStream_t st) {
  constexpr int kKs = D == 128 ? 2 : 5, kVs = D == 128 ? 3 : 5;
  using Geo = TileGeo<D, kKs, kVs>;
  constexpr size_t smem =
      (size_t)Geo::kOffCtl + sizeof(TileCtl<kKs, kVs>) + sizeof(PromptWalk::Shared);
  static_assert(smem <= 232448, "shared memory of a block");
  auto kernel = tile_attn<D, kKs, kVs, PromptWalkD<D>>;
  static std::atomic<uint64_t> done{0};
  if (allow_smem((const void*)kernel, (int)smem, done) != cudaSuccess) return SPEC_ERR_CUDA;
  const int64_t units = ((int64_t)prm.T / (2 * prm.tpt) + prm.B) * prm.Hkv;
  const int grid = (int)(units < kTaCtas ? units : kTaCtas);
  kernel<<<grid, kTaThreads, smem, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int spec_prompt_attention(const void* q, int64_t q_token, const void* k, int64_t k_token,
                                     const void* v, int64_t v_token, const int32_t* seq_start,
                                     int B, int T, int Hq, int Hkv, int D, float scale, void* out,
                                     float* lse, void* stream) {
  if (B < 0 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > kRows)
    return SPEC_ERR_SHAPE;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (q_token < (int64_t)Hq * D || k_token < (int64_t)Hkv * D || v_token < (int64_t)Hkv * D ||
      q_token >= (int64_t)1 << 38 || k_token >= (int64_t)1 << 38 || v_token >= (int64_t)1 << 38)
    return SPEC_ERR_SHAPE;
  if ((q_token | k_token | v_token) % 8 != 0) return SPEC_ERR_UNSUPPORTED;
  // positions (and the 128 keys that a copy may start before the end) are 32-bit
  if (T > SPEC_MAX_POSITIONS || (int64_t)Hq > SPEC_MAX_POSITIONS) return SPEC_ERR_SHAPE;
  if (!(scale > 0.f) || !(scale < 3.4e38f)) return SPEC_ERR_ARG;
  if (B == 0 || T == 0) return SPEC_OK;
  if (!q || !k || !v || !seq_start || !out) return SPEC_ERR_ARG;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out) % 16 != 0 ||
      (uintptr_t)seq_start % 4 != 0 || (uintptr_t)lse % 4 != 0)
    return SPEC_ERR_ARG;
  PromptWalk::Params prm;
  prm.G = Hq / Hkv;
  prm.tpt = kRows / prm.G;
  if (!ta_map(&prm.q, q, D, Hq, T, (int64_t)D * 2, q_token * 2, prm.G, prm.tpt) ||
      !ta_map(&prm.k, k, D, Hkv, T, (int64_t)D * 2, k_token * 2, 1, kKeys) ||
      !ta_map(&prm.v, v, D, Hkv, T, (int64_t)D * 2, v_token * 2, 1, kKeys))
    return SPEC_ERR_CUDA;
  prm.seq_start = seq_start;
  prm.qptr = (const uint16_t*)q;
  prm.kptr = (const uint16_t*)k;
  prm.vptr = (const uint16_t*)v;
  prm.out = (uint16_t*)out;
  prm.lse = lse;
  prm.q_token = q_token;
  prm.k_token = k_token;
  prm.v_token = v_token;
  prm.B = B;
  prm.T = T;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.scale_log2 = fminf(scale * kLog2e, FLT_MAX);
  cudaStream_t st = (cudaStream_t)stream;
  return D == 128 ? launch<128>(prm, st) : launch<64>(prm, st);
}
