// Attention over the 4-bit cache: what its kernels share on the host side.
#pragma once

#include "kernels.h"

namespace sv {

struct Kv4Attn {
  const uint16_t* q;
  const uint8_t *kc, *ks, *vc, *vs;
  const int32_t* prefix_len;
  const uint64_t* mask_bits;
  int B, N, Hq, Hkv, S, R;  // R: query rows per key/value head
  ScoreScale scale;  // scale log2(e) k_unit
  float v_unit;
  uint16_t* out;
  float* lse;  // or null
};

// The tensor-core kernel for many rows per key/value head (kv4_attn_tc.cu): its
// partial results' bytes and its launch.
size_t kv4_tc_ws(int B, int Hkv, int R, int D, int S);
cudaError_t launch_kv4_tc(const Kv4Attn& a, int D, void* ws, cudaStream_t st);

}  // namespace sv
