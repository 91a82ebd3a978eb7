// Rotary positions: the kernel's arguments, shared with the host side.
#pragma once

#include "oscar_internal.cuh"

namespace oscar {

struct RopeArgs {
  uint64_t turn[64];           // speeds, in 2^-64 turns a position
  const __nv_bfloat16* qkv;    // [B·T] rows of Hq + 2 Hkv heads, `row` elements apart
  long long row;
  const int32_t* positions;    // [B]
  const __nv_bfloat16* gamma_q;  // [128], null without norm
  const __nv_bfloat16* gamma_k;
  __nv_bfloat16 *q, *k, *v;
  float eps, size;
  int B, T, Hq, Hkv, layout, dims;
  int parts;  // warps that share a token
};
cudaError_t launch_rope(RopeArgs a, int num_sms, cudaStream_t st, Profiler* prof);

}  // namespace oscar
