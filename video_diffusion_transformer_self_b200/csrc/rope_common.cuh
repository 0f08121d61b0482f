// rope_common.cuh -- the RoPE table reads and the rotation shared by the
// passes over Q and K (rope.cu, block.cu, paged.cu).
#pragma once

#include "wan_internal.cuh"

namespace wan {

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t v) {
  float2 r;
  r.x = __uint_as_float(v << 16);
  r.y = __uint_as_float(v & 0xFFFF0000u);
  return r;
}

// {cos, sin} of absolute pairs p0 and p0 + 1 (p0 even) for the token whose
// band rows are tt (time), th (height), tw (width).
__device__ __forceinline__ float4 pair_cs(int p0, const float4* tt,
                                          const float4* th,
                                          const float4* tw) {
  if (p0 + 1 < 22) return __ldg(tt + (p0 >> 1));
  if (p0 >= 22 && p0 + 1 < 43) return __ldg(th + ((p0 - 22) >> 1));
  if (p0 >= 44) return __ldg(tw + ((p0 - 42) >> 1));
  // p0 = 42: pair 42 is the last height pair, pair 43 the first width pair
  const float4 lo = __ldg(th + 10);  // entries 20, 21 -> pair 42 in .x/.y
  const float4 hi = __ldg(tw);       // entries 0 (pad), 1 -> pair 43 in .z/.w
  return make_float4(lo.x, lo.y, hi.z, hi.w);
}

// (x * f * w_pair) rotated by {cos, sin}, packed to bf16x2.
__device__ __forceinline__ uint32_t norm_rot2(uint32_t v, float f, float w0,
                                              float w1, float co, float si) {
  const float2 x = bf16x2_to_float2(v);
  const float a = x.x * f * w0;
  const float b = x.y * f * w1;
  return pack_bf16x2(fmaf(a, co, -b * si), fmaf(a, si, b * co));
}

}  // namespace wan
