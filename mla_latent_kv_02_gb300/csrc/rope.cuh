// Device side of the decoupled RoPE: one bf16 pair turned by a table entry.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace mla {
namespace dev {

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Pair (x0, x1) turned by (c, s) in fp32, rounded to a bf16 pair.
__device__ __forceinline__ uint32_t rotate_pair(uint32_t x, float2 cs) {
  const float x0 = bf16_lo(x), x1 = bf16_hi(x);
  const float y0 = fmaf(x0, cs.x, -x1 * cs.y);
  const float y1 = fmaf(x0, cs.y, x1 * cs.x);
  return pack_bf16x2(y0, y1);
}

// Four pairs (a uint4) turned by the four table entries t0, t1 (two each).
__device__ __forceinline__ uint4 rotate_pairs4(uint4 x, float4 t0, float4 t1) {
  uint4 y;
  y.x = rotate_pair(x.x, make_float2(t0.x, t0.y));
  y.y = rotate_pair(x.y, make_float2(t0.z, t0.w));
  y.z = rotate_pair(x.z, make_float2(t1.x, t1.y));
  y.w = rotate_pair(x.w, make_float2(t1.z, t1.w));
  return y;
}

}  // namespace dev
}  // namespace mla
