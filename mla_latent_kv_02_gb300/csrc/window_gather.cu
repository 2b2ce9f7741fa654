// Packed gather of the tokens that a chunk under a sliding window with sinks
// reads: of each sequence its sinks and the tokens from its first query row's
// window on, one warp per token, from the bf16 or the FP8 cache to bf16 rows
// (the FP8 latent as code * 2^k, exact in bf16).  HBM-bound: 1152 or 644
// bytes read and 1152 written per token kept.  Rows between two sequences are
// zeros.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace wgather {

using namespace mla::dev;

constexpr int kRowVec = 72;  // 576 bf16 = 72 x 16 B
constexpr int kWarps = 8;

template <bool kF8>
__global__ void __launch_bounds__(kWarps * 32)
    gather_window_kernel(const uint8_t* __restrict__ cache, const float* __restrict__ scales,
                         const __grid_constant__ WindowGather g, uint4* __restrict__ out) {
  if (threadIdx.x == 0) grid_launch_dependents();  // the expansion sets itself up meanwhile
  const int lane = threadIdx.x & 31;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < g.total;
       t += (int64_t)gridDim.x * kWarps) {
    int lo = 0, hi = g.nb - 1;  // the last sequence whose offset is <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (g.off[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    int32_t j = (int32_t)(t - g.off[lo]);
    if (j >= g.n[lo]) {  // between this sequence's rows and the next one's
      for (int k = lane; k < kRowVec; k += 32) out[t * kRowVec + k] = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    if (j >= g.cut[lo]) j += g.shift[lo];
    const int32_t pid = __ldg(g.block_table + (int64_t)g.b[lo] * g.max_pages + j / MLA_PAGE_SIZE);
    if (pid < 0 || (int64_t)pid >= g.num_pages) {
      if (lane == 0) atomicOr(g.dev_err, (int32_t)MLA_DEVERR_PAGE_OOB);
      continue;
    }
    const int64_t slot = (int64_t)pid * MLA_PAGE_SIZE + j % MLA_PAGE_SIZE;
    uint4* dst = out + t * kRowVec;
    if constexpr (kF8) {
      const uint8_t* row = cache + slot * kFp8RowBytes;
      const Fp8Scale sc = fp8_row_scale(__ldg(scales + slot));
      const uint4 c = __ldg(reinterpret_cast<const uint4*>(row) + lane);  // codes [16 lane, 16 lane + 16)
      dst[2 * lane] = dequant8(make_uint2(c.x, c.y), sc);
      dst[2 * lane + 1] = dequant8(make_uint2(c.z, c.w), sc);
      if (lane < 8) dst[64 + lane] = __ldg(reinterpret_cast<const uint4*>(row + kFp8Latent) + lane);
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(cache) + slot * kRowVec;
      for (int k = lane; k < kRowVec; k += 32) dst[k] = __ldg(src + k);
    }
  }
}

}  // namespace wgather

cudaError_t launch_gather_window(const void* cache, const float* scales, bool fp8, const WindowGather& g,
                                 uint16_t* out, cudaStream_t stream) {
  if (g.total <= 0 || g.nb <= 0) return cudaSuccess;
  int64_t blocks = (g.total + wgather::kWarps - 1) / wgather::kWarps;
  if (blocks > 152 * 16) blocks = 152 * 16;
  auto* kern = fp8 ? wgather::gather_window_kernel<true> : wgather::gather_window_kernel<false>;
  kern<<<(int)blocks, wgather::kWarps * 32, 0, stream>>>(static_cast<const uint8_t*>(cache), scales, g,
                                                         reinterpret_cast<uint4*>(out));
  return cudaGetLastError();
}

}  // namespace mla
