// Copies of whole cache pages, in every layer at once: a fork's last page, and
// the moves that bring a pool's used pages together.
//
// [P1] "撕开 DeepSeek MLA 源码…" §3: pages of 64 tokens; §5: 16-byte aligned
// vector access.  The pairs ride in the launch parameters, so that the call
// needs no device memory and can be captured.
//
// Bound by HBM: a page is read once and written once.  A CTA moves 16 KB, four
// 16-byte pieces a thread in flight (five CTAs a bf16 page), so that one page of
// one layer already spreads over SMs and 2 000 pages of four layers (1.18 GB)
// keep them all busy: 168 us, 7.0 TB/s, against 177 at the measured copy rate; one
// page of 60 layers 1.9 us (three pieces 2.0, six 2.4, twelve 2.4), of which most
// is the launch.  Of an NVFP4 cache, whose page is two CTAs: 63 us for the 2 000
// pages of four layers (426 MB), 1.8 for one page of 60.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"

namespace mla {
namespace pages {

constexpr int kThreads = 256, kPieces = 4;  // 16-byte pieces of a thread

template <int kPairs>
struct Pairs {
  int2 p[kPairs];
};

// One CTA: kThreads * kPieces pieces of one page of one layer (x), the pair
// (y), the layer (z).  The FP8 cache's scales go with a page's first CTA.
template <int kPairs>
__global__ void __launch_bounds__(kThreads)
    copy_kernel(const LayerCaches c, int32_t page_bytes, const __grid_constant__ Pairs<kPairs> pairs) {
  const int2 pair = pairs.p[blockIdx.y];
  uint8_t* rows = c.rows + blockIdx.z * c.row_stride;
  const uint4* src = reinterpret_cast<const uint4*>(rows + (int64_t)pair.x * page_bytes);
  uint4* dst = reinterpret_cast<uint4*>(rows + (int64_t)pair.y * page_bytes);
  const int n = page_bytes / 16, k0 = blockIdx.x * kThreads * kPieces + threadIdx.x;
  uint4 v[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j)
    if (k0 + j * kThreads < n) v[j] = __ldg(src + k0 + j * kThreads);
#pragma unroll
  for (int j = 0; j < kPieces; ++j)
    if (k0 + j * kThreads < n) dst[k0 + j * kThreads] = v[j];
  if (c.scales && k0 < MLA_PAGE_SIZE / 4) {
    uint4* sc = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(c.scales) + blockIdx.z * c.scale_stride);
    sc[(int64_t)pair.y * (MLA_PAGE_SIZE / 4) + k0] = __ldg(sc + (int64_t)pair.x * (MLA_PAGE_SIZE / 4) + k0);
  }
}

template <int kPairs>
cudaError_t run(const LayerCaches& c, int page_bytes, const int32_t* src, const int32_t* dst, int n,
                cudaStream_t stream) {
  Pairs<kPairs> p;
  for (int i = 0; i < n; ++i) p.p[i] = make_int2(src[i], dst[i]);
  const int per = kThreads * kPieces * 16;
  copy_kernel<kPairs><<<dim3((page_bytes + per - 1) / per, n, c.layers), kThreads, 0, stream>>>(c, page_bytes, p);
  return cudaGetLastError();
}

}  // namespace pages

cudaError_t launch_copy_pages(const LayerCaches& c, int row_bytes, const int32_t* src, const int32_t* dst, int32_t n,
                              cudaStream_t stream) {
  // 30 KB of the 32 KB of launch parameters, or few pairs, whose parameters the
  // host need not copy (64 pairs: a call of 3.0 us in the small form, 4.6 in the
  // large; the kernels take the same time)
  constexpr int kMost = 3840;
  const int page_bytes = row_bytes * MLA_PAGE_SIZE;
  for (int32_t i = 0; i < n; i += kMost) {
    const int m = std::min<int32_t>(n - i, kMost);
    cudaError_t e = m <= 64 ? pages::run<64>(c, page_bytes, src + i, dst + i, m, stream)
                            : pages::run<kMost>(c, page_bytes, src + i, dst + i, m, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mla
