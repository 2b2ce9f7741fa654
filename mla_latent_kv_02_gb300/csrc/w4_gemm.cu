// Steps A2 and A5 with 4-bit weights: y[t, h, n] = sum_k x[t, h, k] W[h, k, n],
//   W[h, k, n] = s[h, k / G, n] * c[h, k, n],  c a 4-bit two's-complement code.
// Layout (laid out once, mla_pack_w4): words uint32 [128, K/8, N], code of
// k = 8 kb + i in bits [4i, 4i + 4) of word (h, kb, n); scales bf16 [128, K/G, N].
//   A2: K = 128, N = 512;  A5: K = 512, N = 128;  G = 32, 64 or 128.
// Both kernels multiply the integer codes and apply a group's scale to the
// group's fp32 sum, so no weight is rounded: a code times a bf16 scale has up
// to 12 significant bits and would not fit a bf16 operand.
//
// * w4_rows_kernel: up to 8 tokens a block, fp32 on the CUDA cores.  A thread
//   owns one column and 128 values of k (16 words, all requested at once); the
//   K = 512 step joins four threads' sums through shared memory.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace w4 {

using namespace mla::dev;

constexpr int kSlice = 128;        // values of k per thread
constexpr int kWordsPer = kSlice / 8;
constexpr int kRowThreads = 256;

// Eight codes to fp32, exactly: a nibble OR-ed into the mantissa of a power of
// two whose last place it fills reads 2^(23 - 4i) + nibble; the codes are
// offset by 8 first (sign bit flipped).
__device__ __forceinline__ void codes_to_float(uint32_t w, float (&c)[8]) {
  w ^= 0x88888888u;
  const uint32_t hi = w >> 20;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = i < 5 ? 4 * i : 4 * (i - 5);
    const uint32_t bits = ((i < 5 ? w : hi) & (0xFu << at)) | ((uint32_t)(127 + 23 - at) << 23);
    c[i] = __uint_as_float(bits) - (float)((1 << (23 - at)) + 8);
  }
}

template <int N, int K, int TT>
__global__ void __launch_bounds__(kRowThreads)
    w4_rows_kernel(const uint16_t* __restrict__ x, const uint32_t* __restrict__ words,
                   const uint16_t* __restrict__ scales, int group, int32_t T, uint16_t* __restrict__ y) {
  constexpr int kSplits = K / kSlice;              // threads that share a column
  constexpr int kCols = kRowThreads / kSplits;
  __shared__ __align__(16) float xs[TT][K];
  __shared__ float part[kSplits > 1 ? kSplits - 1 : 1][TT][kCols];
  const int h = blockIdx.y, n0 = blockIdx.x * kCols;
  const int64_t t0 = (int64_t)blockIdx.z * TT;
  const int col = threadIdx.x % kCols, ks = threadIdx.x / kCols;
  const int n = n0 + col;
  uint32_t w[kWordsPer];
  const uint32_t* wp = words + ((int64_t)h * (K / 8) + ks * kWordsPer) * N + n;
#pragma unroll
  for (int j = 0; j < kWordsPer; ++j) w[j] = __ldg(wp + (int64_t)j * N);
  for (int i = threadIdx.x; i < TT * K / 2; i += kRowThreads) {
    const int t = i / (K / 2), k2 = i % (K / 2);
    const uint32_t v = t0 + t < T ? __ldg(reinterpret_cast<const uint32_t*>(x) + ((t0 + t) * MLA_NUM_HEADS + h) * (K / 2) + k2) : 0u;
    xs[t][2 * k2] = __uint_as_float(v << 16);
    xs[t][2 * k2 + 1] = __uint_as_float(v & 0xFFFF0000u);
  }
  __syncthreads();
  const uint16_t* sp = scales + ((int64_t)h * (K / group) + ks * kSlice / group) * N + n;
  const int words_per_group = group / 8;
  float acc[TT], sum[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = sum[t] = 0.f;
#pragma unroll
  for (int j = 0; j < kWordsPer; ++j) {
    float c[8];
    codes_to_float(w[j], c);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float4 a = *reinterpret_cast<const float4*>(&xs[t][ks * kSlice + 8 * j]);
      const float4 b = *reinterpret_cast<const float4*>(&xs[t][ks * kSlice + 8 * j + 4]);
      sum[t] = fmaf(a.x, c[0], fmaf(a.y, c[1], fmaf(a.z, c[2], fmaf(a.w, c[3], sum[t]))));
      sum[t] = fmaf(b.x, c[4], fmaf(b.y, c[5], fmaf(b.z, c[6], fmaf(b.w, c[7], sum[t]))));
    }
    if ((j + 1) % words_per_group == 0) {
      const float s = __uint_as_float((uint32_t)__ldg(sp + (int64_t)(j / words_per_group) * N) << 16);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        acc[t] = fmaf(s, sum[t], acc[t]);
        sum[t] = 0.f;
      }
    }
  }
  if (kSplits > 1) {
    if (ks > 0) {
#pragma unroll
      for (int t = 0; t < TT; ++t) part[ks - 1][t][col] = acc[t];
    }
    __syncthreads();
    if (ks > 0) return;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int p = 0; p < kSplits - 1; ++p) acc[t] += part[p][t][col];
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
    if (t0 + t < T) {
      const __nv_bfloat16 v = __float2bfloat16_rn(acc[t]);
      y[((t0 + t) * MLA_NUM_HEADS + h) * N + n] = *reinterpret_cast<const uint16_t*>(&v);
    }
}

template <int N, int K, int TT>
cudaError_t run_rows(const W4Args& a, cudaStream_t stream) {
  constexpr int kCols = kRowThreads / (K / kSlice);
  const dim3 grid(N / kCols, MLA_NUM_HEADS, (unsigned)((a.T + TT - 1) / TT));
  w4_rows_kernel<N, K, TT><<<grid, kRowThreads, 0, stream>>>(a.x, a.words, a.scales, a.group, a.T, a.y);
  return cudaGetLastError();
}

template <int N, int K>
cudaError_t run(const W4Args& a, cudaStream_t stream) {
  if (a.T == 1) return run_rows<N, K, 1>(a, stream);
  if (a.T == 2) return run_rows<N, K, 2>(a, stream);
  if (a.T <= 4) return run_rows<N, K, 4>(a, stream);
  return run_rows<N, K, 8>(a, stream);
}

// The layout above from bf16 weights: s = bf16(amax / 7) of each group of a
// column, code = w / s rounded to nearest even and clamped to [-8, 7] (a
// group whose scale is zero has zero codes).  One thread per (head, group,
// column); run once, when a model is loaded.
__global__ void __launch_bounds__(256)
    w4_pack_kernel(const uint16_t* __restrict__ w, int K, int N, int group, uint32_t* __restrict__ words,
                   uint16_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int n = (int)(i % N);
  const int64_t hg = i / N;  // head * (K / group) + group index
  if (hg >= (int64_t)MLA_NUM_HEADS * (K / group)) return;
  const uint16_t* src = w + hg * group * N + n;
  float amax = 0.f;
  for (int k = 0; k < group; ++k) amax = fmaxf(amax, fabsf(__uint_as_float((uint32_t)src[(int64_t)k * N] << 16)));
  const __nv_bfloat16 sb = __float2bfloat16_rn(amax / 7.f);
  const float s = __bfloat162float(sb);
  scales[i] = *reinterpret_cast<const uint16_t*>(&sb);
  for (int kb = 0; kb < group / 8; ++kb) {
    uint32_t word = 0;
    for (int j = 0; j < 8; ++j) {
      const float v = __uint_as_float((uint32_t)src[(int64_t)(8 * kb + j) * N] << 16);
      const float q = s > 0.f ? fminf(fmaxf(rintf(v / s), -8.f), 7.f) : 0.f;
      word |= ((uint32_t)(int)q & 0xFu) << (4 * j);
    }
    words[(hg * (group / 8) + kb) * N + n] = word;
  }
}

}  // namespace w4

cudaError_t launch_w4_gemm(HeadGemm kind, const W4Args& args, cudaStream_t stream) {
  if (args.T <= 0) return cudaSuccess;
  return kind == HeadGemm::kAbsorbQ ? w4::run<512, 128>(args, stream) : w4::run<128, 512>(args, stream);
}

cudaError_t launch_w4_pack(const uint16_t* w, int K, int N, int group, uint32_t* words, uint16_t* scales,
                           cudaStream_t stream) {
  const int64_t n = (int64_t)MLA_NUM_HEADS * (K / group) * N;
  w4::w4_pack_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(w, K, N, group, words, scales);
  return cudaGetLastError();
}

}  // namespace mla
