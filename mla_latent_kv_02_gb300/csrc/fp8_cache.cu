// FP8 (E4M3) latent cache: the quantising append and the dequantising gather.
//
// [P3] bjbfmj.com/news/60700: the byte formula L x (d_c + d_r) x b counts
// only the elements; quantisation scale factors are stored beside them.
// [P1] "撕开 DeepSeek MLA 源码…", opening section and §5: a quantised gather
// of the latent cache with 16-byte vector loads from 16-byte aligned bases.
//
// Layout: rows uint8 [num_pages][64][640] (512 E4M3 codes, then the 64 bf16
// RoPE values), scales fp32 [num_pages][64] (2^k per token).
//
// * kv_append_fp8: one warp per token.  Lane l holds latent values
//   [8l, 8l+8) and [256+8l, 256+8l+8); a warp max-reduction of |c| gives the
//   row's amax, the scale exponent follows from amax's exponent and mantissa
//   bits, and the scaled values (exact) are rounded to E4M3 by the hardware
//   conversion.  The RoPE key is copied bit for bit.
// * kv_append_rope_fp8: the same append with the RoPE key rotated by its
//   position on the way in, and the queries' RoPE part in the same launch.
// * gather_paged_fp8: one warp per token; lane l loads 16 codes as one
//   16-byte vector and writes 32 bytes of bf16.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace mla {
namespace f8 {

using namespace mla::dev;

constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t abs_max_bf16x2(uint32_t m, uint32_t v) {
  const uint32_t a = v & 0x7FFF7FFFu;
  return max(m, max(a & 0xFFFFu, a >> 16));
}

// Eight bf16 values (a uint4) times 2^n, rounded to eight E4M3 codes (a uint2).
__device__ __forceinline__ uint2 quant8(uint4 v, int n) {
  uint2 r;
  r.x = f32x2_to_e4m3x2(scale_pow2(bf16_lo(v.x), n), scale_pow2(bf16_hi(v.x), n)) |
        (f32x2_to_e4m3x2(scale_pow2(bf16_lo(v.y), n), scale_pow2(bf16_hi(v.y), n)) << 16);
  r.y = f32x2_to_e4m3x2(scale_pow2(bf16_lo(v.z), n), scale_pow2(bf16_hi(v.z), n)) |
        (f32x2_to_e4m3x2(scale_pow2(bf16_lo(v.w), n), scale_pow2(bf16_hi(v.w), n)) << 16);
  return r;
}

// A warp quantises one token's 512 latents (lane l holds values [8l, 8l + 8)
// in a and [256 + 8l, 256 + 8l + 8) in b) into its row and scale.
__device__ __forceinline__ void quant_row(uint4 a, uint4 b, int lane, uint8_t* row, float* scale) {
  uint32_t m = 0;
  m = abs_max_bf16x2(m, a.x);
  m = abs_max_bf16x2(m, a.y);
  m = abs_max_bf16x2(m, a.z);
  m = abs_max_bf16x2(m, a.w);
  m = abs_max_bf16x2(m, b.x);
  m = abs_max_bf16x2(m, b.y);
  m = abs_max_bf16x2(m, b.z);
  m = abs_max_bf16x2(m, b.w);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  const int k = fp8_scale_exponent(__uint_as_float(m << 16));
  *reinterpret_cast<uint2*>(row + 8 * lane) = quant8(a, -k);
  *reinterpret_cast<uint2*>(row + 256 + 8 * lane) = quant8(b, -k);
  if (lane == 0) *scale = k >= -126 ? exp2_int(k) : exp2_int(k + 64) * 0x1p-64f;
}

__global__ void __launch_bounds__(kWarps * 32)
    kv_append_fp8_kernel(const uint4* __restrict__ c_new, const uint4* __restrict__ k_new,
                         const int64_t* __restrict__ slots, int32_t n, uint8_t* __restrict__ rows,
                         float* __restrict__ scales, int64_t num_slots, int32_t* err) {
  const int lane = threadIdx.x & 31;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < n; t += (int64_t)gridDim.x * kWarps) {
    const int64_t slot = __ldg(slots + t);
    if (slot < 0 || slot >= num_slots) {
      if (lane == 0) atomicOr(err, (int32_t)MLA_DEVERR_SLOT_OOB);
      continue;
    }
    const uint4 a = __ldg(c_new + t * 64 + lane);
    const uint4 b = __ldg(c_new + t * 64 + 32 + lane);
    uint8_t* row = rows + slot * kFp8RowBytes;
    quant_row(a, b, lane, row, scales + slot);
    if (lane < 8) reinterpret_cast<uint4*>(row + kFp8Latent)[lane] = __ldg(k_new + t * 8 + lane);
  }
}

// The append with the RoPE key rotated on the way in, and the queries' RoPE
// part rotated in the same launch (q_pe null: keys only).
//   rows[slot] = [E4M3 codes of c | k_pe turned by its position], scales[slot] = 2^k,
//   q_r[t, h] = q_pe[t, h] turned by the same position.
// Blocks [0, key_blocks) take a token per warp; the rest take the queries,
// one thread per 16-byte chunk (four pairs) of a (token, head) row, eight
// threads to a row.  HBM-bound: 128 tokens with their queries, the launch of a
// two-token step of 64 sequences, take 2.2 us on the device, 4.4 MB.
__global__ void __launch_bounds__(kWarps * 32)
    kv_append_rope_fp8_kernel(const uint4* __restrict__ c_new, const uint32_t* __restrict__ k_pe,
                              const uint4* __restrict__ q_pe, const int32_t* __restrict__ positions,
                              const float2* __restrict__ table, int32_t max_pos, const int64_t* __restrict__ slots,
                              int32_t n, int key_blocks, uint8_t* __restrict__ rows, float* __restrict__ scales,
                              uint4* __restrict__ q_r, int64_t num_slots, int32_t* err) {
  if ((int)blockIdx.x < key_blocks) {
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < n; t += (int64_t)key_blocks * kWarps) {
      const int64_t slot = __ldg(slots + t);
      const int32_t p = __ldg(positions + t);
      const bool slot_ok = slot >= 0 && slot < num_slots, pos_ok = p >= 0 && p < max_pos;
      if (!slot_ok || !pos_ok) {
        if (lane == 0)
          atomicOr(err, (int32_t)((slot_ok ? 0u : MLA_DEVERR_SLOT_OOB) | (pos_ok ? 0u : MLA_DEVERR_POS_OOB)));
        continue;
      }
      const uint4 a = __ldg(c_new + t * 64 + lane);
      const uint4 b = __ldg(c_new + t * 64 + 32 + lane);
      const uint32_t r = rotate_pair(__ldg(k_pe + t * 32 + lane), __ldg(table + (int64_t)p * 32 + lane));
      uint8_t* row = rows + slot * kFp8RowBytes;
      quant_row(a, b, lane, row, scales + slot);
      reinterpret_cast<uint32_t*>(row + kFp8Latent)[lane] = r;
    }
    return;
  }
  const float4* table4 = reinterpret_cast<const float4*>(table);
  const int64_t chunks = (int64_t)n * MLA_NUM_HEADS * 8;
  const int64_t step = (int64_t)(gridDim.x - key_blocks) * blockDim.x;
  for (int64_t k = (int64_t)(blockIdx.x - key_blocks) * blockDim.x + threadIdx.x; k < chunks; k += step) {
    const int32_t p = __ldg(positions + k / (MLA_NUM_HEADS * 8));
    const int c = (int)(k & 7);
    if (p < 0 || p >= max_pos) continue;  // reported by the token's key warp
    q_r[k] = rotate_pairs4(__ldg(q_pe + k), __ldg(table4 + (int64_t)p * 16 + 2 * c),
                           __ldg(table4 + (int64_t)p * 16 + 2 * c + 1));
  }
}

__global__ void __launch_bounds__(kWarps * 32)
    gather_fp8_kernel(const uint8_t* __restrict__ rows, const float* __restrict__ scales, int64_t num_pages,
                      const int32_t* __restrict__ block_table, int32_t max_pages, int32_t b, int32_t n_tokens,
                      uint4* __restrict__ out, int32_t* err) {
  const int lane = threadIdx.x & 31;
  for (int64_t j = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); j < n_tokens; j += (int64_t)gridDim.x * kWarps) {
    const int32_t pid = __ldg(block_table + (int64_t)b * max_pages + j / 64);
    if (pid < 0 || (int64_t)pid >= num_pages) {
      if (lane == 0) atomicOr(err, (int32_t)MLA_DEVERR_PAGE_OOB);
      continue;
    }
    const int64_t slot = (int64_t)pid * 64 + j % 64;
    const uint8_t* row = rows + slot * kFp8RowBytes;
    const Fp8Scale sc = fp8_row_scale(__ldg(scales + slot));
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(row) + lane);   // codes [16 lane, 16 lane + 16)
    uint4* dst = out + j * 72;
    dst[2 * lane] = dequant8(make_uint2(c.x, c.y), sc);
    dst[2 * lane + 1] = dequant8(make_uint2(c.z, c.w), sc);
    if (lane < 8) dst[64 + lane] = __ldg(reinterpret_cast<const uint4*>(row + kFp8Latent) + lane);
  }
}

inline int blocks_for(int64_t items) {
  int64_t b = (items + kWarps - 1) / kWarps;
  if (b > 152 * 16) b = 152 * 16;
  return b < 1 ? 1 : (int)b;
}

// Blocks of the rotating append: one token a warp while that fills the GPU,
// then about six, in steps of eight blocks an SM (six are resident: 40 registers
// a thread).  Found by trial on 2^20 tokens of 1.8 KB each: 54 tokens a warp 321
// us, 8 309, 6 302 (6.3 TB/s), 4 315, one 368; two tokens of a warp in flight at
// once 355 (fewer warps fit).
inline int append_blocks(int64_t n) {
  constexpr int64_t kStep = 152 * 8;
  const int64_t few = n / (6 * kWarps) / kStep * kStep;
  const int64_t b = few > blocks_for(n) ? few : blocks_for(n);
  return (int)b;
}

}  // namespace f8

cudaError_t launch_kv_append_fp8(const uint16_t* c_kv_new, const uint16_t* k_r_new, const int64_t* slots, int32_t n,
                                 uint8_t* rows, float* scales, int64_t num_slots, int32_t* dev_err,
                                 cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  f8::kv_append_fp8_kernel<<<f8::blocks_for(n), f8::kWarps * 32, 0, stream>>>(
      reinterpret_cast<const uint4*>(c_kv_new), reinterpret_cast<const uint4*>(k_r_new), slots, n, rows, scales,
      num_slots, dev_err);
  return cudaGetLastError();
}

cudaError_t launch_kv_append_rope_fp8(const uint16_t* c_kv_new, const uint16_t* k_pe_new, const uint16_t* q_pe,
                                      const int32_t* positions, const float* table, int32_t max_pos,
                                      const int64_t* slots, int32_t n, uint8_t* rows, float* scales, uint16_t* q_r,
                                      int64_t num_slots, int32_t* dev_err, cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  const int key_blocks = f8::append_blocks(n);
  int64_t q_blocks = q_pe ? ((int64_t)n * MLA_NUM_HEADS * 8 + 255) / 256 : 0;
  if (q_blocks > 152 * 64) q_blocks = 152 * 64;
  f8::kv_append_rope_fp8_kernel<<<key_blocks + (int)q_blocks, f8::kWarps * 32, 0, stream>>>(
      reinterpret_cast<const uint4*>(c_kv_new), reinterpret_cast<const uint32_t*>(k_pe_new),
      reinterpret_cast<const uint4*>(q_pe), positions, reinterpret_cast<const float2*>(table), max_pos, slots, n,
      key_blocks, rows, scales, reinterpret_cast<uint4*>(q_r), num_slots, dev_err);
  return cudaGetLastError();
}

cudaError_t launch_gather_fp8(const uint8_t* rows, const float* scales, int64_t num_pages,
                              const int32_t* block_table, int32_t max_pages, int32_t b, int32_t n_tokens,
                              uint16_t* out, int32_t* dev_err, cudaStream_t stream) {
  if (n_tokens <= 0) return cudaSuccess;
  f8::gather_fp8_kernel<<<f8::blocks_for(n_tokens), f8::kWarps * 32, 0, stream>>>(
      rows, scales, num_pages, block_table, max_pages, b, n_tokens, reinterpret_cast<uint4*>(out), dev_err);
  return cudaGetLastError();
}

}  // namespace mla
