// Steps A2 and A5 with 4-bit weights: y[t, h, n] = sum_k x[t, h, k] W[h, k, n],
//   W[h, k, n] = s[h, k / G, n] * c[h, k, n],  c a 4-bit two's-complement code.
// Layout (laid out once, mla_pack_w4): words uint32 [128, K/8, N], code of
// k = 8 kb + i in bits [4i, 4i + 4) of word (h, kb, n); scales bf16 [128, K/G, N].
//   A2: K = 128, N = 512;  A5: K = 512, N = 128;  G = 32, 64 or 128.
// Both kernels multiply the integer codes and apply a group's scale to the
// group's fp32 sum, so no weight is rounded: a code times a bf16 scale has up
// to 12 significant bits and would not fit a bf16 operand.
//
// * w4_rows_kernel: up to 32 tokens; the columns are the rows of mma.sync
//   products, the codes go from a word to an operand register without passing
//   through shared memory.
// * w4_gemm_kernel: 128 tokens a tile on the tensor cores (tcgen05).  The codes
//   become exact bf16 integers in shared memory once per head, each group's
//   fp32 sums pass through a slot of tensor memory and are added up under
//   their scales in registers.  See the kernel.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace w4 {

using namespace mla::dev;

// ------------------------------------------------------------------ few tokens
// A warp owns 16 columns of one head and 128 values of k; W^T is the
// left operand of mma.sync (m16n8k16: 16 columns x 16 k), the tokens its eight
// columns, kTiles such tiles of tokens a block.  The order of k inside a
// product is free as long as both operands share it, so nothing is shuffled:
// lane (g, q) = (lane / 4, lane % 4) takes the words of columns g and g + 8 at
// k block 4 j + q, splits each into the pairs (k_i, k_i+4) with a shift and a
// mask, and reads the same eight k of token g as one 16-byte load.
//
// Bound by the 4.2 MB of codes and by latency: a block's loads are all
// requested before the first product, 27 warps an SM for the whole operator.
constexpr int kSlice = 128;         // values of k a warp sums
constexpr int kSteps = kSlice / 32; // words of a column in a slice, four lanes each one
constexpr int kRowThreads = 256;
// More tokens go to tcgen05.  Device us with cold weights, this kernel against
// the 128-token tiles at the same count (absorb, then up; groups of 128 / 64 / 32):
//   16 tokens 5.7 / 5.6 / 6.3 against 8.1 / 10.2 / 12.7; 4.8 / 6.1 / 6.2 against 8.6 / 8.9 / 10.6
//   32 tokens 7.5 / 7.9 / 8.8 against 8.6 / 10.3 / 12.7; 7.1 / 7.5 / 7.5 against 8.6 / 9.0 / 10.6
// The tiles take 8.8 / 10.5 / 13.0 and 8.7 / 9.0 / 10.8 at 33 tokens and up to
// 0.8 us more at 128; this kernel holds at most four token tiles in registers.
constexpr int32_t kRowsMax = 32;

// Pair i of a word (offset binary: sign bits flipped) as bf16: 0x4300 | v is 128 + v.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {
  const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int N, int K, int G, int kTiles>
__global__ void __launch_bounds__(kRowThreads)
    w4_rows_kernel(const uint4* __restrict__ x, const uint32_t* __restrict__ words,
                   const uint16_t* __restrict__ scales, int32_t T, uint16_t* __restrict__ y) {
  constexpr int kSplits = K / kSlice;              // warps that share 16 columns
  constexpr int kCols = 16 * (kRowThreads / 32) / kSplits;
  constexpr int kPerGroup = G / 32;                // steps of a group
  constexpr int kGroups = kSlice / G;              // groups of a slice
  __shared__ float part[kSplits > 1 ? kSplits - 1 : 1][kTiles * 4][kRowThreads / kSplits];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int h = blockIdx.y, ks = warp / (8 / kSplits), tile = warp % (8 / kSplits);
  const int n = blockIdx.x * kCols + tile * 16 + g;
  const uint32_t* wp = words + ((int64_t)h * (K / 8) + ks * (kSlice / 8) + q) * N + n;
  uint32_t w[kSteps][2];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    w[j][0] = __ldg(wp + (int64_t)(4 * j) * N);
    w[j][1] = __ldg(wp + (int64_t)(4 * j) * N + 8);
  }
  float s[kGroups][2];
  const uint16_t* sp = scales + ((int64_t)h * (K / G) + ks * kGroups) * N + n;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    s[i][0] = __uint_as_float((uint32_t)__ldg(sp + i * N) << 16);
    s[i][1] = __uint_as_float((uint32_t)__ldg(sp + i * N + 8) << 16);
  }
  uint4 v[kTiles][kSteps];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      v[t][j] = 8 * t + g < T ? __ldg(x + ((int64_t)(8 * t + g) * MLA_NUM_HEADS + h) * (K / 8) + ks * (kSlice / 8) + 4 * j + q)
                              : make_uint4(0u, 0u, 0u, 0u);
  float acc[kTiles][4], sum[kTiles][4];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = sum[t][i] = 0.f;
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const uint32_t w0 = w[j][0] ^ 0x88888888u, w1 = w[j][1] ^ 0x88888888u;
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // pairs 2 half, 2 half + 1
      const uint32_t a[4] = {code_pair(w0, 2 * half), code_pair(w1, 2 * half), code_pair(w0, 2 * half + 1),
                             code_pair(w1, 2 * half + 1)};
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const uint32_t lo = half ? v[t][j].y : v[t][j].x, hi = half ? v[t][j].w : v[t][j].z;
        mma_16816(sum[t], a, __byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
      }
    }
    if ((j + 1) % kPerGroup == 0) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // rows g (i < 2) and g + 8 of the product are columns n, n + 8
          acc[t][i] = fmaf(s[j / kPerGroup][i >> 1], sum[t][i], acc[t][i]);
          sum[t][i] = 0.f;
        }
    }
  }
  if (kSplits > 1) {
    const int at = tile * 32 + lane;
    if (ks > 0) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[ks - 1][4 * t + i][at] = acc[t][i];
    }
    __syncthreads();
    if (ks > 0) return;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < kSplits - 1; ++p) acc[t][i] += part[p][4 * t + i][at];
  }
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 8 * t + 2 * q + (i & 1);
      if (tok < T) {
        const __nv_bfloat16 r = __float2bfloat16_rn(acc[t][i]);
        y[((int64_t)tok * MLA_NUM_HEADS + h) * N + n + 8 * (i >> 1)] = *reinterpret_cast<const uint16_t*>(&r);
      }
    }
}

template <int N, int K, int G>
cudaError_t run_rows(const W4Args& a, cudaStream_t stream) {
  constexpr int kCols = 16 * (kRowThreads / 32) / (K / kSlice);
  const dim3 grid(N / kCols, MLA_NUM_HEADS);
  const uint4* x = reinterpret_cast<const uint4*>(a.x);
  if (a.T <= 8) w4_rows_kernel<N, K, G, 1><<<grid, kRowThreads, 0, stream>>>(x, a.words, a.scales, a.T, a.y);
  else if (a.T <= 16) w4_rows_kernel<N, K, G, 2><<<grid, kRowThreads, 0, stream>>>(x, a.words, a.scales, a.T, a.y);
  else w4_rows_kernel<N, K, G, 4><<<grid, kRowThreads, 0, stream>>>(x, a.words, a.scales, a.T, a.y);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ many tokens
// A CTA takes a contiguous range of the work units (head, token tile), token
// tiles fastest, so a head's weights are unpacked once into shared memory (128
// KB of exact bf16 integers) and its token tiles stream past them.
//   for each 128-column block of y, for each group g of k:
//     D_slot[128 x 128] = x[128 x G] . C_g[G x 128]     tcgen05, fp32 in TMEM
//     acc += s_g D_slot                                  fp32, in registers
//   y block = bf16(acc)
// TMEM is a ring of four 128-column slots, so the products of one group run
// while the sums of the one before are scaled; every group size has the same
// shape of work.
// Warps: 0 loads x by TMA (chunks of 64 k, a ring of kStages), 1 issues the
// MMAs, 2-9 unpack the weights and scale the sums: two warps per TMEM lane
// quarter (thread = token row), 64 columns each, which store their rows in
// boxes of 32 x 32 by TMA without waiting for one another.
// B is K-major: a word's eight codes are eight consecutive k of a column, one
// 16-byte store into the 128-byte swizzled row of that column.  The words and
// scales of the next head are loaded into registers a head ahead, the first
// head's before the set-up (loading them at the switch, warmed in L2, cost
// 2 % at 2048 tokens).
// The MMA loop is unrolled over a chunk's four steps on precomputed
// descriptors: rolled, with a descriptor built per step, each MMA took 550
// cycles to issue instead of about 70.
// Measured (A5, groups of 128, 2048 tokens, 340 MB): 62 us, 5.5 TB/s, bound by
// the x and y streams; 128 tokens, cold weights: 9.7 us, the chain load ->
// unpack -> products -> scale of a single tile per SM.  Groups of 32 double the
// slots a tile passes through the epilogue: 85 us.
// Every wait is bounded, the ones between the epilogue warps too (mbarriers).
constexpr int kStages = 4;
constexpr int kChunkBytes = 128 * 64 * 2;        // [128 tokens x 64 k] bf16
constexpr int kSlots = 4, kSlotCols = 128;
constexpr int kBoxCols = 32;
constexpr int kBoxBytes = 32 * kBoxCols * 2;     // a warp's output box, 64-byte swizzled rows
constexpr int kEpiWarps = 8, kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 64 + kEpiThreads;

template <int N, int K, int G>
struct Cfg {
  static constexpr int kGroups = K / G, kBlocks = N / kSlotCols, kChunks = K / 64;
  static constexpr int kWChunkBytes = N * 128;                        // [N columns x 64 k] bf16
  static constexpr int kOffA = kChunks * kWChunkBytes;
  static constexpr int kOffOut = kOffA + kStages * kChunkBytes;
  static constexpr int kOffScale = kOffOut + kEpiWarps * kBoxBytes;   // fp32 [kGroups][N]
  static constexpr int kOffBar = kOffScale + kGroups * N * 4;
  static constexpr int kNumBars = 2 * kStages + 2 * kSlots + kChunks + 3;
  static constexpr int kSmem = kOffBar + 8 * kNumBars + 16 + 1024;
  static constexpr int kWords = N * (K / 8) / kEpiThreads;            // words a thread unpacks
  static constexpr int kScales = kGroups * N / kEpiThreads;
  static constexpr uint32_t kIdesc = idesc_bf16_f32(128, kSlotCols, false, false);
  static_assert(kSmem <= 232448, "shared memory layout does not fit");
};

// Eight codes of a word (k ascending) to four bf16 pairs.
__device__ __forceinline__ uint4 codes_to_bf16(uint32_t w) {
  w ^= 0x88888888u;
  uint32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r[j] = code_pair(((w >> (8 * j)) & 0xFFu) * 0x1001u, 0);          // low nibble at 0, high nibble at 16
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int N, int K, int G>
__global__ void __launch_bounds__(kThreads, 1)
    w4_gemm_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap y_map,
                   const uint32_t* __restrict__ words, const uint16_t* __restrict__ scales, int32_t T, int32_t* err) {
  using C = Cfg<N, K, G>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::kOffBar;
  const uint32_t full0 = bars, empty0 = full0 + 8 * kStages, s_full0 = empty0 + 8 * kStages,
                 s_free0 = s_full0 + 8 * kSlots, w_ready0 = s_free0 + 8 * kSlots, head_done = w_ready0 + 8 * C::kChunks,
                 sc_ready = head_done + 8, drain = head_done + 16;
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(gbase + C::kOffBar + 8 * C::kNumBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffBar + 8 * C::kNumBars + 8);
  float* sc = reinterpret_cast<float*>(gbase + C::kOffScale);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (T + 127) / 128, units = MLA_NUM_HEADS * tiles;
  const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);

  // A head's words and scales, this thread's share, into registers.
  const int tid = threadIdx.x - 64;                  // epilogue thread 0 .. 255
  uint32_t w[C::kWords];
  uint16_t sv[C::kScales];
  auto request = [&](int h) {
    const uint32_t* wp = words + (int64_t)h * (K / 8) * N + tid;
    const uint16_t* sp = scales + (int64_t)h * C::kGroups * N + tid;
#pragma unroll
    for (int j = 0; j < C::kWords; ++j) w[j] = __ldg(wp + j * kEpiThreads);
#pragma unroll
    for (int j = 0; j < C::kScales; ++j) sv[j] = __ldg(sp + j * kEpiThreads);
  };
  if (warp >= 2 && u0 < u1) request(u0 / tiles);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(s_full0 + 8 * i, 1);
      mbar_init(s_free0 + 8 * i, kEpiWarps);
    }
    for (int i = 0; i < C::kChunks; ++i) mbar_init(w_ready0 + 8 * i, kEpiWarps);
    mbar_init(head_done, kEpiWarps);
    mbar_init(sc_ready, kEpiWarps);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), kSlots * kSlotCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- x loads
    if (lane == 0) {
      prefetch_tmap(&x_map);
      prefetch_tmap(&y_map);
      uint32_t n = 0;
      bool ok = true;
      for (int u = u0; ok && u < u1; ++u) {
        const int h = u / tiles, m0 = u % tiles * 128;
        for (int kc = 0; kc < C::kChunks; ++kc, ++n) {
          const uint32_t st = n % kStages, use = n / kStages;
          if (use > 0 && !wait_phase(empty0 + 8 * st, (use - 1) & 1u, err, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full0 + 8 * st, (uint32_t)kChunkBytes);
          tma_load_3d(base + C::kOffA + st * kChunkBytes, &x_map, kc * 64, h, m0, full0 + 8 * st);
        }
      }
      for (uint32_t k = n > (uint32_t)kStages ? n - kStages : 0u; k < n; ++k)
        wait_phase_drain(full0 + 8 * (k % kStages), (k / kStages) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      static_assert(C::kBlocks == 1 || C::kChunks <= kStages, "every column block reads the tile's resident chunks");
      const uint64_t adesc0 = sdesc_sw128(base + C::kOffA, 16, 1024), wdesc0 = sdesc_sw128(base, 16, 1024);
      uint32_t n = 0, slot = 0, heads = 0;
      int h_now = -1;
      bool ok = true;
      for (int u = u0; ok && u < u1; ++u, n += C::kChunks) {
        const bool fresh = u / tiles != h_now;       // the head's first tile: its weights arrive chunk by chunk
        if (fresh) {
          h_now = u / tiles;
          ++heads;
        }
        for (int nb = 0; ok && nb < C::kBlocks; ++nb) {
          for (int kc = 0; ok && kc < C::kChunks; ++kc) {
            const uint32_t c = n + kc, st = c % kStages;
            if (nb == 0) {
              ok = (!fresh || wait_phase(w_ready0 + 8 * kc, (heads - 1) & 1u, err, abort_flag)) &&
                   wait_phase(full0 + 8 * st, (c / kStages) & 1u, err, abort_flag);
              if (!ok) break;
            }
            const uint64_t da = adesc0 + (uint64_t)((st * kChunkBytes) >> 4);
            const uint64_t db = wdesc0 + (uint64_t)((kc * C::kWChunkBytes + nb * kSlotCols * 128) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const bool first = G == 128 ? kk == 0 && kc % 2 == 0 : kk % (G / 16) == 0;
              const bool last = G == 128 ? kk == 3 && kc % 2 == 1 : kk % (G / 16) == G / 16 - 1;
              if (first && slot >= (uint32_t)kSlots)
                ok = ok && wait_phase(s_free0 + 8 * (slot % kSlots), (slot / kSlots - 1) & 1u, err, abort_flag);
              if (!ok) break;
              if (kk == 0 || first) tc_fence_after();
              mma_ss(tmem + (slot % kSlots) * kSlotCols, da + (uint64_t)((kk * 32) >> 4), db + (uint64_t)((kk * 32) >> 4),
                     C::kIdesc, first ? 0u : 1u);
              if (last) tc_commit(s_full0 + 8 * (slot++ % kSlots));
            }
            if (ok && nb == C::kBlocks - 1) tc_commit(empty0 + 8 * st);
          }
        }
      }
      tc_commit(drain);  // every MMA has finished before TMEM is released
      wait_phase_drain(drain, 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- weights and epilogue
    const int q4 = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16) + half * 64;
    const uint32_t box = base + C::kOffOut + (warp - 2) * kBoxBytes;
    int h_now = -1;
    uint32_t heads = 0, slot = 0;
    bool ok = true;
    for (int u = u0; ok && u < u1; ++u) {
      const int h = u / tiles, m0 = u % tiles * 128 + q4 * 32;
      if (h != h_now) {
        // Every MMA of the head before has completed (this warp has seen its
        // last slot full); its scales may go once every warp is past them.
        if (h_now >= 0) {
          if (lane == 0) mbar_arrive(head_done);
          ok = __all_sync(0xffffffffu, wait_phase<false, true>(head_done, (heads - 1) & 1u, err, abort_flag));
          if (!ok) break;
        }
        h_now = h;
#pragma unroll
        for (int j = 0; j < C::kScales; ++j) sc[j * kEpiThreads + tid] = __uint_as_float((uint32_t)sv[j] << 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_ready);
        constexpr int kPer = C::kWords / C::kChunks;  // words of a chunk
#pragma unroll
        for (int kc = 0; kc < C::kChunks; ++kc) {
#pragma unroll
          for (int j = kc * kPer; j < (kc + 1) * kPer; ++j) {
            const int at = j * kEpiThreads + tid, n = at % N, kb = at / N;
            const uint4 v = codes_to_bf16(w[j]);
            st_shared_v4(base + kc * C::kWChunkBytes + n * 128 + (((kb & 7) ^ (n & 7)) << 4), v.x, v.y, v.z, v.w);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(w_ready0 + 8 * kc);
        }
        if (h < (u1 - 1) / tiles) request(h + 1);
        ok = __all_sync(0xffffffffu, wait_phase<false, true>(sc_ready, heads & 1u, err, abort_flag));
        if (!ok) break;
        ++heads;
      }
#pragma unroll 1
      for (int nb = 0; ok && nb < C::kBlocks; ++nb) {
        float acc[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = 0.f;
#pragma unroll 1
        for (int g = 0; g < C::kGroups; ++g, ++slot) {
          ok = __all_sync(0xffffffffu, wait_phase<false, true>(s_full0 + 8 * (slot % kSlots), (slot / kSlots) & 1u, err, abort_flag));
          if (!ok) break;
          tc_fence_after();
          const float4* s4 = reinterpret_cast<const float4*>(sc + g * N + nb * kSlotCols + half * 64);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t d[32];
            tmem_ld32_sync(tl + (slot % kSlots) * kSlotCols + 32 * b, d);
            if (b == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(s_free0 + 8 * (slot % kSlots));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 s = s4[8 * b + j];
              float* v = acc + 32 * b + 4 * j;
              v[0] = fmaf(s.x, __uint_as_float(d[4 * j]), v[0]);
              v[1] = fmaf(s.y, __uint_as_float(d[4 * j + 1]), v[1]);
              v[2] = fmaf(s.z, __uint_as_float(d[4 * j + 2]), v[2]);
              v[3] = fmaf(s.w, __uint_as_float(d[4 * j + 3]), v[3]);
            }
          }
        }
        if (!ok) break;
        if (m0 < T) {  // warp-uniform: rows past T are not stored
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (lane == 0) bulk_wait_all_read();  // the box's previous store has read it
            __syncwarp();
            // 64-byte swizzle: row r at 64 r, 16-byte piece c at c ^ ((r / 2) & 3)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float* v = acc + 32 * b + 8 * c;
              st_shared_v4(box + lane * 64u + (((uint32_t)c ^ (((uint32_t)lane >> 1) & 3u)) << 4), pack_bf16x2(v[0], v[1]),
                           pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&y_map, box, nb * kSlotCols + half * 64 + b * kBoxCols, h, m0);
              bulk_commit_group();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all_read();  // the staging box is released at exit
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kSlots * kSlotCols);
  }
}

template <int N, int K, int G>
cudaError_t run_gemm(const W4Args& a, const CUtensorMap& x_map, const CUtensorMap& y_map, cudaStream_t stream) {
  using C = Cfg<N, K, G>;
  auto* kern = w4_gemm_kernel<N, K, G>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int units = MLA_NUM_HEADS * ((a.T + 127) / 128);
  kern<<<units < 152 ? units : 152, kThreads, C::kSmem, stream>>>(x_map, y_map, a.words, a.scales, a.T, a.dev_err);
  return cudaGetLastError();
}

template <int N, int K, int G>
cudaError_t run(const W4Args& a, const CUtensorMap& x_map, const CUtensorMap& y_map, cudaStream_t stream) {
  return a.T <= kRowsMax ? run_rows<N, K, G>(a, stream) : run_gemm<N, K, G>(a, x_map, y_map, stream);
}

template <int N, int K>
cudaError_t run_group(const W4Args& a, const CUtensorMap& x_map, const CUtensorMap& y_map, cudaStream_t stream) {
  if (a.group == 128) return run<N, K, 128>(a, x_map, y_map, stream);
  if (a.group == 64) return run<N, K, 64>(a, x_map, y_map, stream);
  return run<N, K, 32>(a, x_map, y_map, stream);
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

bool w4_uses_maps(int32_t T) { return T > w4::kRowsMax; }

cudaError_t launch_w4_gemm(HeadGemm kind, const W4Args& args, const CUtensorMap& x_map, const CUtensorMap& y_map,
                           cudaStream_t stream) {
  if (args.T <= 0) return cudaSuccess;
  return kind == HeadGemm::kAbsorbQ ? w4::run_group<512, 128>(args, x_map, y_map, stream)
                                    : w4::run_group<128, 512>(args, x_map, y_map, stream);
}

cudaError_t launch_w4_pack(const uint16_t* w, int K, int N, int group, uint32_t* words, uint16_t* scales,
                           cudaStream_t stream) {
  const int64_t n = (int64_t)MLA_NUM_HEADS * (K / group) * N;
  w4::w4_pack_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(w, K, N, group, words, scales);
  return cudaGetLastError();
}

}  // namespace mla
