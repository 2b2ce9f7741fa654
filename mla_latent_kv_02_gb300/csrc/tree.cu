// Trees of drafted tokens over the paged latent cache: the nodes' masks,
// positions and slots before a verification step, and the accepted path's rows
// brought together after it.  The attention between the two is in
// decode_paged.cu (decode_tree_kernel).
//
// [P2] "DeepSeek的推理为什么比别人便宜一个数量级？…": the MTP section drafts a
// chain of tokens for each step; a tree is the same draft with alternatives.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace tree {

constexpr int kMaxNodes = MLA_TREE_MAX_NODES, kMaxWords = kMaxNodes / 64;

// The slot of position pos, or -1 where the table has no page of the pool.
__device__ __forceinline__ int64_t slot_of(const int32_t* __restrict__ row, int32_t max_pages, int64_t num_pages,
                                           int32_t pos) {
  const int32_t page = pos / MLA_PAGE_SIZE;
  const int32_t id = page < max_pages ? __ldg(row + page) : -1;
  return id >= 0 && (int64_t)id < num_pages ? (int64_t)id * MLA_PAGE_SIZE + pos % MLA_PAGE_SIZE : -1;
}

// The masks of a tree are the closure of "parent of": M(i) = {i} ∪ M(parent(i)).
// One CTA a sequence, a thread a node; every node holds the mask and the length
// of a piece of its path and a pointer to the node above the piece, and a round
// joins the piece above, so that a chain of n nodes takes log2 n rounds.  Latency
// bound, three loads behind each other and the rounds: 2.4 us for 64 nodes in a
// stream, 4.5 for 256 trees of 256 (2.8 MB).
__global__ void __launch_bounds__(kMaxNodes) layout_kernel(const TreeLayoutArgs a) {
  __shared__ uint64_t mask[kMaxWords][kMaxNodes];
  __shared__ int16_t up[kMaxNodes], length[kMaxNodes];
  const int b = blockIdx.x, i = threadIdx.x;
  const int32_t q0 = __ldg(a.q_starts + b), q1 = __ldg(a.q_starts + b + 1), len = __ldg(a.seq_lens + b);
  const int32_t n = q1 - q0;
  if (q0 < 0 || q1 < q0 || q1 > a.T || n > 64 * a.words || n > len) {
    if (i == 0) atomicOr(a.dev_err, (int32_t)MLA_DEVERR_TREE);
    return;
  }
  const bool in = i < n;
  int32_t p = in ? __ldg(a.parents + q0 + i) : -1;
  if (p < -1 || p >= i) {
    atomicOr(a.dev_err, (int32_t)MLA_DEVERR_TREE);
    p = -1;
  }
  int64_t at = -1;  // asked for now, used after the rounds
  if (a.slots && in) at = slot_of(a.block_table + (int64_t)b * a.max_pages, a.max_pages, a.num_pages, len - n + i);
  uint64_t m[kMaxWords];
#pragma unroll
  for (int w = 0; w < kMaxWords; ++w) mask[w][i] = m[w] = i / 64 == w ? 1ull << (i % 64) : 0ull;
  int d = 1;
  length[i] = 1;
  up[i] = (int16_t)p;
  while (__syncthreads_or(p >= 0)) {
    int next = -1;
    if (p >= 0) {
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w) m[w] |= mask[w][p];
      d += length[p];
      next = up[p];
    }
    __syncthreads();
    if (p >= 0) {
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w) mask[w][i] = m[w];
      length[i] = (int16_t)d;
      up[i] = (int16_t)next;
    }
    p = next;
  }
  if (!in) return;
  const int64_t row = (int64_t)q0 + i;
#pragma unroll
  for (int w = 0; w < kMaxWords; ++w)
    if (w < a.words) a.masks[row * a.words + w] = m[w];
  if (a.positions) a.positions[row] = len - n + d - 1;
  if (a.slots) {
    if (at < 0) atomicOr(a.dev_err, (int32_t)MLA_DEVERR_PAGE_OOB);
    a.slots[row] = at;
  }
}

// Row r of the kept nodes (ascending, the k_r-th node of the tree) moves from
// slot n0 + k_r to slot n0 + r in every layer.  k_r >= r and rises with r, so a
// row may be written as soon as the rows up to it have been read: a batch is
// loaded, a barrier, and stored, and no batch needs a slot that an earlier one
// wrote.  A CTA takes a sequence (x) in `per` layers (y), layer after layer, so
// that the look-up of its slots, four loads one behind the other, is paid once.
// Four rows a thread in flight: 2.5 us for one sequence in one layer, 8.0 for 64
// in 60 (36.5 MB, 4.6 TB/s; eight rows in flight 8.8: fewer CTAs fit an SM); of an
// FP8 cache 6.6 (20 MB), of an NVFP4 cache 4.3 (13 MB).
template <int kPieces, bool kScales>
struct CompactCfg {
  static constexpr int kPer = kPieces + (kScales ? 1 : 0);  // threads a row: its 16-byte pieces and its scale
  static constexpr int kRows = 256 / kPer;                  // rows at a time
  static constexpr int kBatch = 4;                          // of a thread
};

template <int kPieces, bool kScales>
__global__ void __launch_bounds__(256) compact_kernel(const TreeCompactArgs a, int per) {
  using C = CompactCfg<kPieces, kScales>;
  __shared__ int64_t slot[kMaxNodes];
  __shared__ int16_t node[kMaxNodes];
  const int b = blockIdx.x, layer0 = blockIdx.y * per, t = threadIdx.x;
  const bool first = blockIdx.y == 0;
  const int32_t q0 = __ldg(a.q_starts + b), q1 = __ldg(a.q_starts + b + 1), len = __ldg(a.seq_lens + b);
  const int32_t acc = __ldg(a.accepted + b), n = q1 - q0;
  if (q0 < 0 || q1 < q0 || q1 > a.T || n > 64 * a.words || n > len || acc < -1 || acc >= n) {
    if (t == 0 && first) atomicOr(a.dev_err, (int32_t)MLA_DEVERR_TREE);
    return;
  }
  int kept = 0, rank = 0;
  bool mine = false;
  if (acc >= 0) {
#pragma unroll
    for (int w = 0; w < kMaxWords; ++w) {
      if (w >= a.words || 64 * w > acc) break;
      uint64_t m = __ldg(reinterpret_cast<const unsigned long long*>(a.masks) + ((int64_t)q0 + acc) * a.words + w);
      if (acc - 64 * w < 63) m &= (1ull << (acc - 64 * w + 1)) - 1ull;
      if (t / 64 == w) {
        mine = (m >> (t % 64)) & 1;
        rank = kept + __popcll(m & ((1ull << (t % 64)) - 1ull));
      }
      kept += __popcll(m);
    }
  }
  if (t == 0 && first) a.new_lens[b] = len - n + kept;
  if (t <= acc) {
    slot[t] = slot_of(a.block_table + (int64_t)b * a.max_pages, a.max_pages, a.c.num_pages, len - n + t);
    if (slot[t] < 0 && first && (mine || t < kept)) atomicOr(a.dev_err, (int32_t)MLA_DEVERR_PAGE_OOB);
    if (mine) node[rank] = (int16_t)t;
  }
  __syncthreads();
  const int piece = t % C::kPer, r0 = t / C::kPer;
  const int units = min(per, a.c.layers - layer0) * kept;  // unit u: kept row u % kept of layer layer0 + u / kept
  for (int u0 = 0; u0 < units; u0 += C::kRows * C::kBatch) {
    uint4 v[C::kBatch];
    uint8_t* to[C::kBatch];
#pragma unroll
    for (int j = 0; j < C::kBatch; ++j) {
      const int u = u0 + j * C::kRows + r0;
      to[j] = nullptr;
      if (r0 >= C::kRows || u >= units) continue;
      const int layer = layer0 + u / kept, k = u % kept;
      const int64_t src = slot[node[k]], dst = slot[k];
      if (node[k] == k || src < 0 || dst < 0) continue;
      if (kScales && piece == kPieces) {
        uint8_t* scales = reinterpret_cast<uint8_t*>(a.c.scales) + layer * a.c.scale_stride;
        v[j].x = *reinterpret_cast<const uint32_t*>(scales + src * 4);
        to[j] = scales + dst * 4;
      } else {
        uint8_t* rows = a.c.rows + layer * a.c.row_stride;
        v[j] = *reinterpret_cast<const uint4*>(rows + (src * kPieces + piece) * 16);
        to[j] = rows + (dst * kPieces + piece) * 16;
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < C::kBatch; ++j) {
      if (!to[j]) continue;
      if (kScales && piece == kPieces)
        *reinterpret_cast<uint32_t*>(to[j]) = v[j].x;
      else
        *reinterpret_cast<uint4*>(to[j]) = v[j];
    }
  }
}

// One CTA a page: its 64 rows of E4M3 codes become f16 rows of 576, code * 2^k and
// RoPE, each value as the FP8 decode forms it on chip.  A warp finds the page's
// sequence in the plan's table, 32 entries a look: a grid of sequences by the
// longest one's pages is mostly empty for ragged batches (decode of 255 sequences
// of 1 032 tokens and one of 262 144: 2 023 -> 1 043 us).  A token's scale outside
// the f16 range counts only where a row sees it: every row sees the tokens before
// the tree, and the nodes' masks are asked in that case alone.  Rows past the
// sequence's end become zeros.  Moves 1.8 KB a token: 14 us for 32 832 tokens with
// cold caches, 21 MB from HBM and 38 into L2 (59 by the sectors counted there, half
// as much again as is stored, as for page copies).
__global__ void __launch_bounds__(256) unpack_kernel(const TreeUnpackArgs a) {
  const int t = threadIdx.x;
  const int32_t page = blockIdx.x;
  dev::grid_dependency_wait();
  if (t == 0) dev::grid_launch_dependents();  // the decode may get ready; it waits before it reads a page
  int at = 0;                                 // the last tree whose first page is not behind this one
  for (int n = a.num_trees; n > 1;) {
    const int step = (n + 31) / 32, i = (t & 31) * step;
    const bool le = i < n && __ldg(a.trees + (int64_t)(at + i) * kTreeWords + 1) <= page;
    const int k = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0) * step;
    at += k;
    n = min(step, n - k);
  }
  const int4 lo = __ldg(reinterpret_cast<const int4*>(a.trees) + 2 * at);
  const int4 hi = __ldg(reinterpret_cast<const int4*>(a.trees) + 2 * at + 1);
  const int32_t b = lo.x, base = lo.y, pages = lo.z, n0 = lo.w, len = hi.x, row0 = hi.y, nodes = hi.z;
  const int64_t pg = (int64_t)page - base;    // of the sequence
  if (b < 0 || b >= a.B || base < 0 || pg < 0 || pg >= pages || pages > a.max_pages || n0 < 0 || row0 < 0 || nodes < 0 ||
      nodes > a.T - row0) {
    if (t == 0) atomicOr(a.dev_err, (int32_t)MLA_DEVERR_PLAN);
    return;
  }
  int32_t id = __ldg(a.block_table + (int64_t)b * a.max_pages + pg);
  if (id < 0 || (int64_t)id >= a.num_pages) {
    if (t == 0) atomicOr(a.dev_err, (int32_t)MLA_DEVERR_PAGE_OOB);
    id = 0;
  }
  const uint4* src = reinterpret_cast<const uint4*>(a.rows + (int64_t)id * MLA_PAGE_SIZE * MLA_FP8_ROW_BYTES);
  uint4* dst = a.out + (int64_t)page * MLA_PAGE_SIZE * (MLA_TOKEN_ELEMS / 8);
  // Eight codes and one 16-byte store a thread, two warps a row: a warp stores
  // 512 bytes in one piece (16 codes and two stores left half sectors: 100 MB
  // counted at L2 for 59).
  constexpr int kRows = 8;  // of a thread at a time
  const int piece = t % 64, r0 = t / 64;
  const int last = (int)min((int64_t)len - pg * MLA_PAGE_SIZE, (int64_t)MLA_PAGE_SIZE);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint2 code[kRows];
    float scale[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = 32 * half + r0 + 4 * j;
      code[j] = r < last ? __ldg(reinterpret_cast<const uint2*>(src + r * (MLA_FP8_ROW_BYTES / 16)) + piece) : make_uint2(0u, 0u);
      scale[j] = r < last ? __ldg(a.scales + (int64_t)id * MLA_PAGE_SIZE + r) : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = 32 * half + r0 + 4 * j;
      bool ok;
      const uint32_t f = dev::fp8_f16_factor(scale[j], ok);
      if (!ok) {
        const int k = (int)(pg * MLA_PAGE_SIZE + r - n0);  // its node
        bool seen = k < 0;
        if (k >= 0 && (k >> 6) < a.words)
          for (int i = k + piece; i < nodes; i += 64)
            seen = seen || (__ldg(reinterpret_cast<const unsigned long long*>(a.masks) + ((int64_t)row0 + i) * a.words + (k >> 6)) >> (k & 63) & 1);
        if (seen) atomicOr(a.dev_err, (int32_t)MLA_DEVERR_FP8_RANGE);
      }
      dst[r * (MLA_TOKEN_ELEMS / 8) + piece] =
          make_uint4(dev::mul_f16x2(dev::e4m3x2_to_f16x2(code[j].x & 0xFFFFu), f), dev::mul_f16x2(dev::e4m3x2_to_f16x2(code[j].x >> 16), f),
                     dev::mul_f16x2(dev::e4m3x2_to_f16x2(code[j].y & 0xFFFFu), f), dev::mul_f16x2(dev::e4m3x2_to_f16x2(code[j].y >> 16), f));
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // the 64 RoPE values: eight pieces a row
    const int r = j * 32 + t / 8, q = t % 8;
    uint4 v = r < last ? __ldg(src + r * (MLA_FP8_ROW_BYTES / 16) + 32 + q) : make_uint4(0u, 0u, 0u, 0u);
    v.x = dev::bf16x2_to_f16x2(v.x);
    v.y = dev::bf16x2_to_f16x2(v.y);
    v.z = dev::bf16x2_to_f16x2(v.z);
    v.w = dev::bf16x2_to_f16x2(v.w);
    dst[r * (MLA_TOKEN_ELEMS / 8) + 64 + q] = v;
  }
}

template <int kPieces, bool kScales>
cudaError_t run_compact(const TreeCompactArgs& a, cudaStream_t stream) {
  // up to six CTAs an SM: more layers to a CTA beyond that (64 sequences in 60
  // layers: 8.0 us in a stream, 10.3 with a CTA for each, floor 5.5)
  const int64_t most = 6 * 152;
  const int per = (int)std::min<int64_t>(a.c.layers, ((int64_t)a.B * a.c.layers + most - 1) / most);
  compact_kernel<kPieces, kScales><<<dim3(a.B, (a.c.layers + per - 1) / per), 256, 0, stream>>>(a, per);
  return cudaGetLastError();
}

}  // namespace tree

cudaError_t launch_tree_unpack(const TreeUnpackArgs& args, cudaStream_t stream) {
  return launch_dependent(tree::unpack_kernel, dim3(args.out_pages), 256, 0, true, stream, args);
}

cudaError_t launch_tree_layout(const TreeLayoutArgs& args, cudaStream_t stream) {
  tree::layout_kernel<<<args.B, tree::kMaxNodes, 0, stream>>>(args);
  return cudaGetLastError();
}

cudaError_t launch_tree_compact(const TreeCompactArgs& args, int row_bytes, cudaStream_t stream) {
  if (row_bytes == MLA_FP8_ROW_BYTES) return tree::run_compact<MLA_FP8_ROW_BYTES / 16, true>(args, stream);
  if (row_bytes == MLA_NVFP4_ROW_BYTES) return tree::run_compact<MLA_NVFP4_ROW_BYTES / 16, false>(args, stream);
  return tree::run_compact<MLA_TOKEN_ELEMS * 2 / 16, false>(args, stream);
}

}  // namespace mla
