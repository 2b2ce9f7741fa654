// Internal interface between the C-ABI entry points (mla_api.cu) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mla.h"

namespace mla {

// Records `message` as this thread's mla_last_error() and returns `s`.
mla_status set_last_error(mla_status s, const char* message);

// Layout of the decode plan (int32 words).  Written by the host planner,
// read by the decode and combine kernels.
//   [0] magic  [1] T  [2] B  [3] num_clusters  [4] num_segments
//   [5] num_partials  [6] num_split_rows  [7] max_pages_needed
//   [8..15] reserved
//   seg_off   at kPlanHeader, num_clusters + 1 entries
//   segments  at seg_base, num_segments x 8: {row, b, page_begin, page_end,
//             visible, out_slot (-1 = final), window's or tree's first token,
//             tree: its sequence's first page among the unpacked ones}
//   split rows at split_base, num_split_rows x 4: {row, slot_begin, n_slots, 0}
//   trees     behind them (tree plans only), num_seqs x 8: {b, first unpacked
//             page, pages, first token of the tree, tokens, first row, nodes, 0},
//             one entry for each sequence that has nodes
constexpr int kPlanHeader = 16;
constexpr int kSegWords = 8;
constexpr int kSplitWords = 4;
constexpr int kTreeWords = 8;

struct PlanLayout {
  int64_t seg_off;  // word offsets
  int64_t seg_base;
  int64_t split_base;
  int64_t words;
};
PlanLayout plan_layout(int64_t num_clusters, int64_t num_segments, int64_t num_split_rows);
// Upper bounds used to size the plan buffer.
inline int64_t plan_max_segments(int64_t T, int64_t num_clusters) { return T + num_clusters; }
inline int64_t plan_max_split_rows(int64_t T, int64_t num_clusters) {
  return T < num_clusters ? T : num_clusters;
}
inline int64_t plan_max_partials(int64_t num_clusters) { return 2 * num_clusters; }

// Sliding window with sinks: a row at position p sees the tokens j <= p with
// j < sinks or j >= lo, lo = p - window + 1.  A plan segment carries lo in
// word 6 (0: every token up to p; the planner writes 0 whenever lo <= sinks),
// and its page_begin / page_end count the tiles the row reads: its sink
// pages, then its window pages.
//   * full sink pages 0 .. sinks / 64 - 1, then a page with the last
//     sinks % 64 sinks, unless
//   * that page is the window's first page (`shared`: one tile, two visible
//     pieces), or
//   * the window's first page has room for them before lo (`merged`: the tile
//     is loaded from both pages, its first `split` = sinks % 64 rounded up to
//     eight tokens from the sinks' page and the rest from the window's page).
struct WindowTiles {
  int32_t sink_tiles;  // tiles before the window's first page
  int32_t skip;        // page of tile v: v < sink_tiles ? v : v + skip
  int32_t head;        // sinks visible at the start of tile sink_tiles
  int32_t merged;      // tile sink_tiles takes its first `split` tokens from page sinks / 64
};
__host__ __device__ inline int32_t window_split(int32_t sinks) { return (sinks % 64 + 7) / 8 * 8; }
__host__ __device__ inline WindowTiles window_tiles(int32_t lo, int32_t sinks) {
  WindowTiles w = {0, 0, 0, 0};
  if (lo == 0) return w;
  const int32_t first = lo / 64, full = sinks / 64, rest = sinks % 64;
  const bool shared = rest > 0 && first == full;
  const bool merged = rest > 0 && !shared && window_split(sinks) <= lo % 64;
  w.sink_tiles = full + (rest > 0 && !shared && !merged ? 1 : 0);
  w.skip = first - w.sink_tiles;
  w.head = shared || merged ? rest : 0;
  w.merged = merged ? 1 : 0;
  return w;
}

struct DecodeArgs {
  const uint16_t* q_abs;  // bf16 [T, 128, 512]
  const uint16_t* q_r;    // bf16 [T, 128, 64]
  const int32_t* block_table;
  int32_t max_pages;
  int32_t pad_;
  int64_t num_pages;
  const int32_t* seg_off;
  const int32_t* segs;
  float scale_log2;  // scale * log2(e)
  int32_t pad2_;
  uint16_t* o_lat;     // bf16 [T, 128, 512]
  float* lse;          // [T, 128] or null
  float* part_o;       // fp32 [partials, 128, 512]
  float* part_lse;     // fp32 [partials, 128] (log2 domain)
  int32_t* dev_err;
  // plan summary, used to validate every segment before any access
  int32_t T;
  int32_t B;
  int32_t num_segments;
  int32_t num_partials;
  const float* kv_scales;  // FP8 cache: fp32 [num_pages * 64] token scales (null for bf16)
  // Bound, in SM cycles, of every wait in the decode loop (the drains before
  // exit keep the full default bound).
  uint64_t wait_limit;
  // The deadline is checked when a wait's probe count & wait_every is 0
  // (255 for the default bound; 0, every probe, for a short test bound).
  uint32_t wait_every;
  int32_t pad3_;
};

// Decompress branch over a batch of sequences: sequence i has M query rows
// at positions N - M .. N - 1; its query rows (q_c, q_r, out) start at row
// q_off, its cache rows (gathered rows, K_c, V_c) at token kv_off of the
// packed arrays.  The table rides in the launch parameters.
constexpr int kPrefillMaxSeqs = 64;
struct PrefillSeq {
  int32_t M;
  int32_t N;
  int32_t q_off;
  int32_t kv_off;
};
struct PrefillArgs {
  int32_t nb;           // sequences in seq[]
  float scale_log2;     // scale * log2(e)
  uint16_t* out;        // bf16 [rows, 128, 128]
  int32_t* dev_err;
  int32_t window;       // sliding window with sinks over the packed rows (launch_prefill_window)
  int32_t sinks;
  PrefillSeq seq[kPrefillMaxSeqs];
};

// Gather of the first n[i] cached tokens of sequence b[i] of the block
// table, for i < nb, to rows [off[i], off[i] + n[i]) of one packed output.
struct GatherBatch {
  int32_t nb;
  int32_t pad_;
  int64_t total;        // Σ n[i]
  int32_t b[kPrefillMaxSeqs];
  int32_t n[kPrefillMaxSeqs];
  int64_t off[kPrefillMaxSeqs];
};

// The packed gather of windowed sequences: row j of sequence i comes from
// position j < cut[i] ? j : j + shift[i], for j < n[i]; the rows from there to
// the next sequence's first are zeros.
struct WindowGather {
  int32_t nb;
  int32_t max_pages;
  int64_t total;        // rows, the zeros between sequences included
  int64_t num_pages;
  const int32_t* block_table;
  int32_t* dev_err;
  int32_t b[kPrefillMaxSeqs];
  int32_t n[kPrefillMaxSeqs];
  int32_t cut[kPrefillMaxSeqs];
  int32_t shift[kPrefillMaxSeqs];
  int32_t off[kPrefillMaxSeqs];
};

struct CombineArgs {
  const int32_t* split_rows;
  const float* part_o;
  const float* part_lse;
  uint16_t* o_lat;
  float* lse;
  int32_t T;
  int32_t num_partials;
  int32_t* dev_err;
};

// What the windowed decode takes beside DecodeArgs: the boxes of a merged
// tile, head (split rows) and tail (64 - split rows).  With split == 0 no tile
// is merged and the maps are not read.
struct WindowArgs {
  CUtensorMap kv_head, kv_tail;      // bf16: one 64-column chunk a box; FP8: 256 codes a row
  CUtensorMap rope_head, rope_tail;
  int32_t sinks;
  int32_t split;                     // window_split(sinks)
};

// What the tree decode takes beside DecodeArgs: `words` 64-bit words of mask
// for each row.  A plan segment carries the tree's first token in word 6.
struct TreeArgs {
  const uint64_t* masks;
  int32_t words;
};

// The FP8 cache's pages as f16 rows [page][64][576], for a tree decode that reads
// each of them for several rows.
struct TreeUnpackArgs {
  const uint8_t* rows;
  const float* scales;
  int64_t num_pages;
  const int32_t* block_table;
  const uint64_t* masks;
  const int32_t* trees;        // the plan's table
  uint4* out;
  int32_t* dev_err;
  int32_t max_pages;
  int32_t B;
  int32_t T;
  int32_t words;
  int32_t out_pages;           // those of all the trees' sequences
  int32_t num_trees;
};

// Trees of drafted nodes, a sequence each (tree.cu): sequence b's nodes are
// rows [q_starts[b], q_starts[b + 1]) of T, its last ones of seq_lens[b] tokens.
struct TreeLayoutArgs {
  const int32_t* parents;
  const int32_t* q_starts;
  const int32_t* seq_lens;
  const int32_t* block_table;  // with slots
  int64_t num_pages;
  int32_t max_pages;
  int32_t B;
  int32_t T;
  int32_t words;
  uint64_t* masks;
  int32_t* positions;          // or null
  int64_t* slots;              // or null
  int32_t* dev_err;
};
// The caches of a model's layers as 16-byte pieces of a token's row, and for
// the FP8 cache a scale beside each row (else null).  Strides in bytes.
struct LayerCaches {
  uint8_t* rows;
  float* scales;
  int64_t row_stride;
  int64_t scale_stride;
  int64_t num_pages;
  int32_t layers;
};
struct TreeCompactArgs {
  LayerCaches c;
  const int32_t* block_table;
  const uint64_t* masks;
  const int32_t* q_starts;
  const int32_t* seq_lens;
  const int32_t* accepted;
  int32_t max_pages;
  int32_t B;
  int32_t T;
  int32_t words;
  int32_t* new_lens;
  int32_t* dev_err;
};

// Launches `kern` so that its blocks may take their places while the kernel
// before it on the stream still runs (programmatic: only if that kernel allows
// it); every block must call grid_dependency_wait before it reads or writes
// what that kernel does.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, int threads, int smem, bool programmatic,
                             cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = programmatic ? 1 : 0;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

int decode_smem_bytes();
int decode_threads();
cudaError_t decode_max_clusters(int* out);
// bf16 cache: kv_map 128-byte swizzled boxes of 64 columns x 64 tokens x 4
// chunks (latent), rope_map 64-byte swizzled boxes of 32 columns x 64 tokens.
// FP8 cache (fp8 = true): kv_map uint8 boxes of 256 codes x 64 tokens (no
// swizzle), rope_map as above over the 640-byte rows; args.kv_scales set.
cudaError_t launch_decode(const CUtensorMap& kv_map, const CUtensorMap& rope_map, const DecodeArgs& args,
                          int num_clusters, bool fp8, cudaStream_t stream);
cudaError_t launch_decode_window(const CUtensorMap& kv_map, const CUtensorMap& rope_map, const DecodeArgs& args,
                                 const WindowArgs& window, int num_clusters, bool fp8, cudaStream_t stream);
enum class TreeCache { kBf16, kFp8, kUnpacked };
cudaError_t launch_decode_tree(const CUtensorMap& kv_map, const CUtensorMap& rope_map, const DecodeArgs& args,
                               const TreeArgs& tree, int num_clusters, TreeCache cache, cudaStream_t stream);
cudaError_t launch_tree_unpack(const TreeUnpackArgs& args, cudaStream_t stream);
cudaError_t launch_combine(const CombineArgs& args, int num_split_rows, cudaStream_t stream);

cudaError_t launch_kv_append(const uint16_t* c_kv_new, const uint16_t* k_r_new, const int64_t* slots, int32_t n,
                             uint16_t* kv_cache, int64_t num_slots, int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_rope_table(float* table, int32_t max_pos, double base, cudaStream_t stream);
cudaError_t launch_kv_append_rope(const uint16_t* c_kv_new, const uint16_t* k_pe_new, const int32_t* positions,
                                  const float* table, int32_t max_pos, const int64_t* slots, int32_t n,
                                  uint16_t* kv_cache, int64_t num_slots, int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_rope_q(const uint16_t* q_pe, const int32_t* positions, const float* table, int32_t max_pos,
                          uint16_t* q_r, int32_t T, int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_kv_append_fp8(const uint16_t* c_kv_new, const uint16_t* k_r_new, const int64_t* slots, int32_t n,
                                 uint8_t* rows, float* scales, int64_t num_slots, int32_t* dev_err,
                                 cudaStream_t stream);
cudaError_t launch_kv_append_rope_fp8(const uint16_t* c_kv_new, const uint16_t* k_pe_new, const uint16_t* q_pe,
                                      const int32_t* positions, const float* table, int32_t max_pos,
                                      const int64_t* slots, int32_t n, uint8_t* rows, float* scales, uint16_t* q_r,
                                      int64_t num_slots, int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_gather_fp8(const uint8_t* rows, const float* scales, int64_t num_pages,
                              const int32_t* block_table, int32_t max_pages, int32_t b, int32_t n_tokens,
                              uint16_t* out, int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_kv_append_nvfp4(const uint16_t* c_kv_new, const uint16_t* k_r_new, const int64_t* slots,
                                   int32_t n, float tensor_scale, uint8_t* rows, int64_t num_slots,
                                   int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_gather_nvfp4(const uint8_t* rows, float tensor_scale, int64_t num_pages,
                                const int32_t* block_table, int32_t max_pages, int32_t b, int32_t n_tokens,
                                uint16_t* out, int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_gather_nvfp4_batch(const uint8_t* rows, float tensor_scale, int64_t num_pages,
                                      const int32_t* block_table, int32_t B, int32_t max_pages, const int32_t* seq_ids,
                                      const int64_t* out_offsets, int32_t nb, int64_t total_tokens, uint16_t* out,
                                      int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_gather(const uint16_t* kv_cache, int64_t num_pages, const int32_t* block_table, int32_t max_pages,
                          int32_t b, int32_t n_tokens, uint16_t* out, int32_t* dev_err, cudaStream_t stream);
cudaError_t launch_gather_batch(const uint16_t* kv_cache, int64_t num_pages, const int32_t* block_table,
                                int32_t max_pages, const GatherBatch& g, uint16_t* out, int32_t* dev_err,
                                cudaStream_t stream);

cudaError_t launch_gather_window(const void* cache, const float* scales, bool fp8, const WindowGather& g,
                                 uint16_t* out, cudaStream_t stream);

cudaError_t launch_tree_layout(const TreeLayoutArgs& args, cudaStream_t stream);
// row_bytes: 1152, 640 or 416
cudaError_t launch_tree_compact(const TreeCompactArgs& args, int row_bytes, cudaStream_t stream);
// Pages src[i] to dst[i] in every layer (host arrays of n, read before the call returns).
cudaError_t launch_copy_pages(const LayerCaches& c, int row_bytes, const int32_t* src, const int32_t* dst, int32_t n,
                              cudaStream_t stream);

// Decompress-branch expansion: K_c and V_c in one pass (head-major outputs).
// early: it may start while the kernel before it on the stream still runs.
cudaError_t launch_expand_kv(const CUtensorMap& a_map, const CUtensorMap& k_map, const CUtensorMap& v_map,
                             const CUtensorMap& kc_map, const CUtensorMap& vc_map, int32_t n, int32_t* err,
                             bool early, cudaStream_t stream);
int prefill_smem_bytes();
cudaError_t launch_prefill_attn(const CUtensorMap& q_map, const CUtensorMap& r_map, const CUtensorMap& k_map,
                                const CUtensorMap& kr_map, const CUtensorMap& v_map, const PrefillArgs& args,
                                cudaStream_t stream);
cudaError_t launch_prefill_window(const CUtensorMap& q_map, const CUtensorMap& r_map, const CUtensorMap& k_map,
                                  const CUtensorMap& kr_map, const CUtensorMap& v_map, const PrefillArgs& args,
                                  cudaStream_t stream);

// Per-head GEMM C[t, h, :] = A[t, h, :] · W[h] (bf16 in, fp32 accumulate, bf16 out).
enum class HeadGemm { kAbsorbQ, kUpV };
cudaError_t launch_head_gemm(HeadGemm kind, const CUtensorMap& a_map, const CUtensorMap& w_map,
                             const CUtensorMap& c_map, int32_t T, int32_t* err, cudaStream_t stream);

// The same with 4-bit weights (w4_gemm.cu): words uint32 [128, K/8, N] of
// eight codes along K, scales bf16 [128, K/group, N].
struct W4Args {
  const uint16_t* x;       // bf16 [T, 128, K]
  const uint32_t* words;
  const uint16_t* scales;
  int32_t group;           // 32, 64 or 128
  int32_t T;
  uint16_t* y;             // bf16 [T, 128, N]
  int32_t* dev_err;
};
// x_map, y_map (read only where w4_uses_maps(T)): x as {K, 128 heads, T} in
// boxes of 64 k x 128 tokens, 128-byte swizzle; y as {N, 128, T} in boxes of
// 32 columns x 32 tokens, 64-byte swizzle.
bool w4_uses_maps(int32_t T);
cudaError_t launch_w4_gemm(HeadGemm kind, const W4Args& args, const CUtensorMap& x_map, const CUtensorMap& y_map,
                           cudaStream_t stream);
cudaError_t launch_w4_pack(const uint16_t* w, int K, int N, int group, uint32_t* words, uint16_t* scales,
                           cudaStream_t stream);

}  // namespace mla
