// C-ABI entry points of libmla (declared in include/mla.h): argument
// validation, the page pool, slot mapping, the split-KV planner, TMA tensor
// maps and kernel launches.  No entry point allocates device memory.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <memory>
#include <mutex>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "../../include/mla.h"
#include "internal.h"

namespace {

thread_local std::string g_last_error = "no error";

// Bound of the decode kernel's waits, in SM cycles (about a second at the
// maximum clock); mla_debug_set_decode_wait_limit changes it for tests.
constexpr uint64_t kDefaultDecodeWaitLimit = 1ull << 31;
std::atomic<uint64_t> g_decode_wait_limit{kDefaultDecodeWaitLimit};

mla_status fail(mla_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

mla_status cuda_fail(cudaError_t e, const char* what) {
  return fail(MLA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

#define CHECK_PTR(p)                                                     \
  do {                                                                   \
    if ((p) == nullptr) return fail(MLA_ERR_INVALID_ARG, "%s is NULL", #p); \
  } while (0)
#define CHECK_ALIGN16(p)                                                                          \
  do {                                                                                            \
    if (!aligned16(p)) return fail(MLA_ERR_MISALIGNED, "%s is not 16-byte aligned", #p);          \
  } while (0)

constexpr int64_t kRowBytes = MLA_TOKEN_ELEMS * 2;  // 1152

// ------------------------------------------------------------------ tensor maps
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// bf16 tensor map (128-byte swizzle unless told otherwise); dims innermost
// first, strides in bytes for dims 1..rank-1.
mla_status make_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                    const uint32_t* box, const char* what,
                    CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B,
                    CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  auto fn = encode_fn();
  if (!fn) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(m, dtype, (cuuint32_t)rank, const_cast<void*>(base),
                  reinterpret_cast<const cuuint64_t*>(dims), reinterpret_cast<const cuuint64_t*>(strides),
                  reinterpret_cast<const cuuint32_t*>(box), estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with %d", what, (int)r);
  return MLA_OK;
}

// ------------------------------------------------------------------ planner
struct PlanRow {
  int32_t b;
  int32_t visible;
  int32_t npages;  // tiles the row reads
  int32_t lo;      // the window's first token (0: the row sees every token up to its own), or the tree's
  int32_t base;    // the first unpacked page of the row's sequence (trees)
};

// Minimum 64-token tiles per cluster: below it, the per-range fixed costs
// (query load, epilogue, a combine partial) outweigh the added parallelism.
constexpr int64_t kMinTilesPerCluster = 2;

// What the planned rows see.  window == 0: every token up to the row's own;
// otherwise a sliding window with sinks.  tree: the rows are the nodes of
// trees, masked within them.
struct PlanKind {
  int32_t window = 0;
  int32_t sinks = 0;
  bool tree = false;
  uint32_t magic() const { return tree ? MLA_TREE_PLAN_MAGIC : window > 0 ? MLA_WINDOW_PLAN_MAGIC : MLA_PLAN_MAGIC; }
};

// A tree plan's costs, in tiles (0.85 us).  A piece of a row takes four tiles'
// time beside its tiles: the queries into TMEM and the row out of it are 64 to
// 128 KB a CTA, while the next piece's first tile is under way (two, six and eight
// tiles are within 1 %, as long as rows are dealt out, and contiguous ranges lost
// 5 % without it: 254 rows over 1 024 to 4 096 tokens).
constexpr int64_t kTreeRowTiles = 4;
// No smaller piece is cut off a row that is dealt out (192 rows over 8 192 tokens:
// 279 us, 288 with eight tiles, 292 with two).
constexpr int64_t kTreeCrumb = 16;
// In 64ths of a tile: a partial result, 256 KB written, read and merged; and a
// round of the merge, whose number is that of the pieces of the row with most
// (one row over 8 192 tokens: 25.5 us in 64 pieces, 20.8 in 32, 19.1 in 26, 21.0 in
// 16; four rows over 4 096: 22.6 in 16 pieces each, 19.1 in 11, 20.5 in 8; 32 rows
// over 1 024: 21.6 in two, 22.6 whole).
constexpr int64_t kTreePartial = 5, kTreePiece = 16;
// The share of the L2 cache (129 MB) that a plan counts on for the sequences
// being read at one time.
constexpr int64_t kTreeSharedBytes = 64ll << 20;

// Lanes of a tree plan of fewer rows than clusters.  Rows are planned lane by lane,
// lane j holding the j-th share of every sequence's rows: the clusters of a lane
// walk the sequences together, and every lane at the same time, so that
// num_clusters / lanes sequences are being read at once, each by `lanes` clusters.
// The fewest lanes that keep those in L2, of those that divide the clusters evenly
// (two rows of 32 sequences of 8 192 tokens: 123 us in two lanes, 134 in one; four
// of 16 of 16 384: 214 in four, 240 in one).
int32_t tree_lanes(const int32_t* seq_lens, const int32_t* q_lens, int32_t B, int32_t num_clusters) {
  int64_t tokens = 0, seqs = 0;
  int32_t most = 0;
  for (int32_t b = 0; b < B; ++b)
    if (q_lens[b] > 0) {
      tokens += seq_lens[b];
      ++seqs;
      most = std::max(most, q_lens[b]);
    }
  int32_t lanes = 1;
  for (int32_t l = 1; l <= std::min(most, num_clusters); ++l) {
    if (num_clusters % l) continue;
    lanes = l;
    if (std::min<int64_t>(num_clusters / l, seqs) * (tokens / seqs) * kRowBytes <= kTreeSharedBytes) break;
  }
  return lanes;
}

mla_status build_plan(const int32_t* seq_lens, const int32_t* q_lens, int32_t B, int32_t num_clusters,
                      int32_t* out, size_t out_words, mla_plan_info* info, const PlanKind& kind = {},
                      mla_tree_info* tree_info = nullptr) {
  const int32_t window = kind.window, sinks = kind.sinks;
  if (B < 0) return fail(MLA_ERR_INVALID_ARG, "B = %d is negative", B);
  if (B > 0) {
    CHECK_PTR(seq_lens);
    CHECK_PTR(q_lens);
  }
  if (num_clusters < 1) return fail(MLA_ERR_INVALID_ARG, "num_clusters = %d < 1", num_clusters);
  std::vector<PlanRow> rows;
  std::vector<int32_t> trees;  // the plan's table
  int64_t tree_pages = 0;
  int64_t total = 0;
  int32_t max_pages = 0;
  for (int32_t b = 0; b < B; ++b) {
    const int32_t n = seq_lens[b], q = q_lens[b];
    if (n < 1) return fail(MLA_ERR_INVALID_ARG, "seq_lens[%d] = %d < 1", b, n);
    if (q < 0 || q > n) return fail(MLA_ERR_INVALID_ARG, "q_lens[%d] = %d outside [0, seq_len = %d]", b, q, n);
    if (kind.tree && q > MLA_TREE_MAX_NODES)
      return fail(MLA_ERR_UNSUPPORTED, "q_lens[%d] = %d: a tree has at most %d nodes", b, q, MLA_TREE_MAX_NODES);
    max_pages = std::max<int32_t>(max_pages, (n - 1) / MLA_PAGE_SIZE + 1);
    const int32_t base = (int32_t)std::min<int64_t>(tree_pages, INT32_MAX);
    if (kind.tree && q > 0) {
      const int32_t pages = (n - 1) / MLA_PAGE_SIZE + 1;
      trees.insert(trees.end(), {b, base, pages, n - q, n, (int32_t)rows.size(), q, 0});
      tree_pages += pages;
    }
    for (int32_t i = 0; i < q; ++i) {
      const int32_t vis = n - q + i + 1;
      int32_t np = (vis - 1) / MLA_PAGE_SIZE + 1, lo = kind.tree ? n - q : 0;
      if (window > 0 && vis - (int64_t)window > (int64_t)sinks) {  // tokens between the sinks and the window
        lo = vis - window;
        np -= mla::window_tiles(lo, sinks).skip;
      }
      rows.push_back({b, vis, np, lo, base});
      total += np;
    }
    if ((int64_t)rows.size() > (int64_t)INT32_MAX / MLA_NUM_HEADS)
      return fail(MLA_ERR_INVALID_ARG, "too many query rows");
  }
  const int64_t T = (int64_t)rows.size();
  // The order of the rows and its cut into the clusters' ranges.
  struct Seg {
    int32_t row, b, pb, pe, vis, slot, lo, base;
  };
  std::vector<Seg> segs;
  std::vector<int32_t> seg_off;
  std::vector<int32_t> row_pieces(T, 0);
  auto piece = [&](int32_t rr, int64_t pb, int64_t pe) {
    segs.push_back({rr, rows[rr].b, (int32_t)pb, (int32_t)pe, rows[rr].visible, -1, rows[rr].lo, rows[rr].base});
    ++row_pieces[rr];
  };
  // Rows in the order of `order` as one line of tiles, cut into at most `ranges` equal ranges.
  auto cut = [&](const std::vector<int32_t>& order, int64_t ranges) {
    int64_t all = 0;
    for (int32_t r : order) all += rows[r].npages;
    if (all == 0) return;
    const int64_t per = std::max<int64_t>((all + ranges - 1) / ranges, kMinTilesPerCluster);
    int64_t row_start = 0;
    size_t k = 0;  // index into order
    for (int64_t lo = 0; lo < all; lo += per) {
      const int64_t hi = std::min(all, lo + per);
      seg_off.push_back((int32_t)segs.size());
      while (k < order.size() && row_start + rows[order[k]].npages <= lo) row_start += rows[order[k++]].npages;
      int64_t rs = row_start;
      for (size_t kk = k; kk < order.size() && rs < hi; rs += rows[order[kk++]].npages) {
        const int32_t rr = order[kk];
        const int64_t pb = std::max<int64_t>(lo - rs, 0), pe = std::min<int64_t>(hi - rs, rows[rr].npages);
        if (pe > pb) piece(rr, pb, pe);
      }
    }
  };
  // The same where a piece of a row costs its tiles and kTreeRowTiles more: each
  // range takes pieces up to `budget`, none of under kMinTilesPerCluster tiles
  // unless the row has no more.  Calls begin() for a range and take(row, first,
  // last) for a piece; false when more than `ranges` ranges would be needed.
  auto fill = [&](const std::vector<int32_t>& order, int64_t ranges, int64_t budget, auto begin, auto take) {
    int64_t used = 0, left = 0;
    for (int32_t rr : order) {
      for (int64_t at = 0, n = rows[rr].npages; at < n;) {
        int64_t t = left - kTreeRowTiles;
        if (t < std::min(kMinTilesPerCluster, n - at)) {
          if (++used > ranges) return false;
          begin();
          left = budget;
          t = std::max(left - kTreeRowTiles, kMinTilesPerCluster);
        }
        if (n - at - t < kMinTilesPerCluster) t = n - at;  // no crumb stays behind
        take(rr, at, at + t);
        at += t;
        left -= t + kTreeRowTiles;
      }
    }
    return true;
  };
  // Rows dealt out one after another, each to the range with least so far: a row
  // that passes `budget` goes on in the next range, and no piece under `crumb` tiles
  // is cut off it.  Neighbouring rows, a sequence's, are then read at the same time,
  // from DRAM once, and few are cut (against contiguous ranges: 768 rows over 8 204
  // tokens 1 183 -> 1 131 us, 1 086 over 200 to 20 000 tokens 2 694 -> 2 331, 254 over
  // 1 024 to 4 096 167 -> 151).  Returns the cost of what finds no place, 0 when all
  // is dealt; take(row, range, first, last).  Begins at `from` and leaves there the
  // first row that was not taken whole: up to it a larger budget changes nothing.
  struct Deal {
    std::vector<std::pair<int64_t, int32_t>> open;  // a heap, least first: cost so far, range
    int64_t row = 0;
  };
  auto deal = [&](Deal& from, int64_t budget, auto take) {
    const int64_t crumb = std::min(std::max(budget / 4, kMinTilesPerCluster), kTreeCrumb);
    auto open = from.open;
    bool whole = true;
    auto sink = [&] {  // the first one has grown
      const size_t n = open.size();
      const auto x = open[0];
      size_t i = 0;
      for (size_t k = 1; k < n; k = 2 * i + 1) {
        if (k + 1 < n && open[k + 1] < open[k]) ++k;
        if (!(open[k] < x)) break;
        open[i] = open[k];
        i = k;
      }
      open[i] = x;
    };
    for (int64_t r = from.row; r < T; ++r) {
      for (int64_t at = 0, n = rows[r].npages; at < n;) {
        if (open.empty()) {
          int64_t rest = n - at + kTreeRowTiles;
          for (int64_t k = r + 1; k < T; ++k) rest += rows[k].npages + kTreeRowTiles;
          return rest;
        }
        int64_t t = std::min(budget - open[0].first - kTreeRowTiles, n - at);
        if (whole && t < n) {
          whole = false;
          from = {open, r};
        }
        if (t < std::min(crumb, n - at)) {
          open[0] = open.back();
          open.pop_back();
        } else {
          if (n - at - t < kMinTilesPerCluster) t = n - at;  // no crumb stays behind
          take((int32_t)r, open[0].second, at, at + t);
          at += t;
          open[0].first += t + kTreeRowTiles;
        }
        if (!open.empty()) sink();
      }
    }
    return (int64_t)0;
  };
  // What a plan costs beside its longest range: partial results and the merge.
  struct Merge {
    int64_t partials = 0, most = 0, run = 0;
    int32_t of = -1;
    void add(int32_t row) {  // the pieces of a row come one after another
      run = row == of ? run + 1 : 1;
      of = row;
      partials += run == 1 ? 0 : run == 2 ? 2 : 1;
      most = std::max(most, run);
    }
    int64_t cost(int64_t budget) const { return 64 * budget + kTreePartial * partials + (most > 1 ? kTreePiece * most : 0); }
  };
  if (kind.tree && T >= num_clusters) {
    struct Dealt {
      int32_t row, range;
      int64_t pb, pe;
    };
    std::vector<Dealt> best, now;
    int64_t best_cost = INT64_MAX, best_ranges = 0;
    // All ranges, or fewer that take whole rows alike.
    const int64_t each = (T + num_clusters - 1) / num_clusters, even = (T + each - 1) / each;
    for (int64_t ranges = num_clusters; ranges; ranges = ranges > even ? even : 0) {
      int64_t budget = (total + kTreeRowTiles * T + ranges - 1) / ranges, rest;
      Deal from;
      for (int32_t c = 0; c < ranges; ++c) from.open.push_back({0, c});
      Merge m;
      now.clear();
      while ((rest = (now.resize(from.row), m = {}, deal(from, budget, [&](int32_t row, int32_t c, int64_t pb, int64_t pe) {
                now.push_back({row, c, pb, pe});
                m.add(row);
              }))) > 0)
        budget += 1 + std::min(rest / ranges, budget / 256);
      if (m.cost(budget) < best_cost) {
        best_cost = m.cost(budget);
        best_ranges = ranges;
        best.swap(now);
      }
    }
    // A range's pieces are walked last first: the ones cut short then come at the
    // start, and the ranges do not change rows all at the same time (254 rows 158 ->
    // 153 us, 256 over 4 096 tokens 207 -> 201).
    std::vector<std::vector<const Dealt*>> of(best_ranges);
    for (const Dealt& d : best) of[d.range].push_back(&d);
    for (const auto& range : of) {
      if (range.empty()) continue;
      seg_off.push_back((int32_t)segs.size());
      for (auto d = range.rbegin(); d != range.rend(); ++d) piece((*d)->row, (*d)->pb, (*d)->pe);
    }
  } else if (kind.tree) {
    std::vector<int32_t> order;
    order.reserve(rows.size());
    const int32_t lanes = tree_lanes(seq_lens, q_lens, B, num_clusters);
    for (int32_t lane = 0; lane < lanes; ++lane) {
      int32_t r = 0;
      for (int32_t b = 0; b < B; r += q_lens[b++])
        for (int64_t i = (int64_t)q_lens[b] * lane / lanes; i < (int64_t)q_lens[b] * (lane + 1) / lanes; ++i)
          order.push_back(r + (int32_t)i);
    }
    // As many ranges as pay: each further piece of a row is a partial result to
    // write, read and merge.
    int64_t best_ranges = 0, best_budget = 0, best_cost = INT64_MAX;
    for (int64_t ranges = num_clusters; total > 0 && ranges >= 1; ranges = std::min(ranges - 1, ranges * 7 / 8)) {
      int64_t budget = (total + kTreeRowTiles * std::max<int64_t>(T, ranges) + ranges - 1) / ranges;
      Merge m;
      while (m = {}, !fill(order, ranges, budget, [] {}, [&](int32_t rr, int64_t, int64_t) { m.add(rr); })) budget += 1 + budget / 1024;
      if (m.cost(budget) < best_cost) {
        best_cost = m.cost(budget);
        best_ranges = ranges;
        best_budget = budget;
      }
    }
    if (total > 0)
      fill(order, best_ranges, best_budget, [&] { seg_off.push_back((int32_t)segs.size()); }, piece);
  } else {
    // Lanes: when every sequence has the same number Q >= 2 of query rows
    // (multi-token decode), the clusters are split into Q lanes and lane j takes
    // row j of every sequence, cut into equal contiguous tile ranges the same
    // way in every lane.  Cluster c of each lane then reads the same pages at
    // nearly the same time, so the rows of a sequence share one DRAM read of
    // each page through L2.  Otherwise there is one lane over all rows.
    int32_t lanes = 1, q0 = -1;
    bool uniform = true;
    for (int32_t b = 0; b < B; ++b) {
      if (q_lens[b] == 0) continue;
      if (q0 < 0) q0 = q_lens[b];
      uniform = uniform && q_lens[b] == q0;
    }
    if (uniform && q0 >= 2 && num_clusters / q0 >= 1) lanes = q0;
    std::vector<std::vector<int32_t>> lane_rows(lanes);
    int32_t r = 0;
    for (int32_t b = 0; b < B; ++b)
      for (int32_t i = 0; i < q_lens[b]; ++i, ++r) lane_rows[lanes == 1 ? 0 : i].push_back(r);
    for (const std::vector<int32_t>& order : lane_rows) cut(order, num_clusters / lanes);
  }
  const int64_t used = (int64_t)seg_off.size();
  seg_off.push_back((int32_t)segs.size());
  // partial slots for rows cut into several pieces, contiguous per row
  std::vector<int32_t> split;  // {row, slot_begin, n, 0}
  int32_t nslots = 0;
  {
    std::vector<Seg*> cut_up;
    for (auto& s : segs)
      if (row_pieces[s.row] > 1) cut_up.push_back(&s);
    if (kind.tree)  // dealt pieces of a row lie apart
      std::sort(cut_up.begin(), cut_up.end(), [](const Seg* x, const Seg* y) { return x->row != y->row ? x->row < y->row : x->pb < y->pb; });
    int32_t last_row = -1;
    for (Seg* s : cut_up) {
      if (s->row != last_row) {
        split.insert(split.end(), {s->row, nslots, row_pieces[s->row], 0});
        last_row = s->row;
      }
      s->slot = nslots++;
    }
  }
  const int64_t nsplit = (int64_t)split.size() / mla::kSplitWords;
  const mla::PlanLayout L = mla::plan_layout(used, (int64_t)segs.size(), nsplit);
  const int64_t words = L.words + (int64_t)trees.size();
  if ((size_t)words > out_words)
    return fail(MLA_ERR_INVALID_ARG, "plan buffer holds %zu bytes, %lld needed", out_words * 4, (long long)words * 4);
  std::fill(out, out + words, 0);
  const uint32_t magic = kind.magic();
  out[0] = (int32_t)magic;
  out[1] = (int32_t)T;
  out[2] = B;
  out[3] = (int32_t)used;
  out[4] = (int32_t)segs.size();
  out[5] = nslots;
  out[6] = (int32_t)nsplit;
  out[7] = max_pages;
  std::copy(seg_off.begin(), seg_off.end(), out + L.seg_off);
  for (size_t i = 0; i < segs.size(); ++i) {
    int32_t* w = out + L.seg_base + mla::kSegWords * i;
    w[0] = segs[i].row;
    w[1] = segs[i].b;
    w[2] = segs[i].pb;
    w[3] = segs[i].pe;
    w[4] = segs[i].vis;
    w[5] = segs[i].slot;
    w[6] = segs[i].lo;
    w[7] = kind.tree ? segs[i].base : 0;
  }
  std::copy(split.begin(), split.end(), out + L.split_base);
  std::copy(trees.begin(), trees.end(), out + L.words);
  if (info) {
    info->magic = magic;
    info->T = (int32_t)T;
    info->B = B;
    info->num_clusters = (int32_t)used;
    info->num_segments = (int32_t)segs.size();
    info->num_partials = nslots;
    info->num_split_rows = (int32_t)nsplit;
    info->max_pages_needed = max_pages;
    info->total_tiles = total;
    info->plan_bytes = (size_t)words * 4;
  }
  if (tree_info) {
    tree_info->max_nodes = 0;
    for (size_t i = 6; i < trees.size(); i += mla::kTreeWords) tree_info->max_nodes = std::max(tree_info->max_nodes, trees[i]);
    tree_info->num_trees = (int32_t)(trees.size() / mla::kTreeWords);
    tree_info->total_pages = tree_pages;
  }
  return MLA_OK;
}

// The factor of an exponent of 2.  The kernels take it in fp16 too, where less than
// 2^-24 would be 0, and 0 times the -infinity of a hidden score is no weight of 0;
// raised to 2^-24 it moves no score that fits fp16 by more than 2^-8.
float scale_log2(float scale) { return std::max((float)((double)scale * 1.4426950408889634), 0x1p-24f); }

// A call whose body may run out of host memory: no exception passes.
template <typename F>
mla_status no_throw(F&& body) {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return fail(MLA_ERR_NO_SPACE, "out of host memory");
  }
}

// A tree decode unpacks at most so many pages of the FP8 cache (4.8 GB).
constexpr int64_t kMostUnpackedPages = 1 << 16;
constexpr int64_t kUnpackTiles = 512;

size_t workspace_bytes_for(int64_t partials) {
  return (size_t)partials * (MLA_NUM_HEADS * MLA_LATENT_DIM * 4 + MLA_NUM_HEADS * 4);
}

}  // namespace

namespace mla {
mla_status set_last_error(mla_status s, const char* message) { return fail(s, "%s", message); }

PlanLayout plan_layout(int64_t num_clusters, int64_t num_segments, int64_t num_split_rows) {
  PlanLayout L;
  L.seg_off = kPlanHeader;
  L.seg_base = (L.seg_off + num_clusters + 1 + 7) / 8 * 8;
  L.split_base = L.seg_base + kSegWords * num_segments;
  L.words = L.split_base + kSplitWords * num_split_rows;
  return L;
}
}  // namespace mla

struct mla_pool {
  std::vector<int32_t> refs;  // holders of each page, 0: free
  int32_t free_count = 0;
};

extern "C" {

const char* mla_last_error(void) { return g_last_error.c_str(); }

const char* mla_status_string(mla_status s) {
  switch (s) {
    case MLA_OK: return "MLA_OK";
    case MLA_ERR_INVALID_ARG: return "MLA_ERR_INVALID_ARG";
    case MLA_ERR_MISALIGNED: return "MLA_ERR_MISALIGNED";
    case MLA_ERR_UNSUPPORTED: return "MLA_ERR_UNSUPPORTED";
    case MLA_ERR_CUDA: return "MLA_ERR_CUDA";
    case MLA_ERR_DEVICE: return "MLA_ERR_DEVICE";
    case MLA_ERR_TIMEOUT: return "MLA_ERR_TIMEOUT";
    case MLA_ERR_NO_SPACE: return "MLA_ERR_NO_SPACE";
  }
  return "MLA_ERR_UNKNOWN";
}

int32_t mla_version(void) { return 101; }

mla_config mla_config_default(void) {
  mla_config c;
  c.num_heads = MLA_NUM_HEADS;
  c.head_dim_c = MLA_HEAD_DIM_C;
  c.latent_dim = MLA_LATENT_DIM;
  c.rope_dim = MLA_ROPE_DIM;
  c.page_size = MLA_PAGE_SIZE;
  c.scale = (float)(1.0 / std::sqrt((double)(MLA_HEAD_DIM_C + MLA_ROPE_DIM)));
  return c;
}

mla_status mla_config_validate(const mla_config* cfg) {
  CHECK_PTR(cfg);
  if (cfg->num_heads != MLA_NUM_HEADS || cfg->head_dim_c != MLA_HEAD_DIM_C || cfg->latent_dim != MLA_LATENT_DIM ||
      cfg->rope_dim != MLA_ROPE_DIM || cfg->page_size != MLA_PAGE_SIZE)
    return fail(MLA_ERR_UNSUPPORTED, "only heads=128, d_hc=128, d_c=512, d_r=64, page_size=64 are supported");
  if (!(cfg->scale > 0.f) || !std::isfinite(cfg->scale))
    return fail(MLA_ERR_INVALID_ARG, "scale must be finite and positive");
  return MLA_OK;
}

mla_status mla_kv_bytes(int64_t layers, int64_t dc, int64_t dr, int64_t elem_bytes, int64_t tokens, int64_t seqs,
                        uint64_t* out) {
  CHECK_PTR(out);
  if (layers <= 0 || dc <= 0 || elem_bytes <= 0 || tokens <= 0 || seqs <= 0 || dr < 0)
    return fail(MLA_ERR_INVALID_ARG, "invalid dimension");
  uint64_t acc = (uint64_t)layers, t;
  if (__builtin_add_overflow((uint64_t)dc, (uint64_t)dr, &t) || __builtin_mul_overflow(acc, t, &acc) ||
      __builtin_mul_overflow(acc, (uint64_t)elem_bytes, &acc) || __builtin_mul_overflow(acc, (uint64_t)tokens, &acc) ||
      __builtin_mul_overflow(acc, (uint64_t)seqs, &acc))
    return fail(MLA_ERR_INVALID_ARG, "byte count overflows uint64");
  *out = acc;
  return MLA_OK;
}

// ------------------------------------------------------------------ pool
mla_status mla_pool_create(int32_t num_pages, mla_pool** out) {
  CHECK_PTR(out);
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages = %d < 1", num_pages);
  return no_throw([&] {
    auto p = std::make_unique<mla_pool>();
    p->refs.assign((size_t)num_pages, 0);
    p->free_count = num_pages;
    *out = p.release();
    return MLA_OK;
  });
}

// Takes n free pages, lowest first; the caller has seen that there are so many.
static void pool_take(mla_pool* pool, int32_t n, int32_t* ids) {
  int32_t k = 0;
  for (size_t i = 0; i < pool->refs.size() && k < n; ++i)
    if (!pool->refs[i]) {
      pool->refs[i] = 1;
      ids[k++] = (int32_t)i;
    }
  pool->free_count -= n;
}

static mla_status pool_held(const mla_pool* pool, int32_t id) {
  if (id < 0 || (size_t)id >= pool->refs.size()) return fail(MLA_ERR_INVALID_ARG, "page id %d out of range", id);
  if (!pool->refs[id]) return fail(MLA_ERR_INVALID_ARG, "page id %d is not allocated", id);
  return MLA_OK;
}

mla_status mla_pool_alloc(mla_pool* pool, int32_t n, int32_t* ids) {
  CHECK_PTR(pool);
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(ids);
  if (n > pool->free_count)
    return fail(MLA_ERR_NO_SPACE, "%d pages requested, %d free", n, pool->free_count);
  pool_take(pool, n, ids);
  return MLA_OK;
}

mla_status mla_pool_free(mla_pool* pool, const int32_t* ids, int32_t n) {
  CHECK_PTR(pool);
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(ids);
  return no_throw([&] {
    std::vector<uint8_t> seen(pool->refs.size(), 0);
    for (int32_t i = 0; i < n; ++i) {
      const mla_status s = pool_held(pool, ids[i]);
      if (s != MLA_OK) return s;
      if (seen[ids[i]]) return fail(MLA_ERR_INVALID_ARG, "page id %d repeated", ids[i]);
      seen[ids[i]] = 1;
    }
    for (int32_t i = 0; i < n; ++i)
      if (--pool->refs[ids[i]] == 0) ++pool->free_count;
    return MLA_OK;
  });
}

mla_status mla_pool_retain(mla_pool* pool, const int32_t* ids, int32_t n) {
  CHECK_PTR(pool);
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(ids);
  for (int32_t i = 0; i < n; ++i) {
    const mla_status s = pool_held(pool, ids[i]);
    if (s != MLA_OK) return s;
    if (pool->refs[ids[i]] > INT32_MAX - n) return fail(MLA_ERR_INVALID_ARG, "page id %d has too many holders", ids[i]);
  }
  for (int32_t i = 0; i < n; ++i) ++pool->refs[ids[i]];
  return MLA_OK;
}

mla_status mla_pool_refs(const mla_pool* pool, int32_t id, int32_t* out) {
  CHECK_PTR(pool);
  CHECK_PTR(out);
  if (id < 0 || (size_t)id >= pool->refs.size()) return fail(MLA_ERR_INVALID_ARG, "page id %d out of range", id);
  *out = pool->refs[id];
  return MLA_OK;
}

mla_status mla_pool_fork(mla_pool* pool, const int32_t* parent, int32_t n_tokens, int32_t n_children,
                         int32_t max_pages, int32_t* children, int32_t* src, int32_t* dst, int32_t* n_copies) {
  CHECK_PTR(pool);
  CHECK_PTR(n_copies);
  if (n_tokens < 0 || n_children < 0 || max_pages < 0)
    return fail(MLA_ERR_INVALID_ARG, "n_tokens = %d, n_children = %d, max_pages = %d: negative", n_tokens, n_children,
                max_pages);
  const int32_t full = n_tokens / MLA_PAGE_SIZE, pages = full + (n_tokens % MLA_PAGE_SIZE != 0);
  if (pages > max_pages)
    return fail(MLA_ERR_INVALID_ARG, "n_tokens = %d needs more than max_pages = %d pages", n_tokens, max_pages);
  *n_copies = 0;
  if (n_children == 0) return MLA_OK;
  const int32_t copies = pages > full ? n_children : 0;
  if (max_pages > 0) CHECK_PTR(children);
  if (pages > 0) CHECK_PTR(parent);
  if (copies) {
    CHECK_PTR(src);
    CHECK_PTR(dst);
  }
  return no_throw([&] {
    const std::vector<int32_t> held(parent, parent + pages);  // `children` may hold the parent's row
    std::vector<int32_t> sorted(held);
    std::sort(sorted.begin(), sorted.end());
    for (int32_t k = 0; k < pages; ++k) {
      const mla_status s = pool_held(pool, held[k]);
      if (s != MLA_OK) return s;
      if (k && sorted[k] == sorted[k - 1]) return fail(MLA_ERR_INVALID_ARG, "page id %d repeated", sorted[k]);
      if (pool->refs[held[k]] > INT32_MAX - n_children)
        return fail(MLA_ERR_INVALID_ARG, "page id %d has too many holders", held[k]);
    }
    if (copies > pool->free_count)
      return fail(MLA_ERR_NO_SPACE, "%d pages requested, %d free", copies, pool->free_count);
    std::vector<int32_t> fresh((size_t)copies);
    if (copies) pool_take(pool, copies, fresh.data());
    for (int32_t i = 0; i < n_children; ++i) {
      int32_t* row = children + (int64_t)i * max_pages;
      std::fill(row, row + max_pages, -1);
      for (int32_t k = 0; k < full; ++k) row[k] = held[k];
      if (copies) {
        row[full] = fresh[i];
        src[i] = held[full];
        dst[i] = fresh[i];
      }
    }
    for (int32_t k = 0; k < full; ++k) pool->refs[held[k]] += n_children;
    *n_copies = copies;
    return MLA_OK;
  });
}

mla_status mla_pool_compact(mla_pool* pool, int32_t max_moves, int32_t* src, int32_t* dst, int32_t* n_moves) {
  CHECK_PTR(pool);
  CHECK_PTR(n_moves);
  if (max_moves < 0) return fail(MLA_ERR_INVALID_ARG, "max_moves = %d < 0", max_moves);
  if (max_moves > 0) {
    CHECK_PTR(src);
    CHECK_PTR(dst);
  }
  int32_t n = 0;
  int64_t lo = 0, hi = (int64_t)pool->refs.size() - 1;
  while (n < max_moves) {
    while (lo < hi && pool->refs[lo]) ++lo;
    while (lo < hi && !pool->refs[hi]) --hi;
    if (lo >= hi) break;
    std::swap(pool->refs[lo], pool->refs[hi]);
    src[n] = (int32_t)hi;
    dst[n++] = (int32_t)lo;
  }
  *n_moves = n;
  return MLA_OK;
}

mla_status mla_remap_pages(int32_t* block_table, int64_t entries, const int32_t* src, const int32_t* dst, int32_t n) {
  if (n < 0 || entries < 0)
    return fail(MLA_ERR_INVALID_ARG, "n = %d, entries = %lld: negative", n, (long long)entries);
  if (n == 0 || entries == 0) return MLA_OK;
  CHECK_PTR(block_table);
  CHECK_PTR(src);
  CHECK_PTR(dst);
  return no_throw([&] {
    std::vector<std::pair<int32_t, int32_t>> moves((size_t)n);
    for (int32_t i = 0; i < n; ++i) {
      if (src[i] < 0 || dst[i] < 0) return fail(MLA_ERR_INVALID_ARG, "move %d: a page id is negative", i);
      moves[i] = {src[i], dst[i]};
    }
    std::sort(moves.begin(), moves.end());
    for (int32_t i = 1; i < n; ++i)
      if (moves[i].first == moves[i - 1].first) return fail(MLA_ERR_INVALID_ARG, "page id %d repeated", moves[i].first);
    for (int64_t i = 0; i < entries; ++i) {
      const auto at = std::lower_bound(moves.begin(), moves.end(), std::make_pair(block_table[i], INT32_MIN));
      if (at != moves.end() && at->first == block_table[i]) block_table[i] = at->second;
    }
    return MLA_OK;
  });
}

mla_status mla_pool_available(const mla_pool* pool, int32_t* out) {
  CHECK_PTR(pool);
  CHECK_PTR(out);
  *out = pool->free_count;
  return MLA_OK;
}

void mla_pool_destroy(mla_pool* pool) { delete pool; }

mla_status mla_slot_mapping(const int32_t* block_table, int32_t batch, int32_t max_pages, const int32_t* seq_ids,
                            const int32_t* positions, int32_t n, int64_t* slots_out) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(block_table);
  CHECK_PTR(seq_ids);
  CHECK_PTR(positions);
  CHECK_PTR(slots_out);
  if (batch < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "batch and max_pages must be >= 1");
  for (int32_t i = 0; i < n; ++i) {
    const int32_t b = seq_ids[i], pos = positions[i];
    if (b < 0 || b >= batch) return fail(MLA_ERR_INVALID_ARG, "seq_ids[%d] = %d out of range", i, b);
    if (pos < 0 || pos / MLA_PAGE_SIZE >= max_pages)
      return fail(MLA_ERR_INVALID_ARG, "positions[%d] = %d beyond the block table", i, pos);
    const int32_t page = block_table[(int64_t)b * max_pages + pos / MLA_PAGE_SIZE];
    if (page < 0) return fail(MLA_ERR_INVALID_ARG, "no page mapped for sequence %d position %d", b, pos);
    slots_out[i] = (int64_t)page * MLA_PAGE_SIZE + pos % MLA_PAGE_SIZE;
  }
  return MLA_OK;
}

// ------------------------------------------------------------------ device steps
mla_status mla_cache_init(void* kv_cache, int64_t num_pages, void* stream) {
  CHECK_PTR(kv_cache);
  CHECK_ALIGN16(kv_cache);
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages = %lld < 1", (long long)num_pages);
  cudaError_t e = cudaMemsetAsync(kv_cache, 0, (size_t)num_pages * MLA_PAGE_BYTES, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  return MLA_OK;
}

mla_status mla_kv_append(const void* c_kv_new, const void* k_r_new, const int64_t* slots, int32_t n, void* kv_cache,
                         int64_t num_pages, int32_t* dev_err, void* stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(c_kv_new);
  CHECK_PTR(k_r_new);
  CHECK_PTR(slots);
  CHECK_PTR(kv_cache);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(c_kv_new);
  CHECK_ALIGN16(k_r_new);
  CHECK_ALIGN16(kv_cache);
  if (!aligned(slots, 8)) return fail(MLA_ERR_MISALIGNED, "slots is not 8-byte aligned");
  if (!aligned(dev_err, 4)) return fail(MLA_ERR_MISALIGNED, "dev_err is not 4-byte aligned");
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages = %lld < 1", (long long)num_pages);
  cudaError_t e = mla::launch_kv_append((const uint16_t*)c_kv_new, (const uint16_t*)k_r_new, slots, n,
                                        (uint16_t*)kv_cache, num_pages * MLA_PAGE_SIZE, dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
  return MLA_OK;
}

mla_status mla_rope_table(int32_t max_pos, float base, float* table, void* stream) {
  if (max_pos < 0 || max_pos > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "max_pos = %d outside [0, 2^24]", max_pos);
  if (!(base > 1.f) || !std::isfinite(base)) return fail(MLA_ERR_INVALID_ARG, "base must be finite and > 1");
  if (max_pos == 0) return MLA_OK;
  CHECK_PTR(table);
  CHECK_ALIGN16(table);
  cudaError_t e = mla::launch_rope_table(table, max_pos, (double)base, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "rope_table launch");
  return MLA_OK;
}

mla_status mla_kv_append_rope(const void* c_kv_new, const void* k_pe_new, const int32_t* positions, const float* table,
                              int32_t max_pos, const int64_t* slots, int32_t n, void* kv_cache, int64_t num_pages,
                              int32_t* dev_err, void* stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(c_kv_new);
  CHECK_PTR(k_pe_new);
  CHECK_PTR(positions);
  CHECK_PTR(table);
  CHECK_PTR(slots);
  CHECK_PTR(kv_cache);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(c_kv_new);
  CHECK_ALIGN16(k_pe_new);
  CHECK_ALIGN16(kv_cache);
  CHECK_ALIGN16(table);
  if (!aligned(slots, 8)) return fail(MLA_ERR_MISALIGNED, "slots is not 8-byte aligned");
  if (!aligned(positions, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "positions and dev_err must be 4-byte aligned");
  if (max_pos < 1) return fail(MLA_ERR_INVALID_ARG, "max_pos = %d < 1", max_pos);
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages = %lld < 1", (long long)num_pages);
  cudaError_t e = mla::launch_kv_append_rope((const uint16_t*)c_kv_new, (const uint16_t*)k_pe_new, positions, table,
                                             max_pos, slots, n, (uint16_t*)kv_cache, num_pages * MLA_PAGE_SIZE,
                                             dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv_append_rope launch");
  return MLA_OK;
}

mla_status mla_rope_q(const void* q_pe, const int32_t* positions, const float* table, int32_t max_pos, void* q_r,
                      int32_t T, int32_t* dev_err, void* stream) {
  if (T < 0) return fail(MLA_ERR_INVALID_ARG, "T = %d < 0", T);
  if (T == 0) return MLA_OK;
  CHECK_PTR(q_pe);
  CHECK_PTR(positions);
  CHECK_PTR(table);
  CHECK_PTR(q_r);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(q_pe);
  CHECK_ALIGN16(q_r);
  if (!aligned(positions, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "positions and dev_err must be 4-byte aligned");
  CHECK_ALIGN16(table);
  if (max_pos < 1) return fail(MLA_ERR_INVALID_ARG, "max_pos = %d < 1", max_pos);
  const uintptr_t a0 = (uintptr_t)q_pe, b0 = (uintptr_t)q_r, len = (uintptr_t)T * MLA_NUM_HEADS * MLA_ROPE_DIM * 2;
  if (a0 < b0 + len && b0 < a0 + len) return fail(MLA_ERR_INVALID_ARG, "q_pe and q_r overlap");
  cudaError_t e = mla::launch_rope_q((const uint16_t*)q_pe, positions, table, max_pos, (uint16_t*)q_r, T, dev_err,
                                     (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "rope_q launch");
  return MLA_OK;
}

mla_status mla_gather_paged(const void* kv_cache, int64_t num_pages, const int32_t* block_table, int32_t max_pages,
                            int32_t b, int32_t n_tokens, void* out, int32_t* dev_err, void* stream) {
  if (n_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "n_tokens = %d < 0", n_tokens);
  if (n_tokens == 0) return MLA_OK;
  CHECK_PTR(kv_cache);
  CHECK_PTR(block_table);
  CHECK_PTR(out);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(kv_cache);
  CHECK_ALIGN16(out);
  if (num_pages < 1 || max_pages < 1 || b < 0) return fail(MLA_ERR_INVALID_ARG, "bad pool/table sizes");
  if ((n_tokens + MLA_PAGE_SIZE - 1) / MLA_PAGE_SIZE > max_pages)
    return fail(MLA_ERR_INVALID_ARG, "n_tokens = %d needs more than max_pages = %d pages", n_tokens, max_pages);
  cudaError_t e = mla::launch_gather((const uint16_t*)kv_cache, num_pages, block_table, max_pages, b, n_tokens,
                                     (uint16_t*)out, dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "gather launch");
  return MLA_OK;
}

mla_status mla_kv_append_fp8(const void* c_kv_new, const void* k_r_new, const int64_t* slots, int32_t n,
                             void* rows, float* scales, int64_t num_pages, int32_t* dev_err, void* stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(c_kv_new);
  CHECK_PTR(k_r_new);
  CHECK_PTR(slots);
  CHECK_PTR(rows);
  CHECK_PTR(scales);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(c_kv_new);
  CHECK_ALIGN16(k_r_new);
  CHECK_ALIGN16(rows);
  CHECK_ALIGN16(scales);
  if (!aligned(slots, 8)) return fail(MLA_ERR_MISALIGNED, "slots is not 8-byte aligned");
  if (!aligned(dev_err, 4)) return fail(MLA_ERR_MISALIGNED, "dev_err is not 4-byte aligned");
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages = %lld < 1", (long long)num_pages);
  cudaError_t e = mla::launch_kv_append_fp8((const uint16_t*)c_kv_new, (const uint16_t*)k_r_new, slots, n,
                                            (uint8_t*)rows, scales, num_pages * MLA_PAGE_SIZE, dev_err,
                                            (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv_append_fp8 launch");
  return MLA_OK;
}

mla_status mla_kv_append_rope_fp8(const void* c_kv_new, const void* k_pe_new, const void* q_pe,
                                  const int32_t* positions, const float* table, int32_t max_pos,
                                  const int64_t* slots, int32_t n, void* rows, float* scales, int64_t num_pages,
                                  void* q_r, int32_t* dev_err, void* stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(c_kv_new);
  CHECK_PTR(k_pe_new);
  CHECK_PTR(positions);
  CHECK_PTR(table);
  CHECK_PTR(slots);
  CHECK_PTR(rows);
  CHECK_PTR(scales);
  CHECK_PTR(dev_err);
  if ((q_pe == nullptr) != (q_r == nullptr))
    return fail(MLA_ERR_INVALID_ARG, "q_pe and q_r must be given together");
  CHECK_ALIGN16(c_kv_new);
  CHECK_ALIGN16(k_pe_new);
  CHECK_ALIGN16(q_pe);
  CHECK_ALIGN16(q_r);
  CHECK_ALIGN16(table);
  CHECK_ALIGN16(rows);
  CHECK_ALIGN16(scales);
  if (!aligned(slots, 8)) return fail(MLA_ERR_MISALIGNED, "slots is not 8-byte aligned");
  if (!aligned(positions, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "positions and dev_err must be 4-byte aligned");
  if (max_pos < 1) return fail(MLA_ERR_INVALID_ARG, "max_pos = %d < 1", max_pos);
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages = %lld < 1", (long long)num_pages);
  if (q_pe) {
    const uintptr_t a0 = (uintptr_t)q_pe, b0 = (uintptr_t)q_r, len = (uintptr_t)n * MLA_NUM_HEADS * MLA_ROPE_DIM * 2;
    if (a0 < b0 + len && b0 < a0 + len) return fail(MLA_ERR_INVALID_ARG, "q_pe and q_r overlap");
  }
  cudaError_t e = mla::launch_kv_append_rope_fp8((const uint16_t*)c_kv_new, (const uint16_t*)k_pe_new,
                                                 (const uint16_t*)q_pe, positions, table, max_pos, slots, n,
                                                 (uint8_t*)rows, scales, (uint16_t*)q_r, num_pages * MLA_PAGE_SIZE,
                                                 dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv_append_rope_fp8 launch");
  return MLA_OK;
}

mla_status mla_gather_paged_fp8(const void* rows, const float* scales, int64_t num_pages,
                                const int32_t* block_table, int32_t max_pages, int32_t b, int32_t n_tokens,
                                void* out, int32_t* dev_err, void* stream) {
  if (n_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "n_tokens = %d < 0", n_tokens);
  if (n_tokens == 0) return MLA_OK;
  CHECK_PTR(rows);
  CHECK_PTR(scales);
  CHECK_PTR(block_table);
  CHECK_PTR(out);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(rows);
  CHECK_ALIGN16(scales);
  CHECK_ALIGN16(out);
  if (!aligned(block_table, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "block_table and dev_err must be 4-byte aligned");
  if (num_pages < 1 || max_pages < 1 || b < 0) return fail(MLA_ERR_INVALID_ARG, "bad pool/table sizes");
  if ((n_tokens + MLA_PAGE_SIZE - 1) / MLA_PAGE_SIZE > max_pages)
    return fail(MLA_ERR_INVALID_ARG, "n_tokens = %d needs more than max_pages = %d pages", n_tokens, max_pages);
  cudaError_t e = mla::launch_gather_fp8((const uint8_t*)rows, scales, num_pages, block_table, max_pages, b,
                                         n_tokens, (uint16_t*)out, dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "gather_fp8 launch");
  return MLA_OK;
}

mla_status mla_kv_append_nvfp4(const void* c_kv_new, const void* k_r_new, const int64_t* slots, int32_t n,
                               float tensor_scale, void* rows, int64_t num_pages, int32_t* dev_err,
                               void* stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  if (!(tensor_scale > 0.f) || !std::isfinite(tensor_scale))
    return fail(MLA_ERR_INVALID_ARG, "tensor_scale must be finite and > 0");
  CHECK_PTR(c_kv_new);
  CHECK_PTR(k_r_new);
  CHECK_PTR(slots);
  CHECK_PTR(rows);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(c_kv_new);
  CHECK_ALIGN16(k_r_new);
  CHECK_ALIGN16(rows);
  if (!aligned(slots, 8)) return fail(MLA_ERR_MISALIGNED, "slots is not 8-byte aligned");
  if (!aligned(dev_err, 4)) return fail(MLA_ERR_MISALIGNED, "dev_err is not 4-byte aligned");
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages = %lld < 1", (long long)num_pages);
  cudaError_t e = mla::launch_kv_append_nvfp4((const uint16_t*)c_kv_new, (const uint16_t*)k_r_new, slots, n,
                                              tensor_scale, (uint8_t*)rows, num_pages * MLA_PAGE_SIZE, dev_err,
                                              (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv_append_nvfp4 launch");
  return MLA_OK;
}

mla_status mla_gather_paged_nvfp4(const void* rows, float tensor_scale, int64_t num_pages,
                                  const int32_t* block_table, int32_t max_pages, int32_t b, int32_t n_tokens,
                                  void* out, int32_t* dev_err, void* stream) {
  if (n_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "n_tokens = %d < 0", n_tokens);
  if (n_tokens == 0) return MLA_OK;
  if (!(tensor_scale > 0.f) || !std::isfinite(tensor_scale))
    return fail(MLA_ERR_INVALID_ARG, "tensor_scale must be finite and > 0");
  CHECK_PTR(rows);
  CHECK_PTR(block_table);
  CHECK_PTR(out);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(rows);
  CHECK_ALIGN16(out);
  if (!aligned(block_table, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "block_table and dev_err must be 4-byte aligned");
  if (num_pages < 1 || max_pages < 1 || b < 0) return fail(MLA_ERR_INVALID_ARG, "bad pool/table sizes");
  if ((n_tokens + MLA_PAGE_SIZE - 1) / MLA_PAGE_SIZE > max_pages)
    return fail(MLA_ERR_INVALID_ARG, "n_tokens = %d needs more than max_pages = %d pages", n_tokens, max_pages);
  cudaError_t e = mla::launch_gather_nvfp4((const uint8_t*)rows, tensor_scale, num_pages, block_table, max_pages, b,
                                           n_tokens, (uint16_t*)out, dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "gather_nvfp4 launch");
  return MLA_OK;
}

mla_status mla_gather_paged_nvfp4_batch(const void* rows, float tensor_scale, int64_t num_pages,
                                        const int32_t* block_table, int32_t B, int32_t max_pages,
                                        const int32_t* seq_ids, const int64_t* out_offsets, int32_t nb,
                                        int64_t total_tokens, void* out, int32_t* dev_err, void* stream) {
  if (nb < 0 || total_tokens < 0)
    return fail(MLA_ERR_INVALID_ARG, "nb = %d, total_tokens = %lld: negative", nb, (long long)total_tokens);
  if (nb == 0 || total_tokens == 0) return MLA_OK;
  if (!(tensor_scale > 0.f) || !std::isfinite(tensor_scale))
    return fail(MLA_ERR_INVALID_ARG, "tensor_scale must be finite and > 0");
  CHECK_PTR(rows);
  CHECK_PTR(block_table);
  CHECK_PTR(seq_ids);
  CHECK_PTR(out_offsets);
  CHECK_PTR(out);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(rows);
  CHECK_ALIGN16(out);
  if (!aligned(out_offsets, 8)) return fail(MLA_ERR_MISALIGNED, "out_offsets is not 8-byte aligned");
  if (!aligned(block_table, 4) || !aligned(seq_ids, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "block_table, seq_ids and dev_err must be 4-byte aligned");
  if (num_pages < 1 || B < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "bad pool/table sizes");
  if (total_tokens > ((int64_t)1 << 40)) return fail(MLA_ERR_INVALID_ARG, "total_tokens too large");
  cudaError_t e = mla::launch_gather_nvfp4_batch((const uint8_t*)rows, tensor_scale, num_pages, block_table, B,
                                                 max_pages, seq_ids, out_offsets, nb, total_tokens, (uint16_t*)out,
                                                 dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "gather_nvfp4_batch launch");
  return MLA_OK;
}

// Decompress-branch workspace: gathered rows [N, 576] (rounded up to 16 B),
// then K_c and V_c [N, 128, 128] bf16.
static size_t prefill_rows_bytes(int64_t N) { return ((size_t)N * kRowBytes + 15) / 16 * 16; }
static size_t prefill_ws_bytes(int64_t N) {
  return prefill_rows_bytes(N) + 2 * (size_t)N * MLA_NUM_HEADS * MLA_HEAD_DIM_C * 2;
}

static mla_status head_gemm(mla::HeadGemm kind, const void* a, const void* w, void* c, int32_t T, int32_t* dev_err,
                            void* stream) {
  if (T < 0) return fail(MLA_ERR_INVALID_ARG, "T = %d < 0", T);
  if (T == 0) return MLA_OK;
  CHECK_PTR(a);
  CHECK_PTR(w);
  CHECK_PTR(c);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(a);
  CHECK_ALIGN16(w);
  CHECK_ALIGN16(c);
  if (T > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "T = %d too large", T);
  const bool absorb = kind == mla::HeadGemm::kAbsorbQ;
  const uint64_t K = absorb ? MLA_HEAD_DIM_C : MLA_LATENT_DIM;
  const uint64_t N = absorb ? MLA_LATENT_DIM : MLA_HEAD_DIM_C;
  CUtensorMap amap, wmap;
  // activations [T, 128, K]; box = 64 of K x 1 head x 128 tokens
  const uint64_t adims[3] = {K, MLA_NUM_HEADS, (uint64_t)T};
  const uint64_t astr[2] = {K * 2, K * 2 * MLA_NUM_HEADS};
  const uint32_t abox[3] = {64, 1, 128};
  // weights [128, K, N]; box = 64 of N x 64 of K x 1 head
  const uint64_t wdims[3] = {N, K, MLA_NUM_HEADS};
  const uint64_t wstr[2] = {N * 2, N * 2 * K};
  const uint32_t wbox[3] = {64, 64, 1};
  // outputs [T, 128, N]; box = 64 of N x 1 head x 128 tokens (TMA store)
  const uint64_t cdims[3] = {N, MLA_NUM_HEADS, (uint64_t)T};
  const uint64_t cstr[2] = {N * 2, N * 2 * MLA_NUM_HEADS};
  CUtensorMap cmap;
  mla_status s = make_map(&amap, a, 3, adims, astr, abox, "activations");
  if (s != MLA_OK) return s;
  s = make_map(&wmap, w, 3, wdims, wstr, wbox, "weights");
  if (s != MLA_OK) return s;
  s = make_map(&cmap, c, 3, cdims, cstr, abox, "outputs");
  if (s != MLA_OK) return s;
  cudaError_t e = mla::launch_head_gemm(kind, amap, wmap, cmap, T, dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, absorb ? "absorb_q launch" : "up_v launch");
  return MLA_OK;
}

static mla_status window_check(int32_t window, int32_t sinks) {
  if (window < 1) return fail(MLA_ERR_INVALID_ARG, "window = %d < 1", window);
  if (sinks < 0) return fail(MLA_ERR_INVALID_ARG, "sinks = %d < 0", sinks);
  return MLA_OK;
}

// ------------------------------------------------------------------ decompress branch
int32_t mla_prefill_threshold(void) { return MLA_PREFILL_THRESHOLD; }

int32_t mla_branch_for(int32_t q_len) { return q_len >= MLA_PREFILL_THRESHOLD ? MLA_BRANCH_DECOMPRESS : MLA_BRANCH_ABSORB; }

static mla_status expand_kv(const void* rows, int32_t n, const void* w_uk, const void* w_uv, void* k_c, void* v_c,
                            int32_t* dev_err, bool early, void* stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(rows);
  CHECK_PTR(w_uk);
  CHECK_PTR(w_uv);
  CHECK_PTR(k_c);
  CHECK_PTR(v_c);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(rows);
  CHECK_ALIGN16(w_uk);
  CHECK_ALIGN16(w_uv);
  CHECK_ALIGN16(k_c);
  CHECK_ALIGN16(v_c);
  if (!aligned(dev_err, 4)) return fail(MLA_ERR_MISALIGNED, "dev_err is not 4-byte aligned");
  if (n > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "n = %d too large", n);
  CUtensorMap amap, kmap, vmap;
  // latent part of the rows [n, 576] as {512, 1 (shared by every head), n}
  const uint64_t adims[3] = {MLA_LATENT_DIM, 1, (uint64_t)n};
  const uint64_t astr[2] = {(uint64_t)kRowBytes, (uint64_t)kRowBytes};
  const uint32_t abox[3] = {64, 1, 128};
  mla_status s = make_map(&amap, rows, 3, adims, astr, abox, "latent rows");
  if (s != MLA_OK) return s;
  // W_UK [128, 128 (d_hc), 512 (d_c)] read K-major: box 64 of d_c x 64 of d_hc (one CTA's half) x 1 head
  const uint64_t kdims[3] = {MLA_LATENT_DIM, MLA_HEAD_DIM_C, MLA_NUM_HEADS};
  const uint64_t kstr[2] = {MLA_LATENT_DIM * 2, (uint64_t)MLA_LATENT_DIM * 2 * MLA_HEAD_DIM_C};
  const uint32_t kbox[3] = {64, 64, 1};
  s = make_map(&kmap, w_uk, 3, kdims, kstr, kbox, "W_UK (K-major)");
  if (s != MLA_OK) return s;
  // W_UV [128, 512 (d_c), 128 (d_hc)] as in step A5
  const uint64_t vdims[3] = {MLA_HEAD_DIM_C, MLA_LATENT_DIM, MLA_NUM_HEADS};
  const uint64_t vstr[2] = {MLA_HEAD_DIM_C * 2, (uint64_t)MLA_HEAD_DIM_C * 2 * MLA_LATENT_DIM};
  const uint32_t vbox[3] = {64, 64, 1};
  s = make_map(&vmap, w_uv, 3, vdims, vstr, vbox, "W_UV");
  if (s != MLA_OK) return s;
  // K_c, V_c [128 heads, n, 128] as {128, n, 128 heads}: box 64 x 128 tokens x 1 head (TMA stores)
  const uint64_t odims[3] = {MLA_HEAD_DIM_C, (uint64_t)n, MLA_NUM_HEADS};
  const uint64_t ostr[2] = {MLA_HEAD_DIM_C * 2, (uint64_t)n * MLA_HEAD_DIM_C * 2};
  const uint32_t obox[3] = {64, 128, 1};
  CUtensorMap kcmap, vcmap;
  s = make_map(&kcmap, k_c, 3, odims, ostr, obox, "K_c");
  if (s != MLA_OK) return s;
  s = make_map(&vcmap, v_c, 3, odims, ostr, obox, "V_c");
  if (s != MLA_OK) return s;
  cudaError_t e = mla::launch_expand_kv(amap, kmap, vmap, kcmap, vcmap, n, dev_err, early, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "expand_kv launch");
  return MLA_OK;
}

mla_status mla_expand_kv(const void* rows, int32_t n, const void* w_uk, const void* w_uv, void* k_c, void* v_c,
                         int32_t* dev_err, void* stream) {
  return expand_kv(rows, n, w_uk, w_uv, k_c, v_c, dev_err, false, stream);
}

// Tensor maps over the packed arrays of a batch (T rows of queries, N cached
// tokens in all) and the attention launch.
static mla_status prefill_attention_launch(const void* q_c, const void* q_r, int64_t T, const void* rows,
                                           const void* k_c, const void* v_c, int64_t N, const mla::PrefillArgs& a,
                                           void* stream) {
  CUtensorMap qm, rm, km, krm, vm;
  const uint32_t box3[3] = {64, 1, 128};
  const uint64_t qd[3] = {MLA_HEAD_DIM_C, MLA_NUM_HEADS, (uint64_t)T};
  const uint64_t qs[2] = {MLA_HEAD_DIM_C * 2, (uint64_t)MLA_HEAD_DIM_C * 2 * MLA_NUM_HEADS};
  const uint64_t rd[3] = {MLA_ROPE_DIM, MLA_NUM_HEADS, (uint64_t)T};
  const uint64_t rs[2] = {MLA_ROPE_DIM * 2, (uint64_t)MLA_ROPE_DIM * 2 * MLA_NUM_HEADS};
  const uint64_t kd[3] = {MLA_HEAD_DIM_C, (uint64_t)N, MLA_NUM_HEADS};   // head-major K_c / V_c
  const uint64_t ks[2] = {MLA_HEAD_DIM_C * 2, (uint64_t)MLA_HEAD_DIM_C * 2 * (uint64_t)N};
  const uint32_t kbox[3] = {64, 128, 1};
  const uint64_t krd[2] = {MLA_TOKEN_ELEMS, (uint64_t)N};
  const uint64_t krs[1] = {(uint64_t)kRowBytes};
  const uint32_t box2[2] = {64, 128};
  mla_status s = make_map(&qm, q_c, 3, qd, qs, box3, "q_c");
  if (s == MLA_OK) s = make_map(&rm, q_r, 3, rd, rs, box3, "q_r");
  if (s == MLA_OK) s = make_map(&km, k_c, 3, kd, ks, kbox, "K_c");
  if (s == MLA_OK) s = make_map(&vm, v_c, 3, kd, ks, kbox, "V_c");
  if (s == MLA_OK) s = make_map(&krm, rows, 2, krd, krs, box2, "k_R rows");
  if (s != MLA_OK) return s;
  cudaError_t e = a.window > 0 ? mla::launch_prefill_window(qm, rm, km, krm, vm, a, (cudaStream_t)stream)
                               : mla::launch_prefill_attn(qm, rm, km, krm, vm, a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefill attention launch");
  return MLA_OK;
}

mla_status mla_prefill_attention(const void* q_c, const void* q_r, int32_t M, const void* rows, const void* k_c,
                                 const void* v_c, int32_t N, float scale, void* out, int32_t* dev_err,
                                 void* stream) {
  if (M < 0 || N < 0) return fail(MLA_ERR_INVALID_ARG, "M = %d, N = %d: negative", M, N);
  if (M == 0) return MLA_OK;
  if (M > N) return fail(MLA_ERR_INVALID_ARG, "M = %d query rows exceed the N = %d cached tokens", M, N);
  if (N > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "N = %d too large", N);
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(MLA_ERR_INVALID_ARG, "scale must be finite and positive");
  CHECK_PTR(q_c);
  CHECK_PTR(q_r);
  CHECK_PTR(rows);
  CHECK_PTR(k_c);
  CHECK_PTR(v_c);
  CHECK_PTR(out);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(q_c);
  CHECK_ALIGN16(q_r);
  CHECK_ALIGN16(rows);
  CHECK_ALIGN16(k_c);
  CHECK_ALIGN16(v_c);
  CHECK_ALIGN16(out);
  if (!aligned(dev_err, 4)) return fail(MLA_ERR_MISALIGNED, "dev_err is not 4-byte aligned");
  mla::PrefillArgs a = {};
  a.nb = 1;
  a.seq[0] = {M, N, 0, 0};
  a.scale_log2 = scale_log2(scale);
  a.out = (uint16_t*)out;
  a.dev_err = dev_err;
  return prefill_attention_launch(q_c, q_r, M, rows, k_c, v_c, N, a, stream);
}

mla_status mla_prefill_workspace_size(int32_t N, size_t* bytes) {
  CHECK_PTR(bytes);
  if (N < 0) return fail(MLA_ERR_INVALID_ARG, "N = %d < 0", N);
  *bytes = prefill_ws_bytes(N);
  return MLA_OK;
}

mla_status mla_prefill_batch_workspace_size(const int32_t* n_tokens, int32_t nb, size_t* bytes) {
  CHECK_PTR(bytes);
  if (nb < 0 || nb > mla::kPrefillMaxSeqs)
    return fail(MLA_ERR_INVALID_ARG, "nb = %d outside [0, %d]", nb, mla::kPrefillMaxSeqs);
  if (nb > 0) CHECK_PTR(n_tokens);
  int64_t total = 0;
  for (int32_t i = 0; i < nb; ++i) {
    if (n_tokens[i] < 0) return fail(MLA_ERR_INVALID_ARG, "n_tokens[%d] = %d < 0", i, n_tokens[i]);
    total += n_tokens[i];
  }
  if (total > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "%lld cached tokens in all: too many", (long long)total);
  *bytes = prefill_ws_bytes(total);
  return MLA_OK;
}

mla_status mla_prefill_decompress_batch(const void* q_c, const void* q_r, const int32_t* seq_ids,
                                        const int32_t* q_starts, const int32_t* q_lens, const int32_t* n_tokens,
                                        int32_t nb, const void* kv_cache, int64_t num_pages,
                                        const int32_t* block_table, int32_t batch, int32_t max_pages,
                                        const void* w_uk, const void* w_uv, float scale, void* workspace,
                                        size_t ws_bytes, void* out, int32_t* dev_err, void* stream) {
  if (nb < 0 || nb > mla::kPrefillMaxSeqs)
    return fail(MLA_ERR_INVALID_ARG, "nb = %d outside [0, %d]", nb, mla::kPrefillMaxSeqs);
  if (nb == 0) return MLA_OK;
  CHECK_PTR(seq_ids);
  CHECK_PTR(q_starts);
  CHECK_PTR(q_lens);
  CHECK_PTR(n_tokens);
  CHECK_PTR(q_c);
  CHECK_PTR(q_r);
  CHECK_PTR(kv_cache);
  CHECK_PTR(block_table);
  CHECK_PTR(w_uk);
  CHECK_PTR(w_uv);
  CHECK_PTR(workspace);
  CHECK_PTR(out);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(q_c);
  CHECK_ALIGN16(q_r);
  CHECK_ALIGN16(kv_cache);
  CHECK_ALIGN16(w_uk);
  CHECK_ALIGN16(w_uv);
  CHECK_ALIGN16(workspace);
  CHECK_ALIGN16(out);
  if (!aligned(block_table, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "block_table and dev_err must be 4-byte aligned");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(MLA_ERR_INVALID_ARG, "scale must be finite and positive");
  if (num_pages < 1 || batch < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "bad pool/table sizes");
  mla::GatherBatch g = {};
  mla::PrefillArgs a = {};
  int64_t total = 0, rows_end = 0;
  for (int32_t i = 0; i < nb; ++i) {
    const int32_t b = seq_ids[i], M = q_lens[i], N = n_tokens[i], q0 = q_starts[i];
    if (b < 0 || b >= batch) return fail(MLA_ERR_INVALID_ARG, "seq_ids[%d] = %d outside [0, %d)", i, b, batch);
    if (M < 1 || N < M)
      return fail(MLA_ERR_INVALID_ARG, "sequence %d: q_len %d must be in [1, n_tokens = %d]", i, M, N);
    if ((N + MLA_PAGE_SIZE - 1) / MLA_PAGE_SIZE > max_pages)
      return fail(MLA_ERR_INVALID_ARG, "sequence %d: %d tokens need more than max_pages = %d pages", i, N, max_pages);
    if (q0 < 0) return fail(MLA_ERR_INVALID_ARG, "q_starts[%d] = %d < 0", i, q0);
    g.b[i] = b;
    g.n[i] = N;
    g.off[i] = total;
    a.seq[i] = {M, N, q0, (int32_t)total};
    total += N;
    rows_end = std::max<int64_t>(rows_end, (int64_t)q0 + M);
  }
  if (total > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "%lld cached tokens in all: too many", (long long)total);
  if (rows_end > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "query rows past 2^24");
  if (ws_bytes < prefill_ws_bytes(total))
    return fail(MLA_ERR_INVALID_ARG, "workspace holds %zu bytes, %lld cached tokens need %zu", ws_bytes,
                (long long)total, prefill_ws_bytes(total));
  g.nb = nb;
  g.total = total;
  a.nb = nb;
  a.scale_log2 = scale_log2(scale);
  a.out = (uint16_t*)out;
  a.dev_err = dev_err;
  uint8_t* ws = (uint8_t*)workspace;
  void* rows = ws;
  void* k_c = ws + prefill_rows_bytes(total);
  void* v_c = (uint8_t*)k_c + (size_t)total * MLA_NUM_HEADS * MLA_HEAD_DIM_C * 2;
  cudaError_t e = mla::launch_gather_batch((const uint16_t*)kv_cache, num_pages, block_table, max_pages, g,
                                           (uint16_t*)rows, dev_err, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "batched gather launch");
  mla_status s = mla_expand_kv(rows, (int32_t)total, w_uk, w_uv, k_c, v_c, dev_err, stream);
  if (s != MLA_OK) return s;
  return prefill_attention_launch(q_c, q_r, rows_end, rows, k_c, v_c, total, a, stream);
}

// The tokens of one sequence that a chunk's window and sinks keep, packed:
// row j holds position j < cut ? j : j + shift.  A sequence's rows start at a
// multiple of the attention's 128-token key tiles, after rows of zeros, so that
// no tile of one sequence holds another's tokens: masked there, a NaN of
// another sequence would still reach this one's output.
constexpr int64_t kKeyTile = 128;
struct KeptTokens {
  int32_t n, cut, shift;
};
static int64_t packed_start(int64_t total) { return (total + kKeyTile - 1) / kKeyTile * kKeyTile; }
static KeptTokens kept_tokens(int32_t M, int32_t N, int32_t window, int32_t sinks) {
  const int64_t lo = (int64_t)N - M + 1 - window;  // the first row's window starts here
  if (lo <= sinks) return {N, N, 0};
  return {(int32_t)(sinks + N - lo), sinks, (int32_t)(lo - sinks)};
}

mla_status mla_prefill_window_workspace_size(const int32_t* q_lens, const int32_t* n_tokens, int32_t nb,
                                             int32_t window, int32_t sinks, size_t* bytes) {
  CHECK_PTR(bytes);
  if (nb < 0 || nb > mla::kPrefillMaxSeqs)
    return fail(MLA_ERR_INVALID_ARG, "nb = %d outside [0, %d]", nb, mla::kPrefillMaxSeqs);
  mla_status s = window_check(window, sinks);
  if (s != MLA_OK) return s;
  if (nb > 0) {
    CHECK_PTR(q_lens);
    CHECK_PTR(n_tokens);
  }
  int64_t total = 0;
  for (int32_t i = 0; i < nb; ++i) {
    if (q_lens[i] < 1 || n_tokens[i] < q_lens[i])
      return fail(MLA_ERR_INVALID_ARG, "sequence %d: q_len %d must be in [1, n_tokens = %d]", i, q_lens[i], n_tokens[i]);
    total = packed_start(total) + kept_tokens(q_lens[i], n_tokens[i], window, sinks).n;
  }
  if (total > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "%lld kept tokens in all: too many", (long long)total);
  *bytes = prefill_ws_bytes(total);
  return MLA_OK;
}

static mla_status prefill_window(const void* q_c, const void* q_r, const int32_t* seq_ids, const int32_t* q_starts,
                                 const int32_t* q_lens, const int32_t* n_tokens, int32_t nb, int32_t window,
                                 int32_t sinks, const void* cache, const float* scales, bool fp8, int64_t num_pages,
                                 const int32_t* block_table, int32_t batch, int32_t max_pages, const void* w_uk,
                                 const void* w_uv, float scale, void* workspace, size_t ws_bytes, void* out,
                                 int32_t* dev_err, void* stream) {
  if (nb < 0 || nb > mla::kPrefillMaxSeqs)
    return fail(MLA_ERR_INVALID_ARG, "nb = %d outside [0, %d]", nb, mla::kPrefillMaxSeqs);
  mla_status s = window_check(window, sinks);
  if (s != MLA_OK) return s;
  if (nb == 0) return MLA_OK;
  CHECK_PTR(seq_ids);
  CHECK_PTR(q_starts);
  CHECK_PTR(q_lens);
  CHECK_PTR(n_tokens);
  CHECK_PTR(q_c);
  CHECK_PTR(q_r);
  CHECK_PTR(cache);
  CHECK_PTR(block_table);
  CHECK_PTR(w_uk);
  CHECK_PTR(w_uv);
  CHECK_PTR(workspace);
  CHECK_PTR(out);
  CHECK_PTR(dev_err);
  if (fp8) {
    CHECK_PTR(scales);
    CHECK_ALIGN16(scales);
  }
  CHECK_ALIGN16(q_c);
  CHECK_ALIGN16(q_r);
  CHECK_ALIGN16(cache);
  CHECK_ALIGN16(w_uk);
  CHECK_ALIGN16(w_uv);
  CHECK_ALIGN16(workspace);
  CHECK_ALIGN16(out);
  if (!aligned(block_table, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "block_table and dev_err must be 4-byte aligned");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(MLA_ERR_INVALID_ARG, "scale must be finite and positive");
  if (num_pages < 1 || batch < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "bad pool/table sizes");
  mla::WindowGather g = {};
  mla::PrefillArgs a = {};
  int64_t total = 0, rows_end = 0;
  for (int32_t i = 0; i < nb; ++i) {
    const int32_t b = seq_ids[i], M = q_lens[i], N = n_tokens[i], q0 = q_starts[i];
    if (b < 0 || b >= batch) return fail(MLA_ERR_INVALID_ARG, "seq_ids[%d] = %d outside [0, %d)", i, b, batch);
    if (M < 1 || N < M)
      return fail(MLA_ERR_INVALID_ARG, "sequence %d: q_len %d must be in [1, n_tokens = %d]", i, M, N);
    if ((N - 1) / MLA_PAGE_SIZE >= max_pages)
      return fail(MLA_ERR_INVALID_ARG, "sequence %d: %d tokens need more than max_pages = %d pages", i, N, max_pages);
    if (q0 < 0) return fail(MLA_ERR_INVALID_ARG, "q_starts[%d] = %d < 0", i, q0);
    const KeptTokens k = kept_tokens(M, N, window, sinks);
    total = packed_start(total);
    g.b[i] = b;
    g.n[i] = k.n;
    g.cut[i] = k.cut;
    g.shift[i] = k.shift;
    g.off[i] = (int32_t)total;
    a.seq[i] = {M, k.n, q0, (int32_t)total};
    total += k.n;
    rows_end = std::max<int64_t>(rows_end, (int64_t)q0 + M);
    if (total > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "%lld kept tokens in all: too many", (long long)total);
  }
  if (rows_end > (1 << 24)) return fail(MLA_ERR_INVALID_ARG, "query rows past 2^24");
  int32_t order[mla::kPrefillMaxSeqs];  // by first row: two chunks on one row of the output would race for it
  for (int32_t i = 0; i < nb; ++i) order[i] = i;
  std::sort(order, order + nb, [=](int32_t x, int32_t y) { return q_starts[x] < q_starts[y]; });
  for (int32_t i = 1; i < nb; ++i) {
    const int32_t x = order[i - 1], y = order[i];
    if (q_starts[y] - q_starts[x] < q_lens[x])
      return fail(MLA_ERR_INVALID_ARG, "the query rows of sequences %d and %d overlap", x, y);
  }
  if (ws_bytes < prefill_ws_bytes(total))
    return fail(MLA_ERR_INVALID_ARG, "workspace holds %zu bytes, %lld kept tokens need %zu", ws_bytes,
                (long long)total, prefill_ws_bytes(total));
  g.nb = nb;
  g.max_pages = max_pages;
  g.total = total;
  g.num_pages = num_pages;
  g.block_table = block_table;
  g.dev_err = dev_err;
  a.nb = nb;
  a.scale_log2 = scale_log2(scale);
  a.out = (uint16_t*)out;
  a.dev_err = dev_err;
  a.window = std::min(window, 1 << 25);  // past the kept tokens (at most 2^24) a window is all the same; positions minus it stay in 32 bits
  a.sinks = std::min(sinks, 1 << 25);
  uint8_t* rows = (uint8_t*)workspace;
  uint8_t* k_c = rows + prefill_rows_bytes(total);
  uint8_t* v_c = k_c + (size_t)total * MLA_NUM_HEADS * MLA_HEAD_DIM_C * 2;
  cudaError_t e = mla::launch_gather_window(cache, scales, fp8, g, (uint16_t*)rows, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "window gather launch");
  s = expand_kv(rows, (int32_t)total, w_uk, w_uv, k_c, v_c, dev_err, true, stream);
  if (s != MLA_OK) return s;
  return prefill_attention_launch(q_c, q_r, rows_end, rows, k_c, v_c, total, a, stream);
}

mla_status mla_prefill_window_batch(const void* q_c, const void* q_r, const int32_t* seq_ids, const int32_t* q_starts,
                                    const int32_t* q_lens, const int32_t* n_tokens, int32_t nb, int32_t window,
                                    int32_t sinks, const void* kv_cache, int64_t num_pages, const int32_t* block_table,
                                    int32_t batch, int32_t max_pages, const void* w_uk, const void* w_uv, float scale,
                                    void* workspace, size_t ws_bytes, void* out, int32_t* dev_err, void* stream) {
  return prefill_window(q_c, q_r, seq_ids, q_starts, q_lens, n_tokens, nb, window, sinks, kv_cache, nullptr, false,
                        num_pages, block_table, batch, max_pages, w_uk, w_uv, scale, workspace, ws_bytes, out, dev_err,
                        stream);
}

mla_status mla_prefill_window_batch_fp8(const void* q_c, const void* q_r, const int32_t* seq_ids,
                                        const int32_t* q_starts, const int32_t* q_lens, const int32_t* n_tokens,
                                        int32_t nb, int32_t window, int32_t sinks, const void* rows,
                                        const float* scales, int64_t num_pages, const int32_t* block_table,
                                        int32_t batch, int32_t max_pages, const void* w_uk, const void* w_uv,
                                        float scale, void* workspace, size_t ws_bytes, void* out, int32_t* dev_err,
                                        void* stream) {
  return prefill_window(q_c, q_r, seq_ids, q_starts, q_lens, n_tokens, nb, window, sinks, rows, scales, true,
                        num_pages, block_table, batch, max_pages, w_uk, w_uv, scale, workspace, ws_bytes, out, dev_err,
                        stream);
}

mla_status mla_prefill_decompress(const void* q_c, const void* q_r, int32_t M, const void* kv_cache, int64_t num_pages,
                                  const int32_t* block_table, int32_t max_pages, int32_t b, int32_t N,
                                  const void* w_uk, const void* w_uv, float scale, void* workspace, size_t ws_bytes,
                                  void* out, int32_t* dev_err, void* stream) {
  if (M < 0 || N < 0) return fail(MLA_ERR_INVALID_ARG, "M = %d, N = %d: negative", M, N);
  if (M == 0) return MLA_OK;
  if (M > N) return fail(MLA_ERR_INVALID_ARG, "M = %d query rows exceed the N = %d cached tokens", M, N);
  if (b < 0) return fail(MLA_ERR_INVALID_ARG, "b = %d < 0", b);
  const int32_t zero = 0;
  // one sequence: its block-table row b, its query rows at the start of q_c / q_r / out
  return mla_prefill_decompress_batch(q_c, q_r, &b, &zero, &M, &N, 1, kv_cache, num_pages, block_table, b + 1,
                                      max_pages, w_uk, w_uv, scale, workspace, ws_bytes, out, dev_err, stream);
}

mla_status mla_absorb_q(const void* q_c, const void* w_uk, void* q_abs, int32_t T, int32_t* dev_err, void* stream) {
  return head_gemm(mla::HeadGemm::kAbsorbQ, q_c, w_uk, q_abs, T, dev_err, stream);
}

mla_status mla_up_v(const void* o_lat, const void* w_uv, void* out, int32_t T, int32_t* dev_err, void* stream) {
  return head_gemm(mla::HeadGemm::kUpV, o_lat, w_uv, out, T, dev_err, stream);
}

static mla_status w4_group_check(int32_t group) {
  if (group != 32 && group != 64 && group != 128)
    return fail(MLA_ERR_UNSUPPORTED, "group = %d: 32, 64 and 128 are supported", group);
  return MLA_OK;
}

static mla_status w4_gemm(mla::HeadGemm kind, const void* x, const void* words, const void* scales, int32_t group,
                          void* y, int32_t T, int32_t* dev_err, void* stream) {
  if (T < 0) return fail(MLA_ERR_INVALID_ARG, "T = %d < 0", T);
  mla_status s = w4_group_check(group);
  if (s != MLA_OK) return s;
  if (T == 0) return MLA_OK;
  CHECK_PTR(x);
  CHECK_PTR(words);
  CHECK_PTR(scales);
  CHECK_PTR(y);
  CHECK_PTR(dev_err);
  CHECK_ALIGN16(x);
  CHECK_ALIGN16(words);
  CHECK_ALIGN16(scales);
  CHECK_ALIGN16(y);
  if (!aligned(dev_err, 4)) return fail(MLA_ERR_MISALIGNED, "dev_err is not 4-byte aligned");
  if (T > (1 << 18)) return fail(MLA_ERR_INVALID_ARG, "T = %d too large", T);
  const bool absorb = kind == mla::HeadGemm::kAbsorbQ;
  const uintptr_t row = (uintptr_t)MLA_NUM_HEADS * 2 * (uintptr_t)T;
  const uintptr_t x0 = (uintptr_t)x, x_bytes = row * (absorb ? MLA_HEAD_DIM_C : MLA_LATENT_DIM);
  const uintptr_t y0 = (uintptr_t)y, y_bytes = row * (absorb ? MLA_LATENT_DIM : MLA_HEAD_DIM_C);
  if (x0 < y0 + y_bytes && y0 < x0 + x_bytes) return fail(MLA_ERR_INVALID_ARG, "the input and the output overlap");
  mla::W4Args a = {};
  a.x = (const uint16_t*)x;
  a.words = (const uint32_t*)words;
  a.scales = (const uint16_t*)scales;
  a.group = group;
  a.T = T;
  a.y = (uint16_t*)y;
  a.dev_err = dev_err;
  CUtensorMap xm = {}, ym = {};
  if (mla::w4_uses_maps(T)) {
    const uint64_t K = absorb ? MLA_HEAD_DIM_C : MLA_LATENT_DIM, N = absorb ? MLA_LATENT_DIM : MLA_HEAD_DIM_C;
    const uint64_t xd[3] = {K, MLA_NUM_HEADS, (uint64_t)T}, xs[2] = {K * 2, K * 2 * MLA_NUM_HEADS};
    const uint64_t yd[3] = {N, MLA_NUM_HEADS, (uint64_t)T}, ys[2] = {N * 2, N * 2 * MLA_NUM_HEADS};
    const uint32_t xbox[3] = {64, 1, 128}, ybox[3] = {32, 1, 32};
    s = make_map(&xm, x, 3, xd, xs, xbox, "activations");
    if (s == MLA_OK) s = make_map(&ym, y, 3, yd, ys, ybox, "outputs", CU_TENSOR_MAP_SWIZZLE_64B);
    if (s != MLA_OK) return s;
  }
  cudaError_t e = mla::launch_w4_gemm(kind, a, xm, ym, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, absorb ? "absorb_q_w4 launch" : "up_v_w4 launch");
  return MLA_OK;
}

mla_status mla_absorb_q_w4(const void* q_c, const void* words, const void* scales, int32_t group, void* q_abs,
                           int32_t T, int32_t* dev_err, void* stream) {
  return w4_gemm(mla::HeadGemm::kAbsorbQ, q_c, words, scales, group, q_abs, T, dev_err, stream);
}

mla_status mla_up_v_w4(const void* o_lat, const void* words, const void* scales, int32_t group, void* out, int32_t T,
                       int32_t* dev_err, void* stream) {
  return w4_gemm(mla::HeadGemm::kUpV, o_lat, words, scales, group, out, T, dev_err, stream);
}

mla_status mla_pack_w4(const void* w, int32_t K, int32_t N, int32_t group, void* words, void* scales, void* stream) {
  if (!((K == MLA_HEAD_DIM_C && N == MLA_LATENT_DIM) || (K == MLA_LATENT_DIM && N == MLA_HEAD_DIM_C)))
    return fail(MLA_ERR_UNSUPPORTED, "K = %d, N = %d: 128 x 512 (W_UK) and 512 x 128 (W_UV) are supported", K, N);
  mla_status s = w4_group_check(group);
  if (s != MLA_OK) return s;
  CHECK_PTR(w);
  CHECK_PTR(words);
  CHECK_PTR(scales);
  CHECK_ALIGN16(w);
  CHECK_ALIGN16(words);
  CHECK_ALIGN16(scales);
  cudaError_t e = mla::launch_w4_pack((const uint16_t*)w, K, N, group, (uint32_t*)words, (uint16_t*)scales,
                                      (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "pack_w4 launch");
  return MLA_OK;
}

// ------------------------------------------------------------------ pages and trees
// The caches of `layers` layers: pointers, strides and sizes.
static mla_status check_layers(const mla::LayerCaches& c, int row_bytes, bool fp8) {
  CHECK_PTR(c.rows);
  CHECK_ALIGN16(c.rows);
  if (c.num_pages < 1 || c.num_pages * MLA_PAGE_SIZE > (int64_t)INT32_MAX)
    return fail(MLA_ERR_INVALID_ARG, "num_pages = %lld outside [1, 2^31/64)", (long long)c.num_pages);
  if (c.layers < 1 || c.layers > 65535) return fail(MLA_ERR_INVALID_ARG, "layers = %d outside [1, 65535]", c.layers);
  if (fp8) {
    CHECK_PTR(c.scales);
    CHECK_ALIGN16(c.scales);
  }
  for (int i = 0; i < (fp8 ? 2 : 1) && c.layers > 1; ++i) {
    const int64_t stride = i ? c.scale_stride : c.row_stride;
    const int64_t least = c.num_pages * MLA_PAGE_SIZE * (i ? 4 : row_bytes);
    if (stride % 16) return fail(MLA_ERR_MISALIGNED, "a layer stride of %lld bytes is not a multiple of 16", (long long)stride);
    if (stride < least || stride > INT64_MAX / c.layers)
      return fail(MLA_ERR_INVALID_ARG, "a layer stride of %lld bytes: a layer's pages take %lld", (long long)stride,
                  (long long)least);
  }
  return MLA_OK;
}

static mla_status copy_pages(const mla::LayerCaches& c, int row_bytes, bool fp8, const int32_t* src, const int32_t* dst,
                             int32_t n, void* stream) {
  if (n < 0) return fail(MLA_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n == 0) return MLA_OK;
  CHECK_PTR(src);
  CHECK_PTR(dst);
  mla_status s = check_layers(c, row_bytes, fp8);
  if (s != MLA_OK) return s;
  return no_throw([&] {
    for (int32_t i = 0; i < n; ++i)
      for (const int32_t id : {src[i], dst[i]})
        if (id < 0 || id >= c.num_pages) return fail(MLA_ERR_INVALID_ARG, "copy %d: page id %d out of range", i, id);
    // The written pages: a bit each, or for few pairs of a large pool a sorted list
    // (two pairs of 4 000 000 pages: 183 us with the bits' predecessor, a byte each).
    if (n <= c.num_pages / 4096) {
      std::vector<int32_t> written(dst, dst + n);
      std::sort(written.begin(), written.end());
      const auto twice = std::adjacent_find(written.begin(), written.end());
      if (twice != written.end()) return fail(MLA_ERR_INVALID_ARG, "page %d is written twice", *twice);
      for (int32_t i = 0; i < n; ++i)
        if (std::binary_search(written.begin(), written.end(), src[i]))
          return fail(MLA_ERR_INVALID_ARG, "copy %d: page %d is read and written", i, src[i]);
    } else {
      std::vector<bool> written((size_t)c.num_pages);
      for (int32_t i = 0; i < n; ++i) {
        if (written[dst[i]]) return fail(MLA_ERR_INVALID_ARG, "page %d is written twice", dst[i]);
        written[dst[i]] = true;
      }
      for (int32_t i = 0; i < n; ++i)
        if (written[src[i]]) return fail(MLA_ERR_INVALID_ARG, "copy %d: page %d is read and written", i, src[i]);
    }
    cudaError_t e = mla::launch_copy_pages(c, row_bytes, src, dst, n, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "copy_pages launch");
    return MLA_OK;
  });
}

mla_status mla_copy_pages(void* kv_cache, int64_t num_pages, int32_t layers, int64_t layer_stride, const int32_t* src,
                          const int32_t* dst, int32_t n, void* stream) {
  return copy_pages({(uint8_t*)kv_cache, nullptr, layer_stride, 0, num_pages, layers}, (int)kRowBytes, false, src, dst, n,
                    stream);
}

mla_status mla_copy_pages_fp8(void* rows, float* scales, int64_t num_pages, int32_t layers, int64_t row_stride,
                              int64_t scale_stride, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  return copy_pages({(uint8_t*)rows, scales, row_stride, scale_stride, num_pages, layers}, MLA_FP8_ROW_BYTES, true, src,
                    dst, n, stream);
}

mla_status mla_copy_pages_nvfp4(void* rows, int64_t num_pages, int32_t layers, int64_t layer_stride, const int32_t* src,
                                const int32_t* dst, int32_t n, void* stream) {
  return copy_pages({(uint8_t*)rows, nullptr, layer_stride, 0, num_pages, layers}, MLA_NVFP4_ROW_BYTES, false, src, dst,
                    n, stream);
}

static mla_status tree_sizes(int32_t B, int32_t T, int32_t words) {
  if (B < 0 || T < 0 || T > INT32_MAX / MLA_NUM_HEADS) return fail(MLA_ERR_INVALID_ARG, "B = %d, T = %d: out of range", B, T);
  if (words < 1 || words > MLA_TREE_MAX_NODES / 64)
    return fail(MLA_ERR_INVALID_ARG, "words = %d outside [1, %d]", words, MLA_TREE_MAX_NODES / 64);
  return MLA_OK;
}

mla_status mla_tree_layout(const int32_t* parents, const int32_t* q_starts, const int32_t* seq_lens, int32_t B,
                           int32_t T, int32_t words, const int32_t* block_table, int32_t max_pages, int64_t num_pages,
                           uint64_t* masks, int32_t* positions, int64_t* slots, int32_t* dev_err, void* stream) {
  mla_status s = tree_sizes(B, T, words);
  if (s != MLA_OK) return s;
  if (B == 0 || T == 0) return MLA_OK;
  CHECK_PTR(parents);
  CHECK_PTR(q_starts);
  CHECK_PTR(seq_lens);
  CHECK_PTR(masks);
  CHECK_PTR(dev_err);
  if (slots) {
    CHECK_PTR(block_table);
    if (num_pages < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "bad pool/table sizes");
  }
  if (!aligned(masks, 8) || !aligned(slots, 8)) return fail(MLA_ERR_MISALIGNED, "masks and slots must be 8-byte aligned");
  if (!aligned(parents, 4) || !aligned(q_starts, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4) ||
      !aligned(positions, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "parents, q_starts, seq_lens, block_table, positions and dev_err must be 4-byte aligned");
  const mla::TreeLayoutArgs a = {parents, q_starts, seq_lens, block_table, num_pages, max_pages, B, T, words,
                                 masks, positions, slots, dev_err};
  cudaError_t e = mla::launch_tree_layout(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "tree_layout launch");
  return MLA_OK;
}

static mla_status tree_compact(const mla::LayerCaches& c, int row_bytes, bool fp8, const int32_t* block_table,
                               int32_t max_pages, const uint64_t* masks, int32_t words, const int32_t* q_starts,
                               const int32_t* seq_lens, const int32_t* accepted, int32_t B, int32_t T,
                               int32_t* new_lens, int32_t* dev_err, void* stream) {
  mla_status s = tree_sizes(B, T, words);
  if (s != MLA_OK) return s;
  if (B == 0) return MLA_OK;
  s = check_layers(c, row_bytes, fp8);
  if (s != MLA_OK) return s;
  CHECK_PTR(block_table);
  if (T > 0) CHECK_PTR(masks);
  CHECK_PTR(q_starts);
  CHECK_PTR(seq_lens);
  CHECK_PTR(accepted);
  CHECK_PTR(new_lens);
  CHECK_PTR(dev_err);
  if (max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "max_pages = %d < 1", max_pages);
  if (!aligned(masks, 8)) return fail(MLA_ERR_MISALIGNED, "masks is not 8-byte aligned");
  if (!aligned(block_table, 4) || !aligned(q_starts, 4) || !aligned(seq_lens, 4) || !aligned(accepted, 4) ||
      !aligned(new_lens, 4) || !aligned(dev_err, 4))
    return fail(MLA_ERR_MISALIGNED, "block_table, q_starts, seq_lens, accepted, new_lens and dev_err must be 4-byte aligned");
  const uintptr_t out = (uintptr_t)new_lens, len = (uintptr_t)B * 4;
  const struct {
    const void* p;
    uintptr_t bytes;
    const char* what;
  } in[] = {{seq_lens, len, "seq_lens"},
            {accepted, len, "accepted"},
            {q_starts, len + 4, "q_starts"},
            {masks, (uintptr_t)T * words * 8, "masks"},
            {block_table, len * max_pages, "block_table"},
            {dev_err, 4, "dev_err"}};
  for (const auto& x : in)
    if (out < (uintptr_t)x.p + x.bytes && (uintptr_t)x.p < out + len)
      return fail(MLA_ERR_INVALID_ARG, "new_lens and %s overlap", x.what);
  const mla::TreeCompactArgs a = {c, block_table, masks, q_starts, seq_lens, accepted, max_pages, B, T, words,
                                  new_lens, dev_err};
  cudaError_t e = mla::launch_tree_compact(a, row_bytes, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "tree_compact launch");
  return MLA_OK;
}

mla_status mla_tree_compact(void* kv_cache, int64_t num_pages, int32_t layers, int64_t layer_stride,
                            const int32_t* block_table, int32_t max_pages, const uint64_t* masks, int32_t words,
                            const int32_t* q_starts, const int32_t* seq_lens, const int32_t* accepted, int32_t B,
                            int32_t T, int32_t* new_lens, int32_t* dev_err, void* stream) {
  return tree_compact({(uint8_t*)kv_cache, nullptr, layer_stride, 0, num_pages, layers}, (int)kRowBytes, false, block_table,
                      max_pages, masks, words, q_starts, seq_lens, accepted, B, T, new_lens, dev_err, stream);
}

mla_status mla_tree_compact_fp8(void* rows, float* scales, int64_t num_pages, int32_t layers, int64_t row_stride,
                                int64_t scale_stride, const int32_t* block_table, int32_t max_pages,
                                const uint64_t* masks, int32_t words, const int32_t* q_starts, const int32_t* seq_lens,
                                const int32_t* accepted, int32_t B, int32_t T, int32_t* new_lens, int32_t* dev_err,
                                void* stream) {
  return tree_compact({(uint8_t*)rows, scales, row_stride, scale_stride, num_pages, layers}, MLA_FP8_ROW_BYTES, true,
                      block_table, max_pages, masks, words, q_starts, seq_lens, accepted, B, T, new_lens, dev_err, stream);
}

mla_status mla_tree_compact_nvfp4(void* rows, int64_t num_pages, int32_t layers, int64_t layer_stride,
                                  const int32_t* block_table, int32_t max_pages, const uint64_t* masks, int32_t words,
                                  const int32_t* q_starts, const int32_t* seq_lens, const int32_t* accepted, int32_t B,
                                  int32_t T, int32_t* new_lens, int32_t* dev_err, void* stream) {
  return tree_compact({(uint8_t*)rows, nullptr, layer_stride, 0, num_pages, layers}, MLA_NVFP4_ROW_BYTES, false,
                      block_table, max_pages, masks, words, q_starts, seq_lens, accepted, B, T, new_lens, dev_err, stream);
}

// ------------------------------------------------------------------ decode
mla_status mla_decode_max_clusters(int32_t* out) {
  CHECK_PTR(out);
  int n = 0;
  cudaError_t e = mla::decode_max_clusters(&n);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
  if (n < 1) return fail(MLA_ERR_CUDA, "the decode kernel cannot be resident on this device");
  *out = n;
  return MLA_OK;
}

mla_status mla_decode_plan_bytes(int32_t T, int32_t num_clusters, size_t* bytes) {
  CHECK_PTR(bytes);
  if (T < 0 || num_clusters < 1) return fail(MLA_ERR_INVALID_ARG, "need T >= 0 and num_clusters >= 1");
  const mla::PlanLayout L = mla::plan_layout(num_clusters, mla::plan_max_segments(T, num_clusters),
                                             mla::plan_max_split_rows(T, num_clusters));
  *bytes = (size_t)L.words * 4;
  return MLA_OK;
}

mla_status mla_decode_workspace_size(int32_t num_clusters, size_t* bytes) {
  CHECK_PTR(bytes);
  if (num_clusters < 1) return fail(MLA_ERR_INVALID_ARG, "num_clusters = %d < 1", num_clusters);
  *bytes = workspace_bytes_for(mla::plan_max_partials(num_clusters));
  return MLA_OK;
}

// build_plan where an exception may not pass.
static mla_status plan_checked(const int32_t* seq_lens, const int32_t* q_lens, int32_t B, int32_t num_clusters,
                               int32_t* out, size_t out_words, mla_plan_info* info, const PlanKind& kind = {},
                               mla_tree_info* tree_info = nullptr) {
  try {
    return build_plan(seq_lens, q_lens, B, num_clusters, out, out_words, info, kind, tree_info);
  } catch (const std::bad_alloc&) {
    return fail(MLA_ERR_NO_SPACE, "out of host memory");
  }
}

mla_status mla_decode_plan_host(const int32_t* seq_lens, const int32_t* q_lens, int32_t B, int32_t num_clusters,
                                void* plan_host, size_t plan_bytes, mla_plan_info* info) {
  CHECK_PTR(plan_host);
  CHECK_PTR(info);
  if (!aligned(plan_host, 4)) return fail(MLA_ERR_MISALIGNED, "plan_host is not 4-byte aligned");
  return plan_checked(seq_lens, q_lens, B, num_clusters, (int32_t*)plan_host, plan_bytes / 4, info);
}

// The uploads copy from memory of the call's own: a captured copy would read it
// again at every replay, long after it is gone.
static mla_status not_captured(void* stream) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing((cudaStream_t)stream, &st);
  if (e != cudaSuccess) {
    cudaGetLastError();  // not left for a later launch to find
    return cuda_fail(e, "stream capture query");
  }
  if (st != cudaStreamCaptureStatusNone)
    return fail(MLA_ERR_UNSUPPORTED, "a plan cannot be uploaded into a stream capture: plan before it, or use the host planner");
  return MLA_OK;
}

// A plan built in memory of the call's own and copied to plan_dev.
static mla_status plan_upload(const int32_t* seq_lens_host, const int32_t* q_lens_host, int32_t B, int32_t num_clusters,
                              void* plan_dev, size_t plan_bytes, mla_plan_info* info, void* stream,
                              const PlanKind& kind = {}, mla_tree_info* tree_info = nullptr) {
  CHECK_PTR(plan_dev);
  CHECK_ALIGN16(plan_dev);
  if (B < 0) return fail(MLA_ERR_INVALID_ARG, "B = %d is negative", B);
  if (num_clusters < 1) return fail(MLA_ERR_INVALID_ARG, "num_clusters = %d < 1", num_clusters);
  if (B > 0) CHECK_PTR(q_lens_host);
  int64_t T = 0;  // the rows bound what a plan can need, however large the buffer
  for (int32_t b = 0; b < B; ++b) T += q_lens_host[b] > 0 ? q_lens_host[b] : 0;
  if (T > INT32_MAX / MLA_NUM_HEADS) return fail(MLA_ERR_INVALID_ARG, "too many query rows");
  size_t need = 0;
  mla_status s = kind.tree ? mla_tree_plan_bytes((int32_t)T, num_clusters, &need)
                           : mla_decode_plan_bytes((int32_t)T, num_clusters, &need);
  if (s != MLA_OK) return s;
  const size_t words = std::min(plan_bytes, need) / 4;
  std::unique_ptr<int32_t[]> host(new (std::nothrow) int32_t[words + 1]);
  if (!host) return fail(MLA_ERR_NO_SPACE, "out of host memory");
  s = plan_checked(seq_lens_host, q_lens_host, B, num_clusters, host.get(), words, info, kind, tree_info);
  if (s == MLA_OK) s = not_captured(stream);
  if (s != MLA_OK) return s;
  // Pageable source: the call returns once the data is staged, so `host` may go.
  cudaError_t e = cudaMemcpyAsync(plan_dev, host.get(), info->plan_bytes, cudaMemcpyHostToDevice, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "plan copy");
  return MLA_OK;
}

mla_status mla_decode_plan(const int32_t* seq_lens_host, const int32_t* q_lens_host, int32_t B, int32_t num_clusters,
                           void* plan_dev, size_t plan_bytes, mla_plan_info* info, void* stream) {
  CHECK_PTR(info);
  return plan_upload(seq_lens_host, q_lens_host, B, num_clusters, plan_dev, plan_bytes, info, stream);
}

mla_status mla_window_plan_host(const int32_t* seq_lens, const int32_t* q_lens, int32_t B, int32_t window,
                                int32_t sinks, int32_t num_clusters, void* plan_host, size_t plan_bytes,
                                mla_window_info* info) {
  CHECK_PTR(plan_host);
  CHECK_PTR(info);
  if (!aligned(plan_host, 4)) return fail(MLA_ERR_MISALIGNED, "plan_host is not 4-byte aligned");
  mla_status s = window_check(window, sinks);
  if (s != MLA_OK) return s;
  s = plan_checked(seq_lens, q_lens, B, num_clusters, (int32_t*)plan_host, plan_bytes / 4, &info->plan,
                   {window, sinks});
  if (s != MLA_OK) return s;
  info->window = window;
  info->sinks = sinks;
  return MLA_OK;
}

mla_status mla_window_plan(const int32_t* seq_lens_host, const int32_t* q_lens_host, int32_t B, int32_t window,
                           int32_t sinks, int32_t num_clusters, void* plan_dev, size_t plan_bytes,
                           mla_window_info* info, void* stream) {
  CHECK_PTR(info);
  mla_status s = window_check(window, sinks);
  if (s == MLA_OK)
    s = plan_upload(seq_lens_host, q_lens_host, B, num_clusters, plan_dev, plan_bytes, &info->plan, stream,
                    {window, sinks});
  if (s != MLA_OK) return s;
  info->window = window;
  info->sinks = sinks;
  return MLA_OK;
}

mla_status mla_tree_plan_bytes(int32_t T, int32_t num_clusters, size_t* bytes) {
  mla_status s = mla_decode_plan_bytes(T, num_clusters, bytes);
  if (s == MLA_OK) *bytes += (size_t)T * mla::kTreeWords * 4;  // each tree has a node at least
  return s;
}

mla_status mla_tree_plan_host(const int32_t* seq_lens, const int32_t* q_lens, int32_t B, int32_t num_clusters,
                              void* plan_host, size_t plan_bytes, mla_tree_info* info) {
  CHECK_PTR(plan_host);
  CHECK_PTR(info);
  if (!aligned(plan_host, 4)) return fail(MLA_ERR_MISALIGNED, "plan_host is not 4-byte aligned");
  return plan_checked(seq_lens, q_lens, B, num_clusters, (int32_t*)plan_host, plan_bytes / 4, &info->plan, {0, 0, true},
                      info);
}

mla_status mla_tree_plan(const int32_t* seq_lens_host, const int32_t* q_lens_host, int32_t B, int32_t num_clusters,
                         void* plan_dev, size_t plan_bytes, mla_tree_info* info, void* stream) {
  CHECK_PTR(info);
  return plan_upload(seq_lens_host, q_lens_host, B, num_clusters, plan_dev, plan_bytes, &info->plan, stream,
                     {0, 0, true}, info);
}

// Whether a tree decode over the FP8 cache unpacks its pages: with three rows to a
// page or more (a sequence's first two may need one page less), and enough tiles
// to pay for a launch.  A tile of f16 rows takes half the time of one that has to
// be converted; unpacked and not, in us: two rows of 16 sequences of 8 192 tokens
// 107 and 100, of 64 of 2 048 tokens 109 and 109; three rows of 16 of 2 048 45 and
// 46, of 8 (792 tiles) 26.5 and 29.1; one sequence: 16 rows over 1 024 tokens (272
// tiles) 20 and 20, 8 over 2 048 (264) 22.2 and 21.6, 12 over 4 096 (780) 26 and
// 30, 64 over 32 768 349 and 688; two sequences, 8 rows over 2 048 (528) 24 and 25.
static bool tree_unpacks(const mla_tree_info& info) {
  return info.num_trees > 0 && info.total_pages > 0 && info.total_pages <= kMostUnpackedPages &&
         info.plan.total_tiles >= kUnpackTiles && info.plan.total_tiles + 2ll * info.num_trees >= 3 * info.total_pages;
}
static size_t unpacked_bytes(const mla_tree_info& info) { return (size_t)info.total_pages * MLA_PAGE_BYTES; }

mla_status mla_tree_workspace_size(const mla_tree_info* info, int32_t fp8, size_t* bytes) {
  CHECK_PTR(info);
  CHECK_PTR(bytes);
  if (info->plan.magic != MLA_TREE_PLAN_MAGIC) return fail(MLA_ERR_INVALID_ARG, "info is not a tree plan summary");
  *bytes = workspace_bytes_for(info->plan.num_partials) + (fp8 && tree_unpacks(*info) ? unpacked_bytes(*info) : 0);
  return MLA_OK;
}

// window: the windowed decode's parameters; tree: the tree decode's; both null
// for full attention.
static mla_status decode_common(const void* q_abs, const void* q_r, const void* kv_cache, const float* kv_scales,
                                int64_t num_pages, const int32_t* block_table, int32_t max_pages,
                                const void* plan_dev, const mla_plan_info* info, float scale, void* workspace,
                                size_t ws_bytes, void* o_lat, float* lse, int32_t* dev_err, void* stream,
                                bool fp8, const mla_window_info* window = nullptr,
                                const mla::TreeArgs* tree = nullptr, const mla_tree_info* tree_info = nullptr) {
  CHECK_PTR(info);
  if (info->magic != (tree ? MLA_TREE_PLAN_MAGIC : window ? MLA_WINDOW_PLAN_MAGIC : MLA_PLAN_MAGIC))
    return fail(MLA_ERR_INVALID_ARG, "info is not a %s plan summary", tree ? "tree" : window ? "window" : "decode");
  if (window) {
    const mla_status ws = window_check(window->window, window->sinks);
    if (ws != MLA_OK) return ws;
  }
  if (info->T == 0 || info->num_clusters == 0) return MLA_OK;
  CHECK_PTR(q_abs);
  CHECK_PTR(q_r);
  CHECK_PTR(kv_cache);
  CHECK_PTR(block_table);
  CHECK_PTR(plan_dev);
  CHECK_PTR(o_lat);
  CHECK_PTR(dev_err);
  if (tree) {
    CHECK_PTR(tree->masks);
    if (!aligned(tree->masks, 8)) return fail(MLA_ERR_MISALIGNED, "masks is not 8-byte aligned");
  }
  CHECK_ALIGN16(q_abs);
  CHECK_ALIGN16(q_r);
  CHECK_ALIGN16(kv_cache);
  CHECK_ALIGN16(plan_dev);
  CHECK_ALIGN16(o_lat);
  if (fp8) {
    CHECK_PTR(kv_scales);
    CHECK_ALIGN16(kv_scales);
  }
  if (!aligned(block_table, 4) || !aligned(dev_err, 4) || (lse && !aligned(lse, 4)))
    return fail(MLA_ERR_MISALIGNED, "block_table, dev_err and lse must be 4-byte aligned");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(MLA_ERR_INVALID_ARG, "scale must be finite and positive");
  if (num_pages < 1 || num_pages * MLA_PAGE_SIZE > (int64_t)INT32_MAX)
    return fail(MLA_ERR_INVALID_ARG, "num_pages = %lld outside [1, 2^31/64)", (long long)num_pages);
  if (max_pages < info->max_pages_needed)
    return fail(MLA_ERR_INVALID_ARG, "block table has %d columns, the plan reads %d", max_pages,
                info->max_pages_needed);
  const size_t need_ws = workspace_bytes_for(info->num_partials);
  if (info->num_partials > 0) {
    CHECK_PTR(workspace);
    CHECK_ALIGN16(workspace);
    if (ws_bytes < need_ws)
      return fail(MLA_ERR_INVALID_ARG, "workspace holds %zu bytes, the plan needs %zu", ws_bytes, need_ws);
  }

  const mla::PlanLayout L = mla::plan_layout(info->num_clusters, info->num_segments, info->num_split_rows);
  const int32_t* plan = (const int32_t*)plan_dev;
  // A tree decode over the FP8 cache reads a page for many rows: where that
  // pays and the workspace has the room, the pages are unpacked to f16 once.
  const bool unpack = fp8 && tree && tree_unpacks(*tree_info) && ws_bytes >= need_ws + unpacked_bytes(*tree_info);
  if (unpack) {
    CHECK_PTR(workspace);
    CHECK_ALIGN16(workspace);
    uint8_t* out = (uint8_t*)workspace + need_ws;
    const mla::TreeUnpackArgs u = {(const uint8_t*)kv_cache, kv_scales, num_pages, block_table, tree->masks, plan + L.words,
                                   (uint4*)out, dev_err, max_pages, info->B, info->T, tree->words,
                                   (int32_t)tree_info->total_pages, tree_info->num_trees};
    cudaError_t e = mla::launch_tree_unpack(u, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "unpack launch");
    kv_cache = out;
    num_pages = tree_info->total_pages;
  }

  CUtensorMap kv_map, rope_map;
  mla_status s;
  if (fp8 && !unpack) {
    // Codes: a CTA's 256 of each token row, 64 rows per box (no swizzle: the
    // converters read them); RoPE halves as bf16 columns 256.. of the rows.
    const uint64_t cdims[2] = {MLA_FP8_ROW_BYTES, (uint64_t)num_pages * MLA_PAGE_SIZE};
    const uint64_t cstr[1] = {MLA_FP8_ROW_BYTES};
    const uint32_t cbox[2] = {256, 64};
    s = make_map(&kv_map, kv_cache, 2, cdims, cstr, cbox, "fp8 codes", CU_TENSOR_MAP_SWIZZLE_NONE,
                 CU_TENSOR_MAP_DATA_TYPE_UINT8);
    if (s != MLA_OK) return s;
    const uint64_t rdims[2] = {MLA_FP8_ROW_BYTES / 2, (uint64_t)num_pages * MLA_PAGE_SIZE};
    const uint32_t rope_box[2] = {32, 64};
    s = make_map(&rope_map, kv_cache, 2, rdims, cstr, rope_box, "fp8 RoPE halves", CU_TENSOR_MAP_SWIZZLE_64B);
    if (s != MLA_OK) return s;
  } else {
    // Latent part as a 3D view {64 elements, token, 64-element chunk}: one box
    // of 4 chunks x 64 tokens lands as 4 consecutive 128-byte-swizzled 8 KB
    // tiles, one TMA instruction per page for a CTA's latent half.
    const uint64_t ldims[3] = {64, (uint64_t)num_pages * MLA_PAGE_SIZE, MLA_LATENT_DIM / 64};
    const uint64_t lstr[2] = {(uint64_t)kRowBytes, 128};
    const uint32_t lbox[3] = {64, 64, 4};
    s = make_map(&kv_map, kv_cache, 3, ldims, lstr, lbox, "kv_cache latent chunks");
    if (s != MLA_OK) return s;
    const uint64_t dims[2] = {MLA_TOKEN_ELEMS, (uint64_t)num_pages * MLA_PAGE_SIZE};
    const uint64_t str[1] = {(uint64_t)kRowBytes};
    const uint32_t rope_box[2] = {32, 64};
    s = make_map(&rope_map, kv_cache, 2, dims, str, rope_box, "kv_cache RoPE halves", CU_TENSOR_MAP_SWIZZLE_64B);
    if (s != MLA_OK) return s;
  }

  // Merged tiles: the sinks' first `split` tokens of a page and the rest of
  // another as boxes of their own.
  mla::WindowArgs win = {};
  if (window) {
    win.sinks = window->sinks;
    win.split = mla::window_split(window->sinks);
    if (win.split > 0 && win.split < MLA_PAGE_SIZE) {
      for (int part = 0; part < 2; ++part) {
        const uint32_t n = (uint32_t)(part ? MLA_PAGE_SIZE - win.split : win.split);
        CUtensorMap* km = part ? &win.kv_tail : &win.kv_head;
        CUtensorMap* rm = part ? &win.rope_tail : &win.rope_head;
        const uint64_t tokens = (uint64_t)num_pages * MLA_PAGE_SIZE;
        const uint32_t rbox[2] = {32, n};
        if (fp8) {
          const uint64_t cdims[2] = {MLA_FP8_ROW_BYTES, tokens}, rdims[2] = {MLA_FP8_ROW_BYTES / 2, tokens};
          const uint64_t str[1] = {MLA_FP8_ROW_BYTES};
          const uint32_t cbox[2] = {256, n};
          s = make_map(km, kv_cache, 2, cdims, str, cbox, "fp8 codes of a merged tile", CU_TENSOR_MAP_SWIZZLE_NONE,
                       CU_TENSOR_MAP_DATA_TYPE_UINT8);
          if (s == MLA_OK) s = make_map(rm, kv_cache, 2, rdims, str, rbox, "RoPE of a merged tile", CU_TENSOR_MAP_SWIZZLE_64B);
        } else {
          const uint64_t ldims[3] = {64, tokens, MLA_LATENT_DIM / 64}, rdims[2] = {MLA_TOKEN_ELEMS, tokens};
          const uint64_t lstr[2] = {(uint64_t)kRowBytes, 128}, rstr[1] = {(uint64_t)kRowBytes};
          const uint32_t lbox[3] = {64, n, 1};
          s = make_map(km, kv_cache, 3, ldims, lstr, lbox, "latent chunk of a merged tile");
          if (s == MLA_OK) s = make_map(rm, kv_cache, 2, rdims, rstr, rbox, "RoPE of a merged tile", CU_TENSOR_MAP_SWIZZLE_64B);
        }
        if (s != MLA_OK) return s;
      }
    }
  }

  float* part_o = (float*)workspace;
  float* part_lse = part_o ? part_o + (size_t)info->num_partials * MLA_NUM_HEADS * MLA_LATENT_DIM : nullptr;

  mla::DecodeArgs a = {};
  a.q_abs = (const uint16_t*)q_abs;
  a.q_r = (const uint16_t*)q_r;
  a.block_table = block_table;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.seg_off = plan + L.seg_off;
  a.segs = plan + L.seg_base;
  a.scale_log2 = scale_log2(scale);
  a.o_lat = (uint16_t*)o_lat;
  a.lse = lse;
  a.part_o = part_o;
  a.part_lse = part_lse;
  a.dev_err = dev_err;
  a.T = info->T;
  a.B = info->B;
  a.num_segments = info->num_segments;
  a.num_partials = info->num_partials;
  a.kv_scales = fp8 && !unpack ? kv_scales : nullptr;
  a.wait_limit = g_decode_wait_limit.load(std::memory_order_relaxed);
  a.wait_every = a.wait_limit < (1ull << 20) ? 0u : 255u;
  const mla::TreeCache cache = unpack ? mla::TreeCache::kUnpacked : fp8 ? mla::TreeCache::kFp8 : mla::TreeCache::kBf16;
  cudaError_t e = tree     ? mla::launch_decode_tree(kv_map, rope_map, a, *tree, info->num_clusters, cache, (cudaStream_t)stream)
                  : window ? mla::launch_decode_window(kv_map, rope_map, a, win, info->num_clusters, fp8, (cudaStream_t)stream)
                           : mla::launch_decode(kv_map, rope_map, a, info->num_clusters, fp8, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  if (info->num_split_rows > 0) {
    mla::CombineArgs c = {};
    c.split_rows = plan + L.split_base;
    c.part_o = part_o;
    c.part_lse = part_lse;
    c.o_lat = (uint16_t*)o_lat;
    c.lse = lse;
    c.T = info->T;
    c.num_partials = info->num_partials;
    c.dev_err = dev_err;
    e = mla::launch_combine(c, info->num_split_rows, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "combine launch");
  }
  return MLA_OK;
}

mla_status mla_decode_paged(const void* q_abs, const void* q_r, const void* kv_cache, int64_t num_pages,
                            const int32_t* block_table, int32_t max_pages, const void* plan_dev,
                            const mla_plan_info* info, float scale, void* workspace, size_t ws_bytes, void* o_lat,
                            float* lse, int32_t* dev_err, void* stream) {
  return decode_common(q_abs, q_r, kv_cache, nullptr, num_pages, block_table, max_pages, plan_dev, info, scale,
                       workspace, ws_bytes, o_lat, lse, dev_err, stream, false);
}

mla_status mla_decode_paged_fp8(const void* q_abs, const void* q_r, const void* rows, const float* scales,
                                int64_t num_pages, const int32_t* block_table, int32_t max_pages,
                                const void* plan_dev, const mla_plan_info* info, float scale, void* workspace,
                                size_t ws_bytes, void* o_lat, float* lse, int32_t* dev_err, void* stream) {
  return decode_common(q_abs, q_r, rows, scales, num_pages, block_table, max_pages, plan_dev, info, scale,
                       workspace, ws_bytes, o_lat, lse, dev_err, stream, true);
}

mla_status mla_decode_window(const void* q_abs, const void* q_r, const void* kv_cache, int64_t num_pages,
                             const int32_t* block_table, int32_t max_pages, const void* plan_dev,
                             const mla_window_info* info, float scale, void* workspace, size_t ws_bytes, void* o_lat,
                             float* lse, int32_t* dev_err, void* stream) {
  CHECK_PTR(info);
  return decode_common(q_abs, q_r, kv_cache, nullptr, num_pages, block_table, max_pages, plan_dev, &info->plan, scale,
                       workspace, ws_bytes, o_lat, lse, dev_err, stream, false, info);
}

mla_status mla_decode_window_fp8(const void* q_abs, const void* q_r, const void* rows, const float* scales,
                                 int64_t num_pages, const int32_t* block_table, int32_t max_pages,
                                 const void* plan_dev, const mla_window_info* info, float scale, void* workspace,
                                 size_t ws_bytes, void* o_lat, float* lse, int32_t* dev_err, void* stream) {
  CHECK_PTR(info);
  return decode_common(q_abs, q_r, rows, scales, num_pages, block_table, max_pages, plan_dev, &info->plan, scale,
                       workspace, ws_bytes, o_lat, lse, dev_err, stream, true, info);
}

static mla_status decode_tree(const void* q_abs, const void* q_r, const void* kv_cache, const float* kv_scales,
                              int64_t num_pages, const int32_t* block_table, int32_t max_pages, const uint64_t* masks,
                              int32_t words, const void* plan_dev, const mla_tree_info* info, float scale,
                              void* workspace, size_t ws_bytes, void* o_lat, float* lse, int32_t* dev_err, void* stream,
                              bool fp8) {
  CHECK_PTR(info);
  if (words < 1 || words > MLA_TREE_MAX_NODES / 64)
    return fail(MLA_ERR_INVALID_ARG, "words = %d outside [1, %d]", words, MLA_TREE_MAX_NODES / 64);
  if (info->max_nodes > 64 * words)
    return fail(MLA_ERR_INVALID_ARG, "the plan has a tree of %d nodes, a mask of %d words holds %d", info->max_nodes,
                words, 64 * words);
  if (info->num_trees < 0 || info->total_pages < 0)
    return fail(MLA_ERR_INVALID_ARG, "info is not a tree plan summary");
  const mla::TreeArgs tree = {masks, words};
  return decode_common(q_abs, q_r, kv_cache, kv_scales, num_pages, block_table, max_pages, plan_dev, &info->plan,
                       scale, workspace, ws_bytes, o_lat, lse, dev_err, stream, fp8, nullptr, &tree, info);
}

mla_status mla_decode_tree(const void* q_abs, const void* q_r, const void* kv_cache, int64_t num_pages,
                           const int32_t* block_table, int32_t max_pages, const uint64_t* masks, int32_t words,
                           const void* plan_dev, const mla_tree_info* info, float scale, void* workspace,
                           size_t ws_bytes, void* o_lat, float* lse, int32_t* dev_err, void* stream) {
  return decode_tree(q_abs, q_r, kv_cache, nullptr, num_pages, block_table, max_pages, masks, words, plan_dev, info,
                     scale, workspace, ws_bytes, o_lat, lse, dev_err, stream, false);
}

mla_status mla_decode_tree_fp8(const void* q_abs, const void* q_r, const void* rows, const float* scales,
                               int64_t num_pages, const int32_t* block_table, int32_t max_pages,
                               const uint64_t* masks, int32_t words, const void* plan_dev, const mla_tree_info* info,
                               float scale, void* workspace, size_t ws_bytes, void* o_lat, float* lse,
                               int32_t* dev_err, void* stream) {
  return decode_tree(q_abs, q_r, rows, scales, num_pages, block_table, max_pages, masks, words, plan_dev, info, scale,
                     workspace, ws_bytes, o_lat, lse, dev_err, stream, true);
}

mla_status mla_debug_set_decode_wait_limit(uint64_t cycles) {
  if (cycles > kDefaultDecodeWaitLimit)
    return fail(MLA_ERR_INVALID_ARG, "wait limit %llu above the default %llu", (unsigned long long)cycles,
                (unsigned long long)kDefaultDecodeWaitLimit);
  g_decode_wait_limit.store(cycles == 0 ? kDefaultDecodeWaitLimit : cycles, std::memory_order_relaxed);
  return MLA_OK;
}

mla_status mla_check(void* stream, const int32_t* dev_err, int32_t* word_out) {
  CHECK_PTR(dev_err);
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int32_t w = 0;
  e = cudaMemcpy(&w, dev_err, sizeof(w), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
  if (word_out) *word_out = w;
  if (w == 0) return MLA_OK;
  if (w & MLA_DEVERR_TIMEOUT) return fail(MLA_ERR_TIMEOUT, "a kernel wait timed out (device error word 0x%x)", w);
  return fail(MLA_ERR_DEVICE, "device error word 0x%x", w);
}

}  // extern "C"
