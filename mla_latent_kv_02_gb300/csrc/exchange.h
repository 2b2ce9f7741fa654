// Where the decode's scores and finished rows lie in an exchange buffer of the
// pair.  Plain arithmetic, so that the model of the protocol, on the CPU, takes
// its byte ranges from here too.
#pragma once
#include <cstdint>

#if defined(__CUDACC__)
#define MLA_EXCHANGE_HD __host__ __device__ __forceinline__
#else
#define MLA_EXCHANGE_HD inline
#endif

namespace mla {
namespace decode {

constexpr int kXHeads = 128, kXTokens = 64;
constexpr int kXBytes = kXHeads * kXTokens * 2;           // one CTA's fp16 partial S (16 KB)

// The scores of a tile cross in parts, each with a barrier of its own.  In two,
// 32 tokens each, the second part's way (an SM sends about 20 bytes a cycle) is
// under the first part's arithmetic: 64 unpacked rows of 32 832 tokens 392 -> 369
// us, 768 rows of 8 204 tokens 1 259 -> 1 229.  Over the FP8 cache, where the
// converters bind and leave fewer registers, one part is faster (320 and 344 us on
// 128 rows of 8 194 tokens).
template <int kParts>
struct Exchange {
  static_assert(kParts == 1 || kParts == 2, "the swizzles below");
  static constexpr int kBytes = kXBytes / kParts;         // [128 heads x 64 / kParts tokens] fp16
  static constexpr int kRow = kXTokens * 2 / kParts;      // a row's scores
  static constexpr int kWarp = 32 * kRow;                 // one warp's 32 rows: one copy to the peer
  static constexpr int kPieces = kRow / 16;               // 16-byte pieces of a row, swizzled
  static constexpr int kWords2 = kXTokens / 2 / kParts;   // fp16x2 words of a row
  static MLA_EXCHANGE_HD constexpr uint32_t swizzle(int h) { return kParts == 1 ? (uint32_t)(h & 7) : (uint32_t)((h >> 1) & 3); }
  // The first byte of what warp q4 stages, sends and receives, in a part.
  static MLA_EXCHANGE_HD constexpr uint32_t share(int q4) { return (uint32_t)(q4 * kWarp); }
  // The first byte of head row h's scores in a part, and piece k of a row swizzled by swz.
  static MLA_EXCHANGE_HD constexpr uint32_t row(int h) { return (uint32_t)(h * kRow); }
  static MLA_EXCHANGE_HD constexpr uint32_t piece(uint32_t k, uint32_t swz) { return (k ^ swz) << 4; }
  // 16-byte piece k of the scores of head row h in part p.
  static MLA_EXCHANGE_HD constexpr uint32_t scores(uint32_t h, uint32_t p, uint32_t k) {
    return p * kBytes + row((int)h) + piece(k, swizzle((int)h));
  }
  // 16-byte piece k of eight of a finished row, row r of warp q4's 32, on its way
  // to memory: in the places of the same warp's scores, so that the four warps of a
  // warpgroup, which nothing joins between a finished row and the scores of their
  // next tile, share no byte.  Rows of a second part change places in pairs: the
  // eight pieces of a row then lie in different banks.
  static MLA_EXCHANGE_HD constexpr uint32_t finished(uint32_t q4, uint32_t r, uint32_t k) {
    return scores(32u * q4 + (r ^ (k / kPieces)), k / kPieces, k % kPieces);
  }
  // Every piece of a finished row lies in its own warp's shares.
  static MLA_EXCHANGE_HD constexpr bool apart() {
    for (uint32_t q4 = 0; q4 < 4; ++q4)
      for (uint32_t r = 0; r < 32; ++r)
        for (uint32_t k = 0; k < 8; ++k) {
          const uint32_t at = finished(q4, r, k), from = k / kPieces * kBytes + share((int)q4);
          if (at < from || at + 16u > from + kWarp) return false;
        }
    return true;
  }
};
static_assert(Exchange<1>::apart() && Exchange<2>::apart(), "a finished row outside its warp's share of an exchange buffer");

}  // namespace decode
}  // namespace mla
