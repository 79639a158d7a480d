// Where a cached sequence's tiles, pages and tokens end: the cache attention's
// integer arithmetic on lengths up to 2^31 - 1, in plain C++ so that it can be
// checked on the host.  Nothing here forms a number above 2^32 - 1 or, signed,
// above 2^31 - 1: a token's index may be past the length by a tile only as a
// difference.
#pragma once

#ifdef __CUDACC__
#define FA_TILE_FN __host__ __device__ __forceinline__ constexpr
#else
#define FA_TILE_FN constexpr
#endif

namespace fa {
namespace cache8 {

// Tiles of `tokens` tokens that hold a length's tokens, and pages of 1 << shift.
FA_TILE_FN int tiles_of(int len, int tokens) {
  return static_cast<int>((static_cast<unsigned>(len) + static_cast<unsigned>(tokens) - 1u) / static_cast<unsigned>(tokens));
}
FA_TILE_FN int pages_of(int len, int shift) {
  return static_cast<int>((static_cast<unsigned>(len) + (1u << shift) - 1u) >> shift);
}
// Tokens from token `row` of tile kt to the sequence's end (0 and less: none).
FA_TILE_FN int tokens_from(int len, int kt, int tokens, int row) { return (len - kt * tokens) - row; }

}  // namespace cache8
}  // namespace fa
