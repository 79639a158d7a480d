// The work items of the chunk attention: which query rows, which key tiles, and how
// they are shared out over the launch's CTAs.  Plain C++, so that it can be checked
// on the host.
//
// A sequence's n new tokens and the G query heads of a key/value head make n · G
// rows, token by token (row f: token f / G, head f mod G of the group).  An item is
// kRows of them over one key/value head; its tiles are the runs of kKeys keys that
// its last row sees, at least one.  The items in the order (sequence, row block,
// key/value head), tile after tile, are cut into runs of equal cost, one a CTA.
#pragma once

#ifdef __CUDACC__
#define FA_CHUNK_FN __host__ __device__ __forceinline__ constexpr
#else
#define FA_CHUNK_FN constexpr
#endif

namespace fa {
namespace chunk8 {

constexpr int kRows = 256, kHalf = 128, kKeys = 128;

// Keys that new token i of n sees, of `len` cached ones (the new tokens are the last of them).
FA_CHUNK_FN int visible(int len, int n, int i, bool causal) {
  if (!causal) return len;
  const long long v = static_cast<long long>(len) - n + i + 1;
  return v < 0 ? 0 : v > len ? len : static_cast<int>(v);
}
FA_CHUNK_FN int tiles(int keys) {
  const int t = static_cast<int>((static_cast<unsigned>(keys) + kKeys - 1u) / kKeys);
  return t < 1 ? 1 : t;
}
// Tiles that the rows [first, first + count) take, 0 if none of them exists (rows = n · G).
FA_CHUNK_FN int row_tiles(int len, int n, int G, int first, int count, bool causal) {
  const int rows = n * G;
  if (first >= rows) return 0;
  const int last = (rows - first < count ? rows : first + count) - 1;
  return tiles(visible(len, n, last / G, causal));
}

// A run is counted in units: one for each tile, and `extra` before an item's first,
// as many as its fixed cost is tiles' time (kItemCost; less where a CTA has fewer tiles
// than that: with little work every tile had better have a CTA of its own).
constexpr int kItemCost = 3;
FA_CHUNK_FN int extra_units(long long all_tiles, long long ctas) {
  return all_tiles / ctas <= kItemCost ? static_cast<int>(all_tiles / ctas) - 1 : kItemCost;
}
// Run c of `ctas` over `total` units begins at run_start(c); unit u lies in run run_of(u).
FA_CHUNK_FN long long run_start(long long c, long long total, long long ctas) { return c * total / ctas; }
FA_CHUNK_FN int run_of(long long u, long long total, long long ctas) {
  return static_cast<int>(((u + 1) * ctas + total - 1) / total - 1);
}

}  // namespace chunk8
}  // namespace fa
