// The work items of the chunk attention: which query rows, which key tiles, and how
// they are shared out over the launch's CTAs.  Plain C++, so that it can be checked
// on the host.
//
// A sequence's n new tokens and the G query heads of a key/value head make n · G
// rows, token by token (row f: token f / G, head f mod G of the group).  An item is
// kRows of them over one key/value head; its tiles are the runs of kKeys keys that
// its last row sees, at least one.  The items in the order (sequence, row block,
// key/value head), tile after tile, are cut into runs of equal cost, one a CTA.
//
// A CTA takes rows as two halves.  Where an item has rows for one half only, both take
// the same rows and every other tile each (`dual`).
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
// Where only the first `n` of `all` new tokens are computed: cached tokens that those can
// see, the sequence as if it ended with them (the mask is counted from its end).
FA_CHUNK_FN int reach(int len, int all, int n, bool causal) {
  if (!causal || all <= n) return len;
  return len < all - n ? 0 : len - (all - n);
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

// Row block rb is a sequence's last, or it has none.
FA_CHUNK_FN bool last_block(int n, int G, int rb) { return n * G - rb * kRows <= kRows; }
// Where the pairs (sequence, row block) that have rows are gone through in order: the row
// block behind rb of its sequence, or of the next sequence with new tokens, which
// next_with(b) finds from b on (`count` if there is none).  As many steps as there are
// pairs with rows, whatever the largest sequence's row blocks are.
template <typename NextWith>
FA_CHUNK_FN void next_pair(int& b, int& rb, int n, int G, NextWith next_with) {
  if (!last_block(n, G, rb)) {
    ++rb;
  } else {
    b = next_with(b + 1);
    rb = 0;
  }
}

// Rows of row block rb fit in one half.
FA_CHUNK_FN bool dual(int n, int G, int rb) { return n * G - rb * kRows <= kHalf; }

// Runs are counted in units: two for a tile of a dual item, three for another's (its
// halves' products, of which a dual item's tile is one), and `extra` before an item's
// first, as many as its fixed cost is (kItemCost; less where a CTA has little more than
// a tile: every one had better have a CTA of its own).  Measured: a tile takes 1.6 us, of
// a dual item 1.1, an item 8 (at d = 64: 1.5, 0.8 and 6).  Sixteen sequences of 1 to 512
// new tokens over 100 to 8,192 took 223 us with a cost of 14, 213 with 18, 219 with 22,
// 227 with 26 (before the tile pass was shortened 259 with 10, 240 with 14, 231 with 18);
// one long document took the same with all.  (One batch at d = 128: for d = 64, where an item
// costs less, and for other mixes the same number is taken.)
constexpr int kMostUnits = 3, kItemCost = 18;
// Where every tile can have a CTA of its own, all count the same, so that it has (counted
// as two, each third tile of few rows shared its CTA with another: 15 heads of one tile
// took 16.1 us instead of 11.9, calls below 5 GFLOP 12 % longer on average).
FA_CHUNK_FN bool few(long long tiles, int most) { return tiles <= most; }
FA_CHUNK_FN int tile_units(bool dual, bool few) { return dual && !few ? 2 : kMostUnits; }
// CTAs that have a run each, of `most`: a run has as many units as a tile and more, so
// that a tile begins in every run between an item's first and last.  all: the units of
// all tiles.
FA_CHUNK_FN int runs(long long all, int most) {
  const long long r = all / kMostUnits;
  return r >= most ? most : r > 0 ? static_cast<int>(r) : all > 0;
}
// Units before an item's first.
FA_CHUNK_FN int extra_units(long long all, int ctas) {
  const long long each = all / ctas - kMostUnits;
  return each < 0 ? 0 : each < kItemCost ? static_cast<int>(each) : kItemCost;
}
// Run c of `ctas` over `total` units begins at run_start(c); unit u lies in run run_of(u).
// A tile is in the run that has its first unit.
FA_CHUNK_FN long long run_start(long long c, long long total, long long ctas) { return c * total / ctas; }
FA_CHUNK_FN int run_of(long long u, long long total, long long ctas) {
  return static_cast<int>(((u + 1) * ctas + total - 1) / total - 1);
}
// Sequences of a few tiles at most, by the caller's limit, are not cut: an item counts as
// one tile, and no partial results have to be joined.  Measured, d = 128, 16 sequences of 30
// new tokens: 16.4 us whole and 21.8 cut at 250 keys, 18.1 and 23.9 at 380; 2 of 8: 15.6 and
// 17.0 at 380, where a fourth tile would bring as much as it costs.
constexpr int kWholeTiles = 3;
FA_CHUNK_FN bool uncut(int max_seqlen) { return max_seqlen <= kWholeTiles * kKeys; }
FA_CHUNK_FN int counted(int tiles, bool uncut) { return uncut && tiles > 0 ? 1 : tiles; }
// Tiles of an item that begin before `units` units from its first one's.
FA_CHUNK_FN int tiles_before(long long units, int per_tile, int tiles, bool uncut) {
  if (uncut) return units <= 0 ? 0 : tiles;
  const long long t = units <= 0 ? 0 : (units + per_tile - 1) / per_tile;
  return t < tiles ? static_cast<int>(t) : tiles;
}

}  // namespace chunk8
}  // namespace fa
