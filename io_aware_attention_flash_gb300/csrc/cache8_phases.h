// Which mbarrier, and which phase parity of it, the roles of the cache
// attention use for tile t (counted through all items of a CTA).  Plain C++, so
// that the order of the roles' waits can be explored on the host.
//
// A wait by parity tells a phase from the one before and the one after it only:
// two phases later it reads as not complete again.  So between a wait and the
// second phase after the awaited one there has to be something that the waiting
// role does in between.
#pragma once

#ifdef __CUDACC__
#define FA_PHASE_FN __host__ __device__ __forceinline__ constexpr
#else
#define FA_PHASE_FN constexpr
#endif

namespace fa {
namespace cache8 {

struct Phase {
  int index;        // of the barriers of its kind
  unsigned parity;  // of the phase that stands for the tile
};

// Number of barriers of each kind.
constexpr int kSBars = 2, kPBars = 2, kPvBars = 2;

// K and V of tile t have landed in its ring stage; the stage's last reader has
// finished with tile t.
FA_PHASE_FN Phase ring(int t, int stages) { return {t % stages, static_cast<unsigned>(t / stages) & 1u}; }
// The scores of tile t are in tensor memory.
FA_PHASE_FN Phase s_full(int t) { return {t & 1, static_cast<unsigned>(t >> 1) & 1u}; }
// P of tile t is in shared memory (and the scores of tile t have been read).  Two
// barriers: the scores of tile t + 1 are issued before P of tile t is awaited, so
// P of tile t + 1 may be complete by then; P of tile t + 2 may not, as the warps
// that form it have waited for the product of tile t.
FA_PHASE_FN Phase p_full(int t) { return {t & 1, static_cast<unsigned>(t >> 1) & 1u}; }
// The product of P and V of tile t is in tensor memory.
FA_PHASE_FN Phase pv_done(int t) { return {t & 1, static_cast<unsigned>(t >> 1) & 1u}; }

}  // namespace cache8
}  // namespace fa
