// Attention of a chunk of new tokens over the 8-bit paged cache, for sm_103a.
//
//   O = softmax(scale Q K^T) V over the tokens a sequence has in the cache, its new
//   ones the last of them (causal: new token i of n sees keys up to len - n + i).
//
// The rows of a product are the new tokens times the G query heads of one key/value
// head, so a tile of keys is read once for all of them, and a chunk of a few tokens
// still fills the tensor core's 128 rows.  A CTA takes 256 rows (two tiles of 128)
// over a run of key tiles; chunk8_items.h says which.  An item that several CTAs
// share leaves partials (m, l, O), which a second kernel joins in the order of the
// keys, so results do not depend on timing.
//
// Keys go to the tensor core as the codes they are stored as: a query row, scaled by
// a power of two, is the sum of two e4m3 terms, so S takes two products at twice
// bf16's rate; the page's scale is a factor of 16 columns or more in the softmax.
// Values are made bf16 in shared memory by warps of their own (an e4m3 value times a
// power of two is a bf16 number: nothing is rounded), since P in two e4m3 terms would
// cost the softmax warps more instructions than the conversion costs those.  With
// both keys and values made bf16, 8192 rows over 32768 keys took 1230 us against
// 750 without any conversion: the issue slots of an SM hold the softmax and one.
//
// Warp roles (16 warps):
//   0-3, 4-7   softmax, one warpgroup a row tile; thread r owns row r of it
//   15         items and K: publishes the CTA's next item, copies the codes of its pages
//              (lane i: page i of the tile) and their scales
//   8          the same of V (one warp for both could not issue the copies of 16-token
//              pages as fast as they land)
//   12         tcgen05.mma issue
//   others     conversion of V tiles: none on the scheduler (warp mod 4) that the MMA
//              warp shares.  They note an item's first token with a value stored as NaN
// The softmax is the forward kernel's: the reference of a row is the maximum of its
// first tile and moves only where a tile's row sum reaches 2^40.
//
// Measured, a call: 2,048 new tokens of 32 heads (8 of keys) over 32,768 at d = 128 in 743
// us, 1430 TFLOP/s, 76 % of the large product's rate; 16 mixed sequences at 965, pieces of
// prompts at d = 64 at 583 TFLOP/s; 4 x 12 tokens over 32,768 in 85 us (3.2 TB/s).  Bound by a
// softmax warp's way through its tile, some 450 instructions at four cycles each (fixed
// latencies, instruction fetch) with the hand-overs around it: without the conversion, the
// exponentials and three quarters of the products the first takes 2 to 4 % less.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "cache8_tiles.h"
#include "chunk8_items.h"
#include "e4m3.cuh"
#include "fa_kernels.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

using chunk8::kHalf;
using chunk8::kKeys;
using chunk8::kRows;

template <int D>
struct ChunkCfg {
  static constexpr int KB = D / 64;                     // 128-byte swizzle blocks of a bf16 row
  static constexpr int BLK_BYTES = kTile * 128;         // one 128-row x 64-col block
  static constexpr int TILE_BYTES = KB * BLK_BYTES;     // one 128 x D tile of bf16
  static constexpr int CODE_BYTES = kKeys * D;          // the same of codes
  static constexpr int NK = D == 128 ? 3 : 6;           // ring of K's codes
  static constexpr int NC = NK;                         // ring of V's codes
  static constexpr int NV = D == 128 ? 2 : 3;           // ring of V in bf16
  // Ring of K's scales.  A slot is written again once the S of NK tiles before has been
  // formed.  By then P of three tiles further back is there (of a dual item, whose halves
  // take turns; else of one), and with it the scales have been read.
  static constexpr int NSC = NK + 3;
  static constexpr int NI = 4;                          // published items
  static constexpr int MAX_PPT = kKeys / 16;            // pages of a tile, at most
  static constexpr int OFF_Q = 0;                       // two row tiles: of each 8 rows the first terms, then the second
  static constexpr int OFF_V = OFF_Q + 2 * TILE_BYTES;
  static constexpr int OFF_K = OFF_V + NV * TILE_BYTES;
  static constexpr int OFF_C = OFF_K + NK * CODE_BYTES;
  static constexpr int OFF_KS = OFF_C + NC * CODE_BYTES;           // [NSC][pages] K's scales
  static constexpr int OFF_VF = OFF_KS + NSC * MAX_PPT * 4;        // [NC][pages] V's two factors, bf16 pairs
  static constexpr int ITEM_INTS = 16;
  static constexpr int OFF_ITEM = OFF_VF + NC * MAX_PPT * 8;
  static constexpr int OFF_SCAN = OFF_ITEM + NI * ITEM_INTS * 4;   // [3][16] sums, then what is found
  static constexpr int OFF_BAR = OFF_SCAN + 50 * 8;
  static constexpr int B_IFULL = 0;
  static constexpr int B_IEMPTY = B_IFULL + NI;
  static constexpr int B_KFULL = B_IEMPTY + NI;
  static constexpr int B_KEMPTY = B_KFULL + NK;
  static constexpr int B_SCFULL = B_KEMPTY + NK;
  static constexpr int B_CFULL = B_SCFULL + NSC;
  static constexpr int B_CEMPTY = B_CFULL + NC;
  static constexpr int B_VFULL = B_CEMPTY + NC;
  static constexpr int B_VEMPTY = B_VFULL + NV;
  static constexpr int B_Q = B_VEMPTY + NV;
  static constexpr int B_SFULL = B_Q + 2;
  static constexpr int B_PFULL = B_SFULL + 2;
  static constexpr int B_ODONE = B_PFULL + 2;
  static constexpr int B_DRAIN = B_ODONE + 2;
  static constexpr int B_RAW = B_DRAIN + 1;             // [8]: a softmax warp's rows of Q have landed
  static constexpr int B_JOIN = B_RAW + 8;              // a dual item's second half is there, and has been read
  static constexpr int NBAR = B_JOIN + 2;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;          // slack to align the base to 1024
  static constexpr int COPY_WARP = 15, V_WARP = 8, MMA_WARP = 12, CONVERT_WARPS = 5;
  static constexpr int NUM_THREADS = 512;
  static constexpr int READERS = 15;                    // warps that take an item: all but the one that publishes it
  // Registers a thread after the split; launched with 128.
  static constexpr int REG_SOFTMAX = 192, REG_OTHER = 64;
  static_assert(2 * REG_SOFTMAX + 2 * REG_OTHER == 4 * 128, "the split takes what the launch gives");
  // How far the MMA warp's loops over the halves and the steps of P V are unrolled: at d = 64
  // hardly, since the code that each scheduler fetches counts for more than the issue of
  // these small products (pieces of prompts 176 us with steps in pairs, 181 one by one, 189
  // unrolled, 204 with the halves unrolled); at d = 128 rolled steps cost 703 -> 763 us on a
  // long document, rolled halves 0.8 %.  Of dual items the halves' loop is rolled for both (1 %
  // over drawn sizes).
  static constexpr int HALF_UNROLL = D == 64 ? 1 : 2, PV_UNROLL = D == 64 ? 2 : kKeys / 16;
  static constexpr uint32_t TMEM_COLS = 512;
  __host__ __device__ static constexpr uint32_t S_COL(int t) { return t * 128; }
  __host__ __device__ static constexpr uint32_t O_COL(int t) { return 256 + t * D; }
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(OFF_K % 1024 == 0 && OFF_C % 1024 == 0 && CODE_BYTES % 1024 == 0, "swizzle atoms");
  static_assert(OFF_ITEM % 16 == 0 && OFF_KS % 16 == 0 && OFF_SCAN % 8 == 0, "vector accesses");
};

// What the roles know of an item.
struct Item {
  int b, hk, rb, k0, tiles, n, len, tok0, cnt0, cnt1, slot;  // slot: of the partial, -1: the item is whole
  bool dual;
};

// A place in a ring of N slots that is gone through in order, and its phase there.
template <int N>
struct Ring {
  int i = 0, phase = 0;
  __device__ __forceinline__ void step(int n = 1) {  // n <= N
    i += n;
    if (i >= N) {
      i -= N;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// New tokens and cached tokens of sequence b, within what the buffers hold and the call
// computes; whether that is all of them.
__device__ __forceinline__ bool chunk_seq(const Chunk8Params& p, int b, int& tok0, int& n, int& len) {
  tok0 = min(max(p.cu_seqlens[b], 0), p.total);
  const int all = min(max(p.cu_seqlens[b + 1], tok0), p.total) - tok0, given = p.seqlens[b];
  n = min(all, p.max_new);
  const long long cap = min(static_cast<long long>(p.table_cols) << p.block_shift, static_cast<long long>(p.max_seqlen));
  const int held = static_cast<int>(min(max(static_cast<long long>(given), 0LL), cap));
  len = chunk8::reach(held, all, n, p.causal);
  return held == given && n == all;
}

// Four codes to bf16 by their bits: sign, and exponent and mantissa four places
// down, which reads as the value times 2^-120 (a subnormal code as a subnormal).
// The first word holds elements 0 and 2, the second 1 and 3: O's dimensions change
// places again at the end.  (The search for NaN is one instruction more a word; of all codes
// again, byte by byte, it was five halves of one: 2 to 4 % of the attention.)
// `top` keeps the largest magnitude (of each half's): NaN, 0x7f, comes out as 480, above all
// numbers' bits.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& even, uint32_t& odd, uint32_t& top) {
  const uint32_t o = (w >> 4) & 0x07f007f0u, e = (w << 4) & 0x07f007f0u;
  odd = o | (w & 0x80008000u);
  even = e | ((w << 8) & 0x80008000u);
  top = __vimax3_u16x2(top, o, e);
}
__device__ __forceinline__ bool nan_among(uint32_t top) { return (top & 0xffffu) == 0x07f0u || (top >> 16) == 0x07f0u; }
__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kOne2 = 0x3f803f80u;
// Bit 7 of each byte: whether that code of four is NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }
constexpr int kNoKey = 0x7fffffff;  // behind every key
// V is kept 2^-kVShift times its value, so that O, up to 2^40 times the largest value
// while it is summed, does not leave fp32; the least of a value's codes, 2^-9 · 2^-64,
// stays a normal bf16 number.
constexpr int kVShift = 48;
// 2^(e + 120 - kVShift) as two bf16 factors, each a pair; e the exponent of a page's scale.
__device__ __forceinline__ uint2 scale_factors(float scale) {
  const int e = static_cast<int>((__float_as_uint(scale) >> 23) & 255u) - 127 + 120 - kVShift;
  const int a = max(min(e, 127), -126), b = max(e - 127, 0);
  return make_uint2(static_cast<uint32_t>(a + 127) * 0x00800080u, static_cast<uint32_t>(b + 127) * 0x00800080u);
}

template <int D>
__global__ void __launch_bounds__(ChunkCfg<D>::NUM_THREADS, 1) fa_chunk8_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                              const Chunk8Params p) {
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = raw_base + pad;
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == C::COPY_WARP && lane == 0) {
    for (int i = 0; i < C::NI; ++i) {
      mbar_init(bar(C::B_IFULL + i), 1);
      mbar_init(bar(C::B_IEMPTY + i), C::READERS);
    }
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(bar(C::B_KFULL + i), 1);
      mbar_init(bar(C::B_KEMPTY + i), 1);
    }
    for (int i = 0; i < C::NSC; ++i) mbar_init(bar(C::B_SCFULL + i), 1);
    for (int i = 0; i < C::NC; ++i) {
      mbar_init(bar(C::B_CFULL + i), 1);
      mbar_init(bar(C::B_CEMPTY + i), C::CONVERT_WARPS);
    }
    for (int i = 0; i < C::NV; ++i) {
      mbar_init(bar(C::B_VFULL + i), C::CONVERT_WARPS);
      mbar_init(bar(C::B_VEMPTY + i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(C::B_Q + t), 128);
      mbar_init(bar(C::B_SFULL + t), 1);
      mbar_init(bar(C::B_PFULL + t), 128);
      mbar_init(bar(C::B_ODONE + t), 1);
      mbar_init(bar(C::B_JOIN + t), 128);
    }
    mbar_init(bar(C::B_DRAIN), 1);
    for (int i = 0; i < 8; ++i) mbar_init(bar(C::B_RAW + i), 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
  }
  // The kernel may start while the one before it in the stream finishes; what that
  // one wrote is read, and tensor memory taken, from here on.
  grid_dependency_wait();
  grid_launch_dependents();

  if (p.zero_tail) {
    // Rows in front of the first sequence and behind the last, shared out over the grid.
    const int front = min(max(p.cu_seqlens[0], 0), p.total), end = min(max(p.cu_seqlens[p.B], front), p.total);
    for (int x = blockIdx.x; x < front + p.total - end; x += gridDim.x) {
      const int row = x < front ? x : x - front + end;
      uint4* o = reinterpret_cast<uint4*>(p.o + static_cast<size_t>(row) * p.H * D);
      for (int i = tid; i < p.H * (D / 8); i += C::NUM_THREADS) o[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int h = tid; h < p.H; h += C::NUM_THREADS) p.lse[static_cast<size_t>(h) * p.total + row] = -CUDART_INF_F;
    }
  }

  // ---- this CTA's place: the tiles and items of all (sequence, row block) pairs
  // counted, then the pair that holds the run's first unit
  const int pairs = p.B * p.row_blocks;
  const bool uncut = chunk8::uncut(p.max_seqlen);
  long long* scan = reinterpret_cast<long long*>(smem + C::OFF_SCAN);
  auto pair_tiles = [&](int x, int& tiles) -> bool {  // whether they are a dual item's
    const int b = x / p.row_blocks, rb = x - b * p.row_blocks;
    int tok0, n, len;
    chunk_seq(p, b, tok0, n, len);
    tiles = chunk8::row_tiles(len, n, p.G, rb * kRows, kRows, p.causal);
    return chunk8::dual(n, p.G, rb);
  };
  auto warp_scan = [&](long long v) {  // inclusive
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += y;
    }
    return v;
  };
  int one = 0;  // pair tid's tiles, if one pass takes all pairs
  bool one_dual = false;
  long long sums[3] = {0, 0, 0};  // tiles, those of dual items, items
  for (int x = tid; x < pairs; x += C::NUM_THREADS) {
    one_dual = pair_tiles(x, one);
    one = chunk8::counted(one, uncut);
    sums[0] += one;
    sums[1] += one_dual ? one : 0;
    sums[2] += one > 0;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sums[k] += __shfl_xor_sync(0xffffffffu, sums[k], off);
    if (lane == 0) scan[16 * k + warp] = sums[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    sums[k] = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[k] += scan[16 * k + i];
    sums[k] *= p.Hk;
  }
  const bool few = chunk8::few(sums[0], static_cast<int>(gridDim.x));
  const long long units_sum = (sums[0] - sums[1]) * chunk8::tile_units(false, few) + sums[1] * chunk8::tile_units(true, few);
  const int ctas = chunk8::runs(units_sum, static_cast<int>(gridDim.x));
  if (tid == 0) p.merge[blockIdx.x * 8] = -1;
  auto report = [&]() {  // lengths out of range, and new tokens past max_new: once
    for (int b = tid; b < p.B; b += C::NUM_THREADS) {
      int tok0, n, len;
      if (!chunk_seq(p, b, tok0, n, len)) atomicOr(p.err, kDevErrPage);
    }
  };
  if (static_cast<int>(blockIdx.x) >= ctas) {
    if (blockIdx.x == 0) report();  // (there is no row to compute)
    return;
  }
  const int extra = chunk8::extra_units(units_sum, ctas);
  const long long total = units_sum + extra * sums[2];
  auto pair_units = [&](int tile_units) -> long long {
    return tile_units > 0 ? static_cast<long long>(p.Hk) * (tile_units + extra) : 0;
  };
  const long long u_lo = chunk8::run_start(blockIdx.x, total, ctas), u_hi = chunk8::run_start(blockIdx.x + 1LL, total, ctas);
  long long* found = scan + 48;  // first unit of the pair; the pair
  {
    long long base = 0;
    for (int x0 = 0; x0 < pairs && base <= u_lo; x0 += C::NUM_THREADS) {
      if (pairs > C::NUM_THREADS) {
        one = 0;
        if (x0 + tid < pairs) one_dual = pair_tiles(x0 + tid, one);
        one = chunk8::counted(one, uncut);
      }
      const long long w = pair_units(one * chunk8::tile_units(one_dual, few));
      long long sum = warp_scan(w);
      __syncthreads();  // (the sums before have been read)
      if (lane == 31) scan[warp] = sum;
      __syncthreads();
      long long all = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const long long v = scan[i];
        if (i < warp) sum += v;
        all += v;
      }
      if (u_lo >= base + sum - w && u_lo < base + sum) {
        found[0] = base + sum - w;
        found[1] = x0 + tid;
      }
      base += all;
    }
  }
  if (blockIdx.x == 0) report();
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The next item of the CTA, as the copying warp publishes it; false at the end.
  int items = 0;
  auto take_item = [&](Item& it) -> bool {
    const int s = items % C::NI;
    bool ok = wait_bounded(bar(C::B_IFULL + s), (items / C::NI) & 1, abort_flag, p.err, p.timeout_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    const int4* src = reinterpret_cast<const int4*>(smem + C::OFF_ITEM + s * C::ITEM_INTS * 4);
    const int4 a = src[0], b = src[1], c = src[2];
    it.b = a.x, it.hk = a.y, it.rb = a.z, it.k0 = a.w;
    it.tiles = b.x, it.n = b.y, it.len = b.z, it.tok0 = b.w;
    it.cnt0 = c.x, it.cnt1 = c.y, it.slot = c.z, it.dual = c.w != 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_IEMPTY + s));
    ++items;
    return it.tiles > 0;
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    // (Ahead of the other roles, and the long code that runs once an item, the items' with
    // K's copies, behind them: where the loops of a tile lie among one another decides how
    // often their instructions are fetched again.  With that between the softmax and the rest 16
    // mixed sequences take 218 to 271 us, by what it holds, instead of 214 to 222, a long
    // document 736 to 769 instead of 731 to 743, pieces of prompts of 64 heads at d = 64 173 to
    // 206 instead of 176; with the softmax behind all others d = 64 takes 3 % longer over drawn
    // sizes.)
    setmaxnreg_inc<C::REG_SOFTMAX>();
    const int t = warp / 4, wq = warp % 4, r = wq * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t tS = lane_addr + C::S_COL(t), tO = lane_addr + C::O_COL(t);
    uint8_t* q_smem = smem + C::OFF_Q + t * C::TILE_BYTES;
    // A warp moves its 32 rows 16 bytes a lane, RPP rows at a time.
    constexpr int CH = D / 8, RPP = 32 / CH;
    const int my_chunk = lane % CH;
    // Phases of what this half waits for once a tile, an item, a load of Q, a join: one
    // register (the tile loop has none to spare).
    uint32_t phases = 0;
    enum { kTile = 1, kItem = 2, kRaw = 4, kJoin = 8, kRawAhead = 16, kRawEver = 32 };
    auto phase = [&](uint32_t of) { return (phases & of) ? 1 : 0; };
    int tile0 = 0;       // tiles of the items before
    bool ok = true;
    auto wait = [&](int i, int phase) {
      ok = ok && wait_bounded(bar(i), phase & 1, abort_flag, p.err, p.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    // An item's fields are read from shared memory where they are needed, which saves the
    // tile loop their registers.
    uint32_t item = 0;
    enum { kHk = 1, kRb, kK0, kTiles, kN, kLen, kTok0, kCnt0, kCnt1, kSlot, kDual, kNan };
    auto field = [&](int i) {
      int v;
      asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(item + 4 * i));
      return v;
    };
    // This half's rows of the item: the first, and behind the last.
    auto first_row = [&]() { return field(kRb) * kRows + (field(kDual) ? 0 : t * kHalf); };
    auto all_rows = [&]() { return field(kN) * p.G; };
    // The warp's rows of Q of an item, all in flight at once.  (Loaded through registers in
    // four batches, each as long as a miss: 5 us an item.)
    auto load_q = [&]() {
      const int first = first_row(), from = first + wq * 32, count = max(min(all_rows() - from, 32), 0);
      const int tok_a = from / p.G, toks = count > 0 ? (from + count - 1) / p.G - tok_a + 1 : 0;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(bar(C::B_RAW + warp), count * (2 * D));
      __syncwarp();
      for (int i = lane; i < toks; i += 32) {
        const int f0 = max((tok_a + i) * p.G, from), f1 = min((tok_a + i + 1) * p.G, from + count);
        bulk_load(sb + C::OFF_Q + t * C::TILE_BYTES + (f0 - first) * (2 * D),
                  p.q + static_cast<size_t>(field(kTok0) + tok_a + i) * p.ldq +
                      (static_cast<size_t>(field(kHk)) * p.G + f0 - (tok_a + i) * p.G) * D,
                  (f1 - f0) * (2 * D), bar(C::B_RAW + warp));
      }
      phases |= kRawEver;
    };
    auto take = [&]() {
      const int cnt = field(kCnt0 + t);
      const int first_tile = tile0;
      tile0 += field(kTiles);
      if (first_row() >= all_rows()) return;
      float m_ref = -CUDART_INF_F, l = 0.f;
      // (of the warp) some reference so large that a product's rounding, 2^-24 of it,
      // counts in the exponent
      bool far = false;
      if (cnt > 0) {
        // ---- Q: each row scaled by a power of two, as two e4m3 terms, in place: 8 rows'
        // terms take the room of the rows
        if (!(phases & kRawAhead)) load_q();  // (else they are on their way already)
        phases &= ~kRawAhead;
        const bool landed = wait(C::B_RAW + warp, phase(kRaw));
        phases ^= kRaw;
        if (!landed) return;
        const int first = first_row(), rows = all_rows();
        // (rolled: run through once an item, unrolled code is all instruction fetches)
        int my_e = 0;  // the exponent of this thread's row
#pragma unroll 1
        for (int r8 = 0; r8 < 32; r8 += 8) {
          constexpr int NB = 8 / RPP;
          uint8_t* rows8 = q_smem + (wq * 32 + r8) * (2 * D);
          uint4 x[NB];
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const int row = i * RPP + lane / CH;
            x[i] = *reinterpret_cast<const uint4*>(rows8 + row * (2 * D) + 16 * my_chunk);
            if (first + wq * 32 + r8 + row >= rows) x[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t top = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) top = __vmaxu2(top, w[u] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
#pragma unroll
            for (int off = CH / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
            // smallest power of two s with max <= 448 s, for any finite row: 2^120 at
            // most, at least 2^-126 (fp32's smallest that is not subnormal)
            const int e = min(scale_exponent(top, -126), 120);
            const int of_row = __shfl_sync(0xffffffffu, e, lane % RPP * CH);
            if (lane / RPP == r8 / RPP + i) my_e = of_row;
            // (infinities, which e4m3 has not, make the row NaN as a whole)
            const float inv = top < 0x7f80u ? exp2_int(-e) : CUDART_NAN_F;
            // (through f16, which holds the scaled values exactly down to 2^-14)
            const uint64_t inv2 = f2_pack(inv, inv);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t h[2], back[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float a, b;
                f2_unpack(fmul2(f2_pack(bf16lo_to_f32(w[2 * u + k]), bf16hi_to_f32(w[2 * u + k])), inv2), a, b);
                h[k] = pack_f16x2(a, b);
              }
              hi[u] = e4m3x4_of_f16(h[0], h[1]);
              f16_of_e4m3x4(hi[u], back[0], back[1]);
              lo[u] = e4m3x4_of_f16(sub_f16x2(h[0], back[0]), sub_f16x2(h[1], back[1]));
            }
            uint8_t* at = rows8 + swz<D>(i * RPP + lane / CH, 8 * my_chunk);
            *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(at + 8 * D) = make_uint2(lo[0], lo[1]);
          }
        }
        const float c_row = exp2_int(my_e) * p.scale_log2;
        fence_proxy_async_smem();
        mbar_arrive(bar(C::B_Q + t));
        // This half's tiles: every one, or every other.  Keys, from the next tile's first, that
        // the row sees, and that the half's first row does (which sees the fewest).
        const int stride = field(kDual) ? 2 : 1, at = field(kDual) ? t : 0;
        const int kv0 = (field(kK0) + at) * kKeys;  // (of a first tile behind the last: not used)
        int sees = (first + r < rows ? chunk8::visible(field(kLen), field(kN), (first + r) / p.G, p.causal) : 0) - kv0;
        int all_see = chunk8::visible(field(kLen), field(kN), first / p.G, p.causal) - kv0;
        Ring<C::NSC> scr;  // the next tile's place among K's scales
        scr.i = (first_tile + at) % C::NSC, scr.phase = (first_tile + at) / C::NSC & 1;
        for (int j = 0; j < cnt; ++j) {
          // the columns' factors: K's scale of each 16 keys, the row's and the softmax's
          // (not below fp32's least normal number: a masked column stays -infinity)
          const int sc = scr.i;
          if (!wait(C::B_SCFULL + sc, scr.phase)) break;
          scr.step(stride);
          const uint32_t k_scale = sb + C::OFF_KS + sc * (C::MAX_PPT * 4);
          float cf[8];
#pragma unroll
          for (int g16 = 0; g16 < 8; ++g16) {
            float v;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(k_scale + (((16 * g16) >> p.block_shift) << 2)));
            cf[g16] = fmaxf(v * c_row, 0x1p-126f);
          }
          if (!wait(C::B_SFULL + t, phase(kTile))) break;
          phases ^= kTile;
          tc_fence_after();
          // The first tile, whose largest score is the reference, and those that a row does not
          // see all of, which are masked in place.  (Rolled, run through a few times an item: the
          // same on the registers below is code that every tile jumps over, which its own
          // instructions' fetch waits for.  239 against 213 us on 16 mixed sequences.)
          if (j == 0 || all_see < kKeys) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t x[16];
              tmem_ld16(tS + 16 * c, x);
              tmem_wait_ld();
              reg_fence(x);
              if (all_see < 16 * c + 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (i >= sees - 16 * c) x[i] = __float_as_uint(-CUDART_INF_F);
                tmem_st16(tS + 16 * c, x);
              }
              if (j == 0) {
                float v, mx[2] = {__uint_as_float(x[0]), __uint_as_float(x[1])};
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(k_scale + (((16 * c) >> p.block_shift) << 2)));
#pragma unroll
                for (int i = 1; i < 8; ++i) mx[i & 1] = fmax3(mx[i & 1], __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                m_ref = fmaxf(m_ref, fmaxf(mx[0], mx[1]) * fmaxf(v * c_row, 0x1p-126f));
              }
            }
            tmem_wait_st();
          }
          uint32_t s[4][32];
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) tmem_ld32(tS + ch * 32, s[ch]);
          tmem_wait_ld();
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) reg_fence(s[ch]);
          // The largest y = s · factor of the row.
          auto row_max = [&]() -> float {
            float m = -CUDART_INF_F;
#pragma unroll
            for (int g16 = 0; g16 < 8; ++g16) {
              const uint32_t* x = s[g16 / 2] + 16 * (g16 % 2);
              float mx[2] = {__uint_as_float(x[0]), __uint_as_float(x[1])};
#pragma unroll
              for (int i = 1; i < 8; ++i) mx[i & 1] = fmax3(mx[i & 1], __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
              m = fmaxf(m, fmaxf(mx[0], mx[1]) * cf[g16]);
            }
            return m;
          };
          // P = 2^(y − m_ref) as bf16 over S; returns the tile's row sum.
          auto p_pass = [&]() -> float {
            const float m = m_ref == -CUDART_INF_F ? 0.f : m_ref;
            const uint64_t nm2 = f2_pack(-m, -m);
            uint64_t cf2[8];
#pragma unroll
            for (int g16 = 0; g16 < 8; ++g16) cf2[g16] = f2_pack(cf[g16], cf[g16]);
            uint64_t ls2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) ls2[k] = f2_pack(0.f, 0.f);
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float x0, x1;
                f2_unpack(ffma2(f2_pack(__uint_as_float(s[ch][2 * e]), __uint_as_float(s[ch][2 * e + 1])),
                                cf2[2 * ch + e / 8], nm2),
                          x0, x1);
                const float p0 = ex2_approx(x0);
                const float p1 = ex2_approx(x1);
                ls2[e & 3] = fadd2(ls2[e & 3], f2_pack(p0, p1));
                pk[e] = pack_bf16x2(p0, p1);
              }
              tmem_st16(tS + ch * 16, pk);
            }
            float ls[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) f2_unpack(ls2[k], ls[2 * k], ls[2 * k + 1]);
            return ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
          };
          auto set_far = [&]() {
            far = __any_sync(0xffffffffu, m_ref != -CUDART_INF_F && !(fabsf(m_ref) < 0x1p20f));
          };
          // Far references: y is formed before the reference is taken off, so that the
          // largest of the row comes to 0 exactly.
          auto form_y = [&]() {
#pragma unroll
            for (int ch = 0; ch < 4; ++ch)
#pragma unroll
              for (int i = 0; i < 32; ++i) s[ch][i] = __float_as_uint(__uint_as_float(s[ch][i]) * cf[2 * ch + i / 16]);
#pragma unroll
            for (int g16 = 0; g16 < 8; ++g16) cf[g16] = 1.f;
          };
          if (j == 0) set_far();
          float lt;
#pragma unroll 1
          for (bool moved = false;; moved = true) {  // (one copy of the pass in the code)
            if (far) form_y();
            lt = p_pass();
            if (moved || !__any_sync(0xffffffffu, !(lt < 0x1p40f))) break;
            const float m_new = fmaxf(m_ref, row_max());
            const float alpha = (m_ref == -CUDART_INF_F) ? 0.f : ex2_approx(m_ref - m_new);
            m_ref = m_new;
            l *= alpha;
            set_far();
#pragma unroll 1
            for (int ch = 0; j > 0 && ch < D / 16; ++ch) {
              uint32_t o[16];
              tmem_ld16(tO + ch * 16, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tO + ch * 16, o);
            }
            tmem_wait_st();
          }
          l += lt;
          sees -= stride * kKeys;
          all_see -= stride * kKeys;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(C::B_PFULL + t));
        }
        // Q's place is free: the next item's, if that is known
        if (const int i = (items + 1) % C::NI;
            ok && __all_sync(0xffffffffu, mbar_test_wait(bar(C::B_IFULL + i), (items + 1) / C::NI & 1))) {
          const uint32_t now = item;
          item = sb + C::OFF_ITEM + i * C::ITEM_INTS * 4;
          if (field(kTiles) > 0 && field(kCnt0 + t) > 0 && first_row() < all_rows()) {
            load_q();
            phases |= kRawAhead;
          }
          item = now;
        }
        if (!ok || !wait(C::B_ODONE + t, phase(kItem))) return;
        phases ^= kItem;
        tc_fence_after();
      }
      // ---- a dual item: the first half's warps, which have the same lanes of tensor memory,
      // take the second half's O with their own; m and l go through its columns of S
      const bool join = field(kDual) && field(kCnt1) > 0;
      float join0 = 1.f, join1 = 0.f;  // factors of the halves' O
      if (join) {
        uint32_t ml[16];
        const uint32_t tM = lane_addr + C::S_COL(1);
        if (t == 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) ml[i] = __float_as_uint(i == 0 ? m_ref : l);
          tmem_st16(tM, ml);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(C::B_JOIN));
          if (wait(C::B_JOIN + 1, phase(kJoin))) tc_fence_after();
          phases ^= kJoin;
          return;
        }
        if (!wait(C::B_JOIN, phase(kJoin))) return;
        phases ^= kJoin;
        tc_fence_after();
        tmem_ld16(tM, ml);
        tmem_wait_ld();
        reg_fence(ml);
        const float m1 = __uint_as_float(ml[0]), m = fmaxf(m_ref, m1);
        join0 = m_ref == -CUDART_INF_F ? 0.f : ex2_approx(m_ref - m);
        join1 = m1 == -CUDART_INF_F ? 0.f : ex2_approx(m1 - m);
        l = fmaf(__uint_as_float(ml[1]), join1, l * join0);
        m_ref = m;
      } else if (field(kDual) && t == 1) {
        return;
      }
      const int first = first_row(), rows = all_rows(), hk = field(kHk), tok0 = field(kTok0), slot = field(kSlot);
      const bool exists = first + r < rows;
      const int tok = (first + r) / p.G, g = first + r - tok * p.G;
      // a row that sees a value stored as NaN (the products have taken it for a number)
      if (const int key = field(kNan); key != kNoKey && chunk8::visible(field(kLen), field(kN), tok, p.causal) > key)
        l = CUDART_NAN_F;
      auto load_o = [&](int c0, uint32_t (&o)[32]) {  // 32 columns of O
        tmem_ld32(tO + c0, o);
        if (join) {
          uint32_t o1[32];
          tmem_ld32(lane_addr + C::O_COL(1) + c0, o1);
          tmem_wait_ld();
          reg_fence(o);
          reg_fence(o1);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(fmaf(__uint_as_float(o[i]), join0, __uint_as_float(o1[i]) * join1));
        } else {
          tmem_wait_ld();
          reg_fence(o);
        }
      };
      const size_t part = static_cast<size_t>(slot < 0 ? 0 : slot) * kRows + t * kHalf + r;
      if (slot < 0) {
        // ---- O / l, row by row (staged for whole lines it would take Q's place, which the
        // next item's rows are on their way to)
        const float inv_l = l == 0.f ? 0.f : exp2_int(kVShift) / l;
        uint4* dst = reinterpret_cast<uint4*>(p.o + (static_cast<size_t>(tok0 + tok) * p.H + hk * p.G + g) * D);
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t o[32];
          load_o(cb * 32, o);
#pragma unroll
          for (int u = 0; u < 4; ++u) {  // a 16-byte chunk; its dimensions change places again
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t* q4 = o + 8 * u + 4 * e;
              w[2 * e] = pack_bf16x2(__uint_as_float(q4[0]) * inv_l, __uint_as_float(q4[2]) * inv_l);
              w[2 * e + 1] = pack_bf16x2(__uint_as_float(q4[1]) * inv_l, __uint_as_float(q4[3]) * inv_l);
            }
            if (exists) dst[cb * 4 + u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        tc_fence_before();
        if (exists)
          p.lse[static_cast<size_t>(hk * p.G + g) * p.total + tok0 + tok] =
              l == 0.f ? -CUDART_INF_F : (m_ref + log2f(l)) * kLn2;
      } else if (exists) {
        reinterpret_cast<float2*>(p.ml_part)[part] = make_float2(l == 0.f ? -CUDART_INF_F : l > 0.f ? m_ref : l, l);  // (NaN: both)
      }
      if (slot >= 0 && cnt > 0) {
        // ---- a partial: four dimensions of 32 rows side by side
        float4* dst = reinterpret_cast<float4*>(p.o_part) + static_cast<size_t>(slot) * (kRows * D / 4) + t * kHalf + r;
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t o[32];
          load_o(cb * 32, o);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (exists)
              dst[(cb * 8 + u) * kRows] = make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 2]),
                                                      __uint_as_float(o[4 * u + 1]), __uint_as_float(o[4 * u + 3]));
        }
        tc_fence_before();
      }
      if (join) {
        tc_fence_before();
        mbar_arrive(bar(C::B_JOIN + 1));
      }
    };
    while (ok) {
      const int i = items % C::NI;
      if (!wait(C::B_IFULL + i, items / C::NI)) break;
      item = sb + C::OFF_ITEM + i * C::ITEM_INTS * 4;
      const bool any = field(kTiles) > 0;
      if (any) take();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::B_IEMPTY + i));
      ++items;
      if (!any) break;
    }
    // A copy issued lands before the CTA may exit, whoever aborted.
    if (phases & kRawEver) wait_drain(bar(C::B_RAW + warp), phase(kRaw) ^ ((phases & kRawAhead) ? 0 : 1), p.err, p.timeout_ns);
  } else {
    setmaxnreg_dec<C::REG_OTHER>();
    if (warp == C::MMA_WARP) {
      // ------------------------------------------------------------ MMA
      // The tensor core's queue holds some 190 cycles of products, and a wait for what
      // is there already, or a commit, costs this thread 50 to 100: each stands between
      // two batches of products, none beside another where that can be had.  (All waits
      // of a tile before its products: 880 us on 8192 rows over 32768 keys; a thread for
      // each row tile, whose products then alternate on the tensor core: 1064.)
      constexpr uint32_t idesc_s = idesc_e4m3(128, 128, false);
      constexpr uint32_t idesc_o = idesc_bf16(128, D, false, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t dQ0 = sdesc8<D>(sb + C::OFF_Q, 16, 16 * D);
      const uint64_t dK0 = sdesc8<D>(sb + C::OFF_K, 16);
      const uint64_t dV0 = sdesc_sw128(sb + C::OFF_V, C::BLK_BYTES, 1024);
      auto issue_s = [&](int t, int ks) {
        const uint64_t dQ = sdesc_add(dQ0, t * C::TILE_BYTES), dK = sdesc_add(dK0, ks * C::CODE_BYTES);
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_e4m3(tm + C::S_COL(t), sdesc_add(dQ, term * 8 * D + kk * 32), sdesc_add(dK, kk * 32), idesc_s,
                     term + kk > 0);
      };
      auto issue_pv = [&](int t, int vs, bool acc) {
        const uint64_t dV = sdesc_add(dV0, vs * C::TILE_BYTES);
#pragma unroll(C::PV_UNROLL)
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(tm + C::O_COL(t), tm + C::S_COL(t) + kk * 8, sdesc_add(dV, kk * 2048), idesc_o,
                 (acc || kk > 0) ? 1u : 0u);
      };
      bool ok = true;
      auto wait = [&](int i, int phase) {  // (the whole warp, which stays together)
        ok = ok && wait_bounded(bar(i), phase & 1, abort_flag, p.err, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      Ring<C::NK> kr;                        // the next tile of K, of V
      Ring<C::NV> vr;
      uint32_t half_phases = 0;  // bit t: of half t's items, bit 2 + t: of its P tiles
      auto wait_half = [&](int b, int t, int bit) {
        const int ph = (half_phases >> (bit + t)) & 1;
        half_phases ^= 1u << (bit + t);
        return wait(b + t, ph);
      };
      auto wait_k = [&]() { return wait(C::B_KFULL + kr.i, kr.phase); };
      auto wait_v = [&]() { return wait(C::B_VFULL + vr.i, vr.phase); };
      auto take_s = [&](int t, bool free_k) {  // S of half t over the K that is next
        tc_fence_after();
        if (elect_one()) {
          issue_s(t, kr.i);
          tc_commit(bar(C::B_SFULL + t));
          if (free_k) tc_commit(bar(C::B_KEMPTY + kr.i));
        }
      };
      Item it;
      while (ok && take_item(it)) {
        const int tiles = __shfl_sync(0xffffffffu, it.tiles, 0);
        const int cnt0 = __shfl_sync(0xffffffffu, it.cnt0, 0), cnt1 = __shfl_sync(0xffffffffu, it.cnt1, 0);
        auto cnt = [&](int t) { return t ? cnt1 : cnt0; };
        if (__shfl_sync(0xffffffffu, it.dual ? 1 : 0, 0) != 0) {
          // The halves take the tiles in turn: K and V of each are free after its half.
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            if (cnt(t) == 0) break;
            if (!wait_k() || !wait_half(C::B_Q, t, 0)) break;
            take_s(t, true);
            kr.step();
          }
          for (int j = 0; ok && j < cnt0; ++j) {
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
              if (j >= cnt(t)) break;
              if (!wait_v() || !wait_half(C::B_PFULL, t, 2)) break;
              tc_fence_after();
              if (elect_one()) {
                issue_pv(t, vr.i, j > 0);
                if (j + 1 == cnt(t)) tc_commit(bar(C::B_ODONE + t));
                tc_commit(bar(C::B_VEMPTY + vr.i));
              }
              vr.step();
              if (j + 1 < cnt(t)) {
                if (!wait_k()) break;
                take_s(t, true);
                kr.step();
              }
            }
          }
          continue;
        }
        if (!wait_k()) break;
#pragma unroll(C::HALF_UNROLL)
        for (int t = 0; t < 2; ++t)
          if (cnt(t) > 0 && wait_half(C::B_Q, t, 0)) take_s(t, false);
        if (!ok) break;
        if (elect_one()) tc_commit(bar(C::B_KEMPTY + kr.i));
        kr.step();
        wait_v();
        for (int j = 0; ok && j < tiles; ++j) {
          const bool more = j + 1 < tiles;
#pragma unroll(C::HALF_UNROLL)
          for (int t = 0; t < 2; ++t) {
            if (j < cnt(t) && wait_half(C::B_PFULL, t, 2)) {
              tc_fence_after();
              if (elect_one()) {
                issue_pv(t, vr.i, j > 0);
                if (j + 1 == cnt(t)) tc_commit(bar(C::B_ODONE + t));
              }
            }
            if (!ok) break;
            if (t == 0) {
              if (more && !wait_k()) break;
            } else {
              if (elect_one()) tc_commit(bar(C::B_VEMPTY + vr.i));
              vr.step();
              if (more && !wait_v()) break;
            }
            if (j + 1 < cnt(t)) take_s(t, false);
          }
          if (ok && more) {
            if (elect_one()) tc_commit(bar(C::B_KEMPTY + kr.i));
            kr.step();
          }
        }
      }
      // every MMA issued so far must finish before tensor memory is released
      if (elect_one()) tc_commit(bar(C::B_DRAIN));
      wait_drain(bar(C::B_DRAIN), 0, p.err, p.timeout_ns);
    } else if (warp != C::COPY_WARP && warp != C::V_WARP) {
      // ---------------------------------------------------------------- conversion
      // A thread's 16-byte chunk of codes becomes two chunks of bf16; a warp takes 32
      // chunks of consecutive rows, every fifth group of them.  The chunks of a
      // quarter-warp lie in two rows, at d = 128 in the two halves of them: neither its
      // reads nor its swizzled writes meet in a bank.
      const int cw = warp < C::MMA_WARP ? warp - 9 : warp - 10;
      constexpr int CPR = D / 16, ROWS = 32 / CPR, GROUPS = kKeys / ROWS;
      int row0, chunk;  // within a group
      if (D == 128) {
        const int rb = (lane >> 2) & 1;
        row0 = ((lane >> 4) & 1) * 2 + rb;
        chunk = (lane & 3) + 4 * (((lane >> 3) & 1) ^ rb);
      } else {
        row0 = lane >> 2;
        chunk = lane & 3;
      }
      const uint32_t in0 = row0 * D + chunk * 16;
      const uint32_t c0 = 2 * (chunk % 4), out0 = (2 * chunk / 8) * C::BLK_BYTES;
      auto place = [&](int row, int half) -> uint32_t { return out0 + row * 128 + (((c0 + half) ^ (row & 7)) << 4); };
      // From a group of the warp's to its next the chunk's place moves by STEP, and its row's
      // last three bits, which the swizzle takes, change by a half where a group has four rows;
      // the second chunk's place is the first's with another lowest bit.
      constexpr uint32_t STEP = C::CONVERT_WARPS * ROWS * 128, FLIP = ROWS == 4 ? 64 : 0;
      static_assert(C::CONVERT_WARPS % 2 == 1 && (ROWS == 4 || ROWS == 8), "rows mod 8 from group to group");
      const uint32_t place0 = place(cw * ROWS + row0, 0);
      int tile = 0;
      Ring<C::NC> cr;
      Ring<C::NV> vr;
      bool ok = true;
      auto wait = [&](int i, int phase) {
        ok = ok && wait_bounded(bar(i), phase & 1, abort_flag, p.err, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      Item it;
      while (ok && take_item(it)) {
        int* first_nan = reinterpret_cast<int*>(smem + C::OFF_ITEM + (items - 1) % C::NI * (C::ITEM_INTS * 4)) + 12;
        for (int kt = it.k0; kt < it.k0 + it.tiles; ++kt, ++tile) {
          const int held = cache8::tokens_from(it.len, kt, kKeys, 0);  // tokens of the tile, if fewer than its rows
          const int st = cr.i, slot = vr.i;
          if (!wait(C::B_CFULL + st, cr.phase)) break;
          if (tile >= C::NV && !wait(C::B_VEMPTY + slot, vr.phase ^ 1)) break;
          const uint8_t* codes = smem + C::OFF_C + st * C::CODE_BYTES + in0;
          const uint2* factors = reinterpret_cast<const uint2*>(smem + C::OFF_VF) + st * C::MAX_PPT;
          uint8_t* out = smem + C::OFF_V + slot * C::TILE_BYTES;
          // (rolled: beside the softmax's code an unrolled loop costs instruction fetches)
          uint4 next = *reinterpret_cast<const uint4*>(codes + cw * ROWS * D);
          uint32_t top = 0, at = sb + C::OFF_V + slot * C::TILE_BYTES + place0;
#pragma unroll 1
          for (int g = cw; g < GROUPS; g += C::CONVERT_WARPS, at = (at + STEP) ^ FLIP) {
            const uint4 now = next;
            const uint32_t f = factors[g * ROWS >> p.block_shift].x;  // (a group lies in one page)
            if (g + C::CONVERT_WARPS < GROUPS)
              next = *reinterpret_cast<const uint4*>(codes + (g + C::CONVERT_WARPS) * ROWS * D);
            const uint32_t in[4] = {now.x, now.y, now.z, now.w};
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              widen4(in[k], v[2 * k], v[2 * k + 1], top);
              v[2 * k] = mul_bf16x2(v[2 * k], f);
              v[2 * k + 1] = mul_bf16x2(v[2 * k + 1], f);
            }
            st_shared_v4(at, v[0], v[1], v[2], v[3]);
            st_shared_v4(at ^ 16u, v[4], v[5], v[6], v[7]);
          }
          // Seldom: slots without a token, which may hold anything, become 0; a scale above
          // 2^55, whose factor does not fit one bf16 number, is a second one; of tokens with a
          // value stored as NaN the first is noted in the item (P of rows that do not see it is
          // 0, which a NaN in the product would not leave so).
          if (held < kKeys || __any_sync(0xffffffffu, factors[lane % C::MAX_PPT].y != kOne2 || nan_among(top))) {
#pragma unroll 1
            for (int g = cw; g < GROUPS; g += C::CONVERT_WARPS) {
              const int row = g * ROWS + row0;
              const uint32_t f = factors[row >> p.block_shift].y;
              const uint4 c = *reinterpret_cast<const uint4*>(codes + g * ROWS * D);
              if (((nan_codes(c.x) | nan_codes(c.y) | nan_codes(c.z) | nan_codes(c.w)) & 0x80808080u) && row < held &&
                  factors[row >> p.block_shift].x != 0)  // (of a page out of range: what was here before)
                atomicMin(first_nan, kt * kKeys + row);
#pragma unroll 1
              for (int half = 0; half < 2; ++half) {
                uint4* at = reinterpret_cast<uint4*>(out + place(row, half));
                const uint4 x = *at;
                *at = row >= held ? make_uint4(0u, 0u, 0u, 0u)
                                  : make_uint4(mul_bf16x2(x.x, f), mul_bf16x2(x.y, f), mul_bf16x2(x.z, f), mul_bf16x2(x.w, f));
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(C::B_CEMPTY + st));
            mbar_arrive(bar(C::B_VFULL + slot));
          }
          cr.step();
          vr.step();
        }
      }
    } else if (warp == C::V_WARP) {
      // ------------------------------------------------------------ copies of V
      const int ppt = kKeys >> p.block_shift, page_bytes = D << p.block_shift, window = 32 / ppt;  // tiles of 32 pages
      Ring<C::NC> cr;
      int tile = 0;
      bool ok = true;
      Item it;
      while (ok && take_item(it)) {
        const int pages = cache8::pages_of(it.len, p.block_shift), end = it.k0 + it.tiles;
        auto load_pages = [&](int kt) {  // lane i: page i of the window at tile kt, -1: none
          return kt + lane / ppt < end && kt * ppt + lane < pages
                     ? p.table[static_cast<size_t>(it.b) * p.table_cols + kt * ppt + lane]
                     : -1;
        };
        auto load_scales = [&](int& page) {  // (a page out of range is reported with K's)
          if (page < 0 || page >= p.num_blocks) page = -1;
          return page >= 0 ? p.v_scale[static_cast<size_t>(page) * p.Hk + it.hk] : 0.f;
        };
        int cur = load_pages(it.k0);
        float scale = load_scales(cur);
        for (int k0 = it.k0; ok && k0 < end; k0 += window) {
          int next = load_pages(min(k0 + window, end));
          float next_scale = 0.f;
          for (int i = 0; i < window && k0 + i < end; ++i, ++tile) {
            const int from = (i * ppt + lane) & 31;
            const int page = __shfl_sync(0xffffffffu, cur, from);
            const float vs = __shfl_sync(0xffffffffu, scale, from);
            const bool mine = lane < ppt && page >= 0;  // (a page out of range reads as zeros: its factor is 0)
            if (tile >= C::NC) ok = wait_bounded(bar(C::B_CEMPTY + cr.i), cr.phase ^ 1, abort_flag, p.err, p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * page_bytes;
            if (lane < C::MAX_PPT)
              reinterpret_cast<uint2*>(smem + C::OFF_VF)[cr.i * C::MAX_PPT + lane] =
                  mine ? scale_factors(vs) : make_uint2(0u, kOne2);
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bar(C::B_CFULL + cr.i), bytes);
            __syncwarp();
            if (mine)
              bulk_load(sb + C::OFF_C + cr.i * C::CODE_BYTES + lane * page_bytes,
                        p.v_codes + (static_cast<size_t>(page) * p.Hk + it.hk) * page_bytes, page_bytes,
                        bar(C::B_CFULL + cr.i));
            cr.step();
            if (i == 0) next_scale = load_scales(next);
          }
          cur = next;
          scale = next_scale;
        }
      }
      // Every copy issued lands before the CTA may exit, whoever aborted.
      for (int s = 0; s < C::NC && s < tile; ++s)
        wait_drain(bar(C::B_CFULL + s), ((tile - 1 - s) / C::NC) & 1, p.err, p.timeout_ns);
    } else {
      // ------------------------------------------------------------ items, copies
      const int ppt = kKeys >> p.block_shift, page_bytes = D << p.block_shift;
      struct Unit {
        int b, hk, rb, k0, k1, nt, n, len, tok0;  // the item (tiles k0 .. k1 of nt)
        bool dual;
        int kt, tiles;                            // first tile of the unit, and how many
        long long last;                           // the first unit of the item's last tile
        int page;                                 // this lane's page (of 32 / ppt tiles), -1: none
        float ks;
      };
      int b = static_cast<int>(found[1]) / p.row_blocks, rb = static_cast<int>(found[1]) - b * p.row_blocks;
      long long x_start = found[0], at = u_lo;  // first unit of the pair; the next unit
      int nt = 0, w = 0, n = 0, len = 0, tok0 = 0;  // (w: units of a tile)
      auto load_pair = [&]() {
        chunk_seq(p, b, tok0, n, len);
        n = __shfl_sync(0xffffffffu, n, 0);  // the warp stays together even if a caller changes the lengths meanwhile
        len = __shfl_sync(0xffffffffu, len, 0);
        nt = chunk8::row_tiles(len, n, p.G, rb * kRows, kRows, p.causal);
        w = chunk8::tile_units(chunk8::dual(n, p.G, rb), few);
      };
      // The first sequence from `from` on that has new tokens, 32 at a time: the other roles
      // wait for an item meanwhile, and a wait has a limit.
      auto next_with = [&](int from) {
        for (; from < p.B; from += 32) {
          int first, rows = 0, held;
          if (from + lane < p.B) chunk_seq(p, from + lane, first, rows, held);
          const unsigned some = __ballot_sync(0xffffffffu, rows > 0);
          if (some) return from + __ffs(some) - 1;
        }
        return p.B;
      };
      load_pair();
      auto next_unit = [&](Unit& u) {
        u.tiles = 0;
        while (u.tiles <= 0) {
          if (at >= u_hi) return;
          while (at >= x_start + pair_units(chunk8::counted(nt, uncut) * w)) {
            x_start += pair_units(chunk8::counted(nt, uncut) * w);
            chunk8::next_pair(b, rb, n, p.G, next_with);
            if (b >= p.B) {
              at = u_hi;
              return;
            }
            load_pair();
          }
          const int own = chunk8::counted(nt, uncut) * w, units = own + extra;  // of an item
          const int hk = static_cast<int>((at - x_start) / units);
          const long long first = x_start + static_cast<long long>(hk) * units + extra;
          u.b = b, u.rb = rb, u.n = n, u.len = len, u.tok0 = tok0, u.nt = nt, u.hk = hk, u.dual = chunk8::dual(n, p.G, rb);
          u.kt = chunk8::tiles_before(at - first, w, nt, uncut);
          u.k0 = chunk8::tiles_before(u_lo - first, w, nt, uncut);
          u.k1 = chunk8::tiles_before(u_hi - first, w, nt, uncut);
          u.tiles = min(u.k1 - u.kt, 32 / ppt);
          u.last = first + static_cast<long long>(nt - 1) * w;
          // (no tile of it begins in what is left of the run: on to the next item, or the end)
          at = u.tiles > 0 && !uncut ? first + static_cast<long long>(u.kt + u.tiles) * w : first + own;
        }
        u.page = -1;
        if (lane < u.tiles * ppt && u.kt * ppt + lane < cache8::pages_of(len, p.block_shift))
          u.page = p.table[static_cast<size_t>(b) * p.table_cols + u.kt * ppt + lane];
      };
      auto load_scales = [&](Unit& u) {
        const bool token = lane < u.tiles * ppt && u.kt * ppt + lane < cache8::pages_of(u.len, p.block_shift);
        u.ks = 0.f;
        if (token && u.page >= 0 && u.page < p.num_blocks) {
          u.ks = p.k_scale[static_cast<size_t>(u.page) * p.Hk + u.hk];
        } else {
          if (token) atomicOr(p.err, kDevErrPage);
          u.page = -1;
        }
      };
      Unit cur, next;
      next_unit(cur);
      if (cur.tiles > 0) load_scales(cur);
      int tile = 0, published = 0;  // tiles issued, items
      bool ok = true;
      auto publish = [&](const Unit& u) {
        const int s = published % C::NI;
        if (published >= C::NI)
          ok = wait_bounded(bar(C::B_IEMPTY + s), (published / C::NI - 1) & 1, abort_flag, p.err, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        if (lane == 0) {
          int4* dst = reinterpret_cast<int4*>(smem + C::OFF_ITEM + s * C::ITEM_INTS * 4);
          int slot = -1, cnt0 = 0, cnt1 = 0;
          if (u.tiles > 0) {
            const bool whole = u.k0 == 0 && u.k1 == u.nt;
            if (!whole) slot = 2 * blockIdx.x + (u.k0 == 0 ? 1 : 0);
            const int first = u.rb * kRows;
            if (u.dual) {
              cnt0 = (u.k1 - u.k0 + 1) / 2;
              cnt1 = (u.k1 - u.k0) / 2;
            } else {
              cnt0 = max(min(u.k1, chunk8::row_tiles(u.len, u.n, p.G, first, kHalf, p.causal)) - u.k0, 0);
              cnt1 = max(min(u.k1, chunk8::row_tiles(u.len, u.n, p.G, first + kHalf, kHalf, p.causal)) - u.k0, 0);
            }
            if (!whole && u.k0 == 0) {
              // begins here and ends in another CTA's run: joined by the second kernel
              int* m = p.merge + blockIdx.x * 8;
              m[1] = u.tok0, m[2] = u.n, m[3] = u.hk, m[4] = u.rb;
              m[0] = chunk8::run_of(u.last, total, ctas);
            }
          }
          dst[0] = make_int4(u.b, u.hk, u.rb, u.k0);
          dst[1] = make_int4(u.tiles > 0 ? u.k1 - u.k0 : 0, u.n, u.len, u.tok0);
          dst[2] = make_int4(cnt0, cnt1, slot, u.tiles > 0 && u.dual);
          dst[3] = make_int4(kNoKey, 0, 0, 0);
          mbar_arrive(bar(C::B_IFULL + s));
        }
        ++published;
      };
      while (ok && cur.tiles > 0) {
        if (cur.kt == cur.k0) publish(cur);
        next_unit(next);
        for (int i = 0; ok && i < cur.tiles; ++i) {
          const int n_pages = min(ppt, cache8::pages_of(cur.len, p.block_shift) - (cur.kt + i) * ppt);
          const int from = (i * ppt + lane) & 31;
          const int page = __shfl_sync(0xffffffffu, cur.page, from);
          const float ks = __shfl_sync(0xffffffffu, cur.ks, from);
          const bool mine = lane < n_pages && page >= 0;
          // a page out of range reads as zeros (the copy's fill)
          const int ks_slot = tile % C::NK;
          if (tile >= C::NK)
            ok = wait_bounded(bar(C::B_KEMPTY + ks_slot), (tile / C::NK - 1) & 1, abort_flag, p.err, p.timeout_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane < C::MAX_PPT)
            reinterpret_cast<float*>(smem + C::OFF_KS)[tile % C::NSC * C::MAX_PPT + lane] = mine ? ks : 1.f;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(C::B_SCFULL + tile % C::NSC));
            mbar_arrive_expect_tx(bar(C::B_KFULL + ks_slot), max(n_pages, 0) * page_bytes);
          }
          __syncwarp();
          if (lane < n_pages)
            tma_load_4d(sb + C::OFF_K + ks_slot * C::CODE_BYTES + lane * page_bytes, &tmK, bar(C::B_KFULL + ks_slot), 0, 0,
                        cur.hk, page >= 0 ? page : p.num_blocks);
          ++tile;
          if (i == 0 && next.tiles > 0) load_scales(next);
        }
        cur = next;
      }
      if (ok) {  // no more items
        cur.tiles = 0;
        publish(cur);
      }
      // Every copy issued lands before the CTA may exit, whoever aborted.
      for (int s = 0; s < C::NK && s < tile; ++s)
        wait_drain(bar(C::B_KFULL + s), ((tile - 1 - s) / C::NK) & 1, p.err, p.timeout_ns);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the items that several CTAs have partial results of.  Block (c0, y): rows
// [16 y, 16 y + 16) of the item whose first part is CTA c0's.  The parts of a row are
// first weighed, all at once (a thread a row and part: few rows have as many as the
// launch has CTAs), then summed by a thread a row and four values, eight parts' loads
// at a time, in the order of the keys.  Bound by the latency of those loads: with 25
// parts of up to 50 rows the whole call takes 28.5 us; 60 with threads that weigh and sum
// part by part.
constexpr int kMergeRows = 16;

template <int D>
__global__ void __launch_bounds__(4 * D) fa_chunk8_merge_kernel(const Chunk8Params p) {
  extern __shared__ float weights[];  // [part][kMergeRows]
  __shared__ float red[D / 4][kMergeRows];
  grid_dependency_wait();
  const int c0 = blockIdx.x;
  const int* m = p.merge + c0 * 8;
  const int parts = m[0] - c0 + 1;
  const int tok0 = m[1], n = m[2], hk = m[3], rb = m[4];
  const int row0 = blockIdx.y * kMergeRows;
  if (m[0] < 0 || rb * kRows + row0 >= n * p.G) return;
  const int r = threadIdx.x % kMergeRows, d4 = threadIdx.x / kMergeRows;
  const int row = row0 + r, f = rb * kRows + row;
  const bool exists = f < n * p.G;
  const float2* ml = reinterpret_cast<const float2*>(p.ml_part);
  const float4* part = reinterpret_cast<const float4*>(p.o_part);
  // a CTA's first slot has the item that it ends or goes through, the second the one that it begins
  auto slot = [&](int i) { return static_cast<size_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)); };
  float top = -CUDART_INF_F;
  for (int i = d4; i < parts; i += D / 4) {
    const float t = exists ? ml[slot(i) * kRows + row].x : -CUDART_INF_F;  // -inf: it sees none of the part's keys
    weights[i * kMergeRows + r] = t;
    top = fmaxf(top, t);
  }
  red[d4][r] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < D / 4; ++i) top = fmaxf(top, red[i][r]);
  __syncthreads();
  float l = 0.f;
  for (int i = d4; i < parts; i += D / 4) {
    const float t = weights[i * kMergeRows + r];
    const float wt = t == -CUDART_INF_F ? 0.f : ex2_approx(t - top);
    weights[i * kMergeRows + r] = wt;
    if (wt != 0.f) l = fmaf(wt, ml[slot(i) * kRows + row].y, l);
  }
  red[d4][r] = l;
  __syncthreads();
  if (!exists) return;
  l = 0.f;
#pragma unroll
  for (int i = 0; i < D / 4; ++i) l += red[i][r];
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = 0; i < parts; ++i) {
    const float wt = weights[i * kMergeRows + r];
    const float4 v = part[(slot(i) * (D / 4) + d4) * kRows + row];
    // what a row that sees none of the keys has in its place is not defined
    const float4 u = wt != 0.f ? v : make_float4(0.f, 0.f, 0.f, 0.f);
    o.x = fmaf(wt, u.x, o.x), o.y = fmaf(wt, u.y, o.y);
    o.z = fmaf(wt, u.z, o.z), o.w = fmaf(wt, u.w, o.w);
  }
  const float inv = l == 0.f ? 0.f : exp2_int(kVShift) / l;
  const int tok = f / p.G, h = hk * p.G + f - tok * p.G;
  *reinterpret_cast<uint2*>(p.o + (static_cast<size_t>(tok0 + tok) * p.H + h) * D + 4 * d4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (d4 == 0)
    p.lse[static_cast<size_t>(h) * p.total + tok0 + tok] = l == 0.f ? -CUDART_INF_F : (top + log2f(l)) * kLn2;
}

template <int D>
cudaError_t launch_chunk(const CUtensorMap& tk, const Chunk8Params& p, int ctas, bool merge, cudaStream_t s) {
  using C = ChunkCfg<D>;
  static SmemLimit smem_limit;
  cudaError_t e = smem_limit.ensure(reinterpret_cast<const void*>(fa_chunk8_kernel<D>), C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  // The softmax warps' larger share of registers comes out of what the CTA was
  // launched with: with fewer the kernel would wait for it without end.
  static const int launch_regs = [] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(fa_chunk8_kernel<D>)) == cudaSuccess ? a.numRegs : 0;
  }();
  if (launch_regs != 128) return cudaErrorInvalidConfiguration;
  e = launch_kernel(fa_chunk8_kernel<D>, dim3(static_cast<unsigned>(ctas)), dim3(C::NUM_THREADS), C::SMEM_BYTES, s, true, tk, p);
  if (e != cudaSuccess || !merge) return e;
  const long long rows = static_cast<long long>(p.max_new < p.total ? p.max_new : p.total) * p.G;  // of a sequence, at most
  const unsigned groups = static_cast<unsigned>(((rows < kRows ? rows : kRows) + kMergeRows - 1) / kMergeRows);
  return launch_kernel(fa_chunk8_merge_kernel<D>, dim3(static_cast<unsigned>(ctas), groups),
                       dim3(4 * D), static_cast<unsigned>(ctas) * kMergeRows * sizeof(float), s, true, p);
}

}  // namespace

cudaError_t launch_cache8_chunk(int d, const CUtensorMap& tk, const Chunk8Params& p, int ctas, bool merge,
                                cudaStream_t s) {
  return d == 64 ? launch_chunk<64>(tk, p, ctas, merge, s) : launch_chunk<128>(tk, p, ctas, merge, s);
}

}  // namespace fa
