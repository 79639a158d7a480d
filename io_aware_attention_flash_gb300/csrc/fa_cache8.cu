// The 8-bit paged key/value cache for sm_103a: storing new tokens, and the
// attention of new tokens over it.
//
// Cache: K and V are pools of pages [num_blocks, Hk, block, d] of e4m3 codes
// with one fp32 scale for each (page, head); a sequence's page table names the
// page of each run of `block` tokens.  A scale is the smallest power of two s
// with max |x| <= 448 s over the page's tokens and head, so dividing by it and
// multiplying by it are exact and the e4m3 rounding (at most 2^-4 of a value,
// 2^-10 s for values below 2^-6 s) is the only one; a general scale would not
// be more accurate, since e4m3 keeps the same relative step at any size.
//
// The store, and the attention of one new token, are bound by DRAM.  Measured on a
// GB300 (a plain copy moves 6.78 TB/s), whole calls: the store of 34,700 tokens of 8
// heads, d = 128, 32 us, 6.5 TB/s; the attention of one token over 4 x 32768 tokens,
// 32 heads, d = 128, 163 us, 6.6 TB/s, over 64 sequences of 100 .. 8192 tokens, 32
// query over 8 heads, 94 us, 5.9 TB/s, and over 16 x 16384 tokens of 8 heads, one
// call behind another, 6.0 TB/s at d = 128 and 4.8 (pages of 16) to 5.3 TB/s (of 64)
// at d = 64, with 1 or 4 query heads a key/value head.  Several new tokens are held
// by the latency of a tile's chain (scores, the exchange of the row maxima, P, the
// product): 4 of 16 sequences, 64 query over 8 heads of 64, take 30 us for 39 MB
// with the issue slots 47 % busy, the tensor pipe 7 % and DRAM 18 %; each of the two
// groups of 16 rows walks the key/value head's tiles for itself.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "cache8_phases.h"
#include "cache8_tiles.h"
#include "e4m3.cuh"
#include "fa_kernels.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

// ----------------------------------------------------------------------------
// Store
// ----------------------------------------------------------------------------
// One group of TG threads quantises the new tokens of one (page, head) of K or
// V: each thread keeps CH 16-byte chunks of them in registers between the
// maximum and the rounding, so the input is read once, and its loads do not
// wait for the page table's.  A page that already holds tokens keeps its scale
// if that suffices; otherwise they are rounded again to the larger one.
// Groups of consecutive heads are consecutive, so a block's loads cover whole
// rows of the token-major input.
template <int CH, int TG, int D, int BLOCK, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) fa_cache8_store_kernel(const Cache8StoreParams p) {
  static_assert(CH * TG * 8 == D * BLOCK, "a group's chunks cover a page and head");
  constexpr int GPB = NT / TG;  // groups per block
  constexpr int C8 = D / 8;     // chunks per token
  __shared__ uint32_t warp_max[NT / 32];
  const int group = threadIdx.x / TG, tid = threadIdx.x % TG;
  // blockIdx.x: (sequence, block of tokens); the groups run over K's heads, then V's
  const int b = blockIdx.x / p.blocks, nth = blockIdx.x - b * p.blocks;
  const int which = blockIdx.y * GPB + group;
  const bool is_v = which >= p.Hk;
  const int head = is_v ? which - p.Hk : which;
  grid_dependency_wait();  // scheduled while the kernel before it in the stream finishes
  int page = -1, old = 0, lo = 0, hi = 0;  // the page; its tokens [0, old) are held, [lo, hi) are new
  int src = 0;                             // input row of slot 0
  if (which < 2 * p.Hk) {
    const int first = min(max(p.cu_seqlens[b], 0), p.total);
    const int count = min(max(p.cu_seqlens[b + 1], first), p.total) - first;
    const int start = p.start[b];
    const long long end = static_cast<long long>(start) + min(count, p.max_new);
    const long long blk = static_cast<long long>(start) / BLOCK + nth;
    if (start < 0) {
      if (count > 0 && tid == 0) atomicOr(p.err, kDevErrPage);
    } else if (count > 0 && blk * BLOCK < end) {
      if (blk < p.table_cols) page = p.table[static_cast<size_t>(b) * p.table_cols + blk];
      const long long base = blk * BLOCK;
      old = static_cast<int>(max(0LL, start - base));
      lo = old;
      hi = static_cast<int>(min(end - base, static_cast<long long>(BLOCK)));
      src = first + static_cast<int>(base - start);
    }
  }
  const bool touched = hi > lo;
  if (TG == NT ? !touched : __syncthreads_or(touched) == 0) return;
  // Chunk c of a thread: token t0 + c · STEP of the page, the same 8 elements.
  static_assert(TG % C8 == 0, "a thread's chunks lie below one another");
  constexpr int STEP = TG / C8;
  const int t0 = tid / C8;
  const long long ld = is_v ? p.ldv : p.ldk;
  const uint16_t* x = (is_v ? p.v : p.k) + (static_cast<long long>(src) + t0) * ld + head * D + (tid % C8) * 8;
  uint4 val[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    val[c] = make_uint4(0u, 0u, 0u, 0u);
    if (t0 + c * STEP >= lo && t0 + c * STEP < hi) val[c] = *reinterpret_cast<const uint4*>(x + c * (STEP * ld));
  }
  const bool live = touched && page >= 0 && page < p.num_blocks;
  if (touched && !live && tid == 0) atomicOr(p.err, kDevErrPage);
  const size_t ph = live ? static_cast<size_t>(page) * p.Hk + head : 0;
  float* scale = (is_v ? p.v_scale : p.k_scale) + ph;
  const float held = live && old > 0 ? *scale : 0.f;
  // Largest magnitude as bf16 bits.  Infinities and NaN do not set the scale
  // (the maximum passes over NaN; where it is infinite, once more without).
  auto largest = [&](bool finite) {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t w[4] = {val[c].x, val[c].y, val[c].z, val[c].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t m = w[u] & 0x7fff7fffu;
        top = max_bf16x2(top, finite ? m & ~__vcmpgeu2(m, 0x7f807f80u) : m);
      }
    }
    return max(top & 0xffffu, top >> 16);
  };
  uint32_t amax = largest(false);
  if (amax >= 0x7f80u) amax = largest(true);
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (TG > 32) {  // (and every thread has read the scale held before one of them writes the new one)
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
    __syncthreads();
    const int w0 = group * (TG / 32);
#pragma unroll
    for (int w = 0; w < TG / 32; ++w) amax = max(amax, warp_max[w0 + w]);
  }
  if (!live) return;
  const float s = fmaxf(exp2_int(scale_exponent(amax, kScaleFloor)), held);
  // 1 / s of a power of two, by its exponent
  const float inv = exp2_int(127 - static_cast<int>((__float_as_uint(s) >> 23) & 255u));
  const bool again = s > held;
  if (tid == 0 && again) *scale = s;
  const uint64_t inv2 = f2_pack(inv, inv);
  auto codes = [&](uint32_t a, uint32_t b) {  // four values, two a word
    float v[4];
    f2_unpack(fmul2(f2_pack(bf16lo_to_f32(a), bf16hi_to_f32(a)), inv2), v[0], v[1]);
    f2_unpack(fmul2(f2_pack(bf16lo_to_f32(b), bf16hi_to_f32(b)), inv2), v[2], v[3]);
    return pack_e4m3x4(v[0], v[1], v[2], v[3]);
  };
  uint2* out = reinterpret_cast<uint2*>((is_v ? p.v_codes : p.k_codes) + ph * (BLOCK * D)) + tid;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int t = t0 + c * STEP;
    if (t >= lo && t < hi) {
      out[c * TG] = make_uint2(codes(val[c].x, val[c].y), codes(val[c].z, val[c].w));
    } else if (t < old && again) {
      const uint2 code = out[c * TG];
      const float f = held * inv;
      float v[4], w[4];
      unpack_e4m3x4(code.x, v);
      unpack_e4m3x4(code.y, w);
      out[c * TG] = make_uint2(pack_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                               pack_e4m3x4(w[0] * f, w[1] * f, w[2] * f, w[3] * f));
    }
  }
}

template <int D, int BLOCK>
cudaError_t launch_store(const Cache8StoreParams& p, cudaStream_t s) {
  constexpr int CHUNKS = D * BLOCK / 8;
  constexpr int TG = CHUNKS <= 256 ? 32 : CHUNKS / 8;
  constexpr int NT = TG > 128 ? TG : 128;
  const long long x = static_cast<long long>(p.B) * p.blocks, y = (2LL * p.Hk * TG + NT - 1) / NT;
  if (x > 0x7fffffffLL || y > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y));
  return launch_kernel(fa_cache8_store_kernel<CHUNKS / TG, TG, D, BLOCK, NT>, grid, dim3(NT), 0, s, true, p);
}

// ----------------------------------------------------------------------------
// Attention over the cache
// ----------------------------------------------------------------------------
// Work: the tiles (128 rows of 128 bytes of K and of V: 128 tokens, at d = 64
// 256) of every (sequence, key/value head, row group), in
// that order, are shared out in equal runs over the launch's CTAs, whatever
// the sequences' lengths; a row group is up to 16 of the (new token, query
// head) rows that attend to one key/value head.  A CTA that has all tiles of
// an item writes its output; an item that several CTAs share leaves partials
// (m, l, O) that the merge kernel combines in the order of the tiles.
//
// Both products run on the tensor core straight from the codes, keys (or, for
// P V, head dimensions) as the 128 rows of A and the queries as B:
//   S^T = K Q^T     A = K tile, K-major;   B = Q,  K-major
//   O^T = V^T P^T   A = V tile, MN-major;  B = P,  MN-major
// with B in e4m3 as well, split into two terms so that nothing is lost to 8
// bits: q / s_q = hi + lo (s_q a power of two for each row; exact for elements
// above 2^-10 of the row's largest, else off by 2^-17 of that) and p = hi + lo, p
// the probability times its page's V scale (off by at most 2^-8 p, as much as
// rounding to bf16 would be, or by 2^-18 of the tile's largest p where that is
// more).  The terms are separate columns of B: one MMA reads A once for both.  K's scale (times softmax
// scale and s_q) multiplies the scores; V's goes into P: with
// y = s c + log2 s_V the tile's largest y of each row is the tile's reference,
// P = 2^(y - y_max) 256, so that a tile of small probabilities (all but the
// first, where one early key takes most of the weight) keeps its relative
// accuracy, and O is rescaled in registers from tile to tile as in the usual
// online softmax.
//
// One or two warpgroups (thread r: key r for scores and P, head dimension r for
// O; two share the rows from 8 on, as a tile's time is the length of one warp's
// instruction chain), a warp that loads (lane i: page i of the tile, its TMA
// copies and its two scales) and one that issues the MMAs.
//
// d = 64: a tile's 128 rows of 128 bytes hold two tokens each, 256 in all, so
// that a tile, its copies and its fixed costs are those of d = 128.  S^T is two
// products, of the rows' first and second 64 bytes; in V^T P^T the rows' 128
// bytes are M, so P's columns come once for the first tokens (read in lanes
// 0-63) and once for the second ones (lanes 64-127), and the two O are added
// once for each item.
constexpr int kRowsMax = 16;
// V's scales further apart than 2^kWide within an item, or above it, take the sum l
// by another way.  Up to there a factor of the usual one leaves fp32 (2^-126) only
// for keys whose weight is below 2^(kWide - 118) of the largest, 2^31 of which are
// nothing.  (A page of zeros, scale 2^-64, beside values up to 28 does not get there.)
constexpr float kWide = 60.f;
// Up to here every warp finds its CTA's first tile by itself, from all lengths, while
// warp 0 allocates: one barrier before the roles part instead of two, and the merge
// finds its place while the attention runs.  With more sequences the lengths are
// summed by all warps together and CTA 0 writes each one's first tile down.
// Measured in a graph, 32 query heads on 8, d = 128, us by itself / together: 1
// sequence of 40 tokens 6.2 / 6.6, 16 7.1 / 7.2, 64 11.1 / 10.7, 128 17.0 / 16.5, 512
// 56 / 48, 4096 630 / 371; of 1000 tokens 8.5 / 8.7, 13.6 / 13.9, 32.4 / 32.7, 51.7 /
// 51.8, 177 / 170, 1532 / 1271.
constexpr int kScanSeqs = 64;

__device__ __forceinline__ int run_start(long long c, int total, int ctas) { return static_cast<int>(c * total / ctas); }
// The CTA whose run holds tile t.
__device__ __forceinline__ int run_of(long long t, int total, int ctas) {
  return static_cast<int>(((t + 1) * ctas + total - 1) / total - 1);
}

// Cached tokens of sequence b: a length below 0 counts as 0, one past
// max_seqlen or the page table as the nearer of the two.
__device__ __forceinline__ int clamp_len(const Cache8DecodeParams& p, int n) {
  const long long cap = min(static_cast<long long>(p.table_cols) * p.block, static_cast<long long>(p.max_seqlen));
  return static_cast<int>(min(max(static_cast<long long>(n), 0LL), cap));
}
__device__ __forceinline__ int cached_len(const Cache8DecodeParams& p, int b) { return clamp_len(p, p.seqlens[b]); }
// Tokens of a tile: 128 rows of 128 bytes.
template <int D>
constexpr int kTokens = kTile * 128 / D;

template <int D>
__device__ __forceinline__ int seq_tiles(const Cache8DecodeParams& p, int b) {
  return cache8::tiles_of(cached_len(p, b), kTokens<D>);
}

// A CTA's walk through its run: the tiles [k0, k1) of one item after another.
template <int D>
struct Walk {
  int t, t_hi, b, seq0;              // next tile, end of the run, sequence and its first tile
  int hk, rg, nt, k0, k1, len;
  // WARP: called by a whole warp, which takes lane 0's lengths, so that it
  // stays together even if a caller changes the lengths meanwhile.
  template <bool WARP>
  __device__ __forceinline__ bool next(const Cache8DecodeParams& p) {
    if (t >= t_hi) return false;
    const int per = p.Hk * p.row_groups;
    auto read = [&]() {
      len = cached_len(p, b);
      if (WARP) len = __shfl_sync(0xffffffffu, len, 0);
      nt = cache8::tiles_of(len, kTokens<D>);
    };
    read();
    while (t >= seq0 + nt * per) {
      seq0 += nt * per;
      if (++b >= p.B) return false;
      read();
    }
    const int item = (t - seq0) / nt;
    k0 = t - seq0 - item * nt;
    k1 = min(nt, k0 + (t_hi - t));
    hk = item / p.row_groups;
    rg = item - hk * p.row_groups;
    t += k1 - k0;
    return true;
  }
};

// The largest value of the warp, in every lane.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Sums over the warp of RP values a lane: value i of all lanes ends in lanes
// 32/RP · i .. +32/RP - 1.  Each step sends half of the values that are
// left to the lane that keeps them (RP - 1 + log2(32/RP) shuffles in all).
template <int RP>
__device__ __forceinline__ float rows_sum(const float (&y)[RP], int lane) {
  float v[RP];
#pragma unroll
  for (int i = 0; i < RP; ++i) v[i] = y[i];
  int n = RP;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (n > 1) {
      n /= 2;
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < RP / 2; ++i)
        if (i < n) {
          const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    }
  }
  return v[0];
}

template <int D, int RP>
struct Dec8Cfg {
  static constexpr int WG = RP >= 8 ? 2 : 1;                 // warpgroups that share the rows
  static constexpr int RW = RP / WG;                         // rows of one
  static constexpr int NCW = 4 * WG;                         // compute warps; then the TMA and the MMA warp
  static constexpr int NUM_WARPS = NCW + 2;
  static constexpr int NUM_THREADS = 32 * NUM_WARPS;
  static constexpr int NP = 128 / D;                         // tokens of a tile's row
  static constexpr int TILE_BYTES = kTile * 128;
  static constexpr int NST = D == 64 && RP == 16 ? 2 : 3;    // ring stages (K and V tile each)
  static constexpr int NS = 2 * RP < 16 ? 16 : 2 * RP;       // columns of S: a warpgroup's rows' hi, then lo terms
  static constexpr int NO = 2 * RP * NP < 16 ? 16 : 2 * RP * NP;
  static constexpr int Q_BYTES = NS * D;
  static constexpr int P_BYTES = NO * kTile;
  static constexpr int MAX_PPT = 8 * NP;                     // pages of a tile, at most
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + NST * TILE_BYTES;
  static constexpr int OFF_Q = OFF_V + NST * TILE_BYTES;
  static constexpr int OFF_P = OFF_Q + Q_BYTES;
  static constexpr int OFF_HALF = OFF_P;                     // between items: [RP][64] O of the second tokens (d = 64)
  static constexpr int OFF_SC = OFF_P + 2 * P_BYTES;         // (two P buffers) [NST][pages][4]: K's scale, 1 / V's, its log2, the tile's largest
  static constexpr int OFF_QS = OFF_SC + NST * MAX_PPT * 16;    // [RP] score factor of each row
  static constexpr int OFF_XCH = OFF_QS + kRowsMax * 4;      // [2][4 warps][RP]
  static constexpr int STAT_WARP = 4 * RW;                   // reference, alpha, weight, step of the running reference of each row
  static constexpr int OFF_STAT = OFF_XCH + 2 * 4 * kRowsMax * 4;  // [2 tiles][NCW][STAT_WARP]
  static constexpr int OFF_SCAN = OFF_STAT + 2 * NCW * STAT_WARP * 4;  // [warps] sums of tiles
  static constexpr int OFF_BAR = (OFF_SCAN + NUM_WARPS * 4 + 7) / 8 * 8;
  static constexpr int B_FULL = 0, B_EMPTY = NST, B_SFULL = 2 * NST, B_PFULL = B_SFULL + cache8::kSBars,
                       B_PVDONE = B_PFULL + cache8::kPBars, B_XCH = B_PVDONE + cache8::kPvBars, B_QREADY = B_XCH + 2, B_DRAIN = B_QREADY + 1, NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;    // slack to align the base to 1024
  static constexpr uint32_t COLS = 2 * NP * NS + 2 * NO;
  static constexpr uint32_t TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : 256;
  static constexpr uint32_t O_COL = 2 * NP * NS;
  static_assert(2 * TMEM_COLS <= 512, "tensor memory for two CTAs on an SM");
  static_assert(2 * (SMEM_BYTES + 1024) <= 233472, "shared memory for two CTAs on an SM");
  static_assert(OFF_Q % 1024 == 0 && OFF_P % 512 == 0, "swizzle atoms");
  static_assert(D == 128 || RP * 64 * 4 <= 2 * P_BYTES, "O of the second tokens fits over P");
};

// 8 or 16 columns of this warp's TMEM lanes.
template <int N>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, uint32_t (&v)[N]) {
  static_assert(N == 8 || N == 16, "shapes in use");
  if constexpr (N == 8) tmem_ld8(taddr, v);
  else tmem_ld16(taddr, v);
  tmem_wait_ld();
  reg_fence(v);
}

// N floats of shared memory, four at a time.
template <int N>
__device__ __forceinline__ void load_row(const float* src, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 x = reinterpret_cast<const float4*>(src)[i];
      v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = src[i];
  }
}

template <int N>
__device__ __forceinline__ void store_row(float* dst, const float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) dst[i] = v[i];
  }
}

// Element-wise arithmetic on rows' values, two at a time (the paired fp32
// instructions halve the issue slots, which bound a tile of 8 rows and more).
template <int N, typename F2, typename F1>
__device__ __forceinline__ void each_pair(F2 two, F1 one) {
#pragma unroll
  for (int q = 0; q + 1 < N; q += 2) two(q);
  if constexpr (N % 2 == 1) one(N - 1);
}

template <int D, int RP>
__global__ void __launch_bounds__(Dec8Cfg<D, RP>::NUM_THREADS, 2)
    fa_cache8_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const Cache8DecodeParams p) {
  using C = Dec8Cfg<D, RP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = raw_base + pad;
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* scan = reinterpret_cast<int*>(smem + C::OFF_SCAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == C::NCW && lane == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar(C::B_FULL + s), 32);
      mbar_init(bar(C::B_EMPTY + s), 1);
    }
    for (int i = 0; i < cache8::kSBars; ++i) mbar_init(bar(C::B_SFULL + i), 1);
    for (int i = 0; i < cache8::kPBars; ++i) mbar_init(bar(C::B_PFULL + i), 32 * C::NCW);
    for (int i = 0; i < cache8::kPvBars; ++i) mbar_init(bar(C::B_PVDONE + i), 1);
    for (int i = 0; i < C::WG; ++i) mbar_init(bar(C::B_XCH + i), 128);
    mbar_init(bar(C::B_QREADY), 32 * C::NCW);
    mbar_init(bar(C::B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp < C::NCW) {  // terms of rows that do not exist stay zero for good
    for (int i = threadIdx.x; i < (C::Q_BYTES + 2 * C::P_BYTES) / 16; i += 32 * C::NCW)
      reinterpret_cast<uint4*>(smem + C::OFF_Q)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  // The kernel may start while the one before it in the stream finishes: what
  // that one wrote is read from here on, and only now may the merge start,
  // which reads the lengths.  TMEM is taken behind the wait too: that kernel's
  // CTAs may still have to allocate theirs, and would wait for this one's.
  grid_dependency_wait();
  grid_launch_dependents();
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  // ---- this CTA's place: all tiles counted, then the sequence of its first one
  const int per = p.Hk * p.row_groups;
  int total = 0;
  if (p.B <= kScanSeqs) {
    for (int b = lane; b < p.B; b += 32) total += seq_tiles<D>(p, b);
    total = __reduce_add_sync(0xffffffffu, total);
  } else {
    int mine = 0;
    for (int b = threadIdx.x; b < p.B; b += C::NUM_THREADS) mine += seq_tiles<D>(p, b);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) scan[warp] = mine;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C::NUM_WARPS; ++i) total += scan[i];
  }
  total *= per;
  const int ctas = min(static_cast<int>(gridDim.x), total);  // every one of them has a tile
  const bool idle = static_cast<int>(blockIdx.x) >= ctas;
  Walk<D> w{};
  if (!idle) {
    w.t = run_start(blockIdx.x, total, ctas);
    w.t_hi = run_start(blockIdx.x + 1LL, total, ctas);
  }
  // CTA 0 reports lengths out of range, and with many sequences writes down
  // each one's first tile for the merge.
  const bool writes = blockIdx.x == 0 && warp == 0;
  if (writes && lane == 0 && p.B > kScanSeqs) p.tile_start[p.B] = total;
  for (int b0 = 0, base = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int n = b < p.B ? seq_tiles<D>(p, b) * per : 0;
    int sum = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += y;
    }
    const int first = base + sum - n;
    if (writes && b < p.B) {
      if (p.B > kScanSeqs) p.tile_start[b] = first;
      if (p.seqlens[b] != cached_len(p, b)) atomicOr(p.err, kDevErrPage);
    }
    const uint32_t here = __ballot_sync(0xffffffffu, n > 0 && w.t >= first && w.t < first + n);
    if (here != 0) {
      w.b = b0 + __ffs(here) - 1;
      w.seq0 = __shfl_sync(0xffffffffu, first, __ffs(here) - 1);
      if (!writes) break;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == C::NCW) {
    // ---------------------------------------------------------------- TMA
    // The run in units of up to 32 pages (32 / ppt tiles) of one item, a page a
    // lane.  A unit's table entries are read two units ahead and its scales
    // one unit ahead, so that the copies wait for neither.  (Against reading both
    // where a unit begins: pages of 16 tokens, d = 128, of which a unit is 4 tiles,
    // 2 % faster with up to 16 rows and 4 % with 32; pages of 64 and 128 alike.)
    const int ppt = kTokens<D> >> p.block_shift;  // pages of a tile
    struct Unit {
      int kt0, tiles, len, hk, page;  // first tile, tiles; page of this lane (num_blocks: none, reads as zeros)
      float ks, vs;
    };
    int left = 0;  // tiles of the current item not yet in a unit
    auto next_unit = [&](Unit& u) {
      if (left == 0) left = w.template next<true>(p) ? w.k1 - w.k0 : 0;
      u.kt0 = w.k1 - left;
      u.tiles = min(left, 32 / ppt);
      u.len = w.len;
      u.hk = w.hk;
      left -= u.tiles;
      u.page = p.num_blocks;
      if (lane < u.tiles * ppt && u.kt0 * ppt + lane < cache8::pages_of(u.len, p.block_shift))
        u.page = p.table[static_cast<size_t>(w.b) * p.table_cols + u.kt0 * ppt + lane];
    };
    auto load_scales = [&](Unit& u) {
      const bool token = lane < u.tiles * ppt && u.kt0 * ppt + lane < cache8::pages_of(u.len, p.block_shift);
      u.ks = u.vs = 0.f;
      if (token && u.page >= 0 && u.page < p.num_blocks) {
        u.ks = p.k_scale[static_cast<size_t>(u.page) * p.Hk + u.hk];
        u.vs = p.v_scale[static_cast<size_t>(u.page) * p.Hk + u.hk];
      } else {
        if (token) atomicOr(p.err, kDevErrPage);
        u.page = p.num_blocks;
      }
    };
    Unit cur, near, far;
    next_unit(cur);
    next_unit(near);
    load_scales(cur);
    int t = 0;
    bool ok = true;
    while (ok && cur.tiles > 0) {
      for (int i = 0; i < cur.tiles; ++i, ++t) {
        const int st = t % C::NST, kt = cur.kt0 + i;
        const int n_pages = min(ppt, cache8::pages_of(cur.len, p.block_shift) - kt * ppt);
        const int from = i * ppt + lane;  // this lane's page of the tile
        const int page = __shfl_sync(0xffffffffu, cur.page, from & 31);
        if (t >= C::NST) ok = wait_bounded(bar(C::B_EMPTY + st), cache8::ring(t - C::NST, C::NST).parity, abort_flag, p.err, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(bar(C::B_FULL + st), n_pages * p.block * D * 2);
        __syncwarp();
        if (lane < n_pages) {
          const uint32_t off = st * C::TILE_BYTES + lane * p.block * D;
          tma_load_4d(sb + C::OFF_K + off, &tmK, bar(C::B_FULL + st), 0, 0, cur.hk, page);
          tma_load_4d(sb + C::OFF_V + off, &tmV, bar(C::B_FULL + st), 0, 0, cur.hk, page);
        }
        if (i == 0) {
          next_unit(far);
          load_scales(near);
        }
        const float ks = __shfl_sync(0xffffffffu, cur.ks, from & 31), vs = __shfl_sync(0xffffffffu, cur.vs, from & 31);
        // V's scale by its exponent, a power of two; 1 for a page of zeros and for none
        const int ve = lane < n_pages && vs > 0.f ? static_cast<int>(__float_as_uint(vs) >> 23) - 127 : 0;
        const float ve_max = warp_max(lane < n_pages ? static_cast<float>(ve) : -CUDART_INF_F);
        if (lane < ppt)
          reinterpret_cast<float4*>(smem + C::OFF_SC)[st * C::MAX_PPT + lane] =
              make_float4(lane < n_pages ? ks : 0.f, exp2_int(-ve), static_cast<float>(ve), ve_max);
        mbar_arrive(bar(C::B_FULL + st));
      }
      cur = near;
      near = far;
    }
    // Every copy issued lands before the CTA may exit, whoever aborted.
    for (int s = 0; s < C::NST && s < t; ++s) {
      const int last = s + ((t - 1 - s) / C::NST) * C::NST;
      wait_drain(bar(C::B_FULL + s), cache8::ring(last, C::NST).parity, p.err, p.timeout_ns);
    }
  } else if (warp == C::NCW + 1) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0 && !idle) {
      constexpr uint32_t idesc_s = idesc_e4m3(128, C::NS, false), idesc_o = idesc_e4m3(128, C::NO, true);
      const uint64_t dK0 = sdesc8<128>(sb + C::OFF_K, 16);
      const uint64_t dV0 = sdesc8<128>(sb + C::OFF_V, 16);  // MN-major: the rows' 128 bytes are M
      const uint64_t dQ = sdesc8<D>(sb + C::OFF_Q, 16);
      const uint64_t dP = sdesc8<C::NO>(sb + C::OFF_P, 16);  // MN-major: a key's columns are a row
      auto issue_s = [&](int u) -> bool {
        const int st = u % C::NST;
        if (!wait_bounded(bar(C::B_FULL + st), cache8::ring(u, C::NST).parity, abort_flag, p.err, p.timeout_ns)) return false;
        tc_fence_after();
#pragma unroll
        for (int pos = 0; pos < C::NP; ++pos)  // d = 64: the rows' first tokens, then their second ones
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_e4m3(tmem + C::NS * (C::NP * (u & 1) + pos), sdesc_add(dK0, st * C::TILE_BYTES + pos * D + kk * 32),
                     sdesc_add(dQ, kk * 32), idesc_s, kk > 0);
        tc_commit(bar(C::B_SFULL + cache8::s_full(u).index));
        return true;
      };
      int t = 0, n_item = 0;
      bool ok = true;
      for (; ok && w.template next<false>(p); ++n_item) {
        ok = wait_bounded(bar(C::B_QREADY), n_item & 1, abort_flag, p.err, p.timeout_ns) && issue_s(t);
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++t) {
          // the next tile's scores run while this tile's P is formed (across
          // items they cannot: the next Q is staged after this item's last S)
          if (kt + 1 < w.k1) ok = issue_s(t + 1);
          const cache8::Phase pf = cache8::p_full(t);
          ok = ok && wait_bounded(bar(C::B_PFULL + pf.index), pf.parity, abort_flag, p.err, p.timeout_ns);
          if (!ok) break;
          tc_fence_after();
          const int st = t % C::NST;
#pragma unroll
          for (int kk = 0; kk < kTile / 32; ++kk)
            mma_e4m3(tmem + C::O_COL + C::NO * (t & 1), sdesc_add(dV0, st * C::TILE_BYTES + kk * 32 * 128),
                     sdesc_add(dP, (t & 1) * C::P_BYTES + kk * 32 * C::NO), idesc_o, kk > 0);
          tc_commit(bar(C::B_PVDONE + cache8::pv_done(t).index));
          tc_commit(bar(C::B_EMPTY + st));
        }
      }
      tc_commit(bar(C::B_DRAIN));
      wait_drain(bar(C::B_DRAIN), 0, p.err, p.timeout_ns);
    }
  } else {
    // ---------------------------------------------------------------- softmax, P, running O
    constexpr int RW = C::RW;
    const int wg = C::WG == 2 ? warp >> 2 : 0, quarter = warp & 3;
    const int row0 = wg * RW;            // first of this warpgroup's rows
    const int r = quarter * 32 + lane;   // TMEM lane: row of the tile (its tokens); head dimension of O (and which token)
    const int half = r / D;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* xch = reinterpret_cast<float*>(smem + C::OFF_XCH);
    float* qs = reinterpret_cast<float*>(smem + C::OFF_QS);
    float* stats = reinterpret_cast<float*>(smem + C::OFF_STAT) + warp * C::STAT_WARP;
    const int xbar = C::B_XCH + wg;
    constexpr int NP = C::NP, TOK = kTokens<D>;
    constexpr int LPR = 32 / RW;  // lanes that keep one row's statistics
    const int my_row = lane / LPR;  // within the warpgroup's rows
    int t = 0, nx = 0, n_item = 0;
    int st = 0;             // tile t's ring stage, and its phase there
    uint32_t st_phase = 0;
    bool ok = true;
    auto wait = [&](int i, uint32_t ph) {
      ok = ok && wait_bounded(bar(i), ph, abort_flag, p.err, p.timeout_ns);
    };
    for (; __all_sync(0xffffffffu, ok) && w.template next<true>(p); ++n_item) {
      const int rows = min(p.rows, p.Nq * p.G - w.rg * p.rows);
      // Row row0 + my_row: its row of q and o, its place in lse, and how many of
      // the last keys it does not see.
      int row_q, row_lse, row_hidden;
      {
        const int f = min(w.rg * p.rows + row0 + my_row, p.Nq * p.G - 1);
        const int i = f / p.G, h = w.hk * p.G + f - i * p.G;
        row_q = (w.b * p.Nq + i) * p.H + h;
        row_lse = (w.b * p.H + h) * p.Nq + i;
        row_hidden = p.causal ? p.Nq - 1 - i : 0;
      }
      // ---- the item's queries as two terms (their last reader, the S of the
      // item before, has completed); a warpgroup's warps take turns at its rows
      {
        constexpr int E = D / 32, NR = (RW + 3) / 4;
        uint32_t raw[NR][E / 2];
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          const int q = quarter + 4 * j;
          const uint16_t* src = p.q + static_cast<size_t>(__shfl_sync(0xffffffffu, row_q, (q * LPR) & 31)) * D + E * lane;
          const bool live = q < RW && row0 + q < rows;
          if constexpr (E == 4) {
            const uint2 x = live ? *reinterpret_cast<const uint2*>(src) : make_uint2(0u, 0u);
            raw[j][0] = x.x, raw[j][1] = x.y;
          } else {
            raw[j][0] = live ? *reinterpret_cast<const uint32_t*>(src) : 0u;
          }
        }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          const int q = quarter + 4 * j;
          if (q >= RW) break;
          uint32_t top = 0;
#pragma unroll
          for (int u = 0; u < E / 2; ++u) top = __vmaxu2(top, raw[j][u] & 0x7fff7fffu);
          const uint32_t mx = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
          // smallest power of two s with max <= 448 s, for any finite row: 2^120 at
          // most, at least 2^-126 (fp32's smallest that is not subnormal)
          const int e2 = min(scale_exponent(mx, -126), 120);
          const float inv = exp2_int(-e2);
          float x[E], h[E];
#pragma unroll
          for (int u = 0; u < E / 2; ++u) {
            x[2 * u] = bf16lo_to_f32(raw[j][u]) * inv;
            x[2 * u + 1] = bf16hi_to_f32(raw[j][u]) * inv;
          }
          uint32_t hi[2] = {}, lo[2] = {};
#pragma unroll
          for (int u = 0; u < E / 2; ++u) {
            hi[u] = pack_e4m3x2(x[2 * u], x[2 * u + 1]);
            unpack_e4m3x2(hi[u], h[2 * u], h[2 * u + 1]);
            lo[u] = pack_e4m3x2(x[2 * u] - h[2 * u], x[2 * u + 1] - h[2 * u + 1]);
          }
          uint8_t* at_hi = smem + C::OFF_Q + swz<D>(2 * row0 + q, E * lane);
          uint8_t* at_lo = smem + C::OFF_Q + swz<D>(2 * row0 + RW + q, E * lane);
          if constexpr (E == 4) {
            *reinterpret_cast<uint32_t*>(at_hi) = hi[0] | (hi[1] << 16);
            *reinterpret_cast<uint32_t*>(at_lo) = lo[0] | (lo[1] << 16);
          } else {
            *reinterpret_cast<uint16_t*>(at_hi) = static_cast<uint16_t>(hi[0]);
            *reinterpret_cast<uint16_t*>(at_lo) = static_cast<uint16_t>(lo[0]);
          }
          if (lane == 0) qs[row0 + q] = exp2_int(e2) * p.scale_log2;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(C::B_QREADY));
      wait(C::B_QREADY, n_item & 1);
      float qf[RW], lsum[RW], ov[RW];
      load_row<RW>(qs + row0, qf);
#pragma unroll
      for (int q = 0; q < RW; ++q) lsum[q] = ov[q] = 0.f;
      float m = -CUDART_INF_F;  // running reference of row my_row
      float ve_hi = -CUDART_INF_F, ve_lo = 0.f;  // log2 of V's scales: the largest; the least of this thread's tokens, and of 1
      constexpr int NL = RP == 1 ? 8 : 2 * RW;  // columns of the warpgroup's rows
      // O of tile u (its statistics are still in their buffer) into the running one.
      auto add_o = [&](int u) {
        const float* stat = stats + (u & 1) * C::NCW * C::STAT_WARP;
        wait(C::B_PVDONE + cache8::pv_done(u).index, cache8::pv_done(u).parity);
        __syncwarp();
        tc_fence_after();
        uint32_t o[NL];
        tmem_cols(lane_addr + C::O_COL + C::NO * (u & 1) + (RP == 1 ? 0 : 2 * RP * half + 2 * row0), o);
        float alpha[RW], wt[RW];
        load_row<RW>(stat + RW, alpha);
        load_row<RW>(stat + 2 * RW, wt);
        each_pair<RW>(
            [&](int q) {
              const uint64_t sum = fadd2(f2_pack(__uint_as_float(o[q]), __uint_as_float(o[q + 1])),
                                         f2_pack(__uint_as_float(o[RW + q]), __uint_as_float(o[RW + q + 1])));
              f2_unpack(ffma2(sum, f2_pack(wt[q], wt[q + 1]),
                              fmul2(f2_pack(ov[q], ov[q + 1]), f2_pack(alpha[q], alpha[q + 1]))),
                        ov[q], ov[q + 1]);
            },
            [&](int q) {
              float sum = __uint_as_float(o[q]) + __uint_as_float(o[q + RW]);
              if (RP == 1 && D == 64) sum = half ? __uint_as_float(o[2]) + __uint_as_float(o[3]) : sum;
              ov[q] = fmaf(sum, wt[q], ov[q] * alpha[q]);
            });
        tc_fence_before();
      };
      // tiles of which some row does not see all keys: from this one on
      const int kt_mask = max(0, w.len - (p.causal ? p.Nq - 1 : 0)) / TOK;
      for (int kt = w.k0; kt < w.k1; ++kt, ++t) {
        wait(C::B_FULL + st, st_phase);
        // K's scale, 1 / V's scale and its log2 of the page of this thread's tokens (and the
        // largest such log2 of the tile's pages)
        const float4 sc = reinterpret_cast<const float4*>(smem + C::OFF_SC)[st * C::MAX_PPT + ((NP * r) >> p.block_shift)];
        const float ks = sc.x, inv_vs = sc.y, vef = sc.z;
        wait(C::B_SFULL + cache8::s_full(t).index, cache8::s_full(t).parity);
        __syncwarp();
        tc_fence_after();
        float y[NP][RW];
#pragma unroll
        for (int pos = 0; pos < NP; ++pos) {
          uint32_t sv[NL];
          tmem_cols(lane_addr + C::NS * (NP * (t & 1) + pos) + 2 * row0, sv);
          each_pair<RW>(
              [&](int q) {
                const uint64_t s = fadd2(f2_pack(__uint_as_float(sv[q]), __uint_as_float(sv[q + 1])),
                                         f2_pack(__uint_as_float(sv[RW + q]), __uint_as_float(sv[RW + q + 1])));
                f2_unpack(ffma2(s, fmul2(f2_pack(ks, ks), f2_pack(qf[q], qf[q + 1])), f2_pack(vef, vef)), y[pos][q],
                          y[pos][q + 1]);
              },
              [&](int q) {
                y[pos][q] = fmaf(__uint_as_float(sv[q]) + __uint_as_float(sv[RW + q]), ks * qf[q], vef);
              });
        }
        if (kt >= kt_mask) {
#pragma unroll
          for (int q = 0; q < RW; ++q) {
            const int end = cache8::tokens_from(w.len, kt, TOK, NP * r) - __shfl_sync(0xffffffffu, row_hidden, q * LPR);
#pragma unroll
            for (int pos = 0; pos < NP; ++pos)
              if (pos >= end) y[pos][q] = -CUDART_INF_F;
          }
        }
        // ---- the tile's largest y of each row: over the warp, then over the
        // four warps; lane q does the rest of row q's statistics and leaves
        // them for its warp
        float* slot = xch + (nx & 1) * 4 * kRowsMax + row0;
        {
          float wm[RW];
#pragma unroll
          for (int q = 0; q < RW; ++q) wm[q] = warp_max(NP == 2 ? fmaxf(y[0][q], y[NP - 1][q]) : y[0][q]);
          if (lane == 0) store_row<RW>(slot + quarter * kRowsMax, wm);
        }
        mbar_arrive(bar(xbar));
        wait(xbar, nx & 1);
        ++nx;
        float* stat = stats + (t & 1) * C::NCW * C::STAT_WARP;
        {
          const int q = my_row;
          const float mt = fmaxf(fmax3(slot[q], slot[kRowsMax + q], slot[2 * kRowsMax + q]), slot[3 * kRowsMax + q]);
          const float m_new = fmaxf(m, mt);
          const bool none = mt == -CUDART_INF_F;
          if (lane % LPR == 0) {
            stat[q] = none ? 0.f : mt - 8.f;
            stat[RW + q] = m == -CUDART_INF_F ? 0.f : ex2_approx(m - m_new);
            stat[2 * RW + q] = none ? 0.f : ex2_approx(mt - m_new - 8.f);
            stat[3 * RW + q] = m == -CUDART_INF_F ? -CUDART_INF_F : m - m_new;
          }
          m = m_new;
          __syncwarp();
        }
        {
          ve_hi = fmaxf(ve_hi, sc.w);
          ve_lo = fminf(ve_lo, vef);
          const bool wide = __any_sync(0xffffffffu, ve_hi - ve_lo > kWide);
          if (wide) {
            // V's scales so far apart that a factor of a key's share of l, 2^(s - m),
            // would leave fp32 though the share does not: as squares of its root
#pragma unroll
            for (int q = 0; q < RW; ++q) {
              const float to = __shfl_sync(0xffffffffu, m, q * LPR), root = ex2_approx(0.5f * stat[3 * RW + q]);
              lsum[q] = lsum[q] * root * root;
#pragma unroll
              for (int pos = 0; pos < NP; ++pos) {
                const float h = y[pos][q] == -CUDART_INF_F ? 0.f : ex2_approx(0.5f * (y[pos][q] - vef - to));
                lsum[q] = fmaf(h, h, lsum[q]);
              }
            }
          }
          const float inv_l = wide ? 0.f : inv_vs;
          float ref[RW], alpha[RW], wt[RW];
          load_row<RW>(stat, ref);
          load_row<RW>(stat + RW, alpha);
          load_row<RW>(stat + 2 * RW, wt);
          if (!wide) {
#pragma unroll
            for (int q = 0; q < RW; ++q) lsum[q] *= alpha[q];
          }
#pragma unroll
          for (int pos = 0; pos < NP; ++pos) {
            uint32_t hi[(RW + 3) / 4], lo[(RW + 3) / 4];
            float(&x)[RW] = y[pos];
            // P = 2^(y - reference), at most 256, and its share of l
            each_pair<RW>(
                [&](int q) {
                  f2_unpack(fsub2(f2_pack(x[q], x[q + 1]), f2_pack(ref[q], ref[q + 1])), x[q], x[q + 1]);
                  x[q] = ex2_approx(x[q]);
                  x[q + 1] = ex2_approx(x[q + 1]);
                  const uint64_t c = fmul2(f2_pack(inv_l, inv_l), f2_pack(wt[q], wt[q + 1]));
                  f2_unpack(ffma2(f2_pack(x[q], x[q + 1]), c, f2_pack(lsum[q], lsum[q + 1])), lsum[q], lsum[q + 1]);
                },
                [&](int q) {
                  x[q] = ex2_approx(x[q] - ref[q]);
                  lsum[q] = fmaf(x[q], inv_l * wt[q], lsum[q]);
                });
            if constexpr (RW % 4 == 0) {
#pragma unroll
              for (int q = 0; q < RW; q += 4) {
                float h[4], e[4];
                hi[q / 4] = pack_e4m3x4(x[q], x[q + 1], x[q + 2], x[q + 3]);
                unpack_e4m3x4(hi[q / 4], h);
                f2_unpack(fsub2(f2_pack(x[q], x[q + 1]), f2_pack(h[0], h[1])), e[0], e[1]);
                f2_unpack(fsub2(f2_pack(x[q + 2], x[q + 3]), f2_pack(h[2], h[3])), e[2], e[3]);
                lo[q / 4] = pack_e4m3x4(e[0], e[1], e[2], e[3]);
              }
            } else {
              float h, unused;
              hi[0] = pack_e4m3x2(x[0], 0.f);
              unpack_e4m3x2(hi[0], h, unused);
              lo[0] = pack_e4m3x2(x[0] - h, 0.f);
            }
            // the token's columns: a warpgroup's rows' hi terms, then their lo
            // terms (d = 64: of the rows' second tokens behind the first ones')
            uint8_t* at = smem + C::OFF_P + (t & 1) * C::P_BYTES + swz<C::NO>(r, 2 * RP * pos + 2 * row0);
            static_assert(RW == 8 || RW == 4 || RW == 1, "row counts that the P layout has");
            if constexpr (RW == 8)
              *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
            else if constexpr (RW == 4)
              *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], lo[0]);
            else
              *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>((hi[0] & 0xffu) | (lo[0] << 8));
          }
        }
        // slots without a token may hold NaN, and 0 · NaN is not 0
        if (wg == 0 && kt >= kt_mask) {
          const int held = cache8::tokens_from(w.len, kt, TOK, NP * r);  // tokens of this row
          uint4* vrow = reinterpret_cast<uint4*>(smem + C::OFF_V + st * C::TILE_BYTES + r * 128);
#pragma unroll
          for (int u = 0; u < 8; ++u)  // 16-byte chunks, swizzled
            if (u * 16 / D >= held) vrow[u ^ (r & 7)] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(C::B_PFULL + cache8::p_full(t).index));
        // The product of the tile before is ready by now: waiting for this one's
        // would leave the warps idle for its whole latency.
        if (kt > w.k0) add_o(t - 1);
        if (++st == C::NST) {
          st = 0;
          st_phase ^= 1u;
        }
      }
      add_o(t - 1);
      // ---- the item's sums: l over the keys, O over the halves
      float* slot = xch + (nx & 1) * 4 * kRowsMax + row0;
      {
        const float l = rows_sum<RW>(lsum, lane);
        if (lane % LPR == 0) slot[quarter * kRowsMax + my_row] = l;
      }
      float* other = reinterpret_cast<float*>(smem + C::OFF_HALF) + row0 * 64 + r % 64;
      if (D == 64 && half) {
#pragma unroll
        for (int q = 0; q < RW; ++q) other[q * 64] = ov[q];
      }
      mbar_arrive(bar(xbar));
      wait(xbar, nx & 1);
      ++nx;
      float* stat = stats;  // the tile loop's statistics of this warp make room for the rows' factors
      const bool whole = w.k0 == 0 && w.k1 == w.nt;
      const float l = (slot[my_row] + slot[kRowsMax + my_row]) + (slot[2 * kRowsMax + my_row] + slot[3 * kRowsMax + my_row]);
      const size_t part0 = (2 * static_cast<size_t>(blockIdx.x) + (w.k0 == 0 ? 1 : 0)) * p.rows + row0;
      if (lane % LPR == 0) {
        stat[my_row] = l > 0.f ? 1.f / l : 0.f;
        reinterpret_cast<int*>(stat)[RW + my_row] = row_q;
        if (quarter == 0 && row0 + my_row < rows) {
          if (whole) {
            p.lse[row_lse] = l > 0.f ? (m + log2f(l)) * kLn2 : -CUDART_INF_F;
          } else {
            p.ml_part[(part0 + my_row) * 2] = m;
            p.ml_part[(part0 + my_row) * 2 + 1] = l;
          }
        }
      }
      __syncwarp();
      if (r < D) {
        float inv[RW];
        load_row<RW>(stat, inv);
#pragma unroll
        for (int q = 0; q < RW; ++q) {
          if (row0 + q >= rows) break;
          const float o = D == 64 ? ov[q] + other[q * 64] : ov[q];
          if (whole)
            p.o[static_cast<size_t>(reinterpret_cast<int*>(stat)[RW + q]) * D + r] =
                static_cast<uint16_t>(pack_bf16x2(o * inv[q], 0.f));
          else
            p.o_part[(part0 + q) * D + r] = o;
        }
      }
      __syncwarp();
      // (what the next item writes over, it writes after all have arrived on
      // its B_QREADY)
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// One warp per (sequence, new token, query head): the partials of an item that
// several CTAs shared, in the order of its tiles; zeros where no key is cached.
// The kernel is scheduled while the attention still runs and finds its item's
// place from the lengths meanwhile (few sequences; else from what CTA 0 of the
// attention wrote); a lane takes each partial's statistics, and the partials
// are then read with several loads in flight.
template <int D>
__global__ void __launch_bounds__(128) fa_cache8_merge_kernel(const Cache8DecodeParams p, int ctas) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long wid = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const bool live = wid < static_cast<long long>(p.B) * p.Nq * p.H;
  const int h = live ? static_cast<int>(wid % p.H) : 0;
  const long long qrow = live ? wid / p.H : 0;
  const int i = static_cast<int>(qrow % p.Nq), b = static_cast<int>(qrow / p.Nq);
  const int per = p.Hk * p.row_groups;
  int s0 = 0, nt = 0, total = 0;
  const bool scan = p.B <= kScanSeqs;
  if (scan) {
    // Before the wait, yet complete: the attention lets this kernel start only
    // behind its own wait for whatever wrote the lengths.  Read from L2.
    auto tiles = [&](int j) { return cache8::tiles_of(clamp_len(p, ld_relaxed_gpu(p.seqlens + j)), kTokens<D>); };
    for (int j = lane; j < p.B; j += 32) {
      const int n = tiles(j);
      total += n;
      s0 += j < b ? n : 0;
    }
    s0 = __reduce_add_sync(0xffffffffu, s0) * per;
    total = __reduce_add_sync(0xffffffffu, total) * per;
    nt = tiles(b);
  }
  grid_dependency_wait();
  if (!live) return;
  if (!scan) {
    s0 = p.tile_start[b];
    nt = (p.tile_start[b + 1] - s0) / per;
    total = p.tile_start[p.B];
  }
  ctas = min(ctas, total);
  const int hk = h / p.G, f = i * p.G + h % p.G, rg = f / p.rows, r = f - rg * p.rows;
  const long long t0 = s0 + static_cast<long long>(hk * p.row_groups + rg) * nt;
  const int c0 = nt ? run_of(t0, total, ctas) : 0, c1 = nt ? run_of(t0 + nt - 1, total, ctas) : -1;
  if (c0 == c1) return;  // written by that CTA
  auto slot = [&](int c) { return (2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0)) * p.rows + r; };
  float mmax = -CUDART_INF_F, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int c = c0 + lane; c <= c1; c += 32) mmax = fmaxf(mmax, p.ml_part[slot(c) * 2]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mmax = fmaxf(mmax, __shfl_xor_sync(0xffffffffu, mmax, off));
  if (mmax != -CUDART_INF_F) {
    for (int cb = c0; cb <= c1; cb += 32) {
      float w = 0.f;  // of partial cb + lane
      if (cb + lane <= c1) {
        const float2 ml = *reinterpret_cast<const float2*>(p.ml_part + slot(cb + lane) * 2);
        const float root = ml.x == -CUDART_INF_F ? 0.f : ex2_approx(0.5f * (ml.x - mmax));
        w = root * root;
        l = fmaf(root, root * ml.y, l);  // (w may be below fp32's range where w · l is not)
      }
      const int n = min(32, c1 - cb + 1);
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const float* op = p.o_part + slot(cb + j) * D + E * lane;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(op);
          acc[0] = fmaf(wj, v.x, acc[0]), acc[1] = fmaf(wj, v.y, acc[1]);
          acc[2] = fmaf(wj, v.z, acc[2]), acc[3] = fmaf(wj, v.w, acc[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(op);
          acc[0] = fmaf(wj, v.x, acc[0]), acc[1] = fmaf(wj, v.y, acc[1]);
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* o = p.o + (qrow * p.H + h) * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0)
    p.lse[(static_cast<size_t>(b) * p.H + h) * p.Nq + i] = l > 0.f ? (mmax + log2f(l)) * kLn2 : -CUDART_INF_F;
}

template <int D, int RP>
cudaError_t launch_decode8(const CUtensorMap& tk, const CUtensorMap& tv, const Cache8DecodeParams& p, int ctas,
                           cudaStream_t s) {
  using C = Dec8Cfg<D, RP>;
  static SmemLimit smem_limit;
  cudaError_t e = smem_limit.ensure(reinterpret_cast<const void*>(fa_cache8_decode_kernel<D, RP>), C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  e = launch_kernel(fa_cache8_decode_kernel<D, RP>, dim3(static_cast<unsigned>(ctas)), dim3(C::NUM_THREADS),
                    C::SMEM_BYTES, s, true, tk, tv, p);
  if (e != cudaSuccess) return e;
  const long long warps = static_cast<long long>(p.B) * p.Nq * p.H;
  return launch_kernel(fa_cache8_merge_kernel<D>, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, s, true, p,
                       ctas);
}

template <int D>
cudaError_t launch_decode8_rows(const CUtensorMap& tk, const CUtensorMap& tv, const Cache8DecodeParams& p, int ctas,
                                cudaStream_t s) {
  if (p.rows <= 1) return launch_decode8<D, 1>(tk, tv, p, ctas, s);
  if (p.rows <= 4) return launch_decode8<D, 4>(tk, tv, p, ctas, s);
  if (p.rows <= 8) return launch_decode8<D, 8>(tk, tv, p, ctas, s);
  return launch_decode8<D, 16>(tk, tv, p, ctas, s);
}

}  // namespace

void cache8_plan(int d, int rows_total, int* groups, int* rows, int* tokens) {
  *groups = (rows_total + kRowsMax - 1) / kRowsMax;
  *rows = (rows_total + *groups - 1) / *groups;
  *tokens = d == 64 ? kTokens<64> : kTokens<128>;
}

cudaError_t launch_cache8_store(int d, int block, const Cache8StoreParams& p, cudaStream_t s) {
  if (d == 64) {
    if (block == 16) return launch_store<64, 16>(p, s);
    if (block == 32) return launch_store<64, 32>(p, s);
    if (block == 64) return launch_store<64, 64>(p, s);
    return launch_store<64, 128>(p, s);
  }
  if (block == 16) return launch_store<128, 16>(p, s);
  if (block == 32) return launch_store<128, 32>(p, s);
  if (block == 64) return launch_store<128, 64>(p, s);
  return launch_store<128, 128>(p, s);
}

cudaError_t launch_cache8_decode(int d, const CUtensorMap& tk, const CUtensorMap& tv, const Cache8DecodeParams& p,
                                 int ctas, cudaStream_t s) {
  return d == 64 ? launch_decode8_rows<64>(tk, tv, p, ctas, s) : launch_decode8_rows<128>(tk, tv, p, ctas, s);
}

}  // namespace fa
