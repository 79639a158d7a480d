// Rotary positions for sm_103a: queries and keys turned by their tokens'
// positions, and the append to the 8-bit paged cache that turns the keys (and
// the call's queries) on the way.
//
// Pair j of a head's dimensions, (a, b), becomes (a cos t - b sin t, b cos t +
// a sin t), t = position · frequency_j; a token may have several positions
// (time, height, width), and each pair belongs to one of them.  The inverse, which
// is also the gradient (the turn is orthogonal), takes -t.
//
// Angles.  A frequency is kept as a fraction of a turn in 64-bit fixed point, F =
// round(frequency / 2 pi · 2^64), so the angle of an integer position is the low 64
// bits of position · F, whole turns falling off the top: exact but for F's own
// rounding, 2^31 · 2^-65 turns at the furthest position.  Of its upper 32 bits what
// lies beside the nearest quarter goes to sincospif, so that the fraction's rounding to
// fp32 costs the angle 2^-25 at most, no more than the sine's and the cosine's own (a
// fraction of the whole turn: 2^-23, and some more keys get a neighbouring code).  One
// sine and cosine serves a token's pair in all heads, of the append's keys in those that a
// block takes.
//
// Both kernels are bound by DRAM: each element is read once and written once.  Measured:
// 16,421 tokens of 32 + 8 heads of 128 turned in 50 us (6.7 TB/s, 99 % of the copy
// rate), 16 prompts of up to 4,096 of them with 8 heads of values appended in 124 us (6.2
// TB/s) to pages of 16 tokens; 64 single tokens in 5.3 us, a launch of dependent loads.
// Larger pages have fewer heads a block (8, 4, 2, 1 at d = 128), so that the keys' angles
// are formed more often: the same prompts take 130, 141 and 182 us with pages of 32, 64 and 128.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "e4m3.cuh"
#include "fa_kernels.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

// Cosine and sine of pair j at position pos.
__device__ __forceinline__ float2 cos_sin(const RotaryParams& r, int j, int pos) {
  const uint64_t turn = r.turns[j] * static_cast<uint64_t>(static_cast<long long>(pos));
  // the nearest quarter of the turn, and the rest, an eighth at most either way
  const uint32_t t = static_cast<uint32_t>(turn >> 32), quarter = (t + (1u << 29)) >> 30;
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(t - (quarter << 30))) * 0x1p-31f, &s, &c);
  if (quarter & 1) {
    const float x = c;
    c = -s;
    s = x;
  }
  if (quarter & 2) c = -c, s = -s;
  return make_float2(c, r.inverse ? -s : s);
}

// Axis of pair j, within the axes there are.
__device__ __forceinline__ int axis_of(const RotaryParams& r, int j) {
  return r.axes == 1 ? 0 : min(max(r.axis[j], 0), r.axes - 1);
}
// Position of token `row` on the axis of pair j.
__device__ __forceinline__ int position_of(const RotaryParams& r, int j, int row, int total) {
  return r.positions[static_cast<size_t>(axis_of(r, j)) * total + row];
}

// A head's dimensions are taken in units of two 16-byte chunks that hold eight
// whole pairs: unit u is chunks u and u + pairs / 8 where a pair has one element in
// each half, chunks 2u and 2u + 1 where pairs are neighbours and behind the turned
// dimensions.
template <bool IL>
__device__ __forceinline__ void unit_chunks(int u, int pairs, int& c0, int& c1) {
  const bool halves = !IL && 8 * u < pairs;
  c0 = halves ? u : 2 * u;
  c1 = halves ? u + pairs / 8 : 2 * u + 1;
}

// Where the angle of a token's pair lies in shared memory: two pairs of each unit beside
// the same two of the next, so that the units' 16-byte reads meet in no bank.  (A unit's
// eight one after another: four-way conflicts, which held the queries' turn at 57 us
// for 380 MB.)
__device__ __forceinline__ int angle_at(int t, int j, int pairs) {
  return ((t * 4 + ((j >> 1) & 3)) * (pairs / 8) + (j >> 3)) * 2 + (j & 1);
}
// The eight of unit u.
__device__ __forceinline__ void load_angles(const float2* cs, int t, int u, int pairs, float2 (&c)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 v = reinterpret_cast<const float4*>(cs)[(t * 4 + e) * (pairs / 8) + u];
    c[2 * e] = make_float2(v.x, v.y);
    c[2 * e + 1] = make_float2(v.z, v.w);
  }
}

__device__ __forceinline__ void unpack8(const uint4& x, float* v) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo_to_f32(w[i]);
    v[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}

// The unit's sixteen elements in 32 bits, turned: y[0..7] its first chunk.
template <bool IL>
__device__ __forceinline__ void turn_unit(const uint4& x0, const uint4& x1, const float2 (&cs)[8], float (&y)[16]) {
  unpack8(x0, y);
  unpack8(x1, y + 8);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = IL ? 2 * e : e, j = IL ? 2 * e + 1 : e + 8;
    const float a = y[i], b = y[j];
    y[i] = fmaf(a, cs[e].x, -(b * cs[e].y));
    y[j] = fmaf(b, cs[e].x, a * cs[e].y);
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Rows [tok0, tok0 + n) of one or two tensors, turned by the angles cs[token][pair],
// which `angles` forms (for the whole block) while the first rows are on their way.  A
// thread keeps its unit of the head and goes through the heads of one token after
// another, two units in flight.
template <int D, bool IL, int NT, typename Angles>
__device__ __forceinline__ void turn_rows(const TurnRows& x, int tok0, int n, const float2* cs, int pairs,
                                          Angles angles) {
  constexpr int U = D / 16, SWEEP = NT / U;
  const int u = threadIdx.x % U, heads = x.heads0 + x.heads1;
  const bool turned = 8 * u < pairs;
  int c0, c1;
  unit_chunks<IL>(u, pairs, c0, c1);
  int tok = 0, h = threadIdx.x / U;
  auto settle = [&]() {
    while (h >= heads && tok < n) {
      h -= heads;
      ++tok;
    }
  };
  struct Unit {
    uint4 a, b;
    uint16_t* dst;
    int tok;
  };
  auto load = [&](Unit& w) -> bool {
    if (tok >= n) return false;
    const bool first = h < x.heads0;
    const int head = first ? h : h - x.heads0;
    const long long row = tok0 + tok;
    const uint16_t* src = (first ? x.src0 + row * x.ld0 : x.src1 + row * x.ld1) + head * D;
    w.dst = (first ? x.dst0 + row * x.heads0 * D : x.dst1 + row * x.heads1 * D) + head * D;
    w.a = *reinterpret_cast<const uint4*>(src + 8 * c0);
    w.b = *reinterpret_cast<const uint4*>(src + 8 * c1);
    w.tok = tok;
    h += SWEEP;
    settle();
    return true;
  };
  auto finish = [&](const Unit& w) {
    uint4 a = w.a, b = w.b;
    if (turned) {
      float2 c[8];
      float y[16];
      load_angles(cs, w.tok, u, pairs, c);
      turn_unit<IL>(a, b, c, y);
      a = pack8(y);
      b = pack8(y + 8);
    }
    *reinterpret_cast<uint4*>(w.dst + 8 * c0) = a;
    *reinterpret_cast<uint4*>(w.dst + 8 * c1) = b;
  };
  settle();
  Unit w0, w1;
  bool one = load(w0), two = load(w1);
  angles();
  while (one) {
    finish(w0);
    if (two) finish(w1);
    one = load(w0);
    two = load(w1);
  }
}

// ----------------------------------------------------------------------------
// Queries and keys of a packed batch
// ----------------------------------------------------------------------------
constexpr int kTurnThreads = 256, kTurnTokens = 4;  // a block's tokens: one angle a thread at 64 pairs

template <int D, bool IL>
__global__ void __launch_bounds__(kTurnThreads) fa_rotary_kernel(const RotaryParams r, const TurnRows x, int total) {
  __shared__ __align__(16) float2 cs[kTurnTokens * (D / 2)];
  grid_dependency_wait();  // scheduled while the kernel before it in the stream finishes
  const int tok0 = blockIdx.x * kTurnTokens;
  const int n = min(kTurnTokens, total - tok0);
  turn_rows<D, IL, kTurnThreads>(x, tok0, n, cs, r.pairs, [&]() {
    for (int i = threadIdx.x; i < n * r.pairs; i += kTurnThreads) {
      const int t = i / r.pairs, j = i - t * r.pairs;
      cs[angle_at(t, j, r.pairs)] = cos_sin(r, j, position_of(r, j, tok0 + t, total));
    }
    __syncthreads();
  });
}

// ----------------------------------------------------------------------------
// Append to the cache
// ----------------------------------------------------------------------------
// The first blocks take a page's new tokens in some heads of K or of V, a group of
// threads (a warp up to 128 units) each (page, head); the others turn the queries.  A
// thread owns NU units, which stay in registers between the largest magnitude and the
// rounding and are on their way while the block's groups form the angles together.
// Keys are turned in 32 bits and rounded once, to their codes; values go the way of
// the plain store.
template <int D, int BLOCK>
struct AppendCfg {
  static constexpr int U = D / 16, UNITS = BLOCK * U;
  static constexpr int NU = UNITS < 128 ? UNITS / 32 : 4;  // units of a thread
  static constexpr int TG = UNITS / NU;                    // threads of a group
  static constexpr int NT = 256;
  static constexpr int HEADS = NT / TG;                    // heads of a block
  static constexpr int TOKENS = NT / 64;                   // queries' tokens of a block
  static constexpr int SMEM = (BLOCK > TOKENS ? BLOCK : TOKENS) * (D / 2) * 8;
};

template <int D, int BLOCK, bool IL>
__global__ void __launch_bounds__(AppendCfg<D, BLOCK>::NT, 4)
    fa_cache8_append_kernel(const Cache8StoreParams p, const RotaryParams r, const TurnRows x, int store_blocks,
                            int zero_tail) {
  using C = AppendCfg<D, BLOCK>;
  constexpr int NT = C::NT, NU = C::NU, TG = C::TG, U = C::U, WG = TG / 32;
  static_assert(TG % 32 == 0 && TG <= NT, "a warp is of one group");
  extern __shared__ __align__(16) float2 cs[];  // cosine, sine (angle_at)
  __shared__ int place[C::TOKENS];
  __shared__ uint32_t warp_max[NT / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();  // scheduled while the kernel before it in the stream finishes
  if (static_cast<int>(blockIdx.x) >= store_blocks) {
    // ---- queries
    // of the block's tokens those of sequences: not in front of the first, nor behind the last
    const int front = min(max(p.cu_seqlens[0], 0), p.total), end = min(max(p.cu_seqlens[p.B], front), p.total);
    const int all0 = (static_cast<int>(blockIdx.x) - store_blocks) * C::TOKENS, all = min(C::TOKENS, p.total - all0);
    const int skip = min(max(front - all0, 0), all), tok0 = all0 + skip;
    const int n = min(all - skip, end - tok0);
    turn_rows<D, IL, NT>(x, tok0, n, cs, r.pairs, [&]() {
      if (!r.positions) {  // a token's place: that of its row behind its sequence's first
        if (threadIdx.x < C::TOKENS) place[threadIdx.x] = 0;
        __syncthreads();
        for (int b = threadIdx.x; b < p.B; b += NT) {
          const int first = p.cu_seqlens[b], behind = p.cu_seqlens[b + 1], start = p.start[b];
#pragma unroll
          for (int t = 0; t < C::TOKENS; ++t)
            if (first <= tok0 + t && tok0 + t < behind)
              place[t] = static_cast<int>(static_cast<uint32_t>(start) + static_cast<uint32_t>(tok0 + t) -
                                          static_cast<uint32_t>(first));
        }
        __syncthreads();
      }
      for (int i = threadIdx.x; i < n * r.pairs; i += NT) {
        const int t = i / r.pairs, j = i - t * r.pairs;
        cs[angle_at(t, j, r.pairs)] = cos_sin(r, j, r.positions ? position_of(r, j, tok0 + t, p.total) : place[t]);
      }
      __syncthreads();
    });
    if (zero_tail) {
      for (int t = 0; t < all; ++t) {
        if (t >= skip && t - skip < n) continue;
        uint4* row = reinterpret_cast<uint4*>(x.dst0 + static_cast<long long>(all0 + t) * x.heads0 * D);
        for (int i = threadIdx.x; i < x.heads0 * (D / 8); i += NT) row[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    return;
  }
  // ---- keys or values of one page
  const int groups = (p.Hk + C::HEADS - 1) / C::HEADS;
  const int id = blockIdx.x, at = id / (2 * groups), g = id - at * 2 * groups;
  const bool is_v = g >= groups;
  const int group = threadIdx.x / TG, tid = threadIdx.x % TG;
  const int head = (is_v ? g - groups : g) * C::HEADS + group;
  const bool has_head = head < p.Hk;
  const int b = at / p.blocks, nth = at - b * p.blocks;
  const int first = min(max(p.cu_seqlens[b], 0), p.total);
  const int count = min(max(p.cu_seqlens[b + 1], first), p.total) - first;
  const int start = p.start[b];
  const long long end = static_cast<long long>(start) + min(count, p.max_new);
  const long long blk = static_cast<long long>(start) / BLOCK + nth;
  const long long base = blk * BLOCK;
  if (start < 0 || count == 0 || base >= end) {
    if (start < 0 && count > 0 && threadIdx.x == 0) atomicOr(p.err, kDevErrPage);
    return;
  }
  const int page = blk < p.table_cols ? p.table[static_cast<size_t>(b) * p.table_cols + blk] : -1;
  const int old = static_cast<int>(max(0LL, start - base));  // tokens [0, old) are held, [old, hi) are new
  const int hi = static_cast<int>(min(end - base, static_cast<long long>(BLOCK)));
  const int src = first + static_cast<int>(base - start);  // input row of slot 0
  const long long ld = is_v ? p.ldv : p.ldk;
  const int u = tid % U;
  int c0, c1;
  if (is_v) c0 = 2 * u, c1 = 2 * u + 1;
  else unit_chunks<IL>(u, r.pairs, c0, c1);
  const bool turned = !is_v && 8 * u < r.pairs;
  int tok[NU];
  bool fresh[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    tok[n] = (tid + n * TG) / U;
    fresh[n] = tok[n] >= old && tok[n] < hi;
  }
  uint4 raw[NU][2];
  const uint16_t* in = (is_v ? p.v : p.k) + static_cast<long long>(src) * ld + head * D;
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    raw[n][0] = raw[n][1] = make_uint4(0u, 0u, 0u, 0u);
    fresh[n] &= has_head;
    if (fresh[n]) {
      raw[n][0] = *reinterpret_cast<const uint4*>(in + tok[n] * ld + 8 * c0);
      raw[n][1] = *reinterpret_cast<const uint4*>(in + tok[n] * ld + 8 * c1);
    }
  }
  if (!is_v) {
    for (int i = threadIdx.x; i < (hi - old) * r.pairs; i += NT) {
      const int t = i / r.pairs, j = i - t * r.pairs;
      cs[angle_at(old + t, j, r.pairs)] =
          cos_sin(r, j, r.positions ? position_of(r, j, src + old + t, p.total) : static_cast<int>(base + old + t));
    }
    __syncthreads();
  }
  const bool live = page >= 0 && page < p.num_blocks;
  if (!live) {
    if (threadIdx.x == 0) atomicOr(p.err, kDevErrPage);
    return;
  }
  const size_t ph = static_cast<size_t>(page) * p.Hk + (has_head ? head : 0);
  float* scale = (is_v ? p.v_scale : p.k_scale) + ph;
  const float held = old > 0 ? *scale : 0.f;
  auto values = [&](int n, float (&y)[16]) {
    if (turned && fresh[n]) {
      float2 c[8];
      load_angles(cs, tok[n], u, r.pairs, c);
      turn_unit<IL>(raw[n][0], raw[n][1], c, y);
    } else {
      unpack8(raw[n][0], y);
      unpack8(raw[n][1], y + 8);
    }
  };
  // The largest magnitude, as fp32 bits.  Infinities and NaN do not set the scale: the
  // maximum passes over NaN; where it is infinite, once more without.
  auto largest = [&](bool finite) -> uint32_t {
    if (is_v) {
      uint32_t top = 0;
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        const uint32_t w[8] = {raw[n][0].x, raw[n][0].y, raw[n][0].z, raw[n][0].w,
                               raw[n][1].x, raw[n][1].y, raw[n][1].z, raw[n][1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t m = w[i] & 0x7fff7fffu;
          top = max_bf16x2(top, finite ? m & ~__vcmpgeu2(m, 0x7f807f80u) : m);
        }
      }
      return max(top & 0xffffu, top >> 16) << 16;
    }
    float top = 0.f;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      float y[16];
      values(n, y);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float a = fabsf(y[i]);
        top = fmaxf(top, finite && !(a < CUDART_INF_F) ? 0.f : a);
      }
    }
    return __float_as_uint(top);
  };
  uint32_t amax = largest(false);
  if (amax >= 0x7f800000u) amax = largest(true);
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (TG > 32) {  // (and every thread has read the scale held before one of them writes the new one)
    if (lane == 0) warp_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WG; ++w) amax = max(amax, warp_max[group * WG + w]);
  } else {
    __syncwarp();
  }
  if (!has_head) return;
  const float s = fmaxf(exp2_int(scale_exponent_f32(amax, kScaleFloor)), held);
  const float inv = exp2_int(127 - static_cast<int>((__float_as_uint(s) >> 23) & 255u));  // 1 / s, a power of two
  const uint64_t inv2 = f2_pack(inv, inv);
  const bool again = s > held;
  if (tid == 0 && again) *scale = s;
  uint8_t* out = (is_v ? p.v_codes : p.k_codes) + ph * (BLOCK * D);
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    uint2* a = reinterpret_cast<uint2*>(out + tok[n] * D + 8 * c0);
    uint2* z = reinterpret_cast<uint2*>(out + tok[n] * D + 8 * c1);
    if (fresh[n]) {
      float y[16];
      values(n, y);
#pragma unroll
      for (int i = 0; i < 16; i += 2) f2_unpack(fmul2(f2_pack(y[i], y[i + 1]), inv2), y[i], y[i + 1]);
      *a = make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
      *z = make_uint2(pack_e4m3x4(y[8], y[9], y[10], y[11]), pack_e4m3x4(y[12], y[13], y[14], y[15]));
    } else if (tok[n] < old && again) {
      // tokens held at a smaller scale are rounded again
      const float f = held * inv;
      const uint2 code[2] = {*a, *z};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v[4], w[4];
        unpack_e4m3x4(code[k].x, v);
        unpack_e4m3x4(code[k].y, w);
        *(k ? z : a) = make_uint2(pack_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                                  pack_e4m3x4(w[0] * f, w[1] * f, w[2] * f, w[3] * f));
      }
    }
  }
}

template <int D, int BLOCK, bool IL>
cudaError_t launch_append(const Cache8StoreParams& p, const RotaryParams& r, const TurnRows& x, int zero_tail,
                          cudaStream_t s) {
  using C = AppendCfg<D, BLOCK>;
  static SmemLimit smem_limit;
  const cudaError_t e = smem_limit.ensure(reinterpret_cast<const void*>(fa_cache8_append_kernel<D, BLOCK, IL>), C::SMEM);
  if (e != cudaSuccess) return e;
  const long long groups = (p.Hk + C::HEADS - 1) / C::HEADS;
  const long long store = static_cast<long long>(p.B) * p.blocks * 2 * groups;
  const long long turn = (p.total - 1) / C::TOKENS + 1;
  if (store + turn > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_kernel(fa_cache8_append_kernel<D, BLOCK, IL>, dim3(static_cast<unsigned>(store + turn)), dim3(C::NT), C::SMEM, s,
                       true, p, r, x, static_cast<int>(store), zero_tail);
}

template <int D, int BLOCK>
cudaError_t launch_append_il(const Cache8StoreParams& p, const RotaryParams& r, const TurnRows& x, int zero_tail,
                             cudaStream_t s) {
  return r.interleaved ? launch_append<D, BLOCK, true>(p, r, x, zero_tail, s)
                       : launch_append<D, BLOCK, false>(p, r, x, zero_tail, s);
}

template <int D>
cudaError_t launch_append_d(int block, const Cache8StoreParams& p, const RotaryParams& r, const TurnRows& x,
                            int zero_tail, cudaStream_t s) {
  if (block == 16) return launch_append_il<D, 16>(p, r, x, zero_tail, s);
  if (block == 32) return launch_append_il<D, 32>(p, r, x, zero_tail, s);
  if (block == 64) return launch_append_il<D, 64>(p, r, x, zero_tail, s);
  return launch_append_il<D, 128>(p, r, x, zero_tail, s);
}

template <int D>
cudaError_t launch_rotary_d(const RotaryParams& r, const TurnRows& x, int total, cudaStream_t s) {
  const dim3 grid((total - 1) / kTurnTokens + 1), block(kTurnThreads);
  return r.interleaved ? launch_kernel(fa_rotary_kernel<D, true>, grid, block, 0, s, true, r, x, total)
                       : launch_kernel(fa_rotary_kernel<D, false>, grid, block, 0, s, true, r, x, total);
}

}  // namespace

cudaError_t launch_rotary(int d, const RotaryParams& r, const TurnRows& x, int total, cudaStream_t s) {
  return d == 64 ? launch_rotary_d<64>(r, x, total, s) : launch_rotary_d<128>(r, x, total, s);
}

cudaError_t launch_cache8_append(int d, int block, const Cache8StoreParams& p, const RotaryParams& r, const TurnRows& x,
                                 int zero_tail, cudaStream_t s) {
  return d == 64 ? launch_append_d<64>(block, p, r, x, zero_tail, s) : launch_append_d<128>(block, p, r, x, zero_tail, s);
}

}  // namespace fa
