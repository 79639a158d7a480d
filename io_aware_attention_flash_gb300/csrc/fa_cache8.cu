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
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "fa_kernels.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

// ----------------------------------------------------------------------------
// Store
// ----------------------------------------------------------------------------
constexpr int kScaleFloor = -64;  // exponent of the smallest scale

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Scale exponent of a maximum magnitude given as bf16 bits: amax = 1.m · 2^E is
// at most 448 · 2^e = 1.75 · 2^(8+e).
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int biased = static_cast<int>(amax_bits >> 7), mant = static_cast<int>(amax_bits & 127u);
  return max(biased - 127 - 8 + (mant > 96 ? 1 : 0), kScaleFloor);
}

// Four floats to four e4m3 codes (nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
// Two e4m3 codes to two floats (exact).
__device__ __forceinline__ void unpack_e4m3x2(uint32_t code2, float& a, float& b) {
  uint32_t h2;
  const uint16_t c = static_cast<uint16_t>(code2);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
  asm("{.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}" : "=f"(a), "=f"(b) : "r"(h2));
}

// One group of TG threads quantises the new tokens of one (page, head) of K or
// V: each thread keeps CH 16-byte chunks of them in registers between the
// maximum and the rounding, so the input is read once.  A page that already
// holds tokens keeps its scale if that suffices; otherwise they are rounded
// again to the larger one.  Groups of consecutive heads are consecutive, so a
// warp's loads cover whole rows of the token-major input.
template <int CH, int TG, int D, int BLOCK>
__global__ void __launch_bounds__(256) fa_cache8_store_kernel(const Cache8StoreParams p) {
  static_assert(CH * TG * 8 == D * BLOCK, "a group's chunks cover a page and head");
  constexpr int GPB = 256 / TG;  // groups per block
  constexpr int C8 = D / 8;      // chunks per token
  __shared__ uint32_t warp_max[8];
  const int group = threadIdx.x / TG, tid = threadIdx.x % TG;
  const long long item = static_cast<long long>(blockIdx.x) * GPB + group;
  // item = ((sequence · blocks + block) · 2 + V) · Hk + head
  const int head = static_cast<int>(item % p.Hk);
  const long long rest = item / p.Hk;
  const bool is_v = rest & 1;
  const int nth = static_cast<int>((rest >> 1) % p.blocks);
  const int b = static_cast<int>((rest >> 1) / p.blocks);
  int page = -1, old = 0, lo = 0, hi = 0;  // the page; its tokens [0, old) are held, [lo, hi) are new
  int src = 0;                             // input row of slot 0
  if (b < p.B) {
    const int first = min(max(__ldg(p.cu_seqlens + b), 0), p.total);
    const int count = min(max(__ldg(p.cu_seqlens + b + 1), first), p.total) - first;
    const int start = __ldg(p.start + b);
    const long long end = static_cast<long long>(start) + min(count, p.max_new);
    const long long blk = static_cast<long long>(start) / BLOCK + nth;
    if (start < 0) {
      if (count > 0 && nth == 0 && tid == 0) atomicOr(p.err, kDevErrPage);
    } else if (count > 0 && blk * BLOCK < end) {
      page = blk < p.table_cols ? __ldg(p.table + static_cast<size_t>(b) * p.table_cols + blk) : -1;
      if (page < 0 || page >= p.num_blocks) {
        if (tid == 0) atomicOr(p.err, kDevErrPage);
        page = -1;
      }
      const long long base = blk * BLOCK;
      old = static_cast<int>(max(0LL, start - base));
      lo = old;
      hi = static_cast<int>(min(end - base, static_cast<long long>(BLOCK)));
      src = first + static_cast<int>(base - start);
    }
  }
  const uint16_t* x = is_v ? p.v : p.k;
  const long long ld = is_v ? p.ldv : p.ldk;
  uint4 val[CH];
  uint32_t amax2 = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int chunk = c * TG + tid, t = chunk / C8;
    val[c] = make_uint4(0u, 0u, 0u, 0u);
    if (page >= 0 && t >= lo && t < hi)
      val[c] = *reinterpret_cast<const uint4*>(x + (static_cast<long long>(src) + t) * ld + head * D + (chunk % C8) * 8);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t w[4] = {val[c].x, val[c].y, val[c].z, val[c].w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t m = w[u] & 0x7fff7fffu;
      amax2 = __vmaxu2(amax2, m & ~__vcmpgeu2(m, 0x7f807f80u));  // infinities and NaN do not set the scale
    }
  }
  uint32_t amax = max(amax2 & 0xffffu, amax2 >> 16);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (TG > 32) {
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
    __syncthreads();
    const int w0 = group * (TG / 32);
#pragma unroll
    for (int w = 0; w < TG / 32; ++w) amax = max(amax, warp_max[w0 + w]);
  }
  if (page < 0) return;
  const size_t ph = static_cast<size_t>(page) * p.Hk + head;
  float* scale = (is_v ? p.v_scale : p.k_scale) + ph;
  const float held = old > 0 ? *scale : 0.f;
  const float s = fmaxf(exp2_int(scale_exponent(amax)), held);
  // 1 / s of a power of two, by its exponent
  const float inv = exp2_int(127 - static_cast<int>((__float_as_uint(s) >> 23) & 255u));
  uint2* out = reinterpret_cast<uint2*>((is_v ? p.v_codes : p.k_codes) + ph * (BLOCK * D));
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int chunk = c * TG + tid, t = chunk / C8;
    if (t >= lo && t < hi) {
      out[chunk] = make_uint2(
          pack_e4m3x4(bf16lo_to_f32(val[c].x) * inv, bf16hi_to_f32(val[c].x) * inv, bf16lo_to_f32(val[c].y) * inv,
                      bf16hi_to_f32(val[c].y) * inv),
          pack_e4m3x4(bf16lo_to_f32(val[c].z) * inv, bf16hi_to_f32(val[c].z) * inv, bf16lo_to_f32(val[c].w) * inv,
                      bf16hi_to_f32(val[c].w) * inv));
    } else if (t < old && s > held) {
      const uint2 code = out[chunk];
      const float f = held * inv;
      float v[8];
      unpack_e4m3x2(code.x, v[0], v[1]);
      unpack_e4m3x2(code.x >> 16, v[2], v[3]);
      unpack_e4m3x2(code.y, v[4], v[5]);
      unpack_e4m3x2(code.y >> 16, v[6], v[7]);
      out[chunk] = make_uint2(pack_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                              pack_e4m3x4(v[4] * f, v[5] * f, v[6] * f, v[7] * f));
    }
  }
  if (TG > 32) __syncthreads();  // every thread has read the scale held
  else __syncwarp();
  if (tid == 0) *scale = s;
}

template <int D, int BLOCK>
cudaError_t launch_store(const Cache8StoreParams& p, cudaStream_t s) {
  constexpr int CHUNKS = D * BLOCK / 8;
  constexpr int TG = CHUNKS <= 256 ? 32 : CHUNKS / 8;
  const long long items = static_cast<long long>(p.B) * p.blocks * 2 * p.Hk;
  const long long ctas = (items * TG + 255) / 256;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  fa_cache8_store_kernel<CHUNKS / TG, TG, D, BLOCK><<<static_cast<unsigned>(ctas), 256, 0, s>>>(p);
  return cudaGetLastError();
}

// ----------------------------------------------------------------------------
// Attention over the cache
// ----------------------------------------------------------------------------
// Work: the 128-key tiles of every (sequence, key/value head, row group), in
// that order, are shared out in equal runs over the launch's CTAs, whatever
// the sequences' lengths; a row group is up to kRows of the (new token, query
// head) rows that attend to one key/value head.  A CTA that has all tiles of
// an item writes its output; an item that several CTAs share leaves partials
// (m, l, O) that the merge kernel combines in the order of the tiles.
constexpr int kRows = 8;

struct Work {
  int* start;     // [B + 1] shared memory: first tile of each sequence, then the total
  int total;
};

// Cached tokens of sequence b: a length below 0 counts as 0, one past the page
// table as the table's end.
__device__ __forceinline__ int cached_len(const Cache8DecodeParams& p, int b) {
  const long long cap = static_cast<long long>(p.table_cols) * p.block;
  int n = __ldg(p.seqlens + b);
  if (n < 0 || n > cap || n > p.max_seqlen) {
    atomicOr(p.err, kDevErrPage);
    n = n < 0 ? 0 : static_cast<int>(min(cap, static_cast<long long>(p.max_seqlen)));
  }
  return n;
}

__device__ __forceinline__ int run_start(long long c, int total, int ctas) { return static_cast<int>(c * total / ctas); }
// The CTA whose run holds tile t.
__device__ __forceinline__ int run_of(long long t, int total, int ctas) {
  return static_cast<int>(((t + 1) * ctas + total - 1) / total - 1);
}

// Sum of the tiles of the sequences before b0 .. (whole block; NT threads).
// Returns this CTA's first sequence and the tiles before it through `scan`.
template <int NT>
__device__ __forceinline__ int block_scan_tiles(const Cache8DecodeParams& p, int* warp_sums, bool store) {
  // inclusive scans of NT sequences at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + threadIdx.x;
    int n = b < p.B ? (cached_len(p, b) + kTile - 1) / kTile * p.Hk * p.row_groups : 0;
    const int own = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, n, off);
      if (lane >= off) n += y;
    }
    if (lane == 31) warp_sums[warp] = n;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      before += w < warp ? warp_sums[w] : 0;
      all += warp_sums[w];
    }
    __syncthreads();
    if (store && b < p.B) p.tile_start[b] = base + before + n - own;
    base += all;
  }
  return base;
}

template <int D>
__global__ void __launch_bounds__(128) fa_cache8_decode_kernel(const Cache8DecodeParams p) {
  __shared__ int warp_sums[4];
  __shared__ float qs[kRows][D];
  __shared__ float ps[kRows][kTile];
  __shared__ float red[4][kRows];
  __shared__ float m_s[kRows], l_s[kRows], a_s[kRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Every CTA finds its place by itself: the tiles before each sequence.
  const int total = block_scan_tiles<128>(p, warp_sums, blockIdx.x == 0);
  if (blockIdx.x == 0 && tid == 0) p.tile_start[p.B] = total;
  const int ctas = min(static_cast<int>(gridDim.x), total);  // every one of them has a tile
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  const int t_lo = run_start(blockIdx.x, total, ctas), t_hi = run_start(blockIdx.x + 1LL, total, ctas);
  int b = 0, seq0 = 0;  // sequence of tile t and its first tile
  for (int t = t_lo; t < t_hi;) {
    int nt;
    while (true) {
      nt = (cached_len(p, b) + kTile - 1) / kTile;
      if (t < seq0 + nt * p.Hk * p.row_groups) break;
      seq0 += nt * p.Hk * p.row_groups;
      ++b;
    }
    const int len = cached_len(p, b);
    const int item = (t - seq0) / nt;           // (head, row group)
    const int k0 = (t - seq0) - item * nt;      // first tile of the item in this run
    const int k1 = min(nt, k0 + (t_hi - t));
    const int hk = item / p.row_groups, rg = item - hk * p.row_groups;
    const int rows = min(kRows, p.Nq * p.G - rg * kRows);
    __syncthreads();
    for (int i = tid; i < kRows * D; i += 128) {
      const int r = i / D, f = rg * kRows + r;
      float v = 0.f;
      if (r < rows)
        v = __uint_as_float(static_cast<uint32_t>(
                p.q[((static_cast<size_t>(b) * p.Nq + f / p.G) * p.H + hk * p.G + f % p.G) * D + i % D]) << 16);
      qs[r][i % D] = v;
    }
    if (tid < kRows) {
      m_s[tid] = -CUDART_INF_F;
      l_s[tid] = 0.f;
    }
    float acc[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[r] = 0.f;
    for (int kt = k0; kt < k1; ++kt) {
      __syncthreads();
      const int key = kt * kTile + tid;
      float s[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) s[r] = 0.f;
      int page = -1;
      if (key < len) {
        page = __ldg(p.table + static_cast<size_t>(b) * p.table_cols + key / p.block);
        if (page < 0 || page >= p.num_blocks) {
          atomicOr(p.err, kDevErrPage);
          page = -1;
        }
      }
      if (page >= 0) {
        const uint32_t* row = reinterpret_cast<const uint32_t*>(
            p.k_codes + ((static_cast<size_t>(page) * p.Hk + hk) * p.block + key % p.block) * D);
        for (int c = 0; c < D / 4; ++c) {
          const uint32_t w = row[c];
          float x[4];
          unpack_e4m3x2(w, x[0], x[1]);
          unpack_e4m3x2(w >> 16, x[2], x[3]);
#pragma unroll
          for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[r] = fmaf(qs[r][4 * c + e], x[e], s[r]);
        }
        const float ks = p.k_scale[static_cast<size_t>(page) * p.Hk + hk] * p.scale_log2;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s[r] *= ks;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int last = p.causal ? len - p.Nq + (rg * kRows + r) / p.G : len - 1;
        if (key > last || key >= len) s[r] = -CUDART_INF_F;
        float mx = s[r];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        if (lane == 0) red[warp][r] = mx;
      }
      __syncthreads();
      if (tid < kRows) {
        const float m_new = fmaxf(fmaxf(fmaxf(red[0][tid], red[1][tid]), fmaxf(red[2][tid], red[3][tid])), m_s[tid]);
        a_s[tid] = m_s[tid] == -CUDART_INF_F ? 0.f : ex2_approx(m_s[tid] - m_new);
        m_s[tid] = m_new;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float e = s[r] == -CUDART_INF_F ? 0.f : ex2_approx(s[r] - m_s[r]);
        ps[r][tid] = e;
        float sum = e;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) red[warp][r] = sum;
        acc[r] *= a_s[r];
      }
      __syncthreads();
      if (tid < kRows) l_s[tid] = l_s[tid] * a_s[tid] + ((red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]));
      if (tid < D) {
        const int n = min(kTile, len - kt * kTile);
        for (int j = 0; j < n; ++j) {
          const int kj = kt * kTile + j;
          const int pj = __ldg(p.table + static_cast<size_t>(b) * p.table_cols + kj / p.block);
          if (pj < 0 || pj >= p.num_blocks) continue;
          const size_t ph = static_cast<size_t>(pj) * p.Hk + hk;
          float v, unused;
          unpack_e4m3x2(p.v_codes[(ph * p.block + kj % p.block) * D + tid], v, unused);
          v *= p.v_scale[ph];
#pragma unroll
          for (int r = 0; r < kRows; ++r) acc[r] = fmaf(ps[r][j], v, acc[r]);
        }
      }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == nt;
    for (int r = 0; r < rows; ++r) {
      const int f = rg * kRows + r;
      const size_t qrow = static_cast<size_t>(b) * p.Nq + f / p.G;
      const int h = hk * p.G + f % p.G;
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) a = i == r ? acc[i] : a;
      if (whole) {
        const float l = l_s[r];
        if (tid < D) p.o[(qrow * p.H + h) * D + tid] = static_cast<uint16_t>(pack_bf16x2(l > 0.f ? a / l : 0.f, 0.f));
        if (tid == 0)
          p.lse[(static_cast<size_t>(b) * p.H + h) * p.Nq + f / p.G] =
              l > 0.f ? (m_s[r] + log2f(l)) * kLn2 : -CUDART_INF_F;
      } else {
        const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (k0 == 0 ? 1 : 0)) * kRows + r;
        if (tid < D) p.o_part[slot * D + tid] = a;
        if (tid == 0) {
          p.ml_part[slot * 2] = m_s[r];
          p.ml_part[slot * 2 + 1] = l_s[r];
        }
      }
    }
    t += k1 - k0;
  }
}

// One warp per (sequence, new token, query head): the partials of an item that
// several CTAs shared, in the order of its tiles; zeros where no key is cached.
template <int D>
__global__ void __launch_bounds__(128) fa_cache8_merge_kernel(const Cache8DecodeParams p, int ctas) {
  constexpr int E = D / 32;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const long long wid = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (wid >= static_cast<long long>(p.B) * p.Nq * p.H) return;
  const int h = static_cast<int>(wid % p.H);
  const long long qrow = wid / p.H;
  const int i = static_cast<int>(qrow % p.Nq), b = static_cast<int>(qrow / p.Nq);
  const int total = p.tile_start[p.B];
  ctas = min(ctas, total);
  const int s0 = p.tile_start[b], s1 = p.tile_start[b + 1];
  const int hk = h / p.G, f = i * p.G + h % p.G, rg = f / kRows, r = f - rg * kRows;
  const int nt = (s1 - s0) / (p.Hk * p.row_groups);
  const long long t0 = s0 + static_cast<long long>(hk * p.row_groups + rg) * nt;
  const int c0 = nt ? run_of(t0, total, ctas) : 0, c1 = nt ? run_of(t0 + nt - 1, total, ctas) : -1;
  if (c0 == c1) return;  // written by that CTA
  float m = -CUDART_INF_F, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int c = c0; c <= c1; ++c) {
    const size_t slot = (2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0)) * kRows + r;
    const float mc = p.ml_part[slot * 2], lc = p.ml_part[slot * 2 + 1];
    if (mc == -CUDART_INF_F) continue;
    const float m_new = fmaxf(m, mc);
    const float a = m == -CUDART_INF_F ? 0.f : ex2_approx(m - m_new), w = ex2_approx(mc - m_new);
    m = m_new;
    l = l * a + w * lc;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * p.o_part[slot * D + E * lane + e];
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* o = p.o + (qrow * p.H + h) * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0)
    p.lse[(static_cast<size_t>(b) * p.H + h) * p.Nq + i] = l > 0.f ? (m + log2f(l)) * kLn2 : -CUDART_INF_F;
}

template <int D>
cudaError_t launch_decode8(const Cache8DecodeParams& p, int ctas, cudaStream_t s) {
  fa_cache8_decode_kernel<D><<<ctas, 128, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long warps = static_cast<long long>(p.B) * p.Nq * p.H;
  fa_cache8_merge_kernel<D><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, s>>>(p, ctas);
  return cudaGetLastError();
}

}  // namespace

int cache8_rows() { return kRows; }

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

cudaError_t launch_cache8_decode(int d, const Cache8DecodeParams& p, int ctas, cudaStream_t s) {
  return d == 64 ? launch_decode8<64>(p, ctas, s) : launch_decode8<128>(p, ctas, s);
}

}  // namespace fa
