// e4m3 codes and the powers of two that scale them, as the 8-bit cache keeps them, and
// the tensor core's products of codes.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

constexpr int kScaleFloor = -64;  // exponent of the smallest scale

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Scale exponent of a maximum magnitude given as bf16 bits: amax = 1.m · 2^E is
// at most 448 · 2^e = 1.75 · 2^(8+e); not below `least`.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits, int least) {
  const int biased = static_cast<int>(amax_bits >> 7), mant = static_cast<int>(amax_bits & 127u);
  return max(biased - 127 - 8 + (mant > 96 ? 1 : 0), least);
}

// The same of a maximum given as fp32 bits.
__device__ __forceinline__ int scale_exponent_f32(uint32_t amax_bits, int least) {
  const int biased = static_cast<int>(amax_bits >> 23);
  return max(biased - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0), least);
}

// Floats to e4m3 codes, the first in the lowest byte (nearest even,
// saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Two e4m3 codes to two floats (exact).
__device__ __forceinline__ void unpack_e4m3x2(uint32_t code2, float& a, float& b) {
  uint32_t h2;
  const uint16_t c = static_cast<uint16_t>(code2);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
  asm("{.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}" : "=f"(a), "=f"(b) : "r"(h2));
}

// The larger of two bf16 in each half; of a NaN and a number the number.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Four e4m3 codes to four floats (exact).
__device__ __forceinline__ void unpack_e4m3x4(uint32_t code4, float (&v)[4]) {
  uint32_t a, b;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(a), "=r"(b)
      : "r"(code4));
  asm("{.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}" : "=f"(v[0]), "=f"(v[1]) : "r"(a));
  asm("{.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}" : "=f"(v[2]), "=f"(v[3]) : "r"(b));
}

// D(tmem) (+)= A(smem) B(smem), e4m3 inputs, fp32 accumulate, K = 32 a step.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: e4m3 A and B (formats 0), both of them
// K-major or both MN-major, fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool mn_major) {
  return (1u << 4) | ((mn_major ? 3u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Two floats to f16, the first in the low half; two f16 to two e4m3 codes (saturating)
// and back (exact); a difference.
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4_of_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\t"
      "mov.b32 %0, {l, h};}"
      : "=r"(r)
      : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void f16_of_e4m3x4(uint32_t code4, uint32_t& a, uint32_t& b) {
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(a), "=r"(b)
      : "r"(code4));
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Byte `byte` of row `row` in a tile of W-byte rows swizzled over W bytes (the
// 16-byte chunk's index exclusive-or the address bits above the 128-byte line).
template <int W>
__device__ __forceinline__ uint32_t swz(int row, int byte) {
  constexpr int MASK = W / 16 - 1;
  const int line = row / (128 / W);
  return row * W + ((((byte >> 4) ^ line) & MASK) << 4) + (byte & 15);
}
// Descriptor of an operand in W-byte rows swizzled over W bytes (16: not
// swizzled), 8 rows an atom, the next 8 `next8` bytes on.  K-major: rows are M or N.
// MN-major: rows are K, lbo the distance to the next W bytes of M.
template <int W>
__device__ __forceinline__ uint64_t sdesc8(uint32_t saddr, uint32_t lbo, uint32_t next8 = 8 * W) {
  constexpr uint64_t mode = W == 128 ? 2 : W == 64 ? 4 : W == 32 ? 6 : 0;
  // Without a swizzle the two distances change places in MN-major.
  const uint32_t lead = W == 16 ? next8 : lbo, stride = W == 16 ? lbo : next8;
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((stride >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (mode << 61);
}

}  // namespace fa
