// latent_rows.cuh -- the three formats of a latent cache row and the decoding
// of their pieces (device side, internal).
//
//   bf16  576 values; e4m3  576 codes of value / scale;
//   mx    512 codes, 16 scale bytes (value = code * 2^(byte - 127), 32 latents
//         to a scale), 64 bf16 rotary values.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "latent_math.cuh"
#include "mla_epilogue.h"

namespace mla {

constexpr int kMxScales = 512;             // byte offset of the scale bytes in an mx row
constexpr int kMxPe = 528;                 // byte offset of the rotary values
constexpr int kMxRow = 656;                // bytes of an mx row
constexpr int kMxMinExp = -117;            // scale exponents: the smallest non-zero code, 2^-9, times 2^e stays a
constexpr int kMxMaxExp = 119;             // normal bf16 number, and 448 * 2^e stays finite

__host__ __device__ constexpr int row_bytes(int format) {
  return format == MLA_CACHE_BF16 ? 1152 : format == MLA_CACHE_E4M3 ? 576 : kMxRow;
}

// 16 bytes, or zeros where there is no row; a predicate, not a branch, so that one
// load need not have come before the next is issued.
__device__ __forceinline__ uint4 load16(const uint8_t* row, int at) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.s64 p, %4, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%5];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(row), "l"(row + at)
      : "memory");
  return v;
}

// Two e4m3 codes -> their values as fp16 (exact; NaN stays NaN), low code in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\t"
      "cvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

// Two e4m3 codes times `mul` -> packed bf16.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t c, float mul) {
  float lo, hi;
  f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(c)), lo, hi);
  return pack_bf16x2(__fmul_rn(lo, mul), __fmul_rn(hi, mul));
}

// Sixteen codes (one 16-byte piece) times `mul` -> sixteen bf16 (two 16-byte pieces).
__device__ __forceinline__ void codes_to_bf16(const uint4& c, float mul, uint4& a, uint4& b) {
  a.x = e4m3x2_to_bf16x2(c.x & 0xffffu, mul);
  a.y = e4m3x2_to_bf16x2(c.x >> 16, mul);
  a.z = e4m3x2_to_bf16x2(c.y & 0xffffu, mul);
  a.w = e4m3x2_to_bf16x2(c.y >> 16, mul);
  b.x = e4m3x2_to_bf16x2(c.z & 0xffffu, mul);
  b.y = e4m3x2_to_bf16x2(c.z >> 16, mul);
  b.z = e4m3x2_to_bf16x2(c.w & 0xffffu, mul);
  b.w = e4m3x2_to_bf16x2(c.w >> 16, mul);
}

// 2^(byte - 127) of a scale byte as fp32; 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  byte &= 0xffu;
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fffffffu : byte << 23);
}

// ---- the same conversions without the conversion unit, whose rate bounds a
// kernel that decodes a tile per tile of products.  An e4m3 code s eeee mmm is,
// bit for bit, a bf16 number with its exponent 120 too low, zeros and subnormals
// included: one product with 2^120, exact, puts that right.  Only the NaN code (all ones) comes out as 480.

// Whether one of the sixteen codes is NaN.
__device__ __forceinline__ bool any_nan_code(const uint4& c) {
  constexpr uint32_t kLow = 0x7f7f7f7fu, kOne = 0x01010101u;
  return ((((c.x & kLow) + kOne) | ((c.y & kLow) + kOne) | ((c.z & kLow) + kOne) | ((c.w & kLow) + kOne)) &
          0x80808080u) != 0u;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Four codes -> two words of 16-bit pairs before the product: each code in the
// high byte of its half, exponent and mantissa shifted down by four.
__device__ __forceinline__ void spread_codes(uint32_t c, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(c, 0u, 0x1404), b = __byte_perm(c, 0u, 0x3424);
  lo = ((a >> 4) & 0x07f007f0u) | (a & 0x80008000u);
  hi = ((b >> 4) & 0x07f007f0u) | (b & 0x80008000u);
}

// Sixteen codes without a NaN times `mul2` = {m, m}, m = 2^120 times the scale (a power of two) in bf16.
__device__ __forceinline__ void plain_codes_to_bf16(const uint4& c, uint32_t mul2, uint4& a, uint4& b) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    spread_codes(w[i], lo, hi);
    o[2 * i] = mul_bf16x2(lo, mul2);
    o[2 * i + 1] = mul_bf16x2(hi, mul2);
  }
  a = make_uint4(o[0], o[1], o[2], o[3]);
  b = make_uint4(o[4], o[5], o[6], o[7]);
}

constexpr uint32_t kBf16Pow120 = 0x7b807b80u;  // {2^120, 2^120}

// {m, m}, m = 2^120 * 2^(byte - 127) in bf16, for a scale byte up to kMxPlain
constexpr uint32_t kMxPlain = 134;
__device__ __forceinline__ uint32_t mx_mul2(uint32_t byte) { return (byte + 120u) * 0x00800080u; }

}  // namespace mla
