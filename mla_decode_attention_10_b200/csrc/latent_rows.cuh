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

// Sixteen codes -> sixteen fp16 (exact).
__device__ __forceinline__ void codes_to_f16(const uint4& c, uint4& a, uint4& b) {
  a.x = e4m3x2_to_f16x2(static_cast<uint16_t>(c.x & 0xffffu));
  a.y = e4m3x2_to_f16x2(static_cast<uint16_t>(c.x >> 16));
  a.z = e4m3x2_to_f16x2(static_cast<uint16_t>(c.y & 0xffffu));
  a.w = e4m3x2_to_f16x2(static_cast<uint16_t>(c.y >> 16));
  b.x = e4m3x2_to_f16x2(static_cast<uint16_t>(c.z & 0xffffu));
  b.y = e4m3x2_to_f16x2(static_cast<uint16_t>(c.z >> 16));
  b.z = e4m3x2_to_f16x2(static_cast<uint16_t>(c.w & 0xffffu));
  b.w = e4m3x2_to_f16x2(static_cast<uint16_t>(c.w >> 16));
}

// 2^(byte - 127) of a scale byte as fp32 (bytes 1..254; 0 gives 0, 255 infinity).
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float((byte & 0xffu) << 23); }

}  // namespace mla
