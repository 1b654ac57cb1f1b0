// The 8-bit latent row (640 bytes, and a scale apart from it): 512 E4M3 codes, 64 rotary dims in bf16.
//
// The scale is a power of two of 2^-24 .. 2^7. So a value, code * scale, has the code's four
// significant bits: exact in bf16, which makes the unpacked row an MMA operand without a rounding, and
// the division by the scale is exact too, which leaves the conversion the only rounding of the writer.
// An E4M3 number keeps its relative precision over 15 octaves below the row's largest, so one scale a
// row serves; a row is 20 sectors of 32 bytes, every 64-dim chunk of codes two of them.
#pragma once
#include <cstdint>

namespace ds4f8 {

constexpr int kLatent = 512, kRope = 64, kRowDims = kLatent + kRope;
constexpr int kOffRope = 512, kRowBytes = 640;
constexpr int kMinExp = -24, kMaxExp = 7;

// Four codes to the two halves of f16 pairs (exact).
__device__ __forceinline__ void codes_to_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 v;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return v;
}

}  // namespace ds4f8
