// The 4-bit latent row (416 bytes): 512 integers in -7..7 stored as n + 8, of each eight dims of a
// 32-bit word dim 2p in bits 4p.. and dim 2p + 1 in bits 16 + 4p..; 32 scale codes; 64 bf16.
//
// The order inside a word and the scale format make the way back to bf16 cheap: (w >> 4p) &
// 0x000F000F | 0x43004300 is the adjacent pair (128 + n', 128 + n') in bf16 with n' = n + 8, and one
// packed fma with (s, -136 s) gives both n * s. It is exact: a scale has 4 significant bits, so
// 136 s = 17 * 8 * s has 8, and n * s has at most 7; bf16 holds 8. 13 sectors of 32 bytes hold
// a row, and every 64-dim chunk of codes is one of them.
#pragma once
#include <cstdint>

namespace ds4q {

constexpr int kLatent = 512, kRope = 64, kRowDims = kLatent + kRope;
constexpr int kOffScale = 256, kOffRope = 288, kRowBytes = 416;
constexpr uint32_t kEmptyWord = 0x88888888u;  // eight zeros

// bf16 bits of a scale code, in both halves: 2^(c / 8 - 20) * (1 + (c % 8) / 8).
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t code) {
  return (0x3580u + (code << 4)) * 0x00010001u;
}
__device__ __forceinline__ float scale_f32(uint32_t code) {
  return __uint_as_float((code << 20) + (107u << 23));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// -136 * scale in both halves (exact).
__device__ __forceinline__ uint32_t offset_bf16x2(uint32_t s2) { return mul_bf16x2(s2, 0xC308C308u); }
// Eight integers and their scale to eight bf16 values in dim order.
__device__ __forceinline__ uint4 word_to_bf16(uint32_t w, uint32_t s2, uint32_t c2) {
  uint4 v;
  v.x = fma_bf16x2((w & 0x000F000Fu) | 0x43004300u, s2, c2);
  v.y = fma_bf16x2(((w >> 4) & 0x000F000Fu) | 0x43004300u, s2, c2);
  v.z = fma_bf16x2(((w >> 8) & 0x000F000Fu) | 0x43004300u, s2, c2);
  v.w = fma_bf16x2(((w >> 12) & 0x000F000Fu) | 0x43004300u, s2, c2);
  return v;
}

}  // namespace ds4q
