// The 4-bit latent cache's writer and reader (format: q4_format.cuh): a row is one warp, a lane one
// group of 16 dims (its absmax needs no other lane) and two rotary dims. 65536 rows: read back as bf16
// in 16.4 us, an HBM stream (floor 15.4, part of the rows come from L2), as fp32 in 38 (floor 26.7);
// written from bf16 in 24.6 us (floor 15.4), bound by the half-rate integer pipe (71% busy, DRAM 37%),
// from fp32 in 34.8 (floor 26.7).
//
// Rounding. The scale is the code nearest to absmax / 7 and an integer the one nearest to
// x / scale, ties to even, both decided exactly: the fp32 quotient only proposes, and where it
// lands on or next to a border the remainder of one fma (exact) decides. A product with the
// rounded reciprocal alone gets some ties wrong (15 / 8 * 2 at x = 150 / 32 is one).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "launch.cuh"
#include "ptx.cuh"
#include "q4_format.cuh"

namespace ds4l {

using namespace ds4;
using namespace ds4q;

constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t scale_code(float absmax) {
  const float y = __fdiv_rn(absmax, 7.f);
  const uint32_t u = __float_as_uint(y);
  // exponent and the top three fraction bits: 8 (E + 20) + m; below 0: clamped
  int32_t c = static_cast<int32_t>(u >> 20) - 8 * (127 - 20);
  const uint32_t low = u & 0xFFFFFu;
  const float rem = fmaf(-7.f, y, absmax);
  const bool up = low > 0x80000u || (low == 0x80000u && (rem > 0.f || (rem == 0.f && (c & 1))));
  c += up ? 1 : 0;
  return static_cast<uint32_t>(min(255, max(0, c)));
}

// Eight values to their word. k = round(x / s) is proposed by one fma (x * (1 / s) + 1.5 * 2^23
// rounds the exact product to an integer); the remainder x - k s is exact, and where it passes half
// a scale, or equals it at an odd k, k moves one step towards it. Nibbles are collected in fp32
// (exact: below 2^16), which leaves the half-rate integer pipe to the comparisons; with rintf and
// integer conversions, which run at a quarter of its rate, a call took twice as long.
// h and h_up: half a scale and the next fp32 above it.
__device__ __forceinline__ uint32_t pack_word(const float* x, float s, float r, float h, float h_up) {
  constexpr float kMagic = 12582912.f;
  float f[2] = {8388608.f + 34952.f, 8388608.f + 34952.f};  // 2^23, and 8 in each nibble
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float z = fmaf(x[j], r, kMagic);
    float k = z - kMagic;
    const float e = fmaf(-k, s, x[j]);
    const float limit = (__float_as_uint(z) & 1u) ? h : h_up;
    if (fabsf(e) >= limit) k += copysignf(1.f, e);
    f[j & 1] = fmaf(k, static_cast<float>(1 << (4 * (j >> 1))), f[j & 1]);
  }
  return __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x5410);
}

// One row's inputs of a lane: 16 dims of its group and two rotary ones.
template <bool kBf16>
struct RowIn {
  float4 v[kBf16 ? 2 : 4];  // raw bits for bf16
  float2 rope;
  int64_t dst;

  __device__ __forceinline__ void load(const void* x, int64_t row, int lane) {
    if constexpr (kBf16) {
      const uint16_t* src = static_cast<const uint16_t*>(x) + row * kRowDims;
      v[0] = *(reinterpret_cast<const float4*>(src + lane * 16));
      v[1] = *(reinterpret_cast<const float4*>(src + lane * 16) + 1);
      rope.x = *(reinterpret_cast<const float*>(src + kLatent) + lane);
    } else {
      const float* src = static_cast<const float*>(x) + row * kRowDims;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *(reinterpret_cast<const float4*>(src + lane * 16) + j);
      rope = *(reinterpret_cast<const float2*>(src + kLatent) + lane);
    }
  }
  __device__ __forceinline__ void store(uint8_t* cache, int lane) const {
    float x[16];
    uint32_t rp;
    if constexpr (kBf16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = __float_as_uint((&v[0].x)[j]);
        x[2 * j] = __uint_as_float(w << 16);
        x[2 * j + 1] = __uint_as_float(w & 0xFFFF0000u);
      }
      rp = __float_as_uint(rope.x);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = (&v[0].x)[j];
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(rp) : "f"(rope.y), "f"(rope.x));
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(x[j]));
    const uint32_t code = scale_code(m);
    const float s = scale_f32(code), r = __frcp_rn(s), h = 0.5f * s;
    // A nearest scale leaves |x / s| <= 7 * 17 / 16, which rounds to 7 with or without the clamp;
    // past the largest scale it is needed.
    if (!(m <= 7.25f * s)) {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = fminf(7.f * s, fmaxf(-7.f * s, x[j]));
    }
    const float h_up = __uint_as_float(__float_as_uint(h) + 1);
    uint8_t* out = cache + dst * kRowBytes;
    *reinterpret_cast<uint2*>(out + lane * 8) =
        make_uint2(pack_word(x, s, r, h, h_up), pack_word(x + 8, s, r, h, h_up));
    out[kOffScale + lane] = static_cast<uint8_t>(code);
    reinterpret_cast<uint32_t*>(out + kOffRope)[lane] = rp;
  }
};

// Two rows a warp at a time, their loads in flight together.
constexpr int kWriteRows = 2;

template <bool kBf16>
__global__ void __launch_bounds__(kWarps * 32, 4) quantize_latents_kernel(
    const void* x, int64_t n, const int64_t* slots, int64_t dst_offset, uint8_t* cache,
    int64_t cache_rows) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kWriteRows;
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kWriteRows;
       r0 < n; r0 += step) {
    RowIn<kBf16> in[kWriteRows];
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      in[i].dst = -1;
      if (r0 + i >= n) break;
      in[i].load(x, r0 + i, lane);
      in[i].dst = slots ? slots[r0 + i] : dst_offset + r0 + i;
    }
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i)
      if (in[i].dst >= 0 && in[i].dst < cache_rows) in[i].store(cache, lane);
  }
}

// Four rows a warp at a time.
constexpr int kReadRows = 4;

template <bool kBf16>
__global__ void __launch_bounds__(kWarps * 32, 4) read_latents_kernel(
    const uint8_t* cache, int64_t cache_rows, const int64_t* rows, int64_t start, int64_t n,
    void* out) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kReadRows;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kReadRows;
       i0 < n; i0 += step) {
    uint2 w[kReadRows];
    uint32_t code[kReadRows], rope[kReadRows];
#pragma unroll
    for (int j = 0; j < kReadRows; ++j) {
      w[j] = make_uint2(kEmptyWord, kEmptyWord);
      code[j] = rope[j] = 0;
      if (i0 + j >= n) break;
      const int64_t r = rows ? rows[i0 + j] : start + i0 + j;
      if (r >= 0 && r < cache_rows) {
        const uint8_t* src = cache + r * kRowBytes;
        w[j] = *reinterpret_cast<const uint2*>(src + lane * 8);
        code[j] = src[kOffScale + lane];
        rope[j] = reinterpret_cast<const uint32_t*>(src + kOffRope)[lane];
      }
    }
#pragma unroll
    for (int j = 0; j < kReadRows; ++j) {
      if (i0 + j >= n) break;
      const uint32_t s2 = scale_bf16x2(code[j]), c2 = offset_bf16x2(s2);
      const uint4 a = word_to_bf16(w[j].x, s2, c2), b = word_to_bf16(w[j].y, s2, c2);
      if constexpr (kBf16) {
        uint16_t* dst = static_cast<uint16_t*>(out) + (i0 + j) * kRowDims;
        reinterpret_cast<uint4*>(dst + lane * 16)[0] = a;
        reinterpret_cast<uint4*>(dst + lane * 16)[1] = b;
        reinterpret_cast<uint32_t*>(dst + kLatent)[lane] = rope[j];
      } else {
        float* dst = static_cast<float*>(out) + (i0 + j) * kRowDims;
        const uint32_t p[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<float4*>(dst + lane * 16)[q] = make_float4(
              __uint_as_float(p[2 * q] << 16), __uint_as_float(p[2 * q] & 0xFFFF0000u),
              __uint_as_float(p[2 * q + 1] << 16), __uint_as_float(p[2 * q + 1] & 0xFFFF0000u));
        reinterpret_cast<float2*>(dst + kLatent)[lane] =
            make_float2(__uint_as_float(rope[j] << 16), __uint_as_float(rope[j] & 0xFFFF0000u));
      }
    }
  }
}

// A warp for every `rows` rows (65536 rows: 43 us written and read back; CTAs that stay and loop
// over rows, eight an SM, take 48).
unsigned ctas(int64_t n, int rows) {
  return static_cast<unsigned>(std::min<int64_t>((n + kWarps * rows - 1) / (kWarps * rows), 1 << 30));
}

}  // namespace ds4l

extern "C" int ds4idx_quantize_latents(const void* x, int32_t in_dtype, int64_t n,
                                       const int64_t* slots, int64_t dst_offset, uint8_t* cache,
                                       int64_t cache_rows, void* stream) {
  using namespace ds4l;
  if ((in_dtype != DS4IDX_BF16 && in_dtype != DS4IDX_F32) || n < 0 || cache_rows < 0)
    return DS4IDX_ERR_INVALID_ARG;
  if (!slots && (dst_offset < 0 || dst_offset > cache_rows || n > cache_rows - dst_offset))
    return DS4IDX_ERR_INVALID_ARG;
  if (n == 0) return DS4IDX_OK;
  if (!x || !cache || !aligned_to(x, 16) || !aligned_to(cache, 32) || !aligned_to(slots, 8))
    return DS4IDX_ERR_INVALID_ARG;
  return launch_dependent(in_dtype == DS4IDX_BF16 ? quantize_latents_kernel<true>
                                                  : quantize_latents_kernel<false>,
                          ctas(n, kWriteRows), kWarps * 32, 0, 1, stream, x, n, slots, dst_offset, cache,
                          cache_rows);
}

extern "C" int ds4idx_read_latents(const uint8_t* cache, int64_t cache_rows, const int64_t* rows,
                                   int64_t start, int64_t n, void* out, int32_t out_dtype,
                                   void* stream) {
  using namespace ds4l;
  if ((out_dtype != DS4IDX_BF16 && out_dtype != DS4IDX_F32) || n < 0 || cache_rows < 0)
    return DS4IDX_ERR_INVALID_ARG;
  if (!rows && (start < 0 || start > cache_rows || n > cache_rows - start))
    return DS4IDX_ERR_INVALID_ARG;
  if (n == 0) return DS4IDX_OK;
  if (!out || !cache || !aligned_to(out, 16) || !aligned_to(cache, 32) || !aligned_to(rows, 8))
    return DS4IDX_ERR_INVALID_ARG;
  return launch_dependent(out_dtype == DS4IDX_BF16 ? read_latents_kernel<true>
                                                   : read_latents_kernel<false>,
                          ctas(n, kReadRows), kWarps * 32, 0, 1, stream, cache, cache_rows, rows, start, n,
                          out);
}
