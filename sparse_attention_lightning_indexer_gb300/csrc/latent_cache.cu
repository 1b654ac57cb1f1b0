// The 4-bit latent cache's writer and reader (format: q4_format.cuh). Both are HBM streams: a row
// is one warp, a lane one group of 16 dims (its absmax needs no other lane) and two rotary dims.
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

__device__ __forceinline__ uint32_t code_of(float x, float s, float r) {
  const float y = fminf(8.f, fmaxf(-8.f, x * r));
  float k = rintf(y);
  const float e = fmaf(-k, s, x), d = fabsf(e) - 0.5f * s;
  if (d > 0.f || (d == 0.f && (static_cast<int>(k) & 1))) k += copysignf(1.f, e);
  return static_cast<uint32_t>(min(7, max(-7, static_cast<int>(k))) + 8);
}

__device__ __forceinline__ uint32_t pack_word(const float* x, float s, float r) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) w |= code_of(x[j], s, r) << (4 * (j >> 1) + 16 * (j & 1));
  return w;
}

template <bool kBf16>
__global__ void __launch_bounds__(kWarps * 32) quantize_latents_kernel(
    const void* x, int64_t n, const int64_t* slots, int64_t dst_offset,
    uint8_t* cache, int64_t cache_rows) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < n;
       row += warps) {
    const int64_t dst = slots ? slots[row] : dst_offset + row;
    float v[16];
    uint32_t rope;
    if (kBf16) {
      const uint16_t* src = static_cast<const uint16_t*>(x) + row * kRowDims;
      uint4 a[2];
      a[0] = *(reinterpret_cast<const uint4*>(src + lane * 16));
      a[1] = *(reinterpret_cast<const uint4*>(src + lane * 16) + 1);
      rope = *(reinterpret_cast<const uint32_t*>(src + kLatent) + lane);
      const uint32_t w[8] = {a[0].x, a[0].y, a[0].z, a[0].w, a[1].x, a[1].y, a[1].z, a[1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
      const float* src = static_cast<const float*>(x) + row * kRowDims;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 f = *(reinterpret_cast<const float4*>(src + lane * 16) + j);
        v[4 * j] = f.x;
        v[4 * j + 1] = f.y;
        v[4 * j + 2] = f.z;
        v[4 * j + 3] = f.w;
      }
      const float2 f = *(reinterpret_cast<const float2*>(src + kLatent) + lane);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(rope) : "f"(f.y), "f"(f.x));
    }
    if (dst < 0 || dst >= cache_rows) continue;
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(v[j]));
    const uint32_t code = scale_code(m);
    const float s = scale_f32(code), r = __frcp_rn(s);
    uint8_t* out = cache + dst * kRowBytes;
    *reinterpret_cast<uint2*>(out + lane * 8) = make_uint2(pack_word(v, s, r), pack_word(v + 8, s, r));
    out[kOffScale + lane] = static_cast<uint8_t>(code);
    reinterpret_cast<uint32_t*>(out + kOffRope)[lane] = rope;
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kWarps * 32) read_latents_kernel(
    const uint8_t* cache, int64_t cache_rows, const int64_t* rows,
    int64_t start, int64_t n, void* out) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < n;
       i += warps) {
    const int64_t r = rows ? rows[i] : start + i;
    uint2 w = make_uint2(kEmptyWord, kEmptyWord);
    uint32_t code = 0, rope = 0;
    if (r >= 0 && r < cache_rows) {
      const uint8_t* src = cache + r * kRowBytes;
      w = *reinterpret_cast<const uint2*>(src + lane * 8);
      code = src[kOffScale + lane];
      rope = reinterpret_cast<const uint32_t*>(src + kOffRope)[lane];
    }
    const uint32_t s2 = scale_bf16x2(code), c2 = offset_bf16x2(s2);
    const uint4 a = word_to_bf16(w.x, s2, c2), b = word_to_bf16(w.y, s2, c2);
    if (kBf16) {
      uint16_t* dst = static_cast<uint16_t*>(out) + i * kRowDims;
      reinterpret_cast<uint4*>(dst + lane * 16)[0] = a;
      reinterpret_cast<uint4*>(dst + lane * 16)[1] = b;
      reinterpret_cast<uint32_t*>(dst + kLatent)[lane] = rope;
    } else {
      float* dst = static_cast<float*>(out) + i * kRowDims;
      const uint32_t p[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4*>(dst + lane * 16)[j] = make_float4(
            __uint_as_float(p[2 * j] << 16), __uint_as_float(p[2 * j] & 0xFFFF0000u),
            __uint_as_float(p[2 * j + 1] << 16), __uint_as_float(p[2 * j + 1] & 0xFFFF0000u));
      reinterpret_cast<float2*>(dst + kLatent)[lane] =
          make_float2(__uint_as_float(rope << 16), __uint_as_float(rope & 0xFFFF0000u));
    }
  }
}

// A row a warp while that gives every SM at most eight CTAs; longer calls loop.
unsigned ctas(int64_t n) {
  return static_cast<unsigned>(std::min<int64_t>((n + kWarps - 1) / kWarps, 152 * 8));
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
                          ctas(n), kWarps * 32, 0, 1, stream, x, n, slots, dst_offset, cache,
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
                          ctas(n), kWarps * 32, 0, 1, stream, cache, cache_rows, rows, start, n,
                          out);
}
