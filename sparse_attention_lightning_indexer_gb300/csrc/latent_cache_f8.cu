// The 8-bit latent cache's writer and reader (format: f8_format.cuh): a row is one warp, a lane 16
// adjacent dims and two rotary ones. Both are streams of rows: bound by HBM. A warp has the loads of two rows
// (the reader four) in flight before it uses the first. Measured on the device, partly out of L2: 262144 bf16
// rows written in 66.3 us, 7.10 TB/s, and read in 69.4, 6.78; fp32 rows 106.8 us, 7.24 TB/s, and 113.3, 6.82
// (157 with 16 adjacent dims a lane, whose stores leave gaps of 48 bytes); 65536 bf16 rows both ways
// 37.0 us, 8 rows 3.0.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "f8_format.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace ds4lf {

using namespace ds4;
using namespace ds4f8;

constexpr int kWarps = 8;

// The least e of -24 .. 7 with absmax <= 448 * 2^e (7 where none is): 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(uint32_t absmax) {
  const int e = static_cast<int>(absmax >> 23) - 127 - 8 + ((absmax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(kMaxExp, max(kMinExp, e));
}
__device__ __forceinline__ float power(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}
// Four values to their codes: round to nearest, ties to even, saturated at +-448.
__device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

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
  // All lanes of the warp together.
  __device__ __forceinline__ void store(uint8_t* cache, float* scale, int lane) const {
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
    // magnitudes of fp32 order like their bits
    const int e = scale_exp(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    const float r = power(-e);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = codes(x[4 * j] * r, x[4 * j + 1] * r, x[4 * j + 2] * r, x[4 * j + 3] * r);
    uint8_t* out = cache + dst * kRowBytes;
    reinterpret_cast<uint4*>(out)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
    reinterpret_cast<uint32_t*>(out + kOffRope)[lane] = rp;
    if (lane == 0) scale[dst] = power(e);
  }
};

// Rows a warp takes at a time, their loads in flight together.
constexpr int kWriteRows = 2, kReadRows = 4;

template <bool kBf16>
__global__ void __launch_bounds__(kWarps * 32, 4) quantize_latents_fp8_kernel(
    const void* x, int64_t n, const int64_t* slots, int64_t dst_offset, uint8_t* cache, float* scale,
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
      if (in[i].dst >= 0 && in[i].dst < cache_rows) in[i].store(cache, scale, lane);
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kWarps * 32, 4) read_latents_fp8_kernel(
    const uint8_t* cache, const float* scale, int64_t cache_rows, const int64_t* rows, int64_t start,
    int64_t n, void* out) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kReadRows;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kReadRows;
       i0 < n; i0 += step) {
    uint4 w[kReadRows];
    float s[kReadRows];
    uint32_t rope[kReadRows];
#pragma unroll
    for (int j = 0; j < kReadRows; ++j) {
      w[j] = make_uint4(0, 0, 0, 0);
      s[j] = 0.f;
      rope[j] = 0;
      if (i0 + j >= n) break;
      const int64_t r = rows ? rows[i0 + j] : start + i0 + j;
      if (r >= 0 && r < cache_rows) {
        const uint8_t* src = cache + r * kRowBytes;
        if constexpr (kBf16) {
          w[j] = reinterpret_cast<const uint4*>(src)[lane];
        } else {  // word k: dims 128 k + 4 lane .., so that a store of four values a lane covers whole lines
#pragma unroll
          for (int k = 0; k < 4; ++k) (&w[j].x)[k] = reinterpret_cast<const uint32_t*>(src)[32 * k + lane];
        }
        rope[j] = reinterpret_cast<const uint32_t*>(src + kOffRope)[lane];
        s[j] = scale[r];
      }
    }
#pragma unroll
    for (int j = 0; j < kReadRows; ++j) {
      if (i0 + j >= n) break;
      float v[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t lo, hi;
        codes_to_f16((&w[j].x)[k], lo, hi);
        const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
        v[4 * k] = a.x * s[j];
        v[4 * k + 1] = a.y * s[j];
        v[4 * k + 2] = b.x * s[j];
        v[4 * k + 3] = b.y * s[j];
      }
      if constexpr (kBf16) {
        uint16_t* dst = static_cast<uint16_t*>(out) + (i0 + j) * kRowDims;
        uint32_t p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[k]) : "f"(v[2 * k + 1]), "f"(v[2 * k]));
        reinterpret_cast<uint4*>(dst + lane * 16)[0] = make_uint4(p[0], p[1], p[2], p[3]);
        reinterpret_cast<uint4*>(dst + lane * 16)[1] = make_uint4(p[4], p[5], p[6], p[7]);
        reinterpret_cast<uint32_t*>(dst + kLatent)[lane] = rope[j];
      } else {
        float* dst = static_cast<float*>(out) + (i0 + j) * kRowDims;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          reinterpret_cast<float4*>(dst)[32 * k + lane] =
              make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        reinterpret_cast<float2*>(dst + kLatent)[lane] =
            make_float2(__uint_as_float(rope[j] << 16), __uint_as_float(rope[j] & 0xFFFF0000u));
      }
    }
  }
}

unsigned ctas(int64_t n, int rows) {
  return static_cast<unsigned>(std::min<int64_t>((n + kWarps * rows - 1) / (kWarps * rows), 1 << 30));
}

}  // namespace ds4lf

extern "C" int ds4idx_quantize_latents_fp8(const void* x, int32_t in_dtype, int64_t n,
                                           const int64_t* slots, int64_t dst_offset, uint8_t* cache,
                                           float* scale, int64_t cache_rows, void* stream) {
  using namespace ds4lf;
  if ((in_dtype != DS4IDX_BF16 && in_dtype != DS4IDX_F32) || n < 0 || cache_rows < 0)
    return DS4IDX_ERR_INVALID_ARG;
  if (!slots && (dst_offset < 0 || dst_offset > cache_rows || n > cache_rows - dst_offset))
    return DS4IDX_ERR_INVALID_ARG;
  if (n == 0) return DS4IDX_OK;
  if (!x || !cache || !scale || !aligned_to(x, 16) || !aligned_to(cache, 32) ||
      !aligned_to(scale, 4) || !aligned_to(slots, 8))
    return DS4IDX_ERR_INVALID_ARG;
  return launch_dependent(in_dtype == DS4IDX_BF16 ? quantize_latents_fp8_kernel<true>
                                                  : quantize_latents_fp8_kernel<false>,
                          ctas(n, kWriteRows), kWarps * 32, 0, 1, stream, x, n, slots, dst_offset, cache,
                          scale, cache_rows);
}

extern "C" int ds4idx_read_latents_fp8(const uint8_t* cache, const float* scale, int64_t cache_rows,
                                       const int64_t* rows, int64_t start, int64_t n, void* out,
                                       int32_t out_dtype, void* stream) {
  using namespace ds4lf;
  if ((out_dtype != DS4IDX_BF16 && out_dtype != DS4IDX_F32) || n < 0 || cache_rows < 0)
    return DS4IDX_ERR_INVALID_ARG;
  if (!rows && (start < 0 || start > cache_rows || n > cache_rows - start))
    return DS4IDX_ERR_INVALID_ARG;
  if (n == 0) return DS4IDX_OK;
  if (!out || !cache || !scale || !aligned_to(out, 16) || !aligned_to(cache, 32) ||
      !aligned_to(scale, 4) || !aligned_to(rows, 8))
    return DS4IDX_ERR_INVALID_ARG;
  return launch_dependent(out_dtype == DS4IDX_BF16 ? read_latents_fp8_kernel<true>
                                                   : read_latents_fp8_kernel<false>,
                          ctas(n, kReadRows), kWarps * 32, 0, 1, stream, cache, scale, cache_rows, rows,
                          start, n, out);
}
