// Attention of a tree of drafted tokens over a latent cache: every node of a sequence attends over all
// of the sequence's rows and over the drafted rows on its own path.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "f8_format.cuh"
#include "launch.cuh"
#include "placement.cuh"
#include "ptx.cuh"
#include "q4_format.cuh"

namespace ds4ta {

using namespace ds4;

constexpr int kDims = 576, kLatent = 512, kNodes = 64, kMaxHeads = 128;
constexpr int kRows = 16, kKeys = 16, kThreads = 256;
constexpr int kSmem = 2 * 16 * kDims * 4;
constexpr float kMax = __FLT_MAX__, kNegInf = -__builtin_inff();

struct Params {
  const uint16_t* q;
  const uint8_t* cache;
  const float* scale;
  const int32_t* lens;
  const int64_t* mask;
  uint16_t* out;
  float* lse;
  Placement place;
  int32_t format, N, H;
  float scale_log2;
};

__device__ __forceinline__ float bf16_to_f32(uint32_t u) { return __uint_as_float(u << 16); }

__device__ float value(const Params& p, int64_t r, int d) {
  if (p.format == DS4IDX_CACHE_BF16)
    return bf16_to_f32(reinterpret_cast<const uint16_t*>(p.cache)[r * kDims + d]);
  if (p.format == DS4IDX_CACHE_FP8) {
    const uint8_t* row = p.cache + r * ds4f8::kRowBytes;
    if (d >= kLatent) return bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[d - kLatent + 256]);
    uint32_t lo, hi;
    ds4f8::codes_to_f16(row[d], lo, hi);
    return ds4f8::f16x2_to_f32(lo).x * p.scale[r];
  }
  const uint8_t* row = p.cache + r * ds4q::kRowBytes;
  if (d >= kLatent)
    return bf16_to_f32(reinterpret_cast<const uint16_t*>(row + ds4q::kOffRope)[d - kLatent]);
  const int nib = (d % 8) / 2 + 4 * (d % 2);
  const int u = (row[(d / 8) * 4 + nib / 2] >> (4 * (nib % 2))) & 15;
  return (u - 8) * ds4q::scale_f32(row[ds4q::kOffScale + d / 16]);
}

__global__ void __launch_bounds__(kThreads) tree_attn_kernel(const __grid_constant__ Params p) {
  extern __shared__ float smem[];
  float* sq = smem;
  float* sk = smem + kRows * kDims;
  __shared__ float sp[kRows][kKeys], scorr[kRows], sl[kRows];
  griddep_wait();
  griddep_launch_dependents();
  const int groups = (p.H + kRows - 1) / kRows, tid = threadIdx.x;
  const int h0 = blockIdx.x % groups * kRows;
  const int64_t node = blockIdx.x / groups;
  const int b = static_cast<int>(node / p.N);
  const uint64_t bits = static_cast<uint64_t>(p.mask[node]);
  const TokenPlace tp = place_token(p.place, b);
  const int64_t len = min(max(p.lens[b], 0), 0x7FFFFFFF - kNodes);
  int64_t room = tp.table ? static_cast<int64_t>(p.place.pages) * p.place.page
                          : (tp.row0 < 0 ? 0 : max(p.place.rows - tp.row0, static_cast<int64_t>(0)));
  const int64_t n = bits ? min(len + p.N, room) : 0;
  for (int i = tid; i < kRows * kDims; i += kThreads) {
    const int h = h0 + i / kDims;
    sq[i] = h < p.H ? bf16_to_f32(p.q[(node * p.H + h) * kDims + i % kDims]) : 0.f;
  }
  const int h = tid / 16, k = tid % 16;
  float m = kNegInf, l = 0.f, acc[2][kRows] = {};
  bool any = false;
  for (int64_t s0 = 0; s0 < n; s0 += kKeys) {
    __syncthreads();
    bool seen = false;
    for (int j = 0; j < kKeys; ++j) {
      const int64_t s = s0 + j;
      const int64_t r = s < n && (s < len || (bits >> (s - len) & 1))
                            ? place_row(p.place, tp, static_cast<int32_t>(s)) : -1;
      for (int d = tid; d < kDims; d += kThreads) sk[j * kDims + d] = r >= 0 ? value(p, r, d) : 0.f;
      if (j == k) seen = r >= 0;
    }
    __syncthreads();
    float s = 0.f;
    for (int d = 0; d < kDims; ++d) s = fmaf(sq[h * kDims + d], sk[k * kDims + d], s);
    s *= p.scale_log2;
    float mt = seen ? s : kNegInf;
    for (int o = 8; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    any |= (__ballot_sync(0xffffffffu, seen) & (0xFFFFu << (tid & 16))) != 0;
    const float m_new = any ? fminf(fmaxf(fmaxf(m, mt), -kMax), kMax) : m;
    const float corr = any ? exp2f(m - m_new) : 1.f;
    const float pr = seen ? exp2f(s - m_new) : 0.f;
    float sum = pr;
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * corr + sum;
    m = m_new;
    sp[h][k] = pr;
    if (k == 0) scorr[h] = corr;
    __syncthreads();
    for (int r = 0; r < kRows; ++r)
      for (int e = 0; e < 2; ++e) {
        float a = acc[e][r] * scorr[r];
        for (int j = 0; j < kKeys; ++j) a = fmaf(sp[r][j], sk[j * kDims + tid + e * 256], a);
        acc[e][r] = a;
      }
  }
  if (k == 0) sl[h] = any ? l : kMax;
  if (k == 0 && h0 + h < p.H && p.lse)
    p.lse[node * p.H + h0 + h] = any ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
  __syncthreads();
  for (int r = 0; r < kRows; ++r)
    for (int e = 0; e < 2; ++e)
      if (h0 + r < p.H) {
        uint32_t v;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(0.f), "f"(acc[e][r] / sl[r]));
        p.out[(node * p.H + h0 + r) * kLatent + tid + e * 256] = static_cast<uint16_t>(v);
      }
}

int64_t workspace_bytes(int32_t, int32_t, int32_t, int64_t) { return 0; }

bool sizes_ok(int32_t B, int32_t N, int32_t H, int64_t max_kv_len) {
  return B >= 0 && N >= 1 && N <= kNodes && H >= 1 && H <= kMaxHeads && max_kv_len >= 0 &&
         max_kv_len <= 0x7FFFFFFF && static_cast<int64_t>(B) * N * H <= 0x7FFFFFFF / kMaxHeads;
}

}  // namespace ds4ta

extern "C" int ds4idx_tree_attention_workspace(int32_t B, int32_t n_nodes, int32_t n_heads,
                                               int64_t max_kv_len, int64_t* bytes) {
  using namespace ds4ta;
  if (!bytes || !sizes_ok(B, n_nodes, n_heads, max_kv_len)) return DS4IDX_ERR_INVALID_ARG;
  *bytes = workspace_bytes(B, n_nodes, n_heads, max_kv_len);
  return DS4IDX_OK;
}

extern "C" int ds4idx_tree_attention(const void* q, int32_t format, const void* cache,
                                     const float* scale, int64_t kv_rows, const int32_t* kv_lens,
                                     const int64_t* mask, const ds4idx_placement* where, int32_t B,
                                     int32_t n_nodes, int32_t n_heads, int32_t d_qk, int32_t d_v,
                                     int64_t max_kv_len, float sm_scale, void* out, float* lse,
                                     void* workspace, int64_t workspace_size, void* stream) {
  using namespace ds4ta;
  if (d_qk != kDims || d_v != kLatent) return DS4IDX_ERR_UNSUPPORTED;
  if (!sizes_ok(B, n_nodes, n_heads, max_kv_len) || kv_rows < 1 || kv_rows > 0x7FFFFFFF ||
      format < DS4IDX_CACHE_BF16 || format > DS4IDX_CACHE_Q4 || !(sm_scale > 0.f) ||
      !(sm_scale < 1e30f) || (format == DS4IDX_CACHE_FP8) != (scale != nullptr))
    return DS4IDX_ERR_INVALID_ARG;
  if (B == 0) return DS4IDX_OK;
  const int64_t need = workspace_bytes(B, n_nodes, n_heads, max_kv_len);
  Params p{};
  if (!q || !cache || !kv_lens || !mask || !out || !aligned_to(q, 16) || !aligned_to(cache, 32) ||
      !aligned_to(scale, 4) || !aligned_to(kv_lens, 4) || !aligned_to(mask, 8) ||
      !aligned_to(out, 16) || !aligned_to(lse, 4) || workspace_size < need ||
      (need > 0 && (!workspace || !aligned_to(workspace, 16))) ||
      !make_placement(where, kv_rows, B, &p.place))
    return DS4IDX_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.scale = scale;
  p.lens = kv_lens;
  p.mask = mask;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.format = format;
  p.N = n_nodes;
  p.H = n_heads;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  static std::atomic<uint64_t> done{0};
  if (!allow_shared(tree_attn_kernel, kSmem, done)) return DS4IDX_ERR_CUDA;
  const int64_t grid = static_cast<int64_t>(B) * n_nodes * ((n_heads + kRows - 1) / kRows);
  return launch_dependent(tree_attn_kernel, static_cast<unsigned>(grid), kThreads, kSmem, 1, stream, p);
}
