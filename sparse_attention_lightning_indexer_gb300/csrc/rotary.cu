// Rotary positions for sm_103a: every pair (a, b) of a rotated slice turns by the angle of its
// token's position, y = m (a cos - b sin, a sin + b cos), angle = position * frequency[pair]. Up
// to four tensors of the same tokens (the attention's query and key, the indexer's query and key)
// are rotated by one launch, each in its own layout: interleaved pairs (2i, 2i + 1) or halves
// (i, i + rot_dim / 2). The inverse rotation (angle negated, same m) is the transpose, hence the
// gradient.
//
// Angles. A frequency is kept as a 64-bit fraction of a turn, f = round(inv_freq / 2pi * 2^64), so
// the angle modulo one turn is the low 64 bits of position * f: one integer product, exact in the
// wrap. What is left is |position| times the error of f: 2^-65 turn from its rounding, and that of the
// double formula, a few 2^-53 of it (5.9 measured; the header has the bound). The two top bits give
// the quadrant; the rest, within an eighth of a turn, is converted to fp32 (relative error 2^-24) for
// sincospi.
//
// Bound by HBM (each rotated element read and written once) for chunks and by latency for decode. A
// bf16 chunk of 4095 tokens takes 42.5 us; its floor is 30.5, a copy of the same 128-byte pieces takes
// 33.5, so the pieces account for a quarter of the distance.
// A CTA takes one token and a share of its 16-byte items: the first loads are in flight while 32
// to 128 of its threads compute the token's cosines and sines, once for all heads and tensors.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "launch.cuh"
#include "overlap.h"
#include "ptx.cuh"

namespace ds4r {

using namespace ds4;

constexpr int kMaxTensors = 4;
constexpr int kMaxPairs = 128;
constexpr int kThreads = 256;
constexpr int kBatch = 3;  // items a thread has in flight (chunk of 4095: 2 45 us, 3 43 us, 4 at 3 CTAs an SM 55 us)

struct Tensor {
  const uint8_t* x;
  uint8_t* out;
  int64_t xt, xh, ot, oh;   // strides in bytes
  int32_t items;            // items of one token
  int32_t per_head;         // items of one head
  int32_t mode;             // bit 0: fp32, bit 1: interleaved, bit 2: 16-byte items (else one pair)
};
struct Params {
  Tensor t[kMaxTensors];
  const int64_t* positions;
  int32_t n, pairs, total;  // total: items of one token in all tensors
  float scale, sign;
  uint64_t freq[kMaxPairs];
};

// One item: four 32-bit words from each of up to two places. Interleaved items take one 16-byte
// piece; half-layout items take one from each half; scalar items take one pair.
struct Item {
  const uint8_t* src;
  uint8_t* dst;
  int32_t pair, mode;
  uint4 a, b;
};

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void turn(float a, float b, float2 cs, float& u, float& v) {
  u = a * cs.x - b * cs.y;
  v = a * cs.y + b * cs.x;
}
__device__ __forceinline__ void turn2(uint32_t wa, uint32_t wb, float2 c0, float2 c1, uint32_t& ua,
                                      uint32_t& ub) {
  float u0, v0, u1, v1;
  turn(lo_bf16(wa), lo_bf16(wb), c0, u0, v0);
  turn(hi_bf16(wa), hi_bf16(wb), c1, u1, v1);
  ua = pack_bf16(u0, u1);
  ub = pack_bf16(v0, v1);
}
__device__ __forceinline__ uint32_t turn_pair(uint32_t w, float2 c) {
  float u, v;
  turn(lo_bf16(w), hi_bf16(w), c, u, v);
  return pack_bf16(u, v);
}
__device__ __forceinline__ void turn_f32(uint32_t& a, uint32_t& b, float2 c) {
  float u, v;
  turn(__uint_as_float(a), __uint_as_float(b), c, u, v);
  a = __float_as_uint(u);
  b = __float_as_uint(v);
}

__global__ void __launch_bounds__(kThreads, 5) rotary_kernel(const __grid_constant__ Params p,
                                                          int32_t shares) {
  __shared__ float2 s_cs[kMaxPairs];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x / shares;
  const int share = blockIdx.x % shares;
  const int first = static_cast<int>(static_cast<int64_t>(p.total) * share / shares);
  const int last = static_cast<int>(static_cast<int64_t>(p.total) * (share + 1) / shares);

  auto load = [&](int i, Item& it) {
    int k = 0;
    while (k + 1 < p.n && i >= p.t[k].items) i -= p.t[k++].items;
    const Tensor& q = p.t[k];
    const int head = i / q.per_head, c = i - head * q.per_head;
    const int elem = (q.mode & 1) ? 4 : 2;                // bytes of an element
    const bool inter = q.mode & 2, vec = q.mode & 4;
    const int step = vec ? 16 : (inter ? 2 * elem : elem);  // bytes of an item's (first) piece
    it.mode = q.mode;
    it.pair = vec ? (inter ? c * (8 / elem) : c * (16 / elem)) : c;
    it.src = q.x + t * q.xt + head * q.xh + static_cast<int64_t>(c) * step;
    it.dst = q.out + t * q.ot + head * q.oh + static_cast<int64_t>(c) * step;
    const int half = p.pairs * elem;
    if (vec) {
      it.a = *reinterpret_cast<const uint4*>(it.src);
      if (!inter) it.b = *reinterpret_cast<const uint4*>(it.src + half);
    } else {
      const uint8_t* sb = it.src + (inter ? elem : half);
      if (q.mode & 1) {
        it.a.x = *reinterpret_cast<const uint32_t*>(it.src);
        it.b.x = *reinterpret_cast<const uint32_t*>(sb);
      } else {
        it.a.x = *reinterpret_cast<const uint16_t*>(it.src);
        it.b.x = *reinterpret_cast<const uint16_t*>(sb);
      }
    }
  };
  auto store = [&](Item& it) {
    const bool f32 = it.mode & 1, inter = it.mode & 2, vec = it.mode & 4;
    const float2* cs = s_cs + it.pair;
    const int half = p.pairs * (f32 ? 4 : 2);
    if (!vec) {
      uint8_t* db = it.dst + (inter ? (f32 ? 4 : 2) : half);
      float u, v;
      if (f32) {
        turn(__uint_as_float(it.a.x), __uint_as_float(it.b.x), cs[0], u, v);
        *reinterpret_cast<float*>(it.dst) = u;
        *reinterpret_cast<float*>(db) = v;
      } else {
        turn(lo_bf16(it.a.x), lo_bf16(it.b.x), cs[0], u, v);
        const uint32_t w = pack_bf16(u, v);
        *reinterpret_cast<uint16_t*>(it.dst) = static_cast<uint16_t>(w);
        *reinterpret_cast<uint16_t*>(db) = static_cast<uint16_t>(w >> 16);
      }
      return;
    }
    if (inter) {
      if (f32) {
        turn_f32(it.a.x, it.a.y, cs[0]);
        turn_f32(it.a.z, it.a.w, cs[1]);
      } else {
        it.a = make_uint4(turn_pair(it.a.x, cs[0]), turn_pair(it.a.y, cs[1]),
                          turn_pair(it.a.z, cs[2]), turn_pair(it.a.w, cs[3]));
      }
      *reinterpret_cast<uint4*>(it.dst) = it.a;
      return;
    }
    if (f32) {
      turn_f32(it.a.x, it.b.x, cs[0]);
      turn_f32(it.a.y, it.b.y, cs[1]);
      turn_f32(it.a.z, it.b.z, cs[2]);
      turn_f32(it.a.w, it.b.w, cs[3]);
    } else {
      turn2(it.a.x, it.b.x, cs[0], cs[1], it.a.x, it.b.x);
      turn2(it.a.y, it.b.y, cs[2], cs[3], it.a.y, it.b.y);
      turn2(it.a.z, it.b.z, cs[4], cs[5], it.a.z, it.b.z);
      turn2(it.a.w, it.b.w, cs[6], cs[7], it.a.w, it.b.w);
    }
    *reinterpret_cast<uint4*>(it.dst) = it.a;
    *reinterpret_cast<uint4*>(it.dst + half) = it.b;
  };

  Item it[kBatch];
  int base = first + threadIdx.x;
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (base + j * kThreads < last) load(base + j * kThreads, it[j]);
  if (threadIdx.x < p.pairs) {
    const uint64_t phase = static_cast<uint64_t>(p.positions[t]) * p.freq[threadIdx.x];
    const uint64_t quad = (phase + (1ull << 61)) >> 62;  // nearest quarter turn
    const int64_t rest = static_cast<int64_t>(phase - (quad << 62));
    float s, c;
    sincospif(__ll2float_rn(rest) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    const float cq = (quad & 1) ? -s : c, sq = (quad & 1) ? c : s;
    const float flip = (quad & 2) ? -p.scale : p.scale;
    s_cs[threadIdx.x] = make_float2(cq * flip, sq * flip * p.sign);
  }
  __syncthreads();
  while (true) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (base + j * kThreads < last) store(it[j]);
    base += kBatch * kThreads;
    if (base >= last) break;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (base + j * kThreads < last) load(base + j * kThreads, it[j]);
  }
}

}  // namespace ds4r

extern "C" int ds4idx_rotary_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                                   int64_t original_max_position, double beta_fast,
                                   double beta_slow, uint64_t* freqs, float* scale) {
  constexpr double kPi = 3.14159265358979323846;
  if (rot_dim < 2 || rot_dim > 2 * ds4r::kMaxPairs || rot_dim % 2 || !freqs || !scale ||
      !(base > 1.0) || !std::isfinite(base))
    return DS4IDX_ERR_INVALID_ARG;
  if (scaling < DS4IDX_ROTARY_PLAIN || scaling > DS4IDX_ROTARY_YARN) return DS4IDX_ERR_INVALID_ARG;
  if (scaling != DS4IDX_ROTARY_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
    return DS4IDX_ERR_INVALID_ARG;
  if (scaling == DS4IDX_ROTARY_YARN &&
      !(original_max_position >= 1 && beta_slow > 0.0 && beta_fast >= beta_slow &&
        std::isfinite(beta_fast)))
    return DS4IDX_ERR_INVALID_ARG;
  // YaRN (Peng et al. 2023): pairs that turn more than beta_fast times over the original context
  // keep their frequency, those below beta_slow turns are divided by the factor, a linear ramp
  // over the pair index joins them; cosines and sines are scaled by 0.1 ln(factor) + 1.
  double low = 0.0, high = 0.0;
  if (scaling == DS4IDX_ROTARY_YARN) {
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(static_cast<double>(original_max_position) / (2.0 * kPi * turns)) /
             (2.0 * std::log(base));
    };
    low = std::max(std::floor(pair_of(beta_fast)), 0.0);
    high = std::min(std::ceil(pair_of(beta_slow)), static_cast<double>(rot_dim - 1));
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == DS4IDX_ROTARY_LINEAR) {
      f /= factor;
    } else if (scaling == DS4IDX_ROTARY_YARN) {
      const double r = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      f = f * (1.0 - r) + f / factor * r;
    }
    freqs[i] = static_cast<uint64_t>(std::rint(std::ldexp(f / (2.0 * kPi), 64)));  // below 2^62
  }
  *scale = scaling == DS4IDX_ROTARY_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return DS4IDX_OK;
}

extern "C" int ds4idx_rotary(int32_t n_tensors, const ds4idx_rotary_tensor* tensors, int64_t T,
                             int32_t rot_dim, const int64_t* positions, const uint64_t* freqs,
                             float scale, int32_t inverse, void* stream) {
  using namespace ds4r;
  if (n_tensors < 1 || n_tensors > kMaxTensors || !tensors || T < 0 || T > 0x7FFFFFFF ||
      rot_dim < 2 || rot_dim > 2 * kMaxPairs || rot_dim % 2 || !freqs || !(scale > 0.f) ||
      !std::isfinite(scale))
    return DS4IDX_ERR_INVALID_ARG;
  Params p{};
  p.n = n_tensors;
  p.pairs = rot_dim / 2;
  p.scale = scale;
  p.sign = inverse ? -1.f : 1.f;
  p.positions = positions;
  std::copy(freqs, freqs + p.pairs, p.freq);
  int64_t total = 0;
  for (int k = 0; k < n_tensors; ++k) {
    const ds4idx_rotary_tensor& d = tensors[k];
    if ((d.dtype != DS4IDX_BF16 && d.dtype != DS4IDX_F32) || d.n_heads < 1 || d.n_heads > 65536)
      return DS4IDX_ERR_INVALID_ARG;
    const int elem = d.dtype == DS4IDX_F32 ? 4 : 2;
    if (T > 0 && (!d.x || !d.out || !aligned_to(d.x, elem) || !aligned_to(d.out, elem)))
      return DS4IDX_ERR_INVALID_ARG;
    Tensor& q = p.t[k];
    q.x = static_cast<const uint8_t*>(d.x);
    q.out = static_cast<uint8_t*>(d.out);
    q.xt = d.x_stride_t * elem;
    q.xh = d.x_stride_h * elem;
    q.ot = d.out_stride_t * elem;
    q.oh = d.out_stride_h * elem;
    // 16-byte items where every item of both tensors starts on 16 bytes and is whole; otherwise
    // (odd strides or widths) one pair an item, which moves the same bytes in 2- or 4-byte pieces.
    const int run = (d.interleaved ? rot_dim : rot_dim / 2) * elem;
    const uint64_t steps = static_cast<uint64_t>(q.xt | q.ot) |
                           (d.n_heads > 1 ? static_cast<uint64_t>(q.xh | q.oh) : 0ull);
    const bool vec = run % 16 == 0 && aligned_to(d.x, 16) && aligned_to(d.out, 16) &&
                     (steps & 15u) == 0;
    q.per_head = vec ? run / 16 : p.pairs;
    q.items = q.per_head * d.n_heads;
    q.mode = (d.dtype == DS4IDX_F32 ? 1 : 0) | (d.interleaved ? 2 : 0) | (vec ? 4 : 0);
    total += q.items;
  }
  if (T == 0) return DS4IDX_OK;
  if (!positions || !aligned_to(positions, 8) || total > (1 << 24)) return DS4IDX_ERR_INVALID_ARG;
  // A CTA reads some items before and some after another writes its own: outputs that share bytes
  // with each other or with an input (other than in place) would depend on that order.
  Pieces x[kMaxTensors], out[kMaxTensors];
  for (int k = 0; k < n_tensors; ++k) {
    const ds4idx_rotary_tensor& d = tensors[k];
    const int64_t width = static_cast<int64_t>(rot_dim) * (d.dtype == DS4IDX_F32 ? 4 : 2);
    x[k] = Pieces(d.x, T, p.t[k].xt, d.n_heads, p.t[k].xh, width);
    out[k] = Pieces(d.out, T, p.t[k].ot, d.n_heads, p.t[k].oh, width);
  }
  for (int k = 0; k < n_tensors; ++k) {
    if (overlaps_itself(out[k])) return DS4IDX_ERR_INVALID_ARG;
    for (int j = 0; j < n_tensors; ++j)
      if ((j > k && overlap(out[k], out[j])) ||
          (!(j == k && same(out[k], x[k])) && overlap(out[k], x[j])))
        return DS4IDX_ERR_INVALID_ARG;
  }
  p.total = static_cast<int32_t>(total);
  // Few tokens: split a token's items over CTAs until about two CTAs an SM are busy, each with at
  // least a load a thread. Many tokens: as few CTAs a token as keep kBatch loads a thread.
  const int64_t most = std::max<int64_t>(1, (total + kThreads - 1) / kThreads);
  const int64_t sms = sm_count();
  if (sms == 0) return DS4IDX_ERR_CUDA;
  const int64_t fill = std::min<int64_t>(most, std::max<int64_t>(1, 2 * sms / T));
  const int64_t least = (total + kBatch * kThreads - 1) / (kBatch * kThreads);
  const int64_t shares = std::max<int64_t>(1, std::max(fill, least));
  if (shares * T > 0x7FFFFFFF) return DS4IDX_ERR_INVALID_ARG;
  return launch_dependent(rotary_kernel, static_cast<unsigned>(shares * T), kThreads, 0, 1, stream,
                          p, static_cast<int32_t>(shares));
}
