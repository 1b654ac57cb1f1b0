// Attention of a tree of drafted tokens over a latent cache, for sm_103a: every node of a sequence
// attends over all of the sequence's rows and over the drafted rows on its own path. One latent row per
// position, shared by all heads; 576-wide keys, the first 512 dims are values.
//
// The (node, head) rows of a sequence are taken 128 at a time (the lanes of TMEM). O of 128 rows x 512
// dims fills an SM's TMEM, so a pair of CTAs owns such a tile and a range of keys: one (rank 0) the
// keys' products and the softmax, the other the values' products:
//   S[128 x 64 keys] = Q K^T        rank 0; Q stays in TMEM as the A operand, three tiles of S beside it
//   p = exp2(s - m) in bf16         rank 0; m is left alone until a score passes it by 64
//   O[128 x 512] += P V             rank 1; O fills its TMEM over the whole range
// P, and the factors of O where m was raised, are all that goes from one CTA to the other (16 KB a tile;
// shared memory of the pair moves 18.7 bytes a clock in each direction when all SMs do it). A tile
// takes both CTAs about as long: 36 x 32 and 8 x 128 clocks of products. Splitting the dims instead
// reads and unpacks a row once in the pair, but exchanges S, 32 KB a tile both ways: slower.
// Ranges of a split sequence leave (O, m, l) in fp32, and a second kernel joins them.
//
// Both CTAs read the rows themselves and turn them into bf16 (exact) in a ring of parts, 64 keys x 256
// dims in the 128-byte-swizzled layout that serves as K-major and as MN-major operand.
//
// Warps 0..3: softmax, a row a thread (rank 1: the rescaling of O and the output). Warps 4..11: rows to
// operands. Warp 12 issues tcgen05.mma.
//
// 8-bit rows are f16 in the key product: E4M3 to f16 is one conversion for two values, to bf16 five
// instructions. The row's scale is applied to S, the rotary dims (bf16) are divided by it before, and Q is
// scaled by a power of two to f16's range: all exact, but for what of a row of Q lies 2^38 below its largest
// value. As values they are bf16 (P times the scales would leave f16's range).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "attn_ptx.cuh"
#include "f8_format.cuh"
#include "launch.cuh"
#include "placement.cuh"
#include "ptx.cuh"
#include "q4_format.cuh"

namespace ds4a {
extern uint32_t* sparse_attention_error_word();  // device address of the shared error word
}

namespace ds4ta {

using namespace ds4;

constexpr int kDims = 576, kLatent = 512, kNodes = 64, kMaxHeads = 128;
constexpr int kRows = 128;             // (node, head) rows of a tile = TMEM lanes
constexpr int kKeys = 64;              // keys of a step
constexpr int kHalf = 256;             // latent dims of a part
constexpr int kLoad0 = 4, kLoaders = 8, kMmaWarp = 12;
constexpr int kThreads = 13 * 32;
constexpr int kChunk = kKeys * 128;    // 64 dims of a tile's keys
constexpr int kPart = 4 * kChunk, kParts = 5;
constexpr int kOffRope = kParts * kPart;           // the rotary dims of three tiles' keys (rank 0)
constexpr int kOffP = kOffRope + 3 * kChunk, kP = kRows * kKeys * 2;  // P of two tiles
constexpr int kOffF = kOffP + 2 * kP;              // float [2][128]: factors of O before P V
constexpr int kOffL = kOffF + 2 * kRows * 4;       // float [2][128]: l, m (rank 1)
constexpr int kOffScale = kOffL + 2 * kRows * 4;   // float [8 tiles][64]: scales of the keys (8-bit rows)
constexpr int kOffThere = kOffScale + 8 * kKeys * 4;  // uint32 [8 tiles][2]: keys that are there
constexpr int kOffOdd = kOffThere + 8 * 8;         // uint32 [8 tiles][8 chunks][2]: keys not finite
constexpr int kOffBars = kOffOdd + 8 * 64;
constexpr int kNumBars = 2 * kParts + 1 + 2 * 3 + 4 * 2 + 2;
constexpr int kOffMisc = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffMisc + 16 + 1024;
static_assert(kSmem <= 232448 && kOffBars % 8 == 0, "shared memory");
constexpr uint32_t kColRope = 256, kColS = 320;    // rank 0: Q from column 0, S; rank 1: O from 0
constexpr float kNegInf = -__builtin_inff(), kMax = __FLT_MAX__;
// log2 of what exp2(s - m) may be before m is raised. P and the sums are floating point with 2^127 of
// range, so a stale m costs no precision: 2^64 leaves 2^63 for the count and size of the values. (With 2^8
// some row of 128 raised m in most of the first hundred tiles; a rescaling holds P V up for 4000 clocks,
// and 4 sequences of 64 nodes over 16384 rows took 2.05 ms.)
constexpr float kSlack = 64.f;

struct Params {
  const uint16_t* q;
  const uint8_t* cache;
  const float* scale;
  const int32_t* lens;
  const int64_t* mask;
  uint16_t* out;
  float* lse;
  float* part_o;   // [item][128 column quads][128 rows][4]
  float* part_ml;  // [item][2][128]
  uint32_t* err;
  Placement place;
  int32_t N, H, tiles, splits, steps;  // row tiles a sequence, key ranges, least steps of a range
  float scale_log2;
};

// The range of keys of a work item: steps lo .. lo + n - 1 of 64 positions.
struct Range {
  int32_t len, end;  // rows of the sequence; positions from `end` on are not there
  int32_t lo, n;
  uint64_t seen;     // drafted rows that some node of the tile sees
};

// What every warp works out for itself (warp-uniform): one pass over the tile's masks.
__device__ __forceinline__ Range make_range(const Params& p, int b, int tile, int split, int lane) {
  Range g;
  g.len = min(max(p.lens[b], 0), 0x7FFFFFFF - kNodes);
  const int first = tile * kRows / p.H, last = min(p.N - 1, (tile * kRows + kRows - 1) / p.H);
  uint32_t lo = 0, hi = 0;
  for (int i = first + lane; i <= last; i += 32) {
    const uint64_t m = static_cast<uint64_t>(p.mask[static_cast<int64_t>(b) * p.N + i]);
    lo |= static_cast<uint32_t>(m);
    hi |= static_cast<uint32_t>(m >> 32);
  }
  lo = __reduce_or_sync(0xffffffffu, lo);
  hi = __reduce_or_sync(0xffffffffu, hi);
  const bool any = (lo | hi) != 0u;
  g.seen = (static_cast<uint64_t>(hi) << 32 | lo) & (~0ull >> (64 - p.N));
  const TokenPlace tp = place_token(p.place, b);
  int64_t room = static_cast<int64_t>(p.place.pages) * p.place.page;
  if (!tp.table) room = tp.row0 < 0 ? 0 : p.place.rows - tp.row0;
  const int32_t end = g.len + (64 - __clzll(static_cast<long long>(g.seen)));
  g.end = any ? static_cast<int32_t>(max(min(static_cast<int64_t>(end), room), static_cast<int64_t>(0)))
              : 0;
  const int32_t total = g.end / kKeys + (g.end % kKeys ? 1 : 0);
  const int32_t per = max(p.steps, (total - 1) / p.splits + 1);
  g.lo = static_cast<int32_t>(min(static_cast<int64_t>(total), static_cast<int64_t>(split) * per));
  g.n = min(total - g.lo, per);
  return g;
}

__device__ __forceinline__ void st_peer(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void copy_to_peer(uint32_t dst, uint32_t src, uint32_t bytes,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

// ---- reading rows: what one thread takes of a key, chunk c of 64 dims and, in rank 0, 8 rotary ones,
// raw; unpacked as 8 x 16 bytes of bf16.
template <int kFormat>
struct RowPart {
  static constexpr int kWords = kFormat == DS4IDX_CACHE_BF16 ? 32 : kFormat == DS4IDX_CACHE_FP8 ? 16 : 8;
  uint32_t w[kWords];
  uint32_t scale;
  uint4 rope;

  __device__ __forceinline__ void load(const Params& p, int64_t r, int c, bool rotary) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = kFormat == DS4IDX_CACHE_Q4 ? ds4q::kEmptyWord : 0u;
    scale = 0u;
    rope = make_uint4(0, 0, 0, 0);
    if (r < 0) return;
    const uint8_t* row;
    int at, rot;
    if constexpr (kFormat == DS4IDX_CACHE_BF16) {
      row = p.cache + r * (2 * kDims);
      at = c * 128;
      rot = 2 * kLatent;
    } else if constexpr (kFormat == DS4IDX_CACHE_FP8) {
      row = p.cache + r * ds4f8::kRowBytes;
      at = c * 64;
      rot = ds4f8::kOffRope;
      scale = __float_as_uint(p.scale[r]);
    } else {
      row = p.cache + r * ds4q::kRowBytes;
      at = c * 32;
      rot = ds4q::kOffRope;
      scale = *reinterpret_cast<const uint32_t*>(row + ds4q::kOffScale + 4 * c);
    }
#pragma unroll
    for (int j = 0; j < kWords; j += 8) ld32(row + at + 4 * j, reinterpret_cast<uint32_t(&)[8]>(w[j]));
    if (rotary) rope = *reinterpret_cast<const uint4*>(row + rot + c * 16);
  }
  // Whether a value is not finite (the 4-bit format has none).
  __device__ __forceinline__ bool odd() const {
    bool bad = false;
    if constexpr (kFormat == DS4IDX_CACHE_BF16) {
#pragma unroll
      for (int j = 0; j < kWords; ++j)
        bad |= (w[j] & 0x7F80u) == 0x7F80u || (w[j] & 0x7F800000u) == 0x7F800000u;
    } else if constexpr (kFormat == DS4IDX_CACHE_FP8) {
      bad = (scale & 0x7F800000u) == 0x7F800000u;
#pragma unroll
      for (int j = 0; j < kWords; ++j)
        bad |= __vcmpeq4(w[j] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
    }
    return bad;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = kFormat == DS4IDX_CACHE_Q4 ? ds4q::kEmptyWord : 0u;
    scale = 0u;
  }
  // Four E4M3 codes to bf16: sign and magnitude bits to a bf16's places give value * 2^-120 (bf16's
  // exponent bias is 120 larger), one packed product with scale * 2^120 the value, exactly.
  __device__ __forceinline__ static void unpack(uint32_t c, uint32_t s2, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = __byte_perm(c, 0, 0x1404), b = __byte_perm(c, 0, 0x3424);
    lo = ds4q::mul_bf16x2((a & 0x80008000u) | ((a >> 4) & 0x07F007F0u), s2);
    hi = ds4q::mul_bf16x2((b & 0x80008000u) | ((b >> 4) & 0x07F007F0u), s2);
  }
  // To row `key` of a chunk in shared memory; 8-bit rows in f16 without their scale, or in bf16.
  __device__ __forceinline__ void store(uint32_t chunk, int key, bool f16) const {
    const uint32_t at = chunk + key * 128 + (key & 7) * 16;
    uint32_t s2 = 0;
    if constexpr (kFormat == DS4IDX_CACHE_FP8) s2 = ((scale >> 23) + 120u) * 0x00800080u;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint4 v;
      if constexpr (kFormat == DS4IDX_CACHE_BF16) {
        v = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
      } else if constexpr (kFormat == DS4IDX_CACHE_FP8) {
        if (f16) {
          ds4f8::codes_to_f16(w[2 * u], v.x, v.y);
          ds4f8::codes_to_f16(w[2 * u + 1], v.z, v.w);
        } else {
          unpack(w[2 * u], s2, v.x, v.y);
          unpack(w[2 * u + 1], s2, v.z, v.w);
        }
      } else {
        const int g = u >> 1;
        const uint32_t q2 = __byte_perm(scale, 0, 0x4040u | (g << 8) | g) * 16u + 0x35803580u;
        v = ds4q::word_to_bf16(w[u], q2, ds4q::offset_bf16x2(q2));
      }
      st_shared16(at ^ (16 * u), v);
    }
  }
};

// A range's sum may be far above 1, as its m is stale: its power of two goes into the m that the ranges
// are joined by (0 for a sum of nothing, infinite or NaN).
__device__ __forceinline__ int excess(float l) {
  const int e = static_cast<int>(__float_as_uint(l) >> 23);
  return e == 0 || e >= 255 ? 0 : e - 127;
}
__device__ __forceinline__ float power(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// Two bf16 to two f16, times a power of two.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v, float f) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;"
      : "=r"(d)
      : "f"(__uint_as_float(v & 0xFFFF0000u) * f), "f"(__uint_as_float(v << 16) * f));
  return d;
}

template <int kFormat>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  // both CTAs of a pair have the same dynamic shared-memory base, so the offsets agree
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t smem0 = smem_u32(smem);
  float* s_f = reinterpret_cast<float*>(smem + kOffF);
  float* s_l = reinterpret_cast<float*>(smem + kOffL);
  float* s_scale = reinterpret_cast<float*>(smem + kOffScale);
  volatile uint32_t* s_there = reinterpret_cast<uint32_t*>(smem + kOffThere);
  volatile uint32_t* s_odd = reinterpret_cast<uint32_t*>(smem + kOffOdd);
  uint64_t* part_full = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* part_empty = part_full + kParts;
  uint64_t* q_full = part_empty + kParts;
  uint64_t* s_ready = q_full + 1;   // [3] S of a tile is formed
  uint64_t* s_free = s_ready + 3;   // [3] and read
  uint64_t* p_free = s_free + 3;    // [2] rank 1 is done with P (in rank 0)
  uint64_t* p_full = p_free + 2;    // [2] P has come (in rank 1)
  uint64_t* scaled = p_full + 2;    // [2] O is ready for P V
  uint64_t* pv_done = scaled + 2;   // [2] P V of a tile is done
  uint64_t* l_full = pv_done + 2;   // the rows' sums have come (in rank 1)
  uint64_t* done = l_full + 1;      // every MMA has completed
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile uint32_t* s_abort = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1, item = blockIdx.x >> 1;
  const int split = item % p.splits, tile = item / p.splits % p.tiles, b = item / (p.splits * p.tiles);
  uint32_t* err = p.err;
  constexpr uint32_t kPBytes = kP + kRows * 4;  // what comes with a tile: P and the factors

  if (tid == 0) {
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&part_full[i], kLoaders);
      mbar_init(&part_empty[i], 1);
    }
    mbar_init(q_full, 4);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&s_ready[i], 1);
      mbar_init(&s_free[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_free[i], 4);
      mbar_init(&p_full[i], 1);
      mbar_init(&scaled[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(l_full, 4);
    mbar_init(done, 1);
    *s_abort = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  const Range g = make_range(p, b, tile, split, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  constexpr bool kF16 = kFormat == DS4IDX_CACHE_FP8;  // the key product's type

  if (warp < kLoad0) {
    const int r = tid;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int row = tile * kRows + r, node = row / p.H;
    const bool used = node < p.N;
    const int64_t out_row = static_cast<int64_t>(b) * p.N * p.H + row;
    bool ok = true;
    if (rank == 0) {
      // ---------------- softmax: this thread's row
      uint64_t mask = used ? static_cast<uint64_t>(p.mask[static_cast<int64_t>(b) * p.N + node]) : 0ull;
      const bool padding = mask == 0ull;
      mask &= ~0ull >> (64 - p.N);
      float to_log2 = p.scale_log2;  // of a score, from S
      if (g.n > 0) {
        // Q to TMEM
        const uint4* src = reinterpret_cast<const uint4*>(p.q + out_row * kDims);
        const uint4 zero = make_uint4(0, 0, 0, 0);
        float f = 1.f;
        uint32_t f2 = 0;
        if constexpr (kF16) {
          // the power of two that takes the row's largest value to 2^13 .. 2^14
          uint32_t top = 0;
#pragma unroll 8
          for (int j = 0; j < kDims / 8; ++j) {
            const uint4 x = used ? src[j] : zero;
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                         __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
          }
          const int e = static_cast<int>(max(top & 0xFFFFu, top >> 16) >> 7);   // biased by 127
          const int a = max(-110, min(110, e == 0 ? 0 : 127 + 13 - e));         // (zero: any)
          f = __uint_as_float(static_cast<uint32_t>(127 + a) << 23);
          f2 = static_cast<uint32_t>(127 + a) * 0x00800080u;
          to_log2 *= __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
        }
#pragma unroll 1
        for (int h = 0; h < 8; ++h) {
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 x = used ? src[8 * h + j] : zero;
            v[4 * j] = x.x;
            v[4 * j + 1] = x.y;
            v[4 * j + 2] = x.z;
            v[4 * j + 3] = x.w;
          }
          if constexpr (kF16) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = bf16x2_to_f16x2(v[j], f);
          }
          tmem_st32(lanes + h * 32, v);
        }
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 x = used ? src[64 + j] : zero;
          v[4 * j] = x.x;
          v[4 * j + 1] = x.y;
          v[4 * j + 2] = x.z;
          v[4 * j + 3] = x.w;
        }
        if constexpr (kF16) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = ds4q::mul_bf16x2(v[j], f2);
        }
        tmem_st32(lanes + kColRope, v);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      float m = kNegInf, l = 0.f;
      const uint32_t rows_at = warp * 32 * 128;  // this warp's rows of P
      int slot = 0;                              // i % 3
      uint32_t s_parity = 0;
#pragma unroll 1
      for (int i = 0; i < g.n; ++i) {
        ok = mbar_wait_warp(&s_ready[slot], s_parity, s_abort, err);
        if (!ok) break;
        tc_fence_after();
        float s[kKeys];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          tmem_ld32(lanes + kColS + slot * kKeys + 32 * h, reinterpret_cast<uint32_t(&)[32]>(s[32 * h]));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[slot]);
        if (++slot == 3) slot = 0, s_parity ^= 1u;
        const int at = i & 7;
        if constexpr (kF16) {
          const float4* sc = reinterpret_cast<const float4*>(s_scale + at * kKeys);
#pragma unroll
          for (int j = 0; j < kKeys / 4; ++j) {
            const float4 x = sc[j];
            s[4 * j] *= x.x;
            s[4 * j + 1] *= x.y;
            s[4 * j + 2] *= x.z;
            s[4 * j + 3] *= x.w;
          }
        }
        // which keys this row sees
        const int32_t left = g.len - (g.lo + i) * kKeys;  // rows of the sequence from this tile on
        uint64_t see = padding ? 0ull : ~0ull;
        if (left < kKeys) {
          if (!padding)
            see = left >= 0 ? ((1ull << left) - 1ull) | mask << left : left > -64 ? mask >> -left : 0ull;
          uint64_t bad = 0ull;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            bad |= static_cast<uint64_t>(s_odd[16 * at + 2 * c + 1]) << 32 | s_odd[16 * at + 2 * c];
          if (bad) {
#pragma unroll
            for (int j = 0; j < kKeys; ++j)
              if (bad >> j & 1) s[j] = __uint_as_float(0x7FC00000u);
          }
        }
        see &= static_cast<uint64_t>(s_there[2 * at + 1]) << 32 | s_there[2 * at];
        const bool all = __all_sync(0xffffffffu, see == ~0ull);
        float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
        if (all) {
#pragma unroll
          for (int j = 0; j < kKeys; j += 2) mx[j / 2 & 3] = fmaxf(fmaxf(mx[j / 2 & 3], s[j]), s[j + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < kKeys; ++j) {
            if (see >> j & 1) mx[j & 3] = fmaxf(mx[j & 3], s[j]);
          }
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * to_log2;
        // m is raised where a score passes it by more than the slack. Finite once a key was seen: a
        // score of +-infinity keeps its meaning in s - m.
        float f = 1.f;
        if (see != 0ull && (m == kNegInf || top > m + kSlack)) {
          const float now = fminf(fmaxf(top, -kMax), kMax);
          if (m != kNegInf) {
            f = exp2_approx(0.5f * (m - now));  // its square: what is 2^64 above m may matter 2^-126
            l = l * f * f;                      // above the new one, where 2^(m - now) is long zero
          }
          m = now;
        }
        // P, in the layout of an MMA A operand, and the root of the factor of the O before it
        const int ps = i & 1;
        ok = __all_sync(0xffffffffu, wait_cluster(&p_free[ps], (i >> 1 & 1) ^ 1u, s_abort, err));
        if (!ok) break;
        s_f[ps * kRows + r] = f;
        const uint32_t p_at = smem0 + kOffP + ps * kP + r * 128 + (r & 7) * 16;
        const float off = m == kNegInf ? 0.f : m;  // (a row that has seen nothing: p = 0 below)
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint32_t pk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = 8 * u + 2 * j;
            float p0 = exp2_approx(fmaf(s[k], to_log2, -off));
            float p1 = exp2_approx(fmaf(s[k + 1], to_log2, -off));
            if (!all) {
              p0 = see >> k & 1 ? p0 : 0.f;
              p1 = see >> (k + 1) & 1 ? p1 : 0.f;
            }
            sum[0] += p0;
            sum[1] += p1;
            pk[j] = pack_bf16x2(p0, p1);
          }
          st_shared16(p_at ^ (16 * u), make_uint4(pk[0], pk[1], pk[2], pk[3]));
        }
        l += sum[0] + sum[1];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = peer(smem_u32(&p_full[ps]), 1);
          const uint32_t from = smem0 + kOffP + ps * kP + rows_at;
          copy_to_peer(peer(from, 1), from, 32 * 128, bar);
          const uint32_t f_at = smem_u32(s_f + ps * kRows + warp * 32);
          copy_to_peer(peer(f_at, 1), f_at, 128, bar);
        }
        __syncwarp();
      }
      // ---------------- the rows' sums, to rank 1
      st_peer(peer(smem_u32(s_l + r), 1), l);
      st_peer(peer(smem_u32(s_l + kRows + r), 1), m);
      __syncwarp();
      if (lane == 0) arrive_peer(peer(smem_u32(l_full), 1));
      if (p.splits > 1) {
        const int k = excess(l);
        p.part_ml[static_cast<int64_t>(item) * 2 * kRows + r] = m + static_cast<float>(k);
        p.part_ml[static_cast<int64_t>(item) * 2 * kRows + kRows + r] = l * power(-k);
      } else if (used && p.lse) {
        p.lse[out_row] = m == kNegInf ? kNegInf : (m + __log2f(l)) * 0.69314718055994531f;
      }
    } else {
      // ---------------- O: rescaled where m was raised, at the end written
      uint32_t seen = 0;  // P tiles that have come
      if (tid == 0)
        for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&p_full[i], kPBytes);
#pragma unroll 1
      for (int i = 0; i < g.n; ++i) {
        const int slot = i & 1;
        const uint32_t parity = (i >> 1) & 1;
        ok = mbar_wait_warp(&p_full[slot], parity, s_abort, err);
        if (!ok) break;
        ++seen;
        const float f = s_f[slot * kRows + r];
        if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {  // (P V of the tile before was waited for)
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kLatent; c += 32) {
            uint32_t v[32];
            tmem_ld32(lanes + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f * f);
            tmem_st32(lanes + c, v);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scaled[slot]);
        ok = mbar_wait_warp(&pv_done[slot], parity, s_abort, err);
        if (!ok) break;
        if (tid == 0 && i + 2 < g.n) mbar_arrive_expect_tx(&p_full[slot], kPBytes);
        __syncwarp();
        if (lane == 0) arrive_peer(peer(smem_u32(&p_free[slot]), 0));
      }
      // never leave with copies in flight to here (after an abort: bounded)
      if (!ok && tid == 0)
        for (uint32_t i = seen; i < min(seen + 2, static_cast<uint32_t>(g.n)); ++i)
          mbar_drain(&p_full[i & 1], (i >> 1) & 1);
      __syncwarp();
      ok = __all_sync(0xffffffffu, wait_cluster(l_full, 0u, s_abort, err)) && ok;
      tc_fence_after();
      const float l = s_l[r];
      const bool none = s_l[kRows + r] == kNegInf;
      if (p.splits == 1) {
        const float inv = none ? 0.f : 1.f / l;
        uint16_t* dst = p.out + out_row * kLatent;
#pragma unroll 1
        for (int c = 0; c < kLatent; c += 32) {
          uint32_t v[32], pk[16];
          if (g.n > 0) {
            tmem_ld32(lanes + c, v);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            pk[j / 2] =
                none ? 0u : pack_bf16x2(__uint_as_float(v[j]) * inv, __uint_as_float(v[j + 1]) * inv);
          if (used && ok) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              reinterpret_cast<uint4*>(dst + c)[j] =
                  make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          }
        }
      } else if (g.n > 0 && ok) {
        const float f = power(-excess(l));
        float4* dst =
            reinterpret_cast<float4*>(p.part_o) + static_cast<int64_t>(item) * 128 * kRows + r;
#pragma unroll 1
        for (int c = 0; c < kLatent; c += 32) {
          uint32_t v[32];
          tmem_ld32(lanes + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[(c / 4 + j) * kRows] =
                make_float4(__uint_as_float(v[4 * j]) * f, __uint_as_float(v[4 * j + 1]) * f,
                            __uint_as_float(v[4 * j + 2]) * f, __uint_as_float(v[4 * j + 3]) * f);
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ---------------- rows to bf16: one (key, chunk of 64 dims) a thread in each half of the dims
    const int w = warp - kLoad0, key = (w & 1) * 32 + lane, c = w >> 1;
    const TokenPlace tp = place_token(p.place, b);
    auto row_of = [&](int i) -> int32_t {
      const int32_t s = (g.lo + i) * kKeys + key;
      if (i >= g.n || s >= g.end || (s >= g.len && !(g.seen >> (s - g.len) & 1))) return -1;
      return static_cast<int32_t>(place_row(p.place, tp, s));
    };
    RowPart<kFormat> part[2];                  // reads in flight, of each half the next
    int32_t row = row_of(0), next = row_of(1);  // of the tile that is read, and of the one after it
    bool ok = true;
    int st = 0;           // place in the ring
    uint32_t parity = 1;  // of its part_empty
    int rope = 0;         // i % 3
    auto put = [&](int i, int h, const int32_t here, RowPart<kFormat>& x) {
      ok = mbar_wait_warp(&part_empty[st], parity, s_abort, err);
      if (!ok) return;
      // A drafted row that some rows of the tile see and others do not may hold values that are not
      // finite: cleared, since 0 * NaN would reach all of O, and its scores become NaN instead.
      const int32_t left = g.len - (g.lo + i) * kKeys;
      if (left < kKeys) {
        const bool odd = key >= left && x.odd();
        const uint32_t bits = __ballot_sync(0xffffffffu, odd);
        if (odd) x.clear();
        if (lane == 0) s_odd[16 * (i & 7) + 2 * (4 * h + c) + (w & 1)] = bits;
      }
      if (c == 0 && h == 0) {
        const uint32_t bits = __ballot_sync(0xffffffffu, here >= 0);
        if (lane == 0) s_there[2 * (i & 7) + (w & 1)] = bits;
        if (kF16) s_scale[(i & 7) * kKeys + key] = __uint_as_float(x.scale);
      }
      if (rank == 0) {
        x.store(smem0 + st * kPart + c * kChunk, key, kF16);
        uint4 v = x.rope;
        if constexpr (kF16) {  // divided by the scale
          const uint32_t s2 = (254u - (x.scale >> 23)) * 0x00800080u;
          v = make_uint4(ds4q::mul_bf16x2(v.x, s2), ds4q::mul_bf16x2(v.y, s2), ds4q::mul_bf16x2(v.z, s2),
                         ds4q::mul_bf16x2(v.w, s2));
        }
        st_shared16(smem0 + kOffRope + rope * kChunk + key * 128 + (((4 * h + c) ^ key) & 7) * 16, v);
      } else {
        x.store(smem0 + st * kPart + c * kChunk, key, false);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&part_full[st]);
      if (++st == kParts) st = 0, parity ^= 1u;
    };
    part[0].load(p, row, c, rank == 0);
    part[1].load(p, row, 4 + c, rank == 0);
#pragma unroll 1
    for (int i = 0; i < g.n; ++i) {
      const int32_t here = row;
      row = next;
      next = row_of(i + 2);
      put(i, 0, here, part[0]);
      if (!ok) break;
      part[0].load(p, row, c, rank == 0);
      put(i, 1, here, part[1]);
      if (!ok) break;
      part[1].load(p, row, 4 + c, rank == 0);
      if (++rope == 3) rope = 0;
    }
  } else {
      // ---------------- MMA issue: the warp waits together, one elected lane issues
      const bool lead = elect_one();
      bool ok = true;
      int st = 0;
      uint32_t parity = 0;  // of part_full
      auto commit = [&](uint64_t* bar) {
        if (lead) mma_commit(bar);
      };
      auto part_ready = [&] {
        ok = ok && mbar_wait_warp(&part_full[st], parity, s_abort, err);
        tc_fence_after();
      };
      auto part_taken = [&] {
        commit(&part_empty[st]);
        if (++st == kParts) st = 0, parity ^= 1u;
      };
      if (rank == 0) {
        const uint64_t k0 = smem_desc_sw128(smem0), r0 = smem_desc_sw128(smem0 + kOffRope);
        constexpr uint32_t rope_idesc = instr_desc(1u, 1u, kRows, kKeys);
        constexpr uint32_t idesc = kF16 ? instr_desc(0u, 0u, kRows, kKeys) : rope_idesc;
        if (g.n > 0) ok = mbar_wait_warp(q_full, 0u, s_abort, err);
        int slot = 0;
        uint32_t s_parity = 1;
#pragma unroll 1
        for (int i = 0; ok && i < g.n; ++i) {
          ok = mbar_wait_warp(&s_free[slot], s_parity, s_abort, err);
          const uint32_t d = tmem + kColS + slot * kKeys;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            part_ready();
            if (!ok) break;
            const uint64_t kd = k0 + st * (kPart >> 4);
            if (lead) {
#pragma unroll
              for (int k = 0; k < kHalf / 16; ++k)
                mma_bf16_ts(d, tmem + h * 128 + k * 8, kd + (k >> 2) * (kChunk >> 4) + (k & 3) * 2, idesc,
                            (h | k) ? 1u : 0u);
            }
            if (h == 1 && lead) {
              const uint64_t rd = r0 + slot * (kChunk >> 4);  // (i % 3 = slot)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16_ts(d, tmem + kColRope + k * 8, rd + 2 * k, rope_idesc, 1u);
            }
            part_taken();
          }
          if (!ok) break;
          commit(&s_ready[slot]);
          if (++slot == 3) slot = 0, s_parity ^= 1u;
        }
      } else {
        const uint64_t p0 = smem_desc_sw128(smem0 + kOffP), v0 = smem_desc_mn_sw128(smem0, kChunk);
        constexpr uint32_t idesc = instr_desc(1u, 1u, kRows, kHalf) | (1u << 16);  // B MN-major
#pragma unroll 1
        for (int i = 0; ok && i < g.n; ++i) {
          const int slot = i & 1;
          ok = mbar_wait_warp(&p_full[slot], (i >> 1) & 1, s_abort, err);
          if (!ok) break;
          const float4 f = reinterpret_cast<const float4*>(s_f + slot * kRows)[lane];
          if (__any_sync(0xffffffffu, f.x != 1.f || f.y != 1.f || f.z != 1.f || f.w != 1.f))
            ok = mbar_wait_warp(&scaled[slot], (i >> 1) & 1, s_abort, err);
          const uint64_t pd = p0 + slot * (kP >> 4);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            part_ready();
            if (!ok) break;
            const uint64_t vd = v0 + st * (kPart >> 4);
            if (lead) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16(tmem + h * kHalf, pd + 2 * k, vd + k * (16 * 128 >> 4), idesc, (i | k) ? 1u : 0u);
            }
            part_taken();
          }
          commit(&pv_done[slot]);
        }
      }
      // every MMA has completed before TMEM is released (bounded, also after an abort)
      commit(done);
      if (lead) mbar_drain(done, 0u);
      __syncwarp();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  cluster_sync();  // no CTA leaves while the other may still write, read or arrive here
}

// Joins the ranges of a row tile: a thread four columns of one row. Ranges without a seen key carry
// m = -infinity and no O.
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int quad = blockIdx.x % 128, r = threadIdx.x;  // columns 4 quad ..
  const int64_t group = blockIdx.x / 128;              // (sequence, row tile)
  const int tile = static_cast<int>(group % p.tiles);
  const int64_t b = group / p.tiles;
  const int row = tile * kRows + r;
  if (row >= p.N * p.H) return;
  const float* ml = p.part_ml + group * p.splits * 2 * kRows + r;
  float m = kNegInf;
  for (int i = 0; i < p.splits; ++i) m = fmaxf(m, ml[i * 2 * kRows]);
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                      (group * p.splits * 128 + quad) * kRows + r;
  if (m != kNegInf) {
#pragma unroll 4
    for (int i = 0; i < p.splits; ++i) {
      const float mi = ml[i * 2 * kRows];
      if (mi == kNegInf) continue;
      const float f = exp2_approx(mi - m);
      const float4 v = src[static_cast<int64_t>(i) * 128 * kRows];
      l = fmaf(ml[i * 2 * kRows + kRows], f, l);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
  }
  const bool none = m == kNegInf;
  const float inv = none ? 0.f : 1.f / l;
  const int64_t out_row = b * p.N * p.H + row;
  if (quad == 0 && p.lse) p.lse[out_row] = none ? kNegInf : (m + __log2f(l)) * 0.69314718055994531f;
  *reinterpret_cast<uint2*>(p.out + out_row * kLatent + 4 * quad) =
      none ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// Pairs of CTAs that run at once: one CTA an SM.
int64_t pairs_at_once() { return sm_count() / 2; }

struct Plan {
  int32_t tiles, splits, steps;
  int64_t o_bytes, bytes;
};
// Key ranges: the number whose slowest pair takes the least, in steps of 64 keys (0.8 us); what a range
// costs besides its steps, and what joining costs, as measured.
Plan make_plan(int64_t pairs, int32_t B, int32_t N, int32_t H, int64_t max_kv_len) {
  Plan pl{};
  pl.tiles = (N * H + kRows - 1) / kRows;
  const int64_t items = static_cast<int64_t>(B) * pl.tiles;
  const int64_t steps = std::max<int64_t>(1, (max_kv_len + N + kKeys - 1) / kKeys);
  int64_t best = 0, best_cost = 0;
  for (int64_t n = 1; n <= std::min<int64_t>(steps, 2 * pairs); ++n) {
    const int64_t per = (steps + n - 1) / n, waves = (items * n + pairs - 1) / pairs;
    const int64_t cost = waves * (per + 5) + (n > 1 ? 5 : 0);
    if (best == 0 || cost < best_cost) best = n, best_cost = cost;
  }
  pl.splits = static_cast<int32_t>(best);
  pl.steps = static_cast<int32_t>((steps + best - 1) / best);
  pl.o_bytes = items * best * 2 * 64 * kRows * 16;
  if (best > 1) pl.bytes = pl.o_bytes + items * best * 2 * kRows * 4;
  return pl;
}

bool sizes_ok(int32_t B, int32_t N, int32_t H, int64_t max_kv_len) {
  return B >= 0 && N >= 1 && N <= kNodes && H >= 1 && H <= kMaxHeads && max_kv_len >= 0 &&
         max_kv_len <= 0x7FFFFFFF && static_cast<int64_t>(B) * N * H <= 0x7FFFFFFF / kMaxHeads;
}

template <int kFormat>
int launch(const Params& p, int64_t items, void* stream) {
  static std::atomic<uint64_t> done{0};
  if (!allow_shared(tree_attn_kernel<kFormat>, kSmem, done)) return DS4IDX_ERR_CUDA;
  return launch_dependent(tree_attn_kernel<kFormat>, static_cast<unsigned>(2 * items), kThreads, kSmem,
                          2, stream, p);
}

}  // namespace ds4ta

extern "C" int ds4idx_tree_attention_workspace(int32_t B, int32_t n_nodes, int32_t n_heads,
                                               int64_t max_kv_len, int64_t* bytes) {
  using namespace ds4ta;
  if (!bytes || !sizes_ok(B, n_nodes, n_heads, max_kv_len)) return DS4IDX_ERR_INVALID_ARG;
  const int64_t pairs = pairs_at_once();
  if (pairs < 1) return DS4IDX_ERR_CUDA;
  *bytes = B ? make_plan(pairs, B, n_nodes, n_heads, max_kv_len).bytes : 0;
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
  Params p{};
  if (!q || !cache || !kv_lens || !mask || !out || !aligned_to(q, 16) || !aligned_to(cache, 32) ||
      !aligned_to(scale, 4) || !aligned_to(kv_lens, 4) || !aligned_to(mask, 8) ||
      !aligned_to(out, 16) || !aligned_to(lse, 4) || !aligned_to(workspace, 16) ||
      !make_placement(where, kv_rows, B, &p.place))
    return DS4IDX_ERR_INVALID_ARG;
  const int64_t pairs = pairs_at_once();
  if (pairs < 1) return DS4IDX_ERR_CUDA;
  const Plan pl = make_plan(pairs, B, n_nodes, n_heads, max_kv_len);
  if (pl.bytes > 0 && (!workspace || workspace_size < pl.bytes)) return DS4IDX_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.scale = scale;
  p.lens = kv_lens;
  p.mask = mask;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.o_bytes);
  p.err = ds4a::sparse_attention_error_word();
  if (!p.err) return DS4IDX_ERR_CUDA;
  p.N = n_nodes;
  p.H = n_heads;
  p.tiles = pl.tiles;
  p.splits = pl.splits;
  p.steps = pl.steps;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  const int64_t items = static_cast<int64_t>(B) * pl.tiles * pl.splits;
  if (items * 2 > 0x7FFFFFFF) return DS4IDX_ERR_INVALID_ARG;
  const int st = format == DS4IDX_CACHE_FP8    ? launch<DS4IDX_CACHE_FP8>(p, items, stream)
                 : format == DS4IDX_CACHE_BF16 ? launch<DS4IDX_CACHE_BF16>(p, items, stream)
                                               : launch<DS4IDX_CACHE_Q4>(p, items, stream);
  if (st != DS4IDX_OK || pl.splits == 1) return st;
  return launch_dependent(tree_join_kernel,
                          static_cast<unsigned>(static_cast<int64_t>(B) * pl.tiles * 128), kJoinThreads,
                          0, 1, stream, p);
}
