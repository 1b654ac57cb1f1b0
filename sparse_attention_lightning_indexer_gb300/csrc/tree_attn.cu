// Attention of a tree of drafted tokens over a latent cache, for sm_103a: every node of a sequence
// attends over all of the sequence's rows and over the drafted rows on its own path. One latent row per
// position, shared by all heads; 576-wide keys, the first 512 dims are values.
//
// The (node, head) rows of a sequence are taken 128 at a time (the lanes of TMEM). A pair of CTAs owns
// such a tile and a range of keys, and each CTA half of the dims: O of 128 rows x 512 dims would fill an
// SM's whole TMEM and leave no place for S. With rank r holding latent dims 256 r .. and rotary dims
// 32 r .. of every key:
//   S  each CTA forms S_r[128 x 64 keys] over its 288 dims, sends it to the other and adds what comes:
//      S = S_0 + S_1 is the same number in both, so both hold the same softmax, and nothing else is
//      exchanged. A row of a key is read, unpacked and kept once in the pair, as key and as value.
//   P  p = exp2(s - m) in bf16, m a maximum that is left alone until a score passes it by 2^8;
//   O  O[128 x 256 own dims] += P V, in TMEM over the whole range. A raised m rescales O first.
// Ranges of a split sequence leave (O, m, l) in fp32, and a second kernel joins them.
//
// TMEM: O 256 columns, Q (latent dims, the A operand) 128, S 2 x 64. Shared memory: three stages of 64
// keys in bf16 (36 KB), P and the other CTA's S twice each.
//
// Warps 0..7: softmax, warps 0..3 on even tiles and 4..7 on odd ones, so that the exchange of one tile
// runs behind the arithmetic of another; m is handed from tile to tile. Warps 8..15: read rows, turn
// them into bf16 (exact) and write the 128-byte-swizzled operand. Warp 16 issues tcgen05.mma.
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
constexpr int kHalf = 256;             // latent dims of a CTA
constexpr int kLoad0 = 8, kMmaWarp = 16;
constexpr int kThreads = 17 * 32;
constexpr int kChunk = kKeys * 128;    // 64 dims of a step's keys
constexpr int kOffRope = 4 * kChunk;   // in a stage: the 32 rotary dims, 64-byte swizzle
constexpr int kStage = kOffRope + kKeys * 64, kStages = 3;
constexpr int kOffQRope = kStages * kStage;
constexpr int kOffP = kOffQRope + kRows * 64, kP = kRows * kKeys * 2;
constexpr int kOffX = kOffP + 2 * kP, kX = kRows * kKeys * 4;
constexpr int kOffM = kOffX + 2 * kX;              // float [2][128]: m after an even, an odd tile
constexpr int kOffL = kOffM + 2 * kRows * 4;       // float [2][2][128]: l and its m of both groups
constexpr int kOffKeyBits = kOffL + 4 * kRows * 4; // uint32 [kStages][2] keys that are there
constexpr int kOffOddBits = kOffKeyBits + kStages * 8;  // [kStages][4][2] keys not finite, by chunk
constexpr int kOffBars = kOffOddBits + kStages * 32;
constexpr int kNumBars = 2 * kStages + 1 + 4 * 2 + 1 + 2 * 8 + 8;
constexpr int kOffMisc = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffMisc + 16 + 1024;
static_assert(kSmem <= 232448 && kOffBars % 8 == 0, "shared memory");
constexpr uint32_t kColO = 0, kColQ = 256, kColS = 384;
constexpr float kNegInf = -__builtin_inff(), kMax = __FLT_MAX__;
constexpr float kSlack = 8.f;          // log2 of what a probability may exceed 1 by

struct Params {
  const uint16_t* q;
  const uint8_t* cache;
  const float* scale;
  const int32_t* lens;
  const int64_t* mask;
  uint16_t* out;
  float* lse;
  float* part_o;   // [item][2 ranks][64 column quads][128 rows][4]
  float* part_ml;  // [item][2][128]
  uint32_t* err;
  Placement place;
  int32_t N, H, tiles, splits, steps;  // row tiles a sequence, key ranges, least steps of a range
  float scale_log2;
};

// The range of keys of a work item: steps lo .. lo + n - 1 of 64 positions.
struct Range {
  int64_t len, end;  // rows of the sequence; positions from `end` on are not there
  int64_t lo;
  int32_t n;
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
  g.end = any ? max(min(g.len + (64 - __clzll(static_cast<long long>(g.seen))), room),
                    static_cast<int64_t>(0))
              : 0;
  const int64_t total = (g.end + kKeys - 1) / kKeys;
  const int64_t per = max(static_cast<int64_t>(p.steps), (total + p.splits - 1) / p.splits);
  g.lo = min(total, split * per);
  g.n = static_cast<int32_t>(min(total, g.lo + per) - g.lo);
  return g;
}

// 16 bytes to another CTA's shared memory.
__device__ __forceinline__ void st_peer16(uint32_t at, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ float4 ld_shared16(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_global32(void* at, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// Descriptor of a K-major operand of 64-byte rows in the 64-byte swizzle layout: atoms of 8 rows.
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(512u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(4u) << 61;
  return d;
}

// ---- reading rows: what one thread takes of a key, 64 dims (chunk c of this CTA's half) and 8 rotary
// ones, raw; unpacked as 8 x 16 bytes of bf16.
template <int kFormat>
struct RowPart {
  static constexpr int kWords = kFormat == DS4IDX_CACHE_BF16 ? 32 : kFormat == DS4IDX_CACHE_FP8 ? 16 : 8;
  uint32_t w[kWords];
  uint32_t scale;
  uint4 rope;

  __device__ __forceinline__ void load(const Params& p, int64_t r, int rank, int c) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = kFormat == DS4IDX_CACHE_Q4 ? ds4q::kEmptyWord : 0u;
    scale = 0u;
    rope = make_uint4(0, 0, 0, 0);
    if (r < 0) return;
    const uint8_t* row;
    int at, rot;
    if constexpr (kFormat == DS4IDX_CACHE_BF16) {
      row = p.cache + r * (2 * kDims);
      at = rank * 2 * kHalf + c * 128;
      rot = 2 * kLatent;
    } else if constexpr (kFormat == DS4IDX_CACHE_FP8) {
      row = p.cache + r * ds4f8::kRowBytes;
      at = rank * kHalf + c * 64;
      rot = ds4f8::kOffRope;
      scale = __float_as_uint(p.scale[r]);
    } else {
      row = p.cache + r * ds4q::kRowBytes;
      at = rank * (kHalf / 2) + c * 32;
      rot = ds4q::kOffRope;
      scale = *reinterpret_cast<const uint32_t*>(row + ds4q::kOffScale + 4 * (4 * rank + c));
    }
#pragma unroll
    for (int j = 0; j < kWords; j += 8) ld32(row + at + 4 * j, reinterpret_cast<uint32_t(&)[8]>(w[j]));
    rope = *reinterpret_cast<const uint4*>(row + rot + rank * 64 + c * 16);
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
  // To row `key` of a stage.
  __device__ __forceinline__ void store(uint32_t stage, int key, int c) const {
    const uint32_t at = stage + c * kChunk + key * 128 + (key & 7) * 16;
    uint32_t s2 = 0;
    if constexpr (kFormat == DS4IDX_CACHE_FP8) s2 = ((scale >> 23) + 120u) * 0x00800080u;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint4 v;
      if constexpr (kFormat == DS4IDX_CACHE_BF16) {
        v = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
      } else if constexpr (kFormat == DS4IDX_CACHE_FP8) {
        unpack(w[2 * u], s2, v.x, v.y);
        unpack(w[2 * u + 1], s2, v.z, v.w);
      } else {
        const int g = u >> 1;
        const uint32_t q2 = __byte_perm(scale, 0, 0x4040u | (g << 8) | g) * 16u + 0x35803580u;
        v = ds4q::word_to_bf16(w[u], q2, ds4q::offset_bf16x2(q2));
      }
      st_shared16(at ^ (16 * u), v);
    }
    st_shared16(stage + kOffRope + key * 64 + ((c ^ (key >> 1)) & 3) * 16, rope);
  }
};

template <int kFormat>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  // both CTAs of a pair have the same dynamic shared-memory base, so the offsets agree
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t smem0 = smem_u32(smem);
  float* s_m = reinterpret_cast<float*>(smem + kOffM);
  float* s_l = reinterpret_cast<float*>(smem + kOffL);
  volatile uint32_t* s_there = reinterpret_cast<uint32_t*>(smem + kOffKeyBits);
  volatile uint32_t* s_odd = reinterpret_cast<uint32_t*>(smem + kOffOddBits);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* k_empty = k_full + kStages;
  uint64_t* q_full = k_empty + kStages;
  uint64_t* s_ready = q_full + 1;   // [2] S_r of a tile is formed
  uint64_t* s_free = s_ready + 2;   // [2] and read
  uint64_t* p_full = s_free + 2;    // [2]
  uint64_t* pv_done = p_full + 2;   // [2] P V of a tile is done
  uint64_t* done = pv_done + 2;     // every MMA has completed
  uint64_t* x_full = done + 1;      // [8] by softmax warp: the other CTA's S of its rows has come
  uint64_t* x_empty = x_full + 8;   // [8] the other CTA has read what was sent
  uint64_t* m_full = x_empty + 8;   // [8] the warp's m is in s_m
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile uint32_t* s_abort = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1, item = blockIdx.x >> 1;
  const int split = item % p.splits, tile = item / p.splits % p.tiles, b = item / (p.splits * p.tiles);
  uint32_t* err = p.err;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&k_full[i], 8);
      mbar_init(&k_empty[i], 1);
    }
    mbar_init(q_full, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_ready[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(done, 1);
    for (int i = 0; i < 8; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_empty[i], 1);
      mbar_init(&m_full[i], 1);
    }
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

  if (warp < kLoad0) {
    // ---------------- softmax: this thread's row, the tiles of its group's parity
    const int grp = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int row = tile * kRows + r, node = row / p.H;
    const bool used = node < p.N;
    const int64_t out_row = static_cast<int64_t>(b) * p.N * p.H + row;
    uint64_t mask = used ? static_cast<uint64_t>(p.mask[static_cast<int64_t>(b) * p.N + node]) : 0ull;
    const bool padding = mask == 0ull;
    mask &= ~0ull >> (64 - p.N);
    bool ok = true;
    if (g.n > 0) {
      // Q: latent dims to TMEM (64 columns by each group), rotary dims to shared memory
      const uint4* src = reinterpret_cast<const uint4*>(p.q + out_row * kDims + rank * kHalf + grp * 128);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 x = used ? src[8 * h + j] : make_uint4(0, 0, 0, 0);
          v[4 * j] = x.x;
          v[4 * j + 1] = x.y;
          v[4 * j + 2] = x.z;
          v[4 * j + 3] = x.w;
        }
        tmem_st32(tmem + lanes + kColQ + grp * 64 + h * 32, v);
      }
      const uint4* rot = reinterpret_cast<const uint4*>(p.q + out_row * kDims + kLatent + rank * 32);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int u = grp * 2 + j;
        st_shared16(smem0 + kOffQRope + r * 64 + ((u ^ (r >> 1)) & 3) * 16,
                    used ? rot[u] : make_uint4(0, 0, 0, 0));
      }
      tmem_wait_st();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    float m = kNegInf, l = 0.f;
    const uint32_t x_own = smem0 + kOffX + grp * kX + r * 16;
    const uint32_t x_peer = peer(x_own, rank ^ 1);
    const uint32_t s_col = tmem + lanes + kColS + grp * kKeys;
#pragma unroll 1
    for (int i = grp; i < g.n; i += 2) {
      const uint32_t use = i >> 1;
      const int st = i % kStages;
      // this CTA's part of S to the other one
      ok = ok && mbar_wait_warp(&s_ready[grp], use & 1, s_abort, err) &&
           mbar_wait_warp(&k_full[st], (i / kStages) & 1, s_abort, err) &&
           __all_sync(0xffffffffu, wait_cluster(&x_empty[warp], (use & 1) ^ 1u, s_abort, err));
      if (!ok) break;
      tc_fence_after();
      const int64_t pos = (g.lo + i) * kKeys;
      uint64_t there = static_cast<uint64_t>(s_there[2 * st + 1]) << 32 | s_there[2 * st];
      uint64_t bad = 0ull;  // keys whose score is NaN because of values here
      if (pos + kKeys > g.len) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          bad |= static_cast<uint64_t>(s_odd[8 * st + 2 * c + 1]) << 32 | s_odd[8 * st + 2 * c];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        tmem_ld32(s_col + 32 * h, v);
        tmem_wait_ld();
        if (bad) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (bad >> (32 * h + j) & 1) v[j] = 0x7FC00000u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) st_peer16(x_peer + (8 * h + j) * (kRows * 16), &v[4 * j]);
      }
      __syncwarp();
      if (lane == 0) arrive_peer(peer(smem_u32(&x_full[warp]), rank ^ 1));
      // the sum of both
      ok = __all_sync(0xffffffffu, wait_cluster(&x_full[warp], use & 1, s_abort, err));
      if (!ok) break;
      float s[kKeys];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        tmem_ld32(s_col + 32 * h, v);
        float4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = ld_shared16(x_own + (8 * h + j) * (kRows * 16));
        tmem_wait_ld();
        // (the smaller rank's part first: the same sum, bit for bit, in both CTAs; a sum of two does
        // not depend on the order)
#pragma unroll
        for (int j = 0; j < 32; ++j) s[32 * h + j] = __uint_as_float(v[j]) + (&x[j >> 2].x)[j & 3];
      }
      if (bad) {
#pragma unroll
        for (int j = 0; j < kKeys; ++j)
          if (bad >> j & 1) s[j] = __uint_as_float(0x7FC00000u);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_free[grp]);
        arrive_peer(peer(smem_u32(&x_empty[warp]), rank ^ 1));
      }
      // which keys this row sees
      uint64_t see = padding ? 0ull : ~0ull;
      if (pos + kKeys > g.len && !padding) {
        const int64_t d = g.len - pos;  // < 64
        see = d >= 0 ? (1ull << d) - 1ull | mask << d : d > -64 ? mask >> -d : 0ull;
      }
      see &= there;
      const bool all = __all_sync(0xffffffffu, see == ~0ull);
      float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
      if (all) {
#pragma unroll
        for (int j = 0; j < kKeys; ++j) mx[j & 3] = fmaxf(mx[j & 3], s[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
          if (see >> j & 1) mx[j & 3] = fmaxf(mx[j & 3], s[j]);
        }
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      // m of the tile before; raised where a score passes it by more than the slack. Finite once a key
      // was seen: a score of +-infinity keeps its meaning in s - m.
      float before = kNegInf;
      if (i > 0) {
        ok = mbar_wait_warp(&m_full[warp ^ 4], ((i - 1) >> 1) & 1, s_abort, err);
        if (!ok) break;
        before = s_m[(grp ^ 1) * kRows + r];
      }
      float now = before;
      if (see != 0ull && (before == kNegInf || top > before + kSlack))
        now = fminf(fmaxf(top, -kMax), kMax);
      s_m[grp * kRows + r] = now;
      __syncwarp();
      if (lane == 0) mbar_arrive(&m_full[warp]);
      const bool raise = now != before && before != kNegInf;
      if (__any_sync(0xffffffffu, raise)) {
        // O of the tiles before, all columns of these rows
        ok = mbar_wait_warp(&pv_done[grp ^ 1], ((i - 1) >> 1) & 1, s_abort, err);
        if (!ok) break;
        tc_fence_after();
        const float f = raise ? exp2_approx(before - now) : 1.f;
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + lanes + kColO + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
          tmem_st32(tmem + lanes + kColO + c, v);
        }
        tmem_wait_st();
      }
      if (now != m) {
        l *= exp2_approx(m - now);
        m = now;
      }
      // P, in the layout of an MMA A operand
      ok = mbar_wait_warp(&pv_done[grp], (use & 1) ^ 1u, s_abort, err);
      if (!ok) break;
      const uint32_t p_at = smem0 + kOffP + grp * kP + r * 128 + (r & 7) * 16;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint32_t pk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 8 * u + 2 * j;
          float p0 = exp2_approx(fmaf(s[k], p.scale_log2, -m));
          float p1 = exp2_approx(fmaf(s[k + 1], p.scale_log2, -m));
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
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[grp]);
    }
    // ---------------- both groups' sums, and this group's 128 columns of the output
    s_l[grp * kRows + r] = l;
    s_l[(2 + grp) * kRows + r] = m;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const float last = g.n > 0 ? s_m[((g.n - 1) & 1) * kRows + r] : kNegInf;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float mk = s_l[(2 + k) * kRows + r];
      if (mk != kNegInf) l += s_l[k * kRows + r] * (mk == last ? 1.f : exp2_approx(mk - last));
    }
    if (ok && g.n > 0) ok = mbar_wait_warp(&pv_done[(g.n - 1) & 1], ((g.n - 1) >> 1) & 1, s_abort, err);
    tc_fence_after();
    const bool none = last == kNegInf;
    if (p.splits == 1) {
      if (used && rank == 0 && grp == 0 && p.lse)
        p.lse[out_row] = none ? kNegInf : (last + __log2f(l)) * 0.69314718055994531f;
      const float inv = none ? 0.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t v[32], pk[16];
        if (g.n > 0) {
          tmem_ld32(tmem + lanes + kColO + grp * 128 + c, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int j = 0; j < 32; j += 2)
          pk[j / 2] = none ? 0u : pack_bf16x2(__uint_as_float(v[j]) * inv, __uint_as_float(v[j + 1]) * inv);
        if (used && ok) {
          uint16_t* dst = p.out + out_row * kLatent + rank * kHalf + grp * 128 + c;
          reinterpret_cast<uint4*>(dst)[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          reinterpret_cast<uint4*>(dst)[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          reinterpret_cast<uint4*>(dst)[2] = make_uint4(pk[8], pk[9], pk[10], pk[11]);
          reinterpret_cast<uint4*>(dst)[3] = make_uint4(pk[12], pk[13], pk[14], pk[15]);
        }
      }
    } else {
      if (rank == 0 && grp == 0) {
        p.part_ml[static_cast<int64_t>(item) * 2 * kRows + r] = last;
        p.part_ml[static_cast<int64_t>(item) * 2 * kRows + kRows + r] = l;
      }
      if (g.n > 0 && ok) {
        float4* dst = reinterpret_cast<float4*>(p.part_o) +
                      ((static_cast<int64_t>(item) * 2 + rank) * 64 + grp * 32) * kRows + r;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + lanes + kColO + grp * 128 + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[(c / 4 + j) * kRows] =
                make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                            __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ---------------- rows to bf16: one (key, chunk of 64 dims) a thread, two steps in flight
    const int w = warp - kLoad0, key = (w & 1) * 32 + lane, c = w >> 1;
    const TokenPlace tp = place_token(p.place, b);
    auto row_of = [&](int i) -> int64_t {
      const int64_t s = (g.lo + i) * kKeys + key;
      if (i >= g.n || s >= g.end || (s >= g.len && !(g.seen >> (s - g.len) & 1))) return -1;
      return place_row(p.place, tp, static_cast<int32_t>(s));
    };
    RowPart<kFormat> part[2];
    bool there[2];
    int64_t next = row_of(0);
    auto fetch = [&](int i, RowPart<kFormat>& x, bool& t) {
      t = next >= 0;
      x.load(p, next, rank, c);
      next = row_of(i + 1);
    };
    bool ok = true;
    auto put = [&](int i, RowPart<kFormat>& x, bool t) {
      if (!ok || i >= g.n) return;
      const int st = i % kStages;
      ok = mbar_wait_warp(&k_empty[st], ((i / kStages) & 1) ^ 1u, s_abort, err);
      if (!ok) return;
      // A drafted row that some rows of the tile see and others do not may hold values that are not
      // finite: cleared, since 0 * NaN would reach all of O, and its scores become NaN instead.
      const bool drafts = (g.lo + i) * kKeys + kKeys > g.len;
      if (drafts) {
        const bool odd = (g.lo + i) * kKeys + key >= g.len && x.odd();
        const uint32_t bits = __ballot_sync(0xffffffffu, odd);
        if (odd) x.clear();
        if (lane == 0) s_odd[8 * st + 2 * c + (w & 1)] = bits;
      }
      if (c == 0) {
        const uint32_t bits = __ballot_sync(0xffffffffu, t);
        if (lane == 0) s_there[2 * st + (w & 1)] = bits;
      }
      x.store(smem0 + st * kStage, key, c);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[st]);
    };
    fetch(0, part[0], there[0]);
    fetch(1, part[1], there[1]);
#pragma unroll 1
    for (int i = 0; i < g.n && ok; i += 2) {
      put(i, part[0], there[0]);
      fetch(i + 2, part[0], there[0]);
      put(i + 1, part[1], there[1]);
      fetch(i + 3, part[1], there[1]);
    }
  } else {
    // ---------------- MMA issue: the warp waits together, one elected lane issues
    const bool lead = elect_one();
    bool ok = true;
    const uint64_t k0 = smem_desc_sw128(smem0), v0 = smem_desc_mn_sw128(smem0, kChunk);
    const uint64_t kr0 = smem_desc_sw64(smem0 + kOffRope), qr = smem_desc_sw64(smem0 + kOffQRope);
    const uint64_t p0 = smem_desc_sw128(smem0 + kOffP);
    constexpr uint32_t s_idesc = instr_desc(1u, 1u, kRows, kKeys);
    constexpr uint32_t o_idesc = instr_desc(1u, 1u, kRows, kHalf) | (1u << 16);  // B MN-major
    auto commit = [&](uint64_t* bar) {
      if (lead) mma_commit(bar);
    };
    auto value_product = [&](int i) {
      const int st = i % kStages, slot = i & 1;
      ok = mbar_wait_warp(&p_full[slot], (i >> 1) & 1, s_abort, err);
      if (!ok) return;
      tc_fence_after();
      const uint64_t pd = p0 + slot * (kP >> 4), vd = v0 + st * (kStage >> 4);
      if (lead) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16(tmem + kColO, pd + 2 * k, vd + k * (16 * 128 >> 4), o_idesc, (i | k) ? 1u : 0u);
      }
      commit(&k_empty[st]);
      commit(&pv_done[slot]);
    };
    if (g.n > 0) ok = mbar_wait_warp(q_full, 0u, s_abort, err);
#pragma unroll 1
    for (int i = 0; ok && i < g.n; ++i) {
      const int st = i % kStages, slot = i & 1;
      ok = mbar_wait_warp(&k_full[st], (i / kStages) & 1, s_abort, err) &&
           mbar_wait_warp(&s_free[slot], ((i >> 1) & 1) ^ 1u, s_abort, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + kColS + slot * kKeys;
      const uint64_t kd = k0 + st * (kStage >> 4), kr = kr0 + st * (kStage >> 4);
      if (lead) {
        mma_bf16(d, qr, kr, s_idesc, 0u);
        mma_bf16(d, qr + 2, kr + 2, s_idesc, 1u);
#pragma unroll
        for (int k = 0; k < kHalf / 16; ++k)
          mma_bf16_ts(d, tmem + kColQ + k * 8, kd + (k >> 2) * (kChunk >> 4) + (k & 3) * 2, s_idesc, 1u);
      }
      commit(&s_ready[slot]);
      if (i > 0) value_product(i - 1);
    }
    if (ok && g.n > 0) value_product(g.n - 1);
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
  cluster_sync();  // no CTA leaves while the other may still write or arrive here
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
                      ((group * p.splits * 2 + quad / 64) * 64 + quad % 64) * kRows + r;
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
