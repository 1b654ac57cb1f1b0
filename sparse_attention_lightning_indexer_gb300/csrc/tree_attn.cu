// Attention of a tree of drafted tokens over a latent cache, for sm_103a: every node of a sequence
// attends over all of the sequence's rows and over the drafted rows on its own path. One latent row per
// position, shared by all heads; 576-wide keys, the first 512 dims are values.
//
// The (node, head) rows of a sequence are taken 128 at a time (the lanes of TMEM). O of 128 rows x 512
// dims fills an SM's TMEM, so a pair of CTAs owns such a tile and a range of keys: one (rank 0) the
// keys' products and the softmax, the other the values' products:
//   S[128 x 64 keys] = Q K^T        rank 0; Q stays in TMEM as the A operand, three tiles of S beside it
//   p = exp2(s - m) in bf16         rank 0; m is left alone until a score passes it by 64. The sums of p
//                                   are fp32, and so are m and O.
//   O[128 x 512] += P V             rank 1; O fills its TMEM over the whole range
// P, and the factors of O where m was raised, are all that goes from one CTA to the other: 16 KB a tile,
// stored straight into rank 1's shared memory with the bytes counted at a barrier there (the shared memory of
// a pair moves 18.7 bytes a clock in each direction when all SMs do it). Splitting the dims instead reads and
// unpacks a row once in the pair, but exchanges S, 32 KB a tile both ways, before the softmax can go on: 3.27
// against 2.78 ms when both were first built (4 sequences of 64 nodes over 16384 rows, 128 heads, 8 bits).
// Ranges of a split sequence leave (O, m, l) in fp32, and a second kernel joins them.
//
// What bounds it: a tile of 64 keys takes a pair 2550 clocks, 1.35 us. Rank 0's products take 36 times 57 to
// 64 clocks (32 is the tensor core's rate), its softmax groups 3000 and more each for every other tile. Rank
// 1's shared memory moves 240 KB a tile, 1900 clocks at 128 bytes each: codes in and out, bf16 in, out for the
// products, P. Timing-only copies with one side made light (the first case below, 1.28 ms at that time): half
// of rank 0's products 1.27, no value codes read 1.26, both sides light 0.94. A range costs 16 us besides:
// set-up 2, Q 4, the end of the pipeline 2, O 4, the join 4.
//
// Measured on the device: 4 sequences of 64 nodes, 128 heads, 16384 8-bit rows 1.31 ms, 0.89 PFLOP/s; one
// node over 262144 8-bit rows 99 us, 1.7 TB/s; 13 nodes over 32768 bf16 rows 155 us, 0.77 PFLOP/s; three
// sequences of 31 nodes of 16 heads over 12001 4-bit rows in pages 79 us, where unpacking in both ranks is
// what bounds it (3500 clocks a tile).
//
// Both CTAs read the rows themselves and keep them in a ring of parts, 64 keys x 256 dims in the
// 128-byte-swizzled layout that serves as K-major and as MN-major operand.
//
// Warps 0..7: softmax, a row a thread, warps 0..3 on even tiles and 4..7 on odd ones (rank 1: the
// rescaling of O and the output). Warps 8..15: rows to operands. Warp 16 issues tcgen05.mma. The roles' loops
// are kept rolled: they run side by side out of one instruction cache, and with everything unrolled (126 KB of
// code) more than half of its look-ups missed and a tile took 7000 clocks.
//
// 8-bit rows are operands without their scales, which are powers of two: S is multiplied by them, and so is
// P, exactly where P times the scale is normal. As keys they are E4M3 operands as they stand, and Q, scaled by a
// power of two, is a sum of an E4M3 and an E5M2 operand: two products at twice the rate, and nothing to unpack.
// That sum holds a bf16 exactly, but for what of a row of Q lies 2^13 and more below its largest value: that is off
// by at most 2^-21 of the largest, or of 2^-119 (bf16_to_f8_pair). As values the codes are bf16 (P needs its range
// and bits).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

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
constexpr int kLoad0 = 8, kLoaders = 8, kMmaWarp = 16;
constexpr int kThreads = 17 * 32;
constexpr int kChunk = kKeys * 128;    // 64 dims of a tile's keys
constexpr int kPart = 4 * kChunk, kParts = 3;      // the ring of operands
constexpr int kPart8 = 2 * kChunk, kParts8 = 7;    // of 8-bit keys, 128 dims a chunk (in the same place)
constexpr int kRaw = kKeys * 256, kRaws = 3;       // codes of a part as they are read
constexpr int kOffRaw = kParts * kPart;
constexpr int kOffRope = kOffRaw + kRaws * kRaw;   // the rotary dims of four tiles' keys (rank 0)
constexpr int kP = kRows * kKeys * 2;              // P of a tile
constexpr int kIn = 4;                             // tiles of P on their way to rank 1 or in use there
constexpr int kOffP = kOffRope;                    // in rank 1, which has no rotary dims
constexpr int kOffMade = kOffRope + 4 * kChunk;    // P of an even and of an odd tile as it is made (rank 0)
constexpr int kOffF = kOffP + kIn * kP;
static_assert(kOffMade + 2 * kP <= kOffF, "P");    // kOffF: float [4][128], roots of factors of O before P V
constexpr int kOffM = kOffF + kIn * kRows * 4;       // float [2][128]: m after an even, an odd tile
constexpr int kOffL = kOffM + 2 * kRows * 4;       // float [3][2][128]: both sums, and their m, of both groups
constexpr int kOffScale = kOffL + 6 * kRows * 4;   // float [8 tiles][64]: scales of the keys (8-bit
                                                   // rows), or kRaws tiles' codes of scales (4-bit rows)
constexpr int kOffThere = kOffScale + kRaws * 2048;  // uint64 [8 tiles]: keys that are there
constexpr int kOffBars = kOffThere + 8 * 8;
constexpr int kNumBars = 2 * kParts8 + 1 + 2 * 3 + 4 * kIn + 8 + 2;
static_assert(kParts8 * kPart8 <= kOffRope && kParts8 >= kParts, "8-bit keys");
constexpr int kOffMisc = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffMisc + 16 + 1024;
static_assert(kSmem <= 232448 && kOffBars % 8 == 0, "shared memory");
constexpr uint32_t kColRope = 256, kColS = 320;    // rank 0: Q from column 0, S; rank 1: O from 0
constexpr uint32_t kColLow = 128;                  // the low parts of Q beside 8-bit keys
constexpr uint32_t kColAside = 288;                // 224 columns that hold Q before it is turned
constexpr float kNegInf = -__builtin_inff(), kMax = __FLT_MAX__;
// log2 of what exp2(s - m) may be before m is raised. P and the sums are floating point with 2^127 of
// range, so a stale m costs no precision, but it takes room from the values. Those of 8 and 4 bits are below 2^16,
// which leaves 2^47 for their number. bf16 ones may be anything: 2^48 leaves room for values below 2^49 in
// sequences of any length (2^31 of them) and costs nothing (13 nodes over 32768 rows 155.5 us, 160 with 2^32). (With
// 2^8 some row of 128 raises m in most of the first hundred tiles, and a rescaling holds P V up for 4000 clocks:
// one node over 262144 8-bit rows 150 us where it takes 98, 107 with 2^32; 4 sequences of 64 nodes over 16384
// 1.78, 1.32 and 1.36 ms.)
template <int kFormat>
constexpr float kSlack = kFormat == DS4IDX_CACHE_BF16 ? 48.f : 64.f;

struct Params {
  const uint16_t* q;
  const uint8_t* cache;
  const float* scale;
  const int32_t* lens;
  const int64_t* mask;
  uint16_t* out;
  float* lse;
  float* part_o;   // [item][128 column quads][128 rows][4]
  float* part_ml;  // [item][3][128]: m, l, and the sum of the rounded terms
  uint32_t* err;
  Placement place;
  int32_t N, H, tiles, splits;  // row tiles a sequence, key ranges at most
  int32_t items;                // row tiles of all sequences
  int32_t fill, steps;          // ranges that fill the device once, and the steps from which more may be made
  float scale_log2;      // of a score, from a product: may be subnormal
  float scale_fraction;  // the same, of 0.5 .. 1, times 2^scale_exp
  int32_t scale_exp;
};

// The range of keys of a work item: steps lo .. lo + n - 1 of 64 positions.
struct Range {
  int32_t len, end;  // rows of the sequence; positions from `end` on are not there
  int32_t lo, n;
  int32_t plain;     // the first steps, whose keys are all rows of the sequence
  uint64_t seen;     // drafted rows that some node of the tile sees

  __device__ __forceinline__ int32_t position(int i) const { return (lo + i) * kKeys; }
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
  // By the sequence's own length: the grid is laid out for a bound, which may be far above it.
  const int32_t per = max((total - 1) / p.splits + 1, min((total - 1) / p.fill + 1, p.steps));
  g.lo = static_cast<int32_t>(min(static_cast<int64_t>(total), static_cast<int64_t>(split) * per));
  g.n = min(total - g.lo, per);
  g.plain = max(0, min(g.n, min(g.len, g.end) / kKeys - g.lo));
  return g;
}

// Waits of a whole warp for a phase of a barrier, bounded like every wait of the library: after 2^32 clocks
// (2 s) or when the CTA has given up they return false. What follows a first try that fails is kept out of
// the roles' loops.
template <bool kCluster>
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCluster)  // acquires what another CTA released
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
template <bool kCluster>
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                         uint32_t* err) {
  bool ok = false;
  long long since = 0;
  for (uint32_t i = 1; !__all_sync(0xffffffffu, ok = ok || phase_done<kCluster>(bar, parity)); ++i) {
    if (i & 255u) continue;
    const long long now = clock64();
    if (since == 0) since = now;
    const bool late = now - since > (1ll << 32);
    if (__any_sync(0xffffffffu, late || *abort_flag)) {
      if (late) {
        *abort_flag = 1u;
        atomicOr(err, 1u);
      }
      return false;
    }
  }
  return true;
}
template <bool kCluster>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                           uint32_t* err) {
  if (__all_sync(0xffffffffu, phase_done<kCluster>(smem_u32(bar), parity))) return true;
  return wait_longer<kCluster>(smem_u32(bar), parity, abort_flag, err);
}
__device__ __forceinline__ void st_global32(void* at, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// Stores to another CTA's shared memory that count as bytes at a barrier there: nothing here waits for them.
__device__ __forceinline__ void st_async16(uint32_t at, uint4 v, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
          at),
      "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void st_async4(uint32_t at, float v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(at),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}
// Orders generic accesses to the cluster's shared memory before later ones of MMAs.
__device__ __forceinline__ void fence_proxy_async_cluster() {
  asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
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
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// As mma_bf16 and mma_fp8, the first operand in TMEM: a row a lane, adjacent K elements packed in a column
// of 32 bits.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_fp8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---- reading rows: eight warps, each eight keys of a tile. Eight lanes read 128 adjacent bytes of a row
// (rows in L2, all SMs: 16.7 TB/s; a lane for each key instead, 32 bytes at 32 different lines an access,
// 9.7 TB/s, bound by the L1's look-ups).

// 16 bytes of row r at p, zeros where there is no row. One predicated load into registers that hold them:
// with a branch around it the value is moved where the paths meet, and the move waits for it.
__device__ __forceinline__ uint4 ld_row16(const uint8_t* p, int32_t r) {
  uint4 v = make_uint4(0, 0, 0, 0);
  asm volatile(
      "{\n\t.reg .pred there;\n\tsetp.ge.s32 there, %5, 0;\n\t"
      "@there ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
      : "l"(p), "r"(r));
  return v;
}
// 16 (4) bytes of row r at src to shared memory, zeros where there is no row.
__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src, int32_t r) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(r >= 0 ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int32_t r) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(r >= 0 ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Four E4M3 codes to bf16 (exact), by way of f16 and fp32: the conversions run on more pipes than
// shifting the bits into place would.
__device__ __forceinline__ void codes_to_bf16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  ds4f8::codes_to_f16(c, a, b);
  const float2 u = ds4f8::f16x2_to_f32(a), v = ds4f8::f16x2_to_f32(b);
  lo = pack_bf16x2(u.x, u.y);
  hi = pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ bool odd_f8(const uint4& v) {
  return (__vcmpeq4(v.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(v.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
          __vcmpeq4(v.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(v.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu)) != 0u;
}
__device__ __forceinline__ bool odd_bf16(const uint4& v) {
  auto odd = [](uint32_t u) { return (u & 0x7F80u) == 0x7F80u || (u & 0x7F800000u) == 0x7F800000u; };
  return odd(v.x) || odd(v.y) || odd(v.z) || odd(v.w);
}
template <typename T>
__device__ __forceinline__ void swap_if(bool c, T& a, T& b) {
  const T x = c ? b : a;
  b = c ? a : b;
  a = x;
}

// Who orders the writes of a part before the products that read it, by the proxy fence between them: its
// writers, 300 clocks a part of each loader, or the one warp that issues the products. Beside 4-bit rows the
// loaders are the slower (3 sequences of 31 nodes, 12001 rows: 84 us with their fence, 80 with the other's);
// beside the others the products are (4 of 64 nodes over 16384 8-bit rows: 1.28 and 1.43 ms).
template <int kFormat>
constexpr bool kFenceByMma = kFormat == DS4IDX_CACHE_Q4;

// One loader warp's work. kKey: this CTA forms the key products (and takes the rotary dims), or the
// values'. Codes go to shared memory as they are, by asynchronous copies two tiles ahead, and are turned
// into the operand by the thread that copied them. (Held in registers they were waited for as soon as the
// next ones were on their way, 1600 clocks a tile: the scoreboards are too few to tell them apart.)
template <int kFormat, bool kKey>
__device__ __forceinline__ void load_rows(const Params& p, const Range& g, int b, int w, int lane,
                                          uint8_t* smem, uint64_t* part_full, uint64_t* part_empty,
                                          volatile uint32_t* abort_flag) {
  constexpr bool k8 = kKey && kFormat == DS4IDX_CACHE_FP8;  // the operand is the codes
  constexpr int kStride = kFormat == DS4IDX_CACHE_FP8    ? ds4f8::kRowBytes
                          : kFormat == DS4IDX_CACHE_BF16 ? 2 * kDims
                                                         : ds4q::kRowBytes;
  const uint32_t smem0 = smem_u32(smem);
  const int l8 = lane & 7, sub = lane >> 3;
  const TokenPlace tp = place_token(p.place, b);
  auto row_at = [&](int32_t r) { return p.cache + static_cast<int64_t>(r) * kStride; };
  bool ok = true;
  int st = 0;                 // place in the ring
  uint32_t parity = 1;        // of part_empty
  auto claim = [&] { ok = ok && wait_phase<false>(&part_empty[st], parity, abort_flag, p.err); };
  auto step = [&] {
    if (++st == (k8 ? kParts8 : kParts)) st = 0, parity ^= 1u;
  };
  auto publish = [&](int at) {
    if constexpr (!kFenceByMma<kFormat>) fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&part_full[at]);
  };
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // Keys 8 w + first .. + 3, one for each eight lanes.
  auto quad_bits = [&](bool c) -> uint32_t {
    const uint32_t bits = __ballot_sync(0xffffffffu, c);
    uint32_t keys = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) keys |= bits >> (8 * j) & 0xFFu ? 1u << j : 0u;
    return keys;
  };
  // A drafted row that some rows of the tile see and others do not may hold values that are not finite: as
  // a value what is not is cleared, since 0 * NaN would reach all of O. (The nodes that see it have its
  // scores, and from them NaN.)
  auto drafted = [&](int i, int key) { return g.position(i) + 8 * w + key >= g.len; };
  auto rope_address = [&](int i, int key) {
    return smem0 + kOffRope + (i & 3) * kChunk + (8 * w + key) * 128 + ((l8 ^ key) * 16);
  };
  // This thread's rows (keys sub and 4 + sub) of the tile that is read. Rows that follow one another are
  // stepped through. Otherwise a key's page and its place there are stepped from tile to tile, and its entry
  // of the page table is read a tile ahead.
  const bool steps = tp.table == nullptr;
  const int32_t page = steps ? 1 : p.place.page, pages = tp.ok ? p.place.pages : 0;
  const int32_t page_step = kKeys / page, place_step = kKeys % page;
  // (Unsigned: the tiles read ahead may lie past position 2^31, and there is no page.)
  int32_t row[2], id[2] = {};
  uint32_t page_no[2] = {}, place[2] = {};
  auto look_up = [&](int k) { id[k] = page_no[k] < static_cast<uint32_t>(pages) ? tp.table[page_no[k]] : -1; };
  // Rows of tile i, whose entries are read, and the entries of the tile after it.
  auto find_rows = [&](int i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int32_t s = g.position(i) + 8 * w + 4 * k + sub;
      bool is = i < g.plain || (i < g.n && s < g.end && (s < g.len || (g.seen >> (s - g.len) & 1)));
      int64_t r = tp.row0 + s;  // (contiguous: `end` ends at the pool's last row)
      if (!steps) {
        r = static_cast<int64_t>(id[k]) * page + place[k];
        is = is && id[k] >= 0 && r < p.place.rows;
        page_no[k] += page_step;
        place[k] += place_step;
        if (place[k] >= static_cast<uint32_t>(page)) place[k] -= page, ++page_no[k];
        look_up(k);
      }
      row[k] = is ? static_cast<int32_t>(r) : -1;
    }
  };
  if (!steps) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int32_t s = g.position(0) + 8 * w + 4 * k + sub;
      page_no[k] = s / page;
      place[k] = s % page;
      look_up(k);
    }
  }
  find_rows(0);
  const uint8_t* from[2] = {row_at(max(row[0], 0)) + l8 * 16, row_at(max(row[1], 0)) + l8 * 16};
  int read = 0;        // tiles whose reads are on their way
  auto advance_rows = [&] {
    ++read;
    if (steps && read < g.plain) {
#pragma unroll
      for (int k = 0; k < 2; ++k) row[k] += kKeys, from[k] += kKeys * kStride;
      return;
    }
    find_rows(read);
#pragma unroll
    for (int k = 0; k < 2; ++k) from[k] = row_at(max(row[k], 0)) + l8 * 16;
  };
  auto note_there = [&] {  // of the tile that is read, for the softmax
    if (!kKey || (steps && read < g.plain)) return;
    const uint32_t bits = quad_bits(row[0] >= 0) | quad_bits(row[1] >= 0) << 4;
    if (lane == 0) smem[kOffThere + 8 * (read & 7) + w] = static_cast<uint8_t>(bits);
  };

  if constexpr (k8) {
    // Keys: the codes as they are. A part is two lines of 128 codes (c) of rows sub and 4 + sub (k); five
    // parts are on their way. A tile's scales and rotary dims come with its first half; the rotary dims are
    // divided by the scale in place, by the thread that copied them, with the second.
    constexpr int kLag = 5;
    auto finish = [&](int n, int at) {
      if (n & 1) {
        const float* scales = reinterpret_cast<const float*>(smem + kOffScale) + (n >> 1 & 7) * kKeys + 8 * w;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t rope = rope_address(n >> 1, 4 * k + sub);
          // (a scale that is no power of two, which P and these dims cannot follow, makes NaN of the scores)
          const uint32_t bits = __float_as_uint(scales[4 * k + sub]);
          const uint32_t s2 = bits & 0x807FFFFFu ? 0x7FFF7FFFu : (254u - (bits >> 23)) * 0x00800080u;
          const uint4 x = ld_shared16(rope);
          st_shared16(rope, make_uint4(ds4q::mul_bf16x2(x.x, s2), ds4q::mul_bf16x2(x.y, s2),
                                       ds4q::mul_bf16x2(x.z, s2), ds4q::mul_bf16x2(x.w, s2)));
        }
      }
      publish(at);
    };
    const uint32_t to = smem0 + (8 * w + sub) * 128 + ((l8 ^ sub) * 16);  // key sub; 4 + sub: ^ 64, + 512
    int done = 0;  // place of the part to be published next
#pragma unroll 1
    for (int n = 0; n < 2 * g.n; ++n) {
      claim();
      if (!ok) break;
      const int h = n & 1;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t at = to + st * kPart8 + c * kChunk;
        cp_async16(at, from[0] + (2 * h + c) * 128, row[0]);
        cp_async16((at ^ 64) + 512, from[1] + (2 * h + c) * 128, row[1]);
      }
      if (h == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          cp_async16(rope_address(read, 4 * k + sub), from[k] + ds4f8::kOffRope, row[k]);
        if (l8 < 2) {
          const int32_t r = l8 ? row[1] : row[0];
          cp_async4(smem0 + kOffScale + ((read & 7) * kKeys + 8 * w + 4 * l8 + sub) * 4, p.scale + max(r, 0),
                    r);
        }
        note_there();
      } else {
        advance_rows();
      }
      cp_async_commit();
      step();
      if (n >= kLag) {
        cp_async_wait<kLag>();
        __syncwarp();
        finish(n - kLag, done);
        if (++done == kParts8) done = 0;
      }
    }
    cp_async_wait<0>();
    __syncwarp();
    for (int n = max(0, 2 * g.n - kLag); ok && n < 2 * g.n; ++n) {
      finish(n, done);
      if (++done == kParts8) done = 0;
    }
  } else if constexpr (kFormat == DS4IDX_CACHE_FP8) {
    // Values: a part is two lines of 128 codes (c) of rows sub and 4 + sub (k), 16 codes a lane. Three parts
    // are on their way, each a group of copies.
    const uint32_t raw0 = smem0 + kOffRaw + w * 2048 + lane * 16;  // + raw part, + 1024 c + 512 k
    // Turned are the line's first 64 codes of row `sub` by lanes 0..3 of eight, and the last 64 of the row
    // beside it by lanes 4..7: their 16-byte pieces go to different banks.
    const int turn = sub ^ (l8 >> 2);
    const uint32_t raw1 = smem0 + kOffRaw + w * 2048 + turn * 128 + l8 * 16;
    const uint32_t to = smem0 + (l8 >> 2) * kChunk + (8 * w + turn) * 128 + (((l8 & 3) * 2 ^ turn) * 16);
    int raw_in = 0, raw_out = 0;  // places of the part to be read next, and of the one to be turned next
    auto copy = [&](int h, int c, int k) {
      cp_async16(raw0 + raw_in * kRaw + 1024 * c + 512 * k, from[k] + (2 * h + c) * 128, row[k]);
    };
    auto copied = [&](int h) {
      if (h == 1) advance_rows();
      cp_async_commit();
      if (++raw_in == kRaws) raw_in = 0;
    };
#pragma unroll 1
    for (int n = 0; n < kRaws; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) copy(n & 1, c, 0), copy(n & 1, c, 1);
      copied(n & 1);
    }
    // The half h of tile i; the reads of the part three later go to where its codes were.
    auto part = [&](int i, int h, auto checked) {
      constexpr bool check = decltype(checked)::value;
      cp_async_wait<kRaws - 1>();
      __syncwarp();
      claim();
      if (!ok) return;
      const uint32_t raw = raw1 + raw_out * kRaw;
      if (++raw_out == kRaws) raw_out = 0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint4 x = ld_shared16(raw + 1024 * c + 512 * k);
          if constexpr (check) {
            if (drafted(i, 4 * k + turn) && odd_f8(x)) x = zero;
          }
          const uint32_t at = (to ^ (k * 64)) + st * kPart + 2 * c * kChunk + k * 512;
          uint4 v, u;
          codes_to_bf16(x.x, v.x, v.y);
          codes_to_bf16(x.y, v.z, v.w);
          codes_to_bf16(x.z, u.x, u.y);
          codes_to_bf16(x.w, u.z, u.w);
          st_shared16(at, v);
          st_shared16(at ^ 16, u);
        }
      }
      __syncwarp();  // (another lane's copies go where these codes were)
#pragma unroll
      for (int c = 0; c < 2; ++c) copy(h ^ 1, c, 0), copy(h ^ 1, c, 1);
      copied(h ^ 1);
      publish(st);
      step();
    };
#pragma unroll 1
    for (int n = 0; n < 2 * g.plain && ok; ++n) part(n >> 1, n & 1, std::false_type{});
#pragma unroll 1
    for (int n = 2 * g.plain; n < 2 * g.n && ok; ++n) part(n >> 1, n & 1, std::true_type{});
    cp_async_wait<0>();
  } else if constexpr (kFormat == DS4IDX_CACHE_BF16) {
    // straight to the operand; a part is published when the next one's copies are on their way
    int last = -1;
#pragma unroll 1
    for (int i = 0; i < g.n; ++i) {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        claim();
        if (!ok) break;
        const bool check = !kKey && i >= g.plain;
#pragma unroll 2
        for (int k = 0; k < 8; ++k) {  // rows sub and 4 + sub, a chunk of 64 dims (k >> 1)
          const int key = (k & 1) * 4 + sub;
          const int32_t r = k & 1 ? row[1] : row[0];
          const uint32_t at =
              smem0 + st * kPart + (k >> 1) * kChunk + (8 * w + key) * 128 + ((l8 ^ key) * 16);
          const uint8_t* src = (k & 1 ? from[1] : from[0]) + h * 2 * kHalf + (k >> 1) * 128;
          if (check) {
            const uint4 v = ld_row16(src, r);
            st_shared16(at, drafted(i, key) && odd_bf16(v) ? zero : v);
          } else {
            cp_async16(at, src, r);
          }
          if (kKey && h == 0 && k < 2)
            cp_async16(rope_address(i, key), (k & 1 ? from[1] : from[0]) + 2 * kLatent, r);
        }
        cp_async_commit();
        if (h == 0) note_there();
        if (last >= 0) {
          cp_async_wait<1>();
          publish(last);
        }
        last = st;
        step();
      }
      if (!ok) break;
      advance_rows();
    }
    cp_async_wait<0>();
    if (ok && last >= 0) publish(last);
  } else {
    // Eight lanes copy 128 bytes of codes (c) of rows sub and 4 + sub (k) at a time, four of them their scales.
    // Turned are 32 codes a lane of each, in each half of the dims: those that it copied.
    const int x = l8 >> 1;
    const uint32_t raw0 = smem0 + kOffRaw + w * 2048 + sub * 256 + l8 * 16;  // + raw tile, + 1024 k + 128 c
    const uint32_t raw_scale = smem0 + kOffScale + w * 256;                  // + 2048 raw tile
    int raw_in = 0, raw_out = 0;  // places of the tile to be read next, and of the one to be turned
    auto copy = [&] {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          cp_async16(raw0 + raw_in * kRaw + 1024 * k + 128 * c, from[k] + 128 * c, row[k]);
        if (kKey) cp_async16(rope_address(read, 4 * k + sub), from[k] + ds4q::kOffRope, row[k]);
      }
      const bool upper = l8 & 2;  // of the two rows
      if (l8 < 4)
        cp_async16(raw_scale + raw_in * 2048 + (4 * upper + sub) * 32 + (l8 & 1) * 16,
                   (upper ? from[1] : from[0]) + ds4q::kOffScale - l8 * 16 + (l8 & 1) * 16,
                   upper ? row[1] : row[0]);
      if (++raw_in == kRaws) raw_in = 0;
      note_there();
      cp_async_commit();
    };
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
      copy();
      advance_rows();
    }
#pragma unroll 1
    for (int n = 0; n < 2 * g.n; ++n) {
      const int h = n & 1;
      if (h == 0) cp_async_wait<1>();
      __syncwarp();
      claim();
      if (!ok) break;
      if (h == 0) {  // (a part of this tile has a place: tile i - 2 is done with, its rotary dims too)
        copy();
        advance_rows();
      }
      uint4 codes[2];
      uint32_t scales[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        codes[k] = ld_shared16(raw0 + raw_out * kRaw + 1024 * k + 128 * h);
        scales[k] = *reinterpret_cast<const uint16_t*>(smem + kOffScale + w * 256 + raw_out * 2048 +
                                                       (4 * k + sub) * 32 + (h * 8 + l8) * 2);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int key = 4 * k + sub;
        uint4 c = codes[k];
        uint32_t s = scales[k];
        // piece j ^ x at step j: the lanes of the other chunks write other banks
        swap_if(x & 1, c.x, c.y);
        swap_if(x & 1, c.z, c.w);
        swap_if(x & 2, c.x, c.z);
        swap_if(x & 2, c.y, c.w);
        s = x & 2 ? __byte_perm(s, 0, 0x4401) : s;
        const uint32_t at = smem0 + st * kPart + x * kChunk + (8 * w + key) * 128 +
                            ((((l8 & 1) * 4 + x) ^ key) * 16);
        const uint32_t words[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (a row that is not there: codes and scales of zeros, -8 * 2^-20, finite and not seen)
          const uint32_t s2 = __byte_perm(s, 0, j < 2 ? 0x4040u : 0x4141u) * 16u + 0x35803580u;
          st_shared16(at ^ (16 * j), ds4q::word_to_bf16(words[j], s2, ds4q::offset_bf16x2(s2)));
        }
      }
      publish(st);
      step();
      if (h == 1 && ++raw_out == kRaws) raw_out = 0;
    }
    cp_async_wait<0>();
  }
}

// A range's sum may be far above 1, as its m is stale: its power of two goes into the m that the ranges
// are joined by (0 for a sum of nothing, infinite or NaN).
__device__ __forceinline__ int excess(float l) {
  const int e = static_cast<int>(__float_as_uint(l) >> 23);
  return e == 0 || e >= 255 ? 0 : e - 127;
}
__device__ __forceinline__ float power(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// Two fp32 numbers, as bits, times two others.
__device__ __forceinline__ void mul_pair(uint32_t& a, uint32_t& b, uint32_t x, uint32_t y) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "mul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+r"(a), "+r"(b)
      : "r"(x), "r"(y));
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Four bf16 times a power of two as sums of an E4M3 and an E5M2 number: four significant bits, and three of
// the rest, which hold a bf16's eight exactly where the first is normal, 2^-6 and above; below that the error
// is at most 2^-14.
__device__ __forceinline__ void bf16_to_f8_pair(uint32_t a, uint32_t b, float f, uint32_t& hi, uint32_t& lo) {
  const float x[4] = {__uint_as_float(a << 16) * f, __uint_as_float(a & 0xFFFF0000u) * f,
                      __uint_as_float(b << 16) * f, __uint_as_float(b & 0xFFFF0000u) * f};
  asm("{\n\t.reg .b16 u, v;\n\tcvt.rn.satfinite.e4m3x2.f32 u, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 v, %4, %3;\n\tmov.b32 %0, {u, v};\n\t}"
      : "=r"(hi)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
  uint32_t h0, h1;
  ds4f8::codes_to_f16(hi, h0, h1);
  const float2 y0 = ds4f8::f16x2_to_f32(h0), y1 = ds4f8::f16x2_to_f32(h1);
  asm("{\n\t.reg .b16 u, v;\n\tcvt.rn.satfinite.e5m2x2.f32 u, %2, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 v, %4, %3;\n\tmov.b32 %0, {u, v};\n\t}"
      : "=r"(lo)
      : "f"(x[0] - y0.x), "f"(x[1] - y0.y), "f"(x[2] - y1.x), "f"(x[3] - y1.y));
}

template <int kFormat>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  // both CTAs of a pair have the same dynamic shared-memory base, so the offsets agree
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t smem0 = smem_u32(smem);
  float* s_f = reinterpret_cast<float*>(smem + kOffF);
  float* s_m = reinterpret_cast<float*>(smem + kOffM);
  float* s_l = reinterpret_cast<float*>(smem + kOffL);
  volatile uint64_t* s_there = reinterpret_cast<uint64_t*>(smem + kOffThere);
  uint64_t* part_full = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* part_empty = part_full + kParts8;
  uint64_t* q_full = part_empty + kParts8;
  uint64_t* s_ready = q_full + 1;   // [3] S of a tile is formed
  uint64_t* s_free = s_ready + 3;   // [3] and read
  uint64_t* p_free = s_free + 3;      // [4] rank 1 is done with P (in rank 0)
  uint64_t* p_full = p_free + kIn;  // [4] P has come (in rank 1)
  uint64_t* scaled = p_full + kIn;  // [4] O is ready for P V
  uint64_t* pv_done = scaled + kIn; // [4] P V of a tile is done
  uint64_t* m_full = pv_done + kIn;  // [8] a softmax warp's m is in s_m
  uint64_t* l_full = m_full + 8;    // the rows' sums have come (in rank 1)
  uint64_t* done = l_full + 1;      // every MMA has completed
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile uint32_t* s_abort = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The first ranges of all row tiles come first, so that those without keys are the last.
  const int rank = blockIdx.x & 1, nth = blockIdx.x >> 1, split = nth / p.items, group = nth % p.items;
  const int tile = group % p.tiles, b = group / p.tiles, item = group * p.splits + split;
  uint32_t* err = p.err;
  constexpr uint32_t kPBytes = kP + kRows * 4;  // what comes with a tile: P and the factors

  if (tid == 0) {
    for (int i = 0; i < kParts8; ++i) {
      mbar_init(&part_full[i], kLoaders);
      mbar_init(&part_empty[i], 1);
    }
    mbar_init(q_full, 8);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&s_ready[i], 1);
      mbar_init(&s_free[i], 4);
    }
    for (int i = 0; i < kIn; ++i) {
      mbar_init(&p_free[i], 8);
      mbar_init(&p_full[i], 1);
      mbar_init(&scaled[i], 8);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&m_full[i], 1);
    mbar_init(l_full, 4);
    mbar_init(done, 1);
    *s_abort = 0u;
    fence_mbar_init();
  }
  griddep_wait();
  const Range g = make_range(p, b, tile, split, lane);
  if (g.n == 0 && p.splits > 1) {  // nothing to do (with both barriers, whatever the other CTA finds)
    if (rank == 0 && tid < kRows) p.part_ml[static_cast<int64_t>(item) * 3 * kRows + tid] = kNegInf;
    cluster_sync();
    cluster_sync();
    return;
  }
  if (warp == kMmaWarp) {  // (before the range is known: 4 sequences of 64 nodes over 16384 rows 1% slower)
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  // (Not before every CTA has its tensor memory: a dependent that took it first would wait for this grid.)
  griddep_launch_dependents();
  cluster_sync();  // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  constexpr bool k8 = kFormat == DS4IDX_CACHE_FP8;

  if (warp < kLoad0) {
    const int grp = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
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
        // Q to TMEM by way of shared memory, so that it is read a line at a time: 2.1 us, beside 8-bit rows 4.2.
        // (There reading by the rows' threads took 17, and a pass of its own for the rows' largest values 5.7.)
        const int q_rows = min(kRows, p.N * p.H - tile * kRows);  // of the tile
        const uint8_t* q0 = reinterpret_cast<const uint8_t*>(
            p.q + (static_cast<int64_t>(b) * p.N * p.H + tile * kRows) * kDims);
        // Pieces of 32 dims, the groups in turn, two on their way: this warp's rows, 64 bytes each, in a
        // swizzle that spreads a column over the banks. The rotary dims are the last two.
        const uint32_t stage = smem0 + kOffMade + warp * 4096;
        auto copy_q = [&](int h) {
          if (h < 18) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int at = 8 * k + (lane >> 2), u = lane & 3, from = quad * 32 + at;
              const bool is = from < q_rows;
              cp_async16(stage + (h >> 1 & 1) * 2048 + at * 64 + ((u ^ (at >> 1)) & 3) * 16,
                         q0 + (is ? from : 0) * (2 * kDims) + h * 64 + u * 16, is ? 0 : -1);
            }
          }
          cp_async_commit();
        };
        copy_q(grp);
        copy_q(grp + 2);
        // The next of this group's pieces that are on their way.
        auto take_q = [&](int h, uint32_t(&v)[16]) {
          cp_async_wait<1>();
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 x = ld_shared16(stage + (h >> 1 & 1) * 2048 + lane * 64 + ((u ^ (lane >> 1)) & 3) * 16);
            v[4 * u] = x.x;
            v[4 * u + 1] = x.y;
            v[4 * u + 2] = x.z;
            v[4 * u + 3] = x.w;
          }
          __syncwarp();
          copy_q(h + 4);
        };
        if constexpr (k8) {
          // The pieces wait for the row's largest value, seven of a group's nine where S will be.
          const uint32_t aside = lanes + kColAside + grp * 7 * 16;
          uint32_t top = 0, v[16], latent[16], rope[16];
          auto raise = [&](const uint32_t(&x)[16]) {
#pragma unroll
            for (int j = 0; j < 16; ++j) top = __vmaxu2(top, x[j] & 0x7FFF7FFFu);
          };
#pragma unroll 1
          for (int j = 0; j < 7; ++j) {
            take_q(grp + 2 * j, v);
            raise(v);
            tmem_st16(aside + j * 16, v);
          }
          take_q(grp + 14, latent);
          raise(latent);
          take_q(grp + 16, rope);
          raise(rope);
          top = max(top & 0xFFFFu, top >> 16);
          s_l[grp * kRows + r] = __uint_as_float(top);
          tmem_wait_st();
          asm volatile("bar.sync 1, 256;" ::: "memory");
          // the power of two that takes it to 2^7 .. 2^8, or as near as a normal one whose inverse is normal
          // too does: rows below 2^-119 stay below 2^7. (A row that is not finite is multiplied by 0: NaN, where
          // the conversions would saturate.)
          const int e =
              static_cast<int>(max(top, __float_as_uint(s_l[(grp ^ 1) * kRows + r])) >> 7);  // biased by 127
          const int a = e == 255 ? -127 : min(126, 127 + 7 - e);
          const float f = power(a);
          auto put = [&](int h, const uint32_t(&x)[16]) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) bf16_to_f8_pair(x[2 * j], x[2 * j + 1], f, hi[j], lo[j]);
            tmem_st8(lanes + h * 8, hi);
            tmem_st8(lanes + kColLow + h * 8, lo);
          };
          put(grp + 14, latent);
          const uint32_t f2 = static_cast<uint32_t>(127 + a) * 0x00800080u;
#pragma unroll
          for (int j = 0; j < 16; ++j) rope[j] = ds4q::mul_bf16x2(rope[j], f2);
          tmem_st16(lanes + (grp + 16) * 16, rope);
#pragma unroll 1
          for (int j = 0; j < 7; ++j) {
            tmem_ld16(aside + j * 16, v);
            tmem_wait_ld();
            put(grp + 2 * j, v);
          }
          // (neither 0 nor infinite, which times a masked score's infinity or a score of 0 would be NaN)
          to_log2 = p.scale_fraction * power(max(-125, min(127, p.scale_exp - a)));
        } else {
#pragma unroll 1
          for (int h = grp; h < 18; h += 2) {
            uint32_t v[16];
            take_q(h, v);
            tmem_st16(lanes + h * 16, v);
          }
        }
        cp_async_wait<0>();
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      // Two sums: of the terms as they are, for lse, and of the bf16 terms that the values are multiplied by, for
      // the output. Divided by the latter, a term that outweighs the others loses nothing by its rounding: of
      // random rows with 13 keys that count the output is 1.1 times as far off as its own rounding leaves it,
      // where it is 1.5 times with the former. (The second sum costs 4% where most is to do, 4 sequences of 64
      // nodes over 16384 rows; terms cut to bf16 instead of rounded 3%, and further off where many keys count.)
      float m = kNegInf, l = 0.f, lr = 0.f;
      const uint32_t p_row = peer(smem0 + kOffP + r * 128 + (r & 7) * 16, 1);  // + kP * place
      const uint32_t f_row = peer(smem_u32(s_f + r), 1), bar0 = peer(smem_u32(p_full), 1);
      const uint32_t made = smem0 + kOffMade + grp * kP + r * 128 + (r & 7) * 16;
      auto tile_step = [&](int i, auto masked) {
        constexpr bool kMasked = decltype(masked)::value;
        const int slot = i % 3, at = i & 7, in = i & (kIn - 1);
        ok = wait_phase<false>(&s_ready[slot], (i / 3) & 1, s_abort, err);
        if (!ok) return;
        tc_fence_after();
        // which keys this row sees (all, of padding: what its row becomes is not used)
        uint64_t see = ~0ull;
        if constexpr (kMasked) {
          see = s_there[at];
          if (i >= g.plain) {
            const int32_t left = g.len - g.position(i);  // rows of the sequence from this tile on
            see &= left >= kKeys ? ~0ull
                   : left >= 0   ? ((1ull << left) - 1ull) | mask << left
                   : left > -64  ? mask >> -left
                                 : 0ull;
          }
        }
        // P with this group's m, in the layout of an MMA A operand; once more where m is another one now
        float f = 1.f, sum, sum_r;
        for (int pass = 0;; ++pass) {  // (at most twice)
          const float off = m == kNegInf ? 0.f : -m;
          const uint64_t off2 = pack_f32x2(off, off), scale2 = pack_f32x2(to_log2, to_log2);
          uint64_t sum2 = 0ull, sum2_r = 0ull;
          float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t s[32];  // fp32 bits
            tmem_ld32(lanes + kColS + slot * kKeys + 32 * h, s);
            tmem_wait_ld();
            if constexpr (k8) {
              const uint32_t sc = smem0 + kOffScale + (at * kKeys + 32 * h) * 4;
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const uint4 x = ld_shared16(sc + 4 * j);
                mul_pair(s[j], s[j + 1], x.x, x.y);
                mul_pair(s[j + 2], s[j + 3], x.z, x.w);
              }
            }
            if constexpr (kMasked) {  // a masked score is -infinity: p = 0 whatever m, and no maximum
              const uint32_t on = static_cast<uint32_t>(see >> (32 * h));
#pragma unroll
              for (int j = 0; j < 32; ++j) s[j] = on >> j & 1 ? s[j] : 0xFF800000u;
            }
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              mx[j / 2 & 3] = fmaxf(fmaxf(mx[j / 2 & 3], __uint_as_float(s[j])), __uint_as_float(s[j + 1]));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t pk[4];
              [[maybe_unused]] uint4 sa, sb;
              if constexpr (k8) {
                const uint32_t sc = smem0 + kOffScale + (at * kKeys + 32 * h + 8 * u) * 4;
                sa = ld_shared16(sc);
                sb = ld_shared16(sc + 16);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int k = 8 * u + 2 * j;
                float x0, x1;
                unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])),
                                       scale2, off2),
                             x0, x1);
                const float e0 = exp2_approx(x0), e1 = exp2_approx(x1);
                sum2 = add_f32x2(sum2, pack_f32x2(e0, e1));
                uint32_t r2 = pack_bf16x2(e0, e1);
                sum2_r = add_f32x2(sum2_r, pack_f32x2(__uint_as_float(r2 << 16),
                                                      __uint_as_float(r2 & 0xFFFF0000u)));
                if constexpr (k8) {  // the values are codes as well; a scale's upper half is all of it
                  r2 = ds4q::mul_bf16x2(r2, j == 0   ? __byte_perm(sa.x, sa.y, 0x7632)
                                            : j == 1 ? __byte_perm(sa.z, sa.w, 0x7632)
                                            : j == 2 ? __byte_perm(sb.x, sb.y, 0x7632)
                                                     : __byte_perm(sb.z, sb.w, 0x7632));
                  if constexpr (kMasked)  // (0 times a scale that is not finite)
                    r2 &= (see >> (32 * h + k) & 1 ? 0xFFFFu : 0u) |
                          (see >> (32 * h + k + 1) & 1 ? 0xFFFF0000u : 0u);
                }
                pk[j] = r2;
              }
              st_shared16(made ^ (16 * (4 * h + u)), make_uint4(pk[0], pk[1], pk[2], pk[3]));
            }
          }
          float l0, l1;
          unpack_f32x2(sum2, l0, l1);
          sum = l0 + l1;
          unpack_f32x2(sum2_r, l0, l1);
          sum_r = l0 + l1;
          if (pass == 1) break;
          // m after the tile before, which the other group took; raised where a score passes it by more
          // than the slack. Finite once a key was seen: a score of +-infinity keeps its meaning in s - m.
          float before = kNegInf;
          if (i > 0) {
            ok = wait_phase<false>(&m_full[warp ^ 4], ((i - 1) >> 1) & 1, s_abort, err);
            if (!ok) return;
            before = s_m[(grp ^ 1) * kRows + r];
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * to_log2;
          float now = fminf(fmaxf(top, -kMax), kMax);
          if (see == 0ull || (before != kNegInf && now <= before + kSlack<kFormat>)) now = before;
          s_m[grp * kRows + r] = now;
          __syncwarp();
          if (lane == 0) mbar_arrive(&m_full[warp]);
          // Roots of factors: what is 2^kSlack above an old m may matter 2^-126 above the new one, where
          // 2^(old - new) is long zero.
          if (now != before && before != kNegInf) f = exp2_approx(0.5f * (before - now));
          const bool other = now != m;
          if (other) {
            const float fl = m == kNegInf ? 0.f : exp2_approx(0.5f * (m - now));
            l = l * fl * fl;
            lr = lr * fl * fl;
            m = now;
          }
          if (!__any_sync(0xffffffffu, other)) break;
        }
        l += sum;
        lr += sum_r;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[slot]);
        // this row to rank 1
        ok = wait_phase<true>(&p_free[in], (i / kIn & 1) ^ 1u, s_abort, err);
        if (!ok) return;
        const uint32_t bar = bar0 + in * 8, p_at = p_row + in * kP;
#pragma unroll
        for (int u = 0; u < 8; ++u) st_async16(p_at ^ (16 * u), ld_shared16(made ^ (16 * u)), bar);
        st_async4(f_row + in * kRows * 4, f, bar);
      };
      const bool holes = p.place.table != nullptr;  // a page may be missing among the sequence's rows
#pragma unroll 1
      for (int i = grp; i < g.n && ok; i += 2) {
        if (i < g.plain) {
          if (holes) ok = wait_phase<false>(&s_ready[i % 3], (i / 3) & 1, s_abort, err);
          if (!ok) break;
          if (!holes || s_there[i & 7] == ~0ull) {
            tile_step(i, std::false_type{});
            continue;
          }
        }
        tile_step(i, std::true_type{});
      }
      // ---------------- both groups' sums, to rank 1
      s_l[grp * kRows + r] = l;
      s_l[(2 + grp) * kRows + r] = m;
      s_l[(4 + grp) * kRows + r] = lr;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (grp == 0) {
        m = g.n > 0 ? s_m[((g.n - 1) & 1) * kRows + r] : kNegInf;
        l = lr = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float mk = s_l[(2 + k) * kRows + r];
          const float fl = mk == m ? 1.f : exp2_approx(0.5f * (mk - m));
          if (mk != kNegInf) l += s_l[k * kRows + r] * fl * fl, lr += s_l[(4 + k) * kRows + r] * fl * fl;
        }
        if (padding) m = kNegInf, l = lr = 0.f;
        st_peer(peer(smem_u32(s_l + r), 1), lr);
        st_peer(peer(smem_u32(s_l + kRows + r), 1), m);
        __syncwarp();
        if (lane == 0) arrive_peer(peer(smem_u32(l_full), 1));
        if (p.splits > 1) {
          const int k = excess(lr);
          float* ml = p.part_ml + static_cast<int64_t>(item) * 3 * kRows + r;
          ml[0] = m + static_cast<float>(k);
          ml[kRows] = l * power(-k);
          ml[2 * kRows] = lr * power(-k);
        } else if (used && p.lse) {
          p.lse[out_row] = m == kNegInf ? kNegInf : (m + __log2f(l)) * 0.69314718055994531f;
        }
      }
    } else {
      // ---------------- O: rescaled where m was raised, at the end written; 256 columns a group
      const uint32_t o = lanes + grp * kHalf;
      uint32_t seen = 0;  // tiles of P that have come
      if (tid == 0)
        for (int i = 0; i < kIn; ++i) mbar_arrive_expect_tx(&p_full[i], kPBytes);
#pragma unroll 1
      for (int i = 0; i < g.n; ++i) {
        const int slot = i & (kIn - 1);
        const uint32_t parity = i / kIn & 1;
        ok = wait_phase<true>(&p_full[slot], parity, s_abort, err);
        if (!ok) break;
        ++seen;
        const float f = s_f[slot * kRows + r];
        if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {  // (P V of the tile before was waited for)
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kHalf; c += 32) {
            uint32_t v[32];
            tmem_ld32(o + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f * f);
            tmem_st32(o + c, v);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scaled[slot]);
        ok = wait_phase<false>(&pv_done[slot], parity, s_abort, err);
        if (!ok) break;
        if (tid == 0 && i + kIn < g.n) mbar_arrive_expect_tx(&p_full[slot], kPBytes);
        __syncwarp();
        if (lane == 0) arrive_peer(peer(smem_u32(&p_free[slot]), 0));
      }
      // never leave with stores in flight to here (after an abort: bounded)
      if (!ok && tid == 0)
        for (uint32_t i = seen; i < min(seen + kIn, static_cast<uint32_t>(g.n)); ++i)
          mbar_drain(&p_full[i & (kIn - 1)], i / kIn & 1);
      __syncwarp();
      ok = wait_phase<true>(l_full, 0u, s_abort, err) && ok;
      tc_fence_after();
      const float l = s_l[r];
      const bool none = s_l[kRows + r] == kNegInf;
      if (p.splits == 1) {
        const float inv = none ? 0.f : 1.f / l;
        uint16_t* dst = p.out + out_row * kLatent + grp * kHalf;
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
          uint32_t v[32], pk[16];
          if (g.n > 0) {
            tmem_ld32(o + c, v);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            pk[j / 2] =
                none ? 0u : pack_bf16x2(__uint_as_float(v[j]) * inv, __uint_as_float(v[j + 1]) * inv);
          if (used && ok) {
#pragma unroll
            for (int j = 0; j < 2; ++j) st_global32(dst + c + 16 * j, &pk[8 * j]);
          }
        }
      } else if (g.n > 0 && ok) {
        const float f = power(-excess(l));
        float4* dst =
            reinterpret_cast<float4*>(p.part_o) + (static_cast<int64_t>(item) * 128 + grp * 64) * kRows + r;
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
          uint32_t v[32];
          tmem_ld32(o + c, v);
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
    // ---------------- rows to operands
    if (rank == 0)
      load_rows<kFormat, true>(p, g, b, warp - kLoad0, lane, smem, part_full, part_empty, s_abort);
    else
      load_rows<kFormat, false>(p, g, b, warp - kLoad0, lane, smem, part_full, part_empty, s_abort);
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
        ok = ok && wait_phase<false>(&part_full[st], parity, s_abort, err);
        if constexpr (kFenceByMma<kFormat>) fence_proxy_async_smem();
        tc_fence_after();
      };
      auto part_taken = [&] {
        commit(&part_empty[st]);
        if (++st == (k8 && rank == 0 ? kParts8 : kParts)) st = 0, parity ^= 1u;
      };
      if (rank == 0) {
        const uint64_t k0 = smem_desc_sw128(smem0), r0 = smem_desc_sw128(smem0 + kOffRope);
        constexpr uint32_t idesc = instr_desc(1u, 1u, kRows, kKeys);
        constexpr uint32_t hi_idesc = instr_desc(0u, 0u, kRows, kKeys);  // E4M3 x E4M3
        constexpr uint32_t lo_idesc = instr_desc(1u, 0u, kRows, kKeys);  // E5M2 x E4M3
        if (g.n > 0) ok = wait_phase<false>(q_full, 0u, s_abort, err);
        int slot = 0;
        uint32_t s_parity = 1;
#pragma unroll 1
        for (int i = 0; ok && i < g.n; ++i) {
          ok = wait_phase<false>(&s_free[slot], s_parity, s_abort, err);
          const uint32_t d = tmem + kColS + slot * kKeys;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            part_ready();
            if (!ok) break;
            if constexpr (k8) {
              const uint64_t kd = k0 + st * (kPart8 >> 4);
              if (lead) {
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint32_t col = tmem + h * 64 + c * 32 + k * 8;
                    const uint64_t b_desc = kd + c * (kChunk >> 4) + k * 2;
                    mma_fp8_ts(d, col, b_desc, hi_idesc, (h | c | k) ? 1u : 0u);
                    mma_fp8_ts(d, col + kColLow, b_desc, lo_idesc, 1u);
                  }
                }
              }
            } else {
              const uint64_t kd = k0 + st * (kPart >> 4);
              if (lead) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    mma_bf16_ts(d, tmem + h * 128 + c * 32 + k * 8, kd + c * (kChunk >> 4) + k * 2, idesc,
                                (h | c | k) ? 1u : 0u);
                }
              }
            }
            if (h == 1 && lead) {
              const uint64_t rd = r0 + (i & 3) * (kChunk >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16_ts(d, tmem + kColRope + k * 8, rd + 2 * k, idesc, 1u);
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
          const int slot = i & (kIn - 1);
          const uint32_t parity = i / kIn & 1;
          ok = wait_phase<true>(&p_full[slot], parity, s_abort, err);
          if (!ok) break;
          fence_proxy_async_cluster();
          const float4 f = reinterpret_cast<const float4*>(s_f + slot * kRows)[lane];
          if (__any_sync(0xffffffffu, f.x != 1.f || f.y != 1.f || f.z != 1.f || f.w != 1.f))
            ok = wait_phase<false>(&scaled[slot], parity, s_abort, err);
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

// Joins the ranges of a row tile: four columns of one row by one thread, or, from kJoinMany ranges on, by
// four that take every fourth range each, since reading one range after the other is then what takes the
// time. Measured, whole calls with 128 heads, one thread and four: one node over 64 ranges 39.9 and 28.6 us,
// 5 nodes over 15 71.7 and 68.6, 7 over 10 103.3 and 102.8, 9 over 8 121.6 and 122.9, 13 over 5 177.4 and
// 182.0. Ranges without a seen key carry m = -infinity and no O.
constexpr int kJoinMany = 10;
template <int kJoinParts>
__global__ void __launch_bounds__(kRows * kJoinParts) tree_join_kernel(const __grid_constant__ Params p) {
  __shared__ float s_m[kJoinParts][kRows], s_l[kJoinParts][kRows], s_r[kJoinParts][kRows];
  __shared__ float4 s_o[kJoinParts][kRows];
  griddep_wait();
  griddep_launch_dependents();
  const int quad = blockIdx.x % 128, r = threadIdx.x % kRows, part = threadIdx.x / kRows;  // columns 4 quad ..
  const int64_t group = blockIdx.x / 128;              // (sequence, row tile)
  const int tile = static_cast<int>(group % p.tiles);
  const int64_t b = group / p.tiles;
  const int row = tile * kRows + r;
  const float* ml = p.part_ml + group * p.splits * 3 * kRows + r;
  float m = kNegInf;
#pragma unroll 4
  for (int i = part; i < p.splits; i += kJoinParts) m = fmaxf(m, ml[i * 3 * kRows]);
  s_m[part][r] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kJoinParts; ++k) m = fmaxf(m, s_m[k][r]);
  float l = 0.f, lr = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                      (group * p.splits * 128 + quad) * kRows + r;
#pragma unroll 4
  for (int i = part; i < p.splits; i += kJoinParts) {
    const float mi = ml[i * 3 * kRows];
    if (mi == kNegInf) continue;
    const float f = exp2_approx(mi - m);
    const float4 v = src[static_cast<int64_t>(i) * 128 * kRows];
    l = fmaf(ml[i * 3 * kRows + kRows], f, l);
    lr = fmaf(ml[i * 3 * kRows + 2 * kRows], f, lr);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
  s_l[part][r] = l;
  s_r[part][r] = lr;
  s_o[part][r] = o;
  __syncthreads();
  if (part > 0 || row >= p.N * p.H) return;
#pragma unroll
  for (int k = 1; k < kJoinParts; ++k) {
    const float4 v = s_o[k][r];
    l += s_l[k][r];
    lr += s_r[k][r];
    o.x += v.x;
    o.y += v.y;
    o.z += v.z;
    o.w += v.w;
  }
  const bool none = m == kNegInf;
  const float inv = none ? 0.f : 1.f / lr;
  const int64_t out_row = b * p.N * p.H + row;
  if (quad == 0 && p.lse) p.lse[out_row] = none ? kNegInf : (m + __log2f(l)) * 0.69314718055994531f;
  *reinterpret_cast<uint2*>(p.out + out_row * kLatent + 4 * quad) =
      none ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// Pairs of CTAs that run at once: one CTA an SM.
int64_t pairs_at_once() { return sm_count() / 2; }

struct Plan {
  int32_t tiles, items, splits, fill, steps;
  int64_t o_bytes, bytes;
};
// Key ranges: the number that takes the least time, in steps of 64 keys (1.35 us). A range costs some 14
// steps besides its own (set-up, Q, its part of O, and what its last products wait for), the join 4. Several
// sequences have lengths of their own, so that not every pair of a last round has as much to do: half way
// between full rounds and ranges of three quarters of the longest without a gap. (8 ragged sequences of 7
// nodes and up to 5000 rows: 127 us as one range each, 90 as two, 113 as three; 3 of 31 nodes, 16 heads, 12001
// rows: 139 as three, 80 as six, 109 as nine; 13 nodes over 32768 rows: 247 as three, 156 as five, 179 as ten.)
// The kernel divides each sequence by its own length, the bound may be far above it: into the ranges of the grid, but
// not more than fill the device once while those are shorter than three times what a range costs besides, or six
// times where there are row tiles for all pairs anyway. (Whole calls, bound as long as the longest sequence and far
// above: one node over 8192 rows 28.4 and 29.3 us, 89 to 181 where a range was as long as the bound's; 8 ragged
// sequences of 7 nodes, 800 to 5000 rows, 87 and 84, 128; 32 of 4 nodes over 4096 rows 198 and 225, 254; 64 of one
// node over 1000 rows 37 and 65, 98: seven ranges a sequence, six of them without keys.)
// At most eight rounds of pairs: more would save 0.6% at the most, and eight hold the workspace under 161 MB.
constexpr int64_t kRangeCost = 14, kJoinCost = 4, kRounds = 8;
constexpr int64_t kPartBytes = 2 * 64 * kRows * 16, kPartSums = 3 * kRows * 4;  // of a range
Plan make_plan(int64_t pairs, int32_t B, int32_t N, int32_t H, int64_t max_kv_len) {
  Plan pl{};
  pl.tiles = (N * H + kRows - 1) / kRows;
  const int64_t items = static_cast<int64_t>(B) * pl.tiles;
  const int64_t steps = std::max<int64_t>(1, (max_kv_len + N + kKeys - 1) / kKeys);
  int64_t best = 0, best_cost = 0;
  for (int64_t n = 1; n <= std::min<int64_t>(steps, 2 * pairs); ++n) {
    const int64_t per = (steps + n - 1) / n, waves = (items * n + pairs - 1) / pairs;
    if (n > 1 && waves > kRounds) break;
    int64_t cost = waves * (per + kRangeCost);
    if (B > 1 && waves > 1)
      cost = (cost + std::max(per + kRangeCost, items * n * (3 * per / 4 + kRangeCost) / pairs)) / 2;
    if (n > 1) cost += kJoinCost;
    if (best == 0 || cost < best_cost) best = n, best_cost = cost;
  }
  pl.splits = static_cast<int32_t>(best);
  pl.items = static_cast<int32_t>(items);
  pl.fill = static_cast<int32_t>(std::max<int64_t>(1, pairs / items));
  pl.steps = static_cast<int32_t>(
      std::min((steps + best - 1) / best, (items <= pairs ? 3 : 6) * kRangeCost));
  pl.o_bytes = items * best * kPartBytes;
  if (best > 1) pl.bytes = pl.o_bytes + items * best * kPartSums;
  return pl;
}

// Bytes that suffice for every bound up to max_kv_len. The best number of ranges goes up and down with the bound, a
// limit of it does not go down: with a = items / pairs, n ranges of s steps in all take a s + 14 a n at the least, or
// 7/8 a s + 109/8 a n - 1 where full rounds are weighed against ragged sequences, and the join. They are chosen only
// where that is less than one round's ranges take, s / fill + 19 at the most, or, where a round does not hold one
// range of each row tile, than one range each does, r (s + 14) in r rounds.
int64_t enough_workspace(int64_t pairs, int32_t B, int32_t N, int32_t H, int64_t max_kv_len) {
  const int64_t items = static_cast<int64_t>(B) * ((N * H + kRows - 1) / kRows);
  const double s = static_cast<double>(std::max<int64_t>(1, (max_kv_len + N + kKeys - 1) / kKeys));
  const double a = static_cast<double>(items) / pairs, rounds = std::ceil(a);
  const int64_t fill = std::max<int64_t>(1, pairs / items);
  const double other = items <= pairs ? s / fill + 19 : rounds * (s + kRangeCost);
  const double most = B > 1 ? (other - 0.875 * a * s - kJoinCost + 1) / (13.625 * a)
                            : (other - a * s - kJoinCost) / (kRangeCost * a);
  const double rounds_hold = static_cast<double>(kRounds * pairs / items);
  const int64_t n = static_cast<int64_t>(
      std::min({s, 2.0 * pairs, std::max(rounds_hold, 1.0), std::max(most, static_cast<double>(fill))}));
  return n > 1 ? items * n * (kPartBytes + kPartSums) : 0;
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
  *bytes = B ? enough_workspace(pairs, B, n_nodes, n_heads, max_kv_len) : 0;
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
      !aligned_to(out, 32) || !aligned_to(lse, 4) || !aligned_to(workspace, 16) ||
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
  p.items = pl.items;
  p.fill = pl.fill;
  p.steps = pl.steps;
  // A subnormal scale of products below 2^128 leaves scores off by 2^-22 at most. Beside 8-bit rows, whose
  // queries are scaled as well, it is held in full.
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.scale_fraction = static_cast<float>(std::frexp(
      p.scale_log2 < 0x1p-126f ? sm_scale * 1.4426950408889634 : p.scale_log2, &p.scale_exp));
  const int64_t items = static_cast<int64_t>(B) * pl.tiles * pl.splits;
  if (items * 2 > 0x7FFFFFFF) return DS4IDX_ERR_INVALID_ARG;
  const int st = format == DS4IDX_CACHE_FP8    ? launch<DS4IDX_CACHE_FP8>(p, items, stream)
                 : format == DS4IDX_CACHE_BF16 ? launch<DS4IDX_CACHE_BF16>(p, items, stream)
                                               : launch<DS4IDX_CACHE_Q4>(p, items, stream);
  if (st != DS4IDX_OK || pl.splits == 1) return st;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(B) * pl.tiles * 128);
  return pl.splits < kJoinMany ? launch_dependent(tree_join_kernel<1>, blocks, kRows, 0, 1, stream, p)
                               : launch_dependent(tree_join_kernel<4>, blocks, kRows * 4, 0, 1, stream, p);
}
