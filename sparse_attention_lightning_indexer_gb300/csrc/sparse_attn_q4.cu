// Sparse attention over the selected rows of a 4-bit latent cache, for sm_103a: one latent row
// (q4_format.cuh) per position, shared by all heads; 576-wide keys, the first 512 dims are values.
//
// A cluster of C = 1, 2, 4 or 8 CTAs owns one token. Both products are split without partial sums:
//   A  S[128 heads x 512/C keys] = Q K^T: a CTA takes its share of the list's slots (TMEM columns
//      0 .. 512/C - 1). First the rotary chunk of 64 dims, whose keys are copied as they are, then
//      the 8 latent chunks: worker threads read codes, turn them into bf16 (exact) and write the
//      128-byte-swizzled operand in stages of 64 KB. Q chunks come by TMA.
//   B  softmax: the row maxima and sums of the CTAs meet in each other's shared memory, so every
//      probability is final relative to the list's maximum; P goes as bf16 into shared memory in
//      the layout of an MMA A operand, each CTA's share copied to the others by bulk copies.
//   C  O[128 heads x 512/C dims] = P V over all slots: blocks of 32 or 64 keys of the CTA's value
//      dims are turned into bf16 again, as an MN-major B operand. Nothing is joined afterwards.
// C = 1 fills the GPU for many tokens: its CTAs stay and take tokens in turn, reading the next
// token's first rows behind this one's products. A cluster shortens the chain of phases for few.
//
// Warps 0..15 are the workers (unpacking, softmax, output: TMEM lane quadrant warp % 4, column
// quarter warp / 4), warp 16 issues tcgen05.mma, warp 17 loads Q and the next token's row list.
//
// The unpacked tile serves as K (K-major) and as V (MN-major) in the same layout; it is made
// twice because O takes all 512 TMEM columns at C = 1, so P V starts only after the whole of S is
// read, and 512 unpacked rows (576 KB) do not fit shared memory.
//
// 128 heads, 512 rows: 11.4 us for one token (C = 8; the latency of the phases), 680 us for 4096
// tokens of a 65536-row cache (780 with key weights), 859 TFLOP/s, 0.44 of the measured tensor peak:
// bound by the unpacking on the half-rate integer pipe and by shared memory, of which the MMAs read
// 96 bytes a clock.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include "attn_ptx.cuh"
#include "launch.cuh"
#include "placement.cuh"
#include "ptx.cuh"
#include "q4_format.cuh"

namespace ds4a {
extern uint32_t* sparse_attention_error_word();  // device address of the shared error word
}

namespace ds4qa {

using namespace ds4;
using namespace ds4q;

constexpr int kH = 128;        // MMA M = TMEM lanes; heads beyond n_heads are not stored
constexpr int kK = 512;        // list slots
constexpr int kChunks = 9;     // 64-dim chunks of a key: 8 latent, 1 rotary
constexpr int kWorkers = 512, kMmaWarp = 16;  // warp 17 loads Q
constexpr int kThreads = 18 * 32;
constexpr int kQBytes = kH * 128;
constexpr int kPBlock = kH * 128;            // 64 keys of P
constexpr int kOffV = (kK / 64) * kPBlock;   // P first, then the V blocks
constexpr int kVBytes = 64 * 1024;
constexpr float kNegInf = -__builtin_inff(), kMax = __FLT_MAX__;

template <int C>
struct Cfg {
  static constexpr int NK = kK / C;                     // slots of a CTA
  // One latent stage: KS keys x CW chunks of 64 dims, one (key, chunk) a worker thread, 64 KB.
  static constexpr int KS = NK < 256 ? NK : 256;
  static constexpr int CW = kWorkers / KS;              // 2, 2, 4, 8
  static constexpr int Stages = 8 / CW;                 // per key part
  static constexpr int KeyParts = NK / KS;              // 2 at C = 1
  static constexpr int KSlots = C == 8 ? 1 : 2;
  static constexpr int KSlot = KS * CW * 128;           // 64 KB
  static constexpr int OffQ = KSlots * KSlot;
  // The ring of 16 KB items: a token's rotary key pieces, its rotary Q chunk, its other Q chunks.
  static constexpr int NQS = C == 8 ? 9 : 5;
  static constexpr int RP = NK < 128 ? NK : 128;        // keys of a rotary piece
  static constexpr int RingBytes = OffQ + NQS * kQBytes;
  static constexpr int Region = RingBytes > kOffV + kVBytes ? RingBytes : kOffV + kVBytes;
  // Lanes that share a row: 2 (64 bytes of codes) where a stage has two chunks of 256 keys.
  static constexpr int RowLanes = C <= 2 ? 2 : 1;
  static constexpr int DV = kLatent / C;                // value dims of a CTA
  static constexpr int NB = DV / 64 < 4 ? DV / 64 : 4;  // 64-dim pieces of a V block
  static constexpr int Halves = DV / 64 / NB;           // passes over the keys (2 at C = 1)
  // Keys of a V block. At C = 1 blocks of 32 in four stages: one group's hand-over to the products
  // hides behind three others (4096 tokens 677 us, blocks of 64 in two stages 703). A pair of CTAs
  // gains nothing by that, as its products also wait for P, and pays for twice the hand-overs (37
  // tokens 21.4 us, with 64 keys 20.8).
  static constexpr int VK = C == 1 ? 32 : 64;
  static constexpr int VBlocks = kK / VK;               // at most, per pass
  static constexpr int VStage = NB * VK * 128;
  static constexpr int GV = kVBytes / VStage;           // V blocks in the making = V stages
  static constexpr int VLanes = NB == 4 ? 4 : 1;        // lanes that share a row of a V block
  static constexpr int OCol = C == 1 ? 0 : 256;         // first TMEM column of O
  static constexpr int CP = NK / 4;                     // S columns of a thread
  static constexpr int W = CP < 32 ? CP : 32;
  static constexpr int OP = DV / 4;                     // O columns of a thread
  static constexpr int OW = OP < 32 ? OP : 32;
  // The output is staged over P at C = 1. In a cluster this CTA's copies of P may still be read, so
  // it goes over the V blocks, which hold it (512 / C dims).
  static constexpr int OffO = C == 1 ? 0 : kOffV;
  static_assert(C == 1 || DV / 64 * kPBlock <= kVBytes, "output staging");

  static constexpr int OffRows = Region;
  static constexpr int Bufs = C == 1 ? 2 : 1;           // row lists: this token's and the next's
  static constexpr int OffMask = OffRows + Bufs * kK * 4;
  static constexpr int OffRed = OffMask + Bufs * 64;                     // [2][4][128] max, sum
  static constexpr int OffX = OffRed + 2 * 4 * kH * 4;            // [2][C][128] of the cluster
  static constexpr int OffW = OffX + (C > 1 ? 2 * C * kH * 4 : 0);  // [4][NK] key weights
  static constexpr int OffBars = OffW + 4 * NK * 4;
  static constexpr int NumBars = 2 * NQS + 2 * 2 + 2 * GV + 10 + C;
  static constexpr int OffMisc = OffBars + NumBars * 8;
  static constexpr int Smem = OffMisc + 16 + 1024;
  static_assert(GV * VK * NB == kWorkers && Smem <= 232448, "one (key, chunk) a worker thread");
};

struct Params {
  const uint8_t* cache;
  const int32_t* idx;
  float* lse;
  float* weights;
  uint32_t* err;
  Placement place;
  int32_t T, n_heads, n_sel;
  float scale_log2;
};

// One 32-byte sector. Without allocation in L1: every row is another line, and the few lines that
// the shared memory leaves to L1 would bound the loads in flight (chunk of 4096: 988 -> 838 us).
__device__ __forceinline__ void ld32(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar,
                                            int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* src, const CUtensorMap* m, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}
// Closes this thread's group of bulk stores; waits until all but the last N groups have read
// shared memory.
__device__ __forceinline__ void bulk_store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_store_wait() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// ---- other CTAs of the cluster
// mbar_wait with acquire at cluster scope, for data other CTAs stored here.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity,
                                             volatile uint32_t* abort_flag, uint32_t* err) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 63u) == 0u) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1u;
        atomicOr(err, 1u);
        return false;
      }
    }
  }
}
__device__ __forceinline__ void copy_to_peer(uint32_t dst, uint32_t src, uint32_t bytes,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// One 64-dim chunk of a latent row to the 128 swizzled bytes of row `r` at `base`. Where several
// lanes share a row (each its own chunk, chunks a multiple of 1 KB apart), lane x of them writes
// its 16-byte pieces in the order u ^ x * 8 / kLanes, so that the eight lanes of a store
// wavefront hit eight different banks.
template <int kLanes>
__device__ __forceinline__ void store_chunk(uint32_t base, int r, uint32_t (&codes)[8],
                                            uint32_t scales, int x) {
  int ord = 0;
  if constexpr (kLanes == 2) {
    ord = 4 * x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = codes[j], b = codes[j + 4];
      codes[j] = x ? b : a;
      codes[j + 4] = x ? a : b;
    }
    scales = x ? __funnelshift_l(scales, scales, 16) : scales;  // groups g ^ 2
  } else if constexpr (kLanes == 4) {
    ord = 2 * x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = codes[j], b = codes[j + 4];
      codes[j] = x & 2 ? b : a;
      codes[j + 4] = x & 2 ? a : b;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 4)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t a = codes[j + k], b = codes[j + k + 2];
        codes[j + k] = x & 1 ? b : a;
        codes[j + k + 2] = x & 1 ? a : b;
      }
    scales = __byte_perm(scales, 0, 0x3210u ^ (0x1111u * x));  // groups g ^ x
  }
  const uint32_t at = base + r * 128 + (((r & 7) ^ ord) * 16);  // rows are 128-byte aligned
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    // the scale byte in both halves, to bf16 (q4_format.cuh)
    const uint32_t s2 = __byte_perm(scales, 0, 0x4040u | (g << 8) | g) * 16u + 0x35803580u;
    const uint32_t c2 = offset_bf16x2(s2);
    st_shared16(at ^ (32 * g), word_to_bf16(codes[2 * g], s2, c2));
    st_shared16(at ^ (32 * g + 16), word_to_bf16(codes[2 * g + 1], s2, c2));
  }
}

// Sum over the warp of each of v[0..W-1]: lane l returns the total of v[l % W] (W = 16 or 32),
// added in a fixed order.
template <int W>
__device__ __forceinline__ float column_sums(float (&v)[W], int lane) {
  if (W == 16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], 16);
  }
#pragma unroll
  for (int o = W / 2; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float keep = up ? v[j + o] : v[j], give = up ? v[j] : v[j + o];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[W]) {
  if constexpr (W == 32) tmem_ld32(addr, r);
  else tmem_ld16(addr, r);
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1)
    sparse_attn_q4_kernel(const __grid_constant__ CUtensorMap tmap_q,
                          const __grid_constant__ CUtensorMap tmap_o,
                          const __grid_constant__ Params p) {
  using F = Cfg<C>;
  extern __shared__ uint8_t smem_raw[];
  // every CTA of a cluster has the same dynamic shared-memory base, so the offsets agree
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t smem0 = smem_u32(smem);
  float* s_red = reinterpret_cast<float*>(smem + F::OffRed);
  float* s_x = reinterpret_cast<float*>(smem + F::OffX);
  float* s_w = reinterpret_cast<float*>(smem + F::OffW);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + F::OffBars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + F::NQS;
  uint64_t* k_full = q_empty + F::NQS;
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + F::GV;
  uint64_t* s_ready = v_empty + F::GV;
  uint64_t* m_full = s_ready + 1;
  uint64_t* l_full = s_ready + 2;
  uint64_t* o_ready = s_ready + 4;
  uint64_t* o_free = s_ready + 5;     // O is read, S may be written again
  uint64_t* rows_full = s_ready + 6;  // [2] a later token's row list is in place
  uint64_t* done = s_ready + 8;       // every MMA has completed
  uint64_t* rope_full = s_ready + 9;  // the rotary pieces are in place
  uint64_t* p_full = s_ready + 10;    // [C] P of each CTA's slots is in place here
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + F::OffMisc);
  volatile uint32_t* s_abort = reinterpret_cast<volatile uint32_t*>(smem + F::OffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // C = 1: CTAs that stay, taking tokens blockIdx.x, blockIdx.x + gridDim.x, ...
  const int t_first = blockIdx.x / C, t_step = gridDim.x;
  const int rank = blockIdx.x % C;
  uint32_t* err = p.err;

  if (tid == 0) {
    for (int i = 0; i < F::NQS; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 16);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < F::GV; ++i) {
      mbar_init(&v_full[i], F::VK * F::NB / 32);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(s_ready, 1);
    mbar_init(m_full, 4 * C);
    mbar_init(l_full, 4 * C);
    for (int i = 0; i < C; ++i) mbar_init(&p_full[i], i == rank ? 16 : 1);
    mbar_init(o_ready, 1);
    mbar_init(o_free, 17);
    mbar_init(&rows_full[0], 1);
    mbar_init(&rows_full[1], 1);
    mbar_init(done, 1);
    mbar_init(rope_full, 16);
    *s_abort = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  // The row list of a token: slots j = base + (0 .. 31) by one warp.
  auto load_rows = [&](int t, int buf, int base) {
    const int j = base + lane;
    int64_t r = -1;
    if (j < p.n_sel)
      r = place_row(p.place, place_token(p.place, t),
                    p.idx[static_cast<int64_t>(t) * p.n_sel + j]);
    reinterpret_cast<int32_t*>(smem + F::OffRows)[buf * kK + j] = static_cast<int32_t>(r);
    const uint32_t m = __ballot_sync(0xffffffffu, r >= 0);
    if (lane == 0) reinterpret_cast<uint32_t*>(smem + F::OffMask)[buf * 16 + base / 32] = m;
  };
  if (warp < 16) load_rows(t_first, 0, warp * 32);
  tc_fence_before();
  __syncthreads();
  if constexpr (C > 1) cluster_sync();  // every CTA's barriers are set up
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int slot0 = rank * F::NK;
  // Blocks of 64 slots up to the last used one of a row list.
  auto used_blocks = [&](int buf) {
    const uint32_t* mask = reinterpret_cast<const uint32_t*>(smem + F::OffMask) + buf * 16;
    int n = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (mask[i]) n = i / 2 + 1;
    return n;
  };
  // The order in which P V takes its blocks: this CTA's own first, then as the others' shares come.
  auto block_at = [&](int i) {
    constexpr int per = F::VBlocks / C;
    return C == 1 ? i : ((rank - i / per) & (C - 1)) * per + i % per;
  };
  // This CTA's used slots (by 64).
  auto used_slots = [&](int blocks) { return min(F::NK, max(0, blocks * 64 - slot0)); };

  if (warp < kMmaWarp) {
    bool ok = true;
    auto worker_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWorkers) : "memory"); };
    const int quad = warp & 3, part = warp >> 2;
    const int h = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t scol = tmem + lane_base + part * F::CP;
    int stage = 0;       // latent key stages made so far; stage i sits in slot i % 2
    uint32_t vuse = 0;   // V blocks this group has made so far
    uint32_t it = 0;     // tokens done
    const int ch = F::RowLanes == 2 ? tid & 1 : tid / F::KS;  // this thread's (key, chunk)
    const int kk = F::RowLanes == 2 ? tid >> 1 : tid % F::KS;
    constexpr int Units = F::Stages * F::KeyParts;
    constexpr int PF = Units < 2 ? Units : 2;  // codes in flight
    // Scale words: a whole sector (both lanes of a row read it, each uses every other word) where a
    // thread needs four of them, single words otherwise.
    constexpr int SW = F::RowLanes == 2 ? 8 : F::Stages;
    const uint8_t* krow[F::KeyParts] = {};     // null: an empty slot
    uint32_t codes[PF][8], scales[F::KeyParts][SW] = {};
    // unit u: chunk (u / KeyParts) * CW + ch of key part u % KeyParts
    auto load = [&](int u, uint32_t (&c)[8]) {
      const uint8_t* src = krow[u % F::KeyParts];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = kEmptyWord;
      if (src) ld32(src + ((u / F::KeyParts) * F::CW + ch) * 32, c);
    };
    auto scale_of = [&](int k, int i) -> uint32_t {
      if constexpr (SW == 8) return ch ? scales[k][2 * i + 1] : scales[k][2 * i];
      else return scales[k][i];
    };
    // The rows, scales and first codes of a token whose list is in place.
    auto fetch = [&](int buf) {
      const int32_t* rows = reinterpret_cast<const int32_t*>(smem + F::OffRows) + buf * kK;
#pragma unroll
      for (int k = 0; k < F::KeyParts; ++k) {
        const int32_t r = rows[slot0 + k * F::KS + kk];
        krow[k] = r >= 0 ? p.cache + static_cast<int64_t>(r) * kRowBytes : nullptr;
      }
#pragma unroll
      for (int u = 0; u < PF; ++u) load(u, codes[u]);
#pragma unroll
      for (int k = 0; k < F::KeyParts; ++k) {
#pragma unroll
        for (int i = 0; i < SW; ++i) scales[k][i] = 0u;
        if (krow[k]) {
          if constexpr (SW == 8) {
            ld32(krow[k] + kOffScale, scales[k]);
          } else {
#pragma unroll
            for (int i = 0; i < SW; ++i)
              scales[k][i] =
                  *reinterpret_cast<const uint32_t*>(krow[k] + kOffScale + 4 * (i * F::CW + ch));
          }
        }
      }
    };
    // The rotary dims of a token's keys, copied into the ring behind everything else: eight lanes a
    // row, any row for an empty slot (its scores are masked). All warps share it: one warp's copies
    // of 512 rows take about 11 K clocks, TMA gathers of four rows 13 K.
    uint32_t qn = 0;     // ring items of the tokens before
    auto fetch_rope = [&](int buf) {
      const int32_t* rows = reinterpret_cast<const int32_t*>(smem + F::OffRows) + buf * kK + slot0;
      const int used = used_slots(used_blocks(buf));
#pragma unroll 4
      for (int j = tid >> 3; j < used; j += kWorkers / 8)
        cp_async16(smem + F::OffQ + (qn + j / F::RP) % F::NQS * kQBytes + (j % F::RP) * 128 +
                       (((lane & 7) ^ (j & 7)) * 16),
                   p.cache + static_cast<int64_t>(max(rows[j], 0)) * kRowBytes + kOffRope +
                       (lane & 7) * 16);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch_rope(0);
    fetch(0);
#pragma unroll 1
    for (int t = t_first; t < p.T; t += t_step, ++it) {
      const int buf = F::Bufs == 2 ? it & 1 : 0;
      const int32_t* s_rows = reinterpret_cast<const int32_t*>(smem + F::OffRows) + buf * kK;
      const uint32_t* s_mask = reinterpret_cast<const uint32_t*>(smem + F::OffMask) + buf * 16;
      const int nblk = used_blocks(buf), nc = used_slots(nblk);
      // ---------------- A: latent key stages
      const int parts = (nc + F::KS - 1) / F::KS;
      // The last token's output may still be read from the slots: its half in the slot that comes
      // first was sent first, so that half is waited for before a stage is made, the rest after it.
      int pending = it > 0 ? 2 : 0;
      cp_async_wait<0>();
      if (nc > 0) {
        qn += kChunks + (nc + F::RP - 1) / F::RP;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(rope_full);
#pragma unroll
        for (int u = 0; u < Units; ++u) {
          const int kp = u % F::KeyParts;
          if (kp < parts) {
            if (C == 1 && pending > 0) {
              --pending;
              if (tid == 0) {
                if (pending) bulk_store_wait<1>(); else bulk_store_wait<0>();
              }
              worker_sync();
            }
            const int slot = stage & (F::KSlots - 1);
            if (ok) ok = mbar_wait_warp(&k_empty[slot], ((stage >> 1) & 1) ^ 1u, s_abort, err);
            if (ok) {
              if (kp * F::KS + kk < nc)
                store_chunk<F::RowLanes>(smem0 + slot * F::KSlot + ch * (F::KS * 128), kk,
                                         codes[u % PF], scale_of(kp, u / F::KeyParts), ch);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&k_full[slot]);
            }
            ++stage;
          }
          if (u + PF < Units) load(u + PF, codes[u % PF]);
        }
      }
      if (C == 1 && pending > 0) {  // an empty list made no stage
        if (tid == 0) bulk_store_wait<0>();
        worker_sync();
      }
      // ---------------- B: softmax
      const int nch = min(F::CP, max(0, nc - part * F::CP)) / F::W;  // chunks of W columns
      auto mask_of = [&](int i) -> uint32_t {
        const int s = slot0 + part * F::CP + i * F::W;
        const uint32_t m = s_mask[s >> 5];
        return F::W == 32 ? m : (m >> (s & 16)) & 0xFFFFu;
      };
      constexpr uint32_t kAll = F::W == 32 ? 0xFFFFFFFFu : 0xFFFFu;
      // Value blocks of this thread's group: its codes are read one block ahead.
      const int gv = tid / (F::VK * F::NB), vtid = tid % (F::VK * F::NB);
      const int vnb = F::VLanes == 4 ? vtid & 3 : vtid / F::VK;
      const int vr = F::VLanes == 4 ? vtid >> 2 : vtid % F::VK;
      const int nvb = nblk * (64 / F::VK);                                  // used V blocks
      const int vblocks = gv < nvb ? (nvb - gv + F::GV - 1) / F::GV : 0;    // this group's, per half
      uint32_t vc[2][8], vs[2];
      auto v_load = [&](int n, uint32_t (&codes)[8], uint32_t& sc) {  // n: this group's n-th block
        if (n >= vblocks * F::Halves) return;
        const int half = n >= vblocks ? 1 : 0;
        int kb = gv + F::GV * (n - half * vblocks);
        if constexpr (C > 1) {
#pragma unroll
          for (int i = 0, k = n; i < F::VBlocks; ++i) {
            const int b = block_at(i);
            if (b % F::GV == gv && b < nvb && k-- == 0) kb = b;
          }
        }
        const int32_t r = s_rows[kb * F::VK + vr];
        const int chunk = rank * (F::DV / 64) + half * F::NB + vnb;
#pragma unroll
        for (int j = 0; j < 8; ++j) codes[j] = kEmptyWord;
        sc = 0u;
        if (r >= 0) {
          const uint8_t* row = p.cache + static_cast<int64_t>(r) * kRowBytes;
          ld32(row + chunk * 32, codes);
          sc = *reinterpret_cast<const uint32_t*>(row + kOffScale + 4 * chunk);
        }
      };
      auto v_store = [&](int n, uint32_t (&codes)[8], uint32_t sc) {
        if (n >= vblocks * F::Halves) return;
        if (ok) ok = mbar_wait_warp(&v_empty[gv], (vuse & 1) ^ 1u, s_abort, err);
        ++vuse;
        if (!ok) return;
        store_chunk<F::VLanes>(smem0 + kOffV + gv * F::VStage + vnb * (F::VK * 128), vr, codes, sc,
                               vnb);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[gv]);
      };
      v_load(0, vc[0], vs[0]);
      v_load(1, vc[1], vs[1]);
      if (ok) ok = mbar_wait_warp(s_ready, it & 1, s_abort, err);
      tc_fence_after();
      float mx4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
      if (ok) {
        for (int i = 0; i < nch; ++i) {
          uint32_t r[F::W];
          tmem_ld<F::W>(scol + i * F::W, r);
          tmem_wait_ld();
          const uint32_t vm = mask_of(i);
          if (vm == kAll) {
#pragma unroll
            for (int j = 0; j < F::W; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], __uint_as_float(r[j]));
          } else {
#pragma unroll
            for (int j = 0; j < F::W; ++j)
              mx4[j & 3] = fmaxf(mx4[j & 3], ((vm >> j) & 1u) ? __uint_as_float(r[j]) : kNegInf);
          }
        }
      }
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      s_red[part * kH + h] = mx * p.scale_log2;  // scale > 0: the maximum of the scaled scores
      worker_sync();
      float m = fmaxf(fmaxf(s_red[h], s_red[kH + h]), fmaxf(s_red[2 * kH + h], s_red[3 * kH + h]));
      if constexpr (C > 1) {
        if (part == 0) {
#pragma unroll
          for (int r = 0; r < C; ++r) st_peer(peer(smem_u32(s_x + rank * kH + h), r), m);
          __syncwarp();
          if (lane < C) arrive_peer(peer(smem_u32(m_full), lane));
        }
      }
      // its first block while the maxima travel (the rings are done with)
      v_store(0, vc[0], vs[0]);
      if constexpr (C > 1) {
        ok = __all_sync(0xffffffffu, wait_cluster(m_full, 0u, s_abort, err)) && ok;
#pragma unroll
        for (int r = 0; r < C; ++r) m = fmaxf(m, s_x[r * kH + h]);
      }
      // Finite, so that a score of +-infinity keeps its meaning in s - mm. A sum l that is NaN, infinite
      // or (scores of -infinity alone) zero then gives lse and out by the formulas; only an empty list
      // is set apart, by its mask.
      const float mm = fminf(fmaxf(m, -kMax), kMax);
      float l = 0.f;
      if (ok) {
        for (int i = 0; i < nch; ++i) {
          uint32_t r[F::W];
          tmem_ld<F::W>(scol + i * F::W, r);
          tmem_wait_ld();
          const uint32_t vm = mask_of(i);
          uint32_t pk[F::W / 2];
          // (the branch outside: with a select per element the pass takes twice as long)
          if (vm == kAll) {
#pragma unroll
            for (int j = 0; j < F::W; j += 2) {
              const float p0 = exp2_approx(fmaf(__uint_as_float(r[j]), p.scale_log2, -mm));
              const float p1 = exp2_approx(fmaf(__uint_as_float(r[j + 1]), p.scale_log2, -mm));
              l += p0 + p1;
              pk[j / 2] = pack_bf16x2(p0, p1);
            }
          } else {
#pragma unroll
            for (int j = 0; j < F::W; j += 2) {
              float p0 = exp2_approx(fmaf(__uint_as_float(r[j]), p.scale_log2, -mm));
              float p1 = exp2_approx(fmaf(__uint_as_float(r[j + 1]), p.scale_log2, -mm));
              p0 = ((vm >> j) & 1u) ? p0 : 0.f;
              p1 = ((vm >> (j + 1)) & 1u) ? p1 : 0.f;
              l += p0 + p1;
              pk[j / 2] = pack_bf16x2(p0, p1);
            }
          }
          const int s = slot0 + part * F::CP + i * F::W;
          const uint32_t at = smem0 + (s >> 6) * kPBlock + h * 128 + ((h & 7) ^ ((s & 63) >> 3)) * 16;
#pragma unroll
          for (int u = 0; u < F::W / 8; ++u)
            st_shared16(at ^ (16 * u), make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]));
        }
      }
      s_red[4 * kH + part * kH + h] = l;
      fence_proxy_async_smem();  // P (generic writes) before the MMAs and copies that read it
      tc_fence_before();
      worker_sync();
      l = (s_red[4 * kH + h] + s_red[5 * kH + h]) + (s_red[6 * kH + h] + s_red[7 * kH + h]);
      if constexpr (C > 1) {
        if (part == 0) {
#pragma unroll
          for (int r = 0; r < C; ++r) st_peer(peer(smem_u32(s_x + (C + rank) * kH + h), r), l);
          __syncwarp();
          if (lane < C) arrive_peer(peer(smem_u32(l_full), lane));
        }
        if (lane == 0) mbar_arrive(&p_full[rank]);
        if (warp == 15 && lane > 0 && lane < C) {
          const int to = (rank + lane) & (C - 1);
          if (ok && nc > 0)
            copy_to_peer(peer(smem_u32(smem + (slot0 / 64) * kPBlock), to),
                         smem_u32(smem + (slot0 / 64) * kPBlock), (nc / 64) * kPBlock,
                         peer(smem_u32(&p_full[rank]), to));
          // what the CTA `to` sends here
          mbar_arrive_expect_tx(&p_full[to],
                                min(8 / C, max(0, nblk - to * (8 / C))) * kPBlock);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, wait_cluster(l_full, 0u, s_abort, err)) && ok;
        l = 0.f;
#pragma unroll
        for (int r = 0; r < C; ++r) l += s_x[(C + r) * kH + h];
      }
      // w_j = sum over heads of exp2(s - m) / l, once more from S: at C = 1 before P V may write there,
      // in a cluster (S and O apart) while P V runs. Exactly the terms that l sums, so that a head's
      // weights add up to 1 at scores of any size; exp2(s - (m + log2 l)) would save the product, but
      // the rounding of m + log2 l, 2^-24 of the scores' size, would be left in the weights. (The
      // branch outside, as above: chunk of 4096 with weights 777 us, a select per element 834.)
      auto key_weights = [&] {
        const float part_of = nblk > 0 ? 1.f / l : 0.f;
        for (int i = 0; i < F::CP / F::W; ++i) {
          float v[F::W];
          if (ok && i < nch) {
            uint32_t r[F::W];
            tmem_ld<F::W>(scol + i * F::W, r);
            tmem_wait_ld();
            const uint32_t vm = h < p.n_heads ? mask_of(i) : 0u;
            if (__all_sync(0xffffffffu, vm == kAll)) {
#pragma unroll
              for (int j = 0; j < F::W; ++j)
                v[j] = exp2_approx(fmaf(__uint_as_float(r[j]), p.scale_log2, -mm)) * part_of;
            } else {
#pragma unroll
              for (int j = 0; j < F::W; ++j)
                v[j] = ((vm >> j) & 1u)
                           ? exp2_approx(fmaf(__uint_as_float(r[j]), p.scale_log2, -mm)) * part_of
                           : 0.f;
            }
          } else {
#pragma unroll
            for (int j = 0; j < F::W; ++j) v[j] = 0.f;
          }
          const float sum = column_sums<F::W>(v, lane);
          if (lane < F::W) s_w[quad * F::NK + part * F::CP + i * F::W + lane] = sum;
        }
        tc_fence_before();
        worker_sync();
        if (tid < F::NK && slot0 + tid < p.n_sel)
          p.weights[static_cast<int64_t>(t) * p.n_sel + slot0 + tid] =
              (s_w[tid] + s_w[F::NK + tid]) + (s_w[2 * F::NK + tid] + s_w[3 * F::NK + tid]);
      };
      if (C == 1 && p.weights) key_weights();
      if constexpr (C == 1) {
        if (lane == 0) mbar_arrive(&p_full[0]);
      }
      if (p.lse && rank == 0 && part == 0 && h < p.n_heads)
        p.lse[t * p.n_heads + h] = nblk > 0 ? (m + __log2f(l)) * 0.69314718055994531f : kNegInf;
      // ---------------- C: value blocks, then the output through shared memory
#pragma unroll 1
      for (int n = 1; n < vblocks * F::Halves; n += 2) {
        v_load(n + 1, vc[0], vs[0]);
        v_store(n, vc[1], vs[1]);
        v_load(n + 2, vc[1], vs[1]);
        v_store(n + 1, vc[0], vs[0]);
      }
      if (C > 1 && p.weights) key_weights();
      if constexpr (C == 1) {  // the next token's first reads, behind P V and the output
        if (t + t_step < p.T) {
          if (ok) ok = mbar_wait_warp(&rows_full[buf ^ 1], (it >> 1) & 1, s_abort, err);
          if (ok) fetch(buf ^ 1);
        }
      }
      const float inv = nblk > 0 ? 1.f / l : 0.f;
      if (ok) ok = mbar_wait_warp(o_ready, it & 1, s_abort, err);
      tc_fence_after();
      if (C == 1 && ok && t + t_step < p.T) fetch_rope(buf ^ 1);  // (the ring lies over the V blocks)
      // Output columns of 64 dims each, in F::Halves runs; at C = 1 a run fills one key slot, and the
      // run in the slot that the next token's first stage takes goes first.
      constexpr int RunCols = F::DV / F::Halves, PartCols = RunCols / 4;
#pragma unroll 1
      for (int run = 0; run < F::Halves; ++run) {
        const int half = C == 1 ? (stage & 1) ^ run : run;
        if (ok) {
#pragma unroll 1
          for (int i = 0; i < PartCols / F::OW; ++i) {
            const int col = half * RunCols + part * PartCols + i * F::OW;
            uint32_t r[F::OW], pk[F::OW / 2];
            if (nblk > 0) {
              tmem_ld<F::OW>(tmem + lane_base + F::OCol + col, r);
              tmem_wait_ld();
            }
#pragma unroll
            for (int j = 0; j < F::OW; j += 2)
              pk[j / 2] = nblk > 0 ? pack_bf16x2(__uint_as_float(r[j]) * inv, __uint_as_float(r[j + 1]) * inv)
                                   : 0u;
            const uint32_t at =
                smem0 + F::OffO + (col >> 6) * kPBlock + h * 128 + ((h & 7) ^ ((col & 63) >> 3)) * 16;
#pragma unroll
            for (int u = 0; u < F::OW / 8; ++u)
              st_shared16(at ^ (16 * u),
                          make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]));
          }
        }
        fence_proxy_async_smem();
        if (run == F::Halves - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        worker_sync();
        if (tid == 0) {
          if (ok) {
#pragma unroll 1
            for (int i = 0; i < RunCols / 64; ++i)
              tma_store_2d(smem + F::OffO + (half * (RunCols / 64) + i) * kPBlock, &tmap_o,
                           rank * F::DV + half * RunCols + i * 64,
                           t * p.n_heads);
          }
          bulk_store_commit();
        }
      }
      if constexpr (C > 1) break;
    }
    if (tid == 0) bulk_store_wait<0>();
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issue: the warp waits together and one elected lane issues. Descriptors
    // stay warp-uniform; formed in one thread's registers each MMA would wait for their moves to
    // uniform registers, about 100 clocks, more than an MMA of N = 64 takes.
    const bool lead = elect_one();
    bool ok = true;
    const uint64_t q0 = smem_desc_sw128(smem_u32(smem + F::OffQ));
    const uint64_t k0 = smem_desc_sw128(smem_u32(smem));
    const uint64_t v0 = smem_desc_mn_sw128(smem_u32(smem + kOffV), F::VK * 128);
    constexpr uint32_t o_idesc = instr_desc(1u, 1u, 128, F::NB * 64) | (1u << 16);  // B MN-major
    uint32_t qn = 0, it = 0;  // ring items taken, tokens done
    uint32_t stage = 0;       // latent key stages taken
    uint32_t vn[F::GV] = {};  // blocks taken from each V stage
    uint32_t q_phase = 0;     // bit: the parity of the next Q chunk in a ring place
    uint32_t ropes = 0;       // rotary pieces taken (tokens)
    auto q_ready = [&](uint32_t i) {
      const uint32_t at = i % F::NQS, parity = q_phase >> at & 1u;
      q_phase ^= 1u << at;
      return mbar_wait_warp(&q_full[at], parity, s_abort, err);
    };
    auto k_ready = [&] {
      return mbar_wait_warp(&k_full[stage & (F::KSlots - 1)], (stage >> 1) & 1, s_abort, err);
    };
    // S columns col .. col + n - 1 += ring item i (a Q chunk) x the n keys at byte `at`
    auto product = [&](uint32_t i, int at, int col, int n, bool first) {
      const uint32_t idesc = instr_desc(1u, 1u, 128, n);
      const uint64_t qd = q0 + (i % F::NQS) * (kQBytes >> 4), kd = k0 + (at >> 4);
      if (lead) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_bf16(tmem + col, qd + 2 * s, kd + 2 * s, idesc, first && s == 0 ? 0u : 1u);
      }
    };
    auto commit = [&](uint64_t* bar) {
      if (lead) mma_commit(bar);
    };
#pragma unroll 1
    for (int t = t_first; ok && t < p.T; t += t_step, ++it) {
      const int buf = F::Bufs == 2 ? it & 1 : 0;
      if (it > 0)
        ok = mbar_wait_warp(&rows_full[buf], ((it - 1) >> 1) & 1, s_abort, err) &&
             mbar_wait_warp(o_free, (it - 1) & 1, s_abort, err);
      if (!ok) break;
      tc_fence_after();
      const int nblk = used_blocks(buf), nc = used_slots(nblk);
      if (nc > 0) {
        // the rotary chunk, keys in pieces from the ring
        const uint32_t rope = qn + (nc + F::RP - 1) / F::RP;
        ok = mbar_wait_warp(rope_full, ropes++ & 1, s_abort, err) && q_ready(rope);
        tc_fence_after();
        for (int k = 0; ok && k < nc; k += F::RP, ++qn) {
          product(rope, F::OffQ + (qn % F::NQS) * kQBytes, k, min(F::RP, nc - k), true);
          commit(&q_empty[qn % F::NQS]);
        }
        commit(&q_empty[rope % F::NQS]);
        qn = rope + 1;
        // the latent chunks, key stages as the workers make them
        const int parts = (nc + F::KS - 1) / F::KS;
#pragma unroll 1
        for (int c0 = 0; ok && c0 < 8; c0 += F::CW) {
#pragma unroll 1
          for (int k = 0; ok && k < parts; ++k) {
            ok = k_ready();
            const int slot = stage & (F::KSlots - 1);
#pragma unroll
            for (int c = 0; c < F::CW; ++c) {
              const uint32_t i = qn + c0 + c;
              if (!ok || (k == 0 && !(ok = q_ready(i)))) break;
              tc_fence_after();
              product(i, slot * F::KSlot + c * F::KS * 128, k * F::KS, min(F::KS, nc - k * F::KS),
                      false);
              if (k == parts - 1) commit(&q_empty[i % F::NQS]);
            }
            commit(&k_empty[slot]);
            ++stage;
          }
        }
        qn += kChunks - 1;
      }
      commit(s_ready);
      if (C == 1 && ok) ok = mbar_wait_warp(&p_full[0], it & 1, s_abort, err);
      for (int half = 0; half < F::Halves; ++half) {
#pragma unroll 1
        for (int i0 = 0, taken = 0; ok && i0 < F::VBlocks; i0 += F::GV) {
#pragma unroll
          for (int j = 0; j < F::GV; ++j) {
            const int kb = block_at(i0 + j);
            if (!ok || kb >= nblk * (64 / F::VK)) continue;
            const int st = C == 1 ? j : kb % F::GV;
            if (C > 1 && !(ok = mbar_wait_warp(&p_full[kb / (F::VBlocks / C)], 0u, s_abort, err)))
              break;
            uint32_t use = 0;
#pragma unroll
            for (int v = 0; v < F::GV; ++v)
              if (v == st) use = vn[v]++;
            if (!(ok = mbar_wait_warp(&v_full[st], use & 1, s_abort, err))) break;
            tc_fence_after();
            const int key = kb * F::VK;
            const uint64_t pd = k0 + (key >> 6) * (kPBlock >> 4) + (key & 63) * 2 / 16;
            const uint64_t vd = v0 + st * (F::VStage >> 4);
            if (lead) {
#pragma unroll
              for (int s = 0; s < F::VK / 16; ++s)
                mma_bf16(tmem + F::OCol + half * 256, pd + 2 * s, vd + s * (16 * 128 >> 4), o_idesc,
                         (taken | s) ? 1u : 0u);
            }
            ++taken;
            commit(&v_empty[st]);
          }
        }
      }
      commit(o_ready);
      if constexpr (C > 1) break;
    }
    // every MMA has completed before TMEM is released (bounded, also after an abort)
    commit(done);
    if (lead) {
      mbar_drain(done, 0u);
      // shares of P from other CTAs have landed (bounded)
      if (C > 1 && !ok)
        for (int i = 0; i < C; ++i)
          if (i != rank) mbar_drain(&p_full[i], 0u);
    }
    __syncwarp();
  } else {
    // ---------------- Q chunks and the next token's row list (one warp)
    const uint32_t bytes = static_cast<uint32_t>(p.n_heads) * 128u;
    uint32_t qn = 0, it = 0;  // ring items so far, tokens done
    uint32_t q_phase = 0, q_used = 0;  // bits: parity of the next Q chunk in a place, places used
    bool ok = true;
#pragma unroll 1
    for (int t = t_first; ok && t < p.T; t += t_step, ++it) {
      const int buf = F::Bufs == 2 ? it & 1 : 0;
      const int nc = used_slots(used_blocks(buf));
      const int pieces = (nc + F::RP - 1) / F::RP;
      if (nc > 0) {
        qn += pieces;  // made by the workers
        for (int i = 0; i < kChunks; ++i, ++qn) {
          const uint32_t qs = qn % F::NQS;
          if (!(ok = mbar_wait_warp(&q_empty[qs], ((qn / F::NQS) & 1) ^ 1u, s_abort, err))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[qs], bytes);
            tma_load_2d(smem + F::OffQ + qs * kQBytes, &tmap_q, &q_full[qs],
                        i == 0 ? kLatent : (i - 1) * 64, t * p.n_heads);
            q_phase ^= 1u << qs;
            q_used |= 1u << qs;
          }
        }
      }
      if (C > 1 || !ok) break;
      if (t + t_step < p.T) {  // that list's last readers arrived when they were done with O
        if (it > 0) ok = mbar_wait_warp(o_free, (it - 1) & 1, s_abort, err);
        if (!ok) break;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) load_rows(t + t_step, buf ^ 1, i * 32);
        __syncwarp();
        if (lane == 0) mbar_arrive(&rows_full[buf ^ 1]);
      }
      // the Q ring lies over the V blocks: no load before P V is done
      ok = mbar_wait_warp(o_ready, it & 1, s_abort, err);
      if (ok && lane == 0) mbar_arrive(o_free);
    }
    if (lane == 0)  // never exit with loads in flight
      for (int i = 0; i < F::NQS; ++i)
        if (q_used >> i & 1u) mbar_drain(&q_full[i], (q_phase >> i & 1u) ^ 1u);
    __syncwarp();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if constexpr (C > 1) cluster_sync();  // no CTA leaves while another may still write or read here
}

PFN_cuTensorMapEncodeTiled_v12000 g_enc = nullptr;
std::once_flag g_enc_once;

// A [rows, width] bf16 tensor in boxes of box_rows x 64, 128-byte swizzle.
bool encode(CUtensorMap* m, const void* base, int32_t width, int64_t rows, int32_t box_rows) {
  std::call_once(g_enc_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult r{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      g_enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * 2};
  cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1u, 1u};
  return g_enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How many clusters of C CTAs run at once on the current device (asked once per device; 0: an error).
template <int C>
int64_t clusters_at_once() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  static std::atomic<uint64_t> done{0};
  if (!allow_shared(sparse_attn_q4_kernel<C>, Cfg<C>::Smem, done)) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<C>::Smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, sparse_attn_q4_kernel<C>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int C>
int launch(const CUtensorMap& tq, const CUtensorMap& to, const Params& p, int64_t T, void* stream) {
  static std::atomic<uint64_t> done{0};
  if (!allow_shared(sparse_attn_q4_kernel<C>, Cfg<C>::Smem, done)) return DS4IDX_ERR_CUDA;
  // One CTA an SM fits. More tokens than SMs: the CTAs stay and take the tokens in turn.
  const int64_t grid = C == 1 ? std::min<int64_t>(T, sm_count()) : T * C;
  if (grid == 0) return DS4IDX_ERR_CUDA;
  return launch_dependent(sparse_attn_q4_kernel<C>, static_cast<unsigned>(grid), kThreads,
                          Cfg<C>::Smem, C, stream, tq, to, p);
}

}  // namespace ds4qa

extern "C" int ds4idx_sparse_attention_q4(const void* q, const uint8_t* cache, int64_t kv_rows,
                                          const int32_t* idx, const ds4idx_placement* where,
                                          int64_t T, int32_t n_heads, int32_t d_qk, int32_t d_v,
                                          int32_t n_sel, float sm_scale, void* out, float* lse,
                                          float* weights, void* stream) {
  using namespace ds4qa;
  if (d_qk != kRowDims || d_v != kLatent) return DS4IDX_ERR_UNSUPPORTED;
  if (n_heads < 1 || n_heads > kH || n_sel < 1 || n_sel > kK || T < 0 || T > 0x7FFFFFFF / kH ||
      kv_rows < 1 || kv_rows > 0x7FFFFFFF || !(sm_scale > 0.f) || !(sm_scale < 1e30f))
    return DS4IDX_ERR_INVALID_ARG;
  if (T == 0) return DS4IDX_OK;
  Params p{};
  if (!q || !cache || !idx || !out || !aligned_to(q, 16) || !aligned_to(cache, 32) ||
      !aligned_to(idx, 4) || !aligned_to(out, 32) || !aligned_to(lse, 4) ||
      !aligned_to(weights, 4) || !make_placement(where, kv_rows, T, &p.place))
    return DS4IDX_ERR_INVALID_ARG;
  CUtensorMap tq, to;
  if (!encode(&tq, q, kRowDims, T * n_heads, n_heads) ||
      !encode(&to, out, kLatent, T * n_heads, n_heads))
    return DS4IDX_ERR_CUDA;
  p.cache = cache;
  p.idx = idx;
  p.lse = lse;
  p.weights = weights;
  p.err = ds4a::sparse_attention_error_word();
  if (!p.err) return DS4IDX_ERR_CUDA;
  p.T = static_cast<int32_t>(T);
  p.n_heads = n_heads;
  p.n_sel = n_sel;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  // The widest cluster of which all tokens run at once (15 of 8, 36 of 4 and 76 of 2 on the GPU asked
  // first; it depends on which SMs a part has). 512 rows, 128 heads, us for 8 / 4 / 2 / 1 CTAs a token:
  // 12.9 / 13.4 / 17.4 / 25.8 at 12 tokens, 23 / 13.4 / 17.3 / 25.8 at 16, 35 / 18.2 / 17.6 / 25.8 at 37
  // (26 instead of 18.2 where a second round is needed), 71 / 39 / 34 / 26.5 at 77.
  if (T <= clusters_at_once<8>()) return launch<8>(tq, to, p, T, stream);
  if (T <= clusters_at_once<4>()) return launch<4>(tq, to, p, T, stream);
  if (T <= clusters_at_once<2>()) return launch<2>(tq, to, p, T, stream);
  return launch<1>(tq, to, p, T, stream);
}
