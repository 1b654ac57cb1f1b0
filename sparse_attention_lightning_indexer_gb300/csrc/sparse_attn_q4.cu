// Sparse attention over the selected rows of a 4-bit latent cache, for sm_103a: one latent row
// (q4_format.cuh) per position, shared by all heads; 576-wide keys, the first 512 dims are values.
//
// A cluster of C = 1, 2, 4 or 8 CTAs owns one token. Both products are split without partial sums:
//   A  S[128 heads x 512/C keys] = Q K^T: a CTA takes its share of the list's slots (TMEM columns
//      0 .. 512/C - 1). 9 chunks of 64 dims pass through two rings in shared memory: the Q chunk by
//      TMA, the key chunk by the worker threads, which read a row's 32 bytes of codes, turn them
//      into bf16 (exact) and write the 128-byte-swizzled operand.
//   B  softmax: the row maxima and sums of the CTAs meet in each other's shared memory, so every
//      probability is final relative to the list's maximum; P goes as bf16 into shared memory in
//      the layout of an MMA A operand, each CTA's share copied to the others by bulk copies.
//   C  O[128 heads x 512/C dims] = P V over all slots: blocks of 64 keys of the CTA's value dims are
//      turned into bf16 again, as an MN-major B operand. Nothing is joined afterwards.
// C = 1 fills the GPU for many tokens; a cluster shortens the chain of phases for few.
//
// Warps 0..15 are the workers (unpacking, softmax, output: TMEM lane quadrant warp % 4, column
// quarter warp / 4), warp 16 issues tcgen05.mma, warp 17 loads Q.
//
// The unpacked tile serves as K (K-major) and as V (MN-major) in the same layout; it is made
// twice because O takes all 512 TMEM columns at C = 1, so P V starts only after the whole of S is
// read, and 512 unpacked rows (576 KB) do not fit shared memory.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

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
constexpr float kNegInf = -__builtin_inff();

template <int C>
struct Cfg {
  static constexpr int NK = kK / C;                     // slots of a CTA
  static constexpr int KBytes = NK * 128;               // one key chunk
  static constexpr int NKS = C == 1 ? 2 : C == 2 ? 3 : C == 4 ? 5 : 9;
  static constexpr int NQS = C == 1 ? 4 : C == 2 ? 6 : C == 4 ? 7 : 8;
  static constexpr int OffQ = NKS * KBytes;
  static constexpr int RingBytes = OffQ + NQS * kQBytes;
  static constexpr int Region = RingBytes > kOffV + kVBytes ? RingBytes : kOffV + kVBytes;
  static constexpr int G = C;                           // worker groups: key chunks in the making
  static constexpr int CPT = 8 / G;                     // latent chunks of a thread
  static constexpr int DV = kLatent / C;                // value dims of a CTA
  static constexpr int NB = DV / 64 < 4 ? DV / 64 : 4;  // 64-dim pieces of a V block
  static constexpr int Halves = DV / 64 / NB;           // passes over the keys (2 at C = 1)
  static constexpr int GV = 8 / NB;                     // V blocks in the making = V stages
  static constexpr int VStage = NB * 64 * 128;
  static constexpr int OCol = C == 1 ? 0 : 256;         // first TMEM column of O
  static constexpr int CP = NK / 4;                     // S columns of a thread
  static constexpr int W = CP < 32 ? CP : 32;
  static constexpr int OP = NB * 64 / 4;                // O columns of a thread per half
  static constexpr int OW = OP < 32 ? OP : 32;

  static constexpr int OffRows = Region;
  static constexpr int OffMask = OffRows + kK * 4;
  static constexpr int OffRed = OffMask + 64;                     // [2][4][128] max, sum
  static constexpr int OffX = OffRed + 2 * 4 * kH * 4;            // [2][C][128] of the cluster
  static constexpr int OffW = OffX + (C > 1 ? 2 * C * kH * 4 : 0);  // [4][NK] key weights
  static constexpr int OffBars = OffW + 4 * NK * 4;
  static constexpr int NumBars = 2 * NQS + 2 * NKS + 2 * GV + 6;
  static constexpr int OffMisc = OffBars + NumBars * 8;
  static constexpr int Smem = OffMisc + 16 + 1024;
  static_assert(GV * VStage == kVBytes && Smem <= 232448, "shared memory");
};

struct Params {
  const uint8_t* cache;
  const int32_t* idx;
  uint16_t* out;
  float* lse;
  float* weights;
  uint32_t* err;
  Placement place;
  int32_t n_heads, n_sel;
  float scale_log2;
};

__device__ __forceinline__ void ld32(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void st32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar,
                                            int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle layout: blocks of 64 N
// (64 keys x 128 bytes apart), atoms of 8 keys along K.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((64u * 128u) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- other CTAs of the cluster
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_peer(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive_peer(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_to_peer(uint32_t dst, uint32_t src, uint32_t bytes,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
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

// One 64-dim chunk of a latent row to the 128 swizzled bytes of row `r` at `base`.
__device__ __forceinline__ void store_chunk(uint8_t* base, int r, const uint32_t (&codes)[8],
                                            uint32_t scales) {
  uint8_t* row = base + r * 128;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t s2 = scale_bf16x2((scales >> (8 * g)) & 0xFFu), c2 = offset_bf16x2(s2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int u = 2 * g + h;
      *reinterpret_cast<uint4*>(row + ((u ^ (r & 7)) * 16)) = word_to_bf16(codes[u], s2, c2);
    }
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
                          const __grid_constant__ Params p) {
  using F = Cfg<C>;
  extern __shared__ uint8_t smem_raw[];
  // every CTA of a cluster has the same dynamic shared-memory base, so the offsets agree
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  int32_t* s_rows = reinterpret_cast<int32_t*>(smem + F::OffRows);
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + F::OffMask);
  float* s_red = reinterpret_cast<float*>(smem + F::OffRed);
  float* s_x = reinterpret_cast<float*>(smem + F::OffX);
  float* s_w = reinterpret_cast<float*>(smem + F::OffW);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + F::OffBars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + F::NQS;
  uint64_t* k_full = q_empty + F::NQS;
  uint64_t* k_empty = k_full + F::NKS;
  uint64_t* v_full = k_empty + F::NKS;
  uint64_t* v_empty = v_full + F::GV;
  uint64_t* s_ready = v_empty + F::GV;
  uint64_t* m_full = s_ready + 1;
  uint64_t* l_full = s_ready + 2;
  uint64_t* p_full = s_ready + 3;
  uint64_t* o_ready = s_ready + 4;  // [2]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + F::OffMisc);
  volatile uint32_t* s_abort = reinterpret_cast<volatile uint32_t*>(smem + F::OffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t = blockIdx.x / C;
  const int rank = blockIdx.x % C;
  uint32_t* err = p.err;

  if (tid == 0) {
    for (int i = 0; i < F::NQS; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < F::NKS; ++i) {
      mbar_init(&k_full[i], 16 / F::G);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < F::GV; ++i) {
      mbar_init(&v_full[i], 2 * F::NB);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(s_ready, 1);
    mbar_init(m_full, 4 * C);
    mbar_init(l_full, 4 * C);
    mbar_init(p_full, 16 + (C > 1 ? 1 : 0));
    mbar_init(&o_ready[0], 1);
    mbar_init(&o_ready[1], 1);
    *s_abort = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  if (tid < kK) {
    int64_t r = -1;
    if (tid < p.n_sel) {
      const TokenPlace tp = place_token(p.place, t);
      r = place_row(p.place, tp, p.idx[t * p.n_sel + tid]);
    }
    s_rows[tid] = static_cast<int32_t>(r);
    const uint32_t m = __ballot_sync(0xffffffffu, r >= 0);
    if (lane == 0) s_mask[warp] = m;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (C > 1) cluster_sync();  // every CTA's barriers are set up
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  int nblk = 0;  // blocks of 64 slots up to the last used one
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (s_mask[i]) nblk = i / 2 + 1;
  const int slot0 = rank * F::NK;
  const int nc = min(F::NK, max(0, nblk * 64 - slot0));  // this CTA's used slots (by 64)

  if (warp < kMmaWarp) {
    bool ok = true;
    // ---------------- A: key chunks
    if (nc > 0) {
      const int kk = tid % F::NK, grp = tid / F::NK;
      const int32_t row_id = kk < nc ? s_rows[slot0 + kk] : -1;
      const bool live = row_id >= 0;
      const uint8_t* row = p.cache + static_cast<int64_t>(live ? row_id : 0) * kRowBytes;
      constexpr int PF = F::CPT < 3 ? F::CPT : 3;  // chunks in flight
      uint32_t codes[PF][8], scales[F::CPT];
#pragma unroll
      for (int i = 0; i < PF; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) codes[i][j] = kEmptyWord;
        if (live) ld32(row + (grp + F::G * i) * 32, codes[i]);
      }
#pragma unroll
      for (int i = 0; i < F::CPT; ++i)
        scales[i] = live ? *reinterpret_cast<const uint32_t*>(row + kOffScale + 4 * (grp + F::G * i))
                         : 0u;
#pragma unroll
      for (int i = 0; i < F::CPT; ++i) {
        const int c = grp + F::G * i, st = c % F::NKS;
        if (ok) ok = mbar_wait_warp(&k_empty[st], ((c / F::NKS) & 1) ^ 1u, s_abort, err);
        if (ok) {
          if (kk < nc) store_chunk(smem + st * F::KBytes, kk, codes[i % PF], scales[i]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[st]);
        }
        if (i + PF < F::CPT && live) ld32(row + (grp + F::G * (i + PF)) * 32, codes[i % PF]);
      }
      if (grp == 0 && ok) {  // the rotary chunk, bf16 as it is
        uint32_t r[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int k = 0; k < 8; ++k) r[j][k] = 0u;
          if (live) ld32(row + kOffRope + 32 * j, r[j]);
        }
        constexpr int c = kChunks - 1, st = c % F::NKS;
        ok = mbar_wait_warp(&k_empty[st], ((c / F::NKS) & 1) ^ 1u, s_abort, err);
        if (ok) {
          uint8_t* dst = smem + st * F::KBytes + kk * 128;
          if (kk < nc) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(dst + ((u ^ (kk & 7)) * 16)) =
                  make_uint4(r[u / 2][4 * (u & 1)], r[u / 2][4 * (u & 1) + 1],
                             r[u / 2][4 * (u & 1) + 2], r[u / 2][4 * (u & 1) + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[st]);
        }
      }
    }
    // ---------------- B: softmax
    const int quad = warp & 3, part = warp >> 2;
    const int h = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const int nch = min(F::CP, max(0, nc - part * F::CP)) / F::W;  // chunks of W columns
    const uint32_t scol = tmem + lane_base + part * F::CP;
    auto mask_of = [&](int i) -> uint32_t {
      const int s = slot0 + part * F::CP + i * F::W;
      const uint32_t m = s_mask[s >> 5];
      return F::W == 32 ? m : (m >> (s & 16)) & 0xFFFFu;
    };
    constexpr uint32_t kAll = F::W == 32 ? 0xFFFFFFFFu : 0xFFFFu;
    auto worker_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWorkers) : "memory"); };
    ok = mbar_wait_warp(s_ready, 0u, s_abort, err) && ok;
    tc_fence_after();
    float mx = kNegInf;
    if (ok) {
      for (int i = 0; i < nch; ++i) {
        uint32_t r[F::W];
        tmem_ld<F::W>(scol + i * F::W, r);
        tmem_wait_ld();
        const uint32_t vm = mask_of(i);
        if (vm == kAll) {
#pragma unroll
          for (int j = 0; j < F::W; ++j) mx = fmaxf(mx, __uint_as_float(r[j]));
        } else {
#pragma unroll
          for (int j = 0; j < F::W; ++j)
            mx = fmaxf(mx, ((vm >> j) & 1u) ? __uint_as_float(r[j]) : kNegInf);
        }
      }
    }
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
    // The V blocks this group makes first, while the maxima travel (the rings are done with).
    const int gv = tid / (64 * F::NB), vr = tid % 64, vnb = (tid / 64) % F::NB;
    int vuse = 0;
    auto v_load = [&](int half, int kb, uint32_t (&codes)[8], uint32_t& sc) {
      const int32_t r = s_rows[kb * 64 + vr];
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
    auto v_store = [&](const uint32_t (&codes)[8], uint32_t sc) {
      if (ok) ok = mbar_wait_warp(&v_empty[gv], (vuse & 1) ^ 1u, s_abort, err);
      ++vuse;
      if (!ok) return;
      store_chunk(smem + kOffV + gv * F::VStage + vnb * (64 * 128), vr, codes, sc);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[gv]);
    };
    uint32_t vc[8], vs;
    if (gv < nblk) {
      v_load(0, gv, vc, vs);
      v_store(vc, vs);
    }
    if constexpr (C > 1) {
      ok = __all_sync(0xffffffffu, wait_cluster(m_full, 0u, s_abort, err)) && ok;
#pragma unroll
      for (int r = 0; r < C; ++r) m = fmaxf(m, s_x[r * kH + h]);
    }
    const float mm = m == kNegInf ? 0.f : m;
    float l = 0.f;
    if (ok) {
      for (int i = 0; i < nch; ++i) {
        uint32_t r[F::W];
        tmem_ld<F::W>(scol + i * F::W, r);
        tmem_wait_ld();
        const uint32_t vm = mask_of(i);
        uint32_t pk[F::W / 2];
#pragma unroll
        for (int j = 0; j < F::W; j += 2) {
          float p0 = exp2_approx(fmaf(__uint_as_float(r[j]), p.scale_log2, -mm));
          float p1 = exp2_approx(fmaf(__uint_as_float(r[j + 1]), p.scale_log2, -mm));
          if (vm != kAll) {
            p0 = ((vm >> j) & 1u) ? p0 : 0.f;
            p1 = ((vm >> (j + 1)) & 1u) ? p1 : 0.f;
          }
          l += p0 + p1;
          pk[j / 2] = pack_bf16x2(p0, p1);
        }
        const int s = slot0 + part * F::CP + i * F::W;
        uint8_t* row = smem + (s >> 6) * kPBlock + h * 128;
#pragma unroll
        for (int u = 0; u < F::W / 8; ++u) {
          const int cc = ((s & 63) >> 3) + u;
          *reinterpret_cast<uint4*>(row + ((cc ^ (h & 7)) * 16)) =
              make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        }
      }
    }
    s_red[4 * kH + part * kH + h] = l;
    fence_proxy_async_smem();  // P (generic writes) before the MMAs and copies that read it
    tc_fence_before();
    worker_sync();
    l = (s_red[4 * kH + h] + s_red[5 * kH + h]) + (s_red[6 * kH + h] + s_red[7 * kH + h]);
    if constexpr (C > 1) {
      if (tid < C && tid != rank && ok && nc > 0) {
        copy_to_peer(peer(smem_u32(smem + (slot0 / 64) * kPBlock), tid),
                     smem_u32(smem + (slot0 / 64) * kPBlock), (nc / 64) * kPBlock,
                     peer(smem_u32(p_full), tid));
      }
      if (tid == 0) mbar_arrive_expect_tx(p_full, (nblk - nc / 64) * kPBlock);
      if (lane == 0) mbar_arrive(p_full);
      if (part == 0) {
#pragma unroll
        for (int r = 0; r < C; ++r) st_peer(peer(smem_u32(s_x + (C + rank) * kH + h), r), l);
        __syncwarp();
        if (lane < C) arrive_peer(peer(smem_u32(l_full), lane));
      }
      ok = __all_sync(0xffffffffu, wait_cluster(l_full, 0u, s_abort, err)) && ok;
      l = 0.f;
#pragma unroll
      for (int r = 0; r < C; ++r) l += s_x[(C + r) * kH + h];
    }
    if (p.weights) {
      // w_j = sum over heads of exp2(s - m) / l, once more from S (intact until P V starts)
      const float off = l > 0.f && h < p.n_heads ? mm + __log2f(l) : __int_as_float(0x7f800000);
      for (int i = 0; i < F::CP / F::W; ++i) {
        float v[F::W];
        if (ok && i < nch) {
          uint32_t r[F::W];
          tmem_ld<F::W>(scol + i * F::W, r);
          tmem_wait_ld();
          const uint32_t vm = mask_of(i);
#pragma unroll
          for (int j = 0; j < F::W; ++j)
            v[j] = ((vm >> j) & 1u) && h < p.n_heads
                       ? exp2_approx(fmaf(__uint_as_float(r[j]), p.scale_log2, -off))
                       : 0.f;
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
        p.weights[t * p.n_sel + slot0 + tid] =
            (s_w[tid] + s_w[F::NK + tid]) + (s_w[2 * F::NK + tid] + s_w[3 * F::NK + tid]);
    }
    if constexpr (C == 1) {
      if (lane == 0) mbar_arrive(p_full);
    }
    if (p.lse && rank == 0 && part == 0 && h < p.n_heads)
      p.lse[t * p.n_heads + h] = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : kNegInf;
    // ---------------- C: value blocks, then the output
#pragma unroll 1
    for (int n = (gv < nblk ? 1 : 0), half = 0; half < F::Halves; ++half, n = 0) {
#pragma unroll 1
      for (int kb = gv + F::GV * n; kb < nblk; kb += F::GV) {
        v_load(half, kb, vc, vs);
        v_store(vc, vs);
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t* orow = p.out + (t * p.n_heads + h) * kLatent + rank * F::DV;
#pragma unroll 1
    for (int half = 0; half < F::Halves; ++half) {
      if (nblk > 0 && ok) {
        ok = mbar_wait_warp(&o_ready[half], 0u, s_abort, err);
        tc_fence_after();
      }
      if (!ok) break;
#pragma unroll 1
      for (int i = 0; i < F::OP / F::OW; ++i) {
        const int col = half * F::NB * 64 + part * F::OP + i * F::OW;
        uint32_t r[F::OW], pk[F::OW / 2];
        if (nblk > 0) {
          tmem_ld<F::OW>(tmem + lane_base + F::OCol + col, r);
          tmem_wait_ld();
        }
#pragma unroll
        for (int j = 0; j < F::OW; j += 2)
          pk[j / 2] = nblk > 0 ? pack_bf16x2(__uint_as_float(r[j]) * inv, __uint_as_float(r[j + 1]) * inv)
                               : 0u;
        if (h < p.n_heads) {
#pragma unroll
          for (int u = 0; u < F::OW / 16; ++u) st32(orow + col + 16 * u, pk + 8 * u);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issue (one thread)
    if (lane == 0) {
      bool ok = true;
      if (nc > 0) {
        for (int c = 0; c < kChunks; ++c) {
          const int qs = c % F::NQS, ks = c % F::NKS;
          ok = mbar_wait(&q_full[qs], (c / F::NQS) & 1, s_abort, err) &&
               mbar_wait(&k_full[ks], (c / F::NKS) & 1, s_abort, err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t qa = smem_u32(smem + F::OffQ + qs * kQBytes);
          const uint32_t kb = smem_u32(smem + ks * F::KBytes);
          for (int k0 = 0; k0 < nc; k0 += 256) {
            const uint32_t idesc = instr_desc(1u, 1u, 128, min(256, nc - k0));
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_bf16(tmem + k0, smem_desc_sw128(qa + s * 32),
                       smem_desc_sw128(kb + k0 * 128 + s * 32), idesc, (c | s) ? 1u : 0u);
          }
          mma_commit(&q_empty[qs]);
          mma_commit(&k_empty[ks]);
        }
      }
      mma_commit(s_ready);
      if (nblk > 0) {
        constexpr uint32_t idesc = instr_desc(1u, 1u, 128, F::NB * 64) | (1u << 16);  // B MN-major
        if (ok) {
          if constexpr (C > 1) ok = wait_cluster(p_full, 0u, s_abort, err);
          else ok = mbar_wait(p_full, 0u, s_abort, err);
        }
        tc_fence_after();
        const uint32_t pa = smem_u32(smem);
        for (int half = 0; half < F::Halves; ++half) {
          for (int kb = 0; ok && kb < nblk; ++kb) {
            const int st = kb % F::GV;
            const int use = half * ((nblk - st + F::GV - 1) / F::GV) + kb / F::GV;
            if (!(ok = mbar_wait(&v_full[st], use & 1, s_abort, err))) break;
            tc_fence_after();
            const uint32_t vb = smem_u32(smem + kOffV + st * F::VStage);
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_bf16(tmem + F::OCol + half * 256, smem_desc_sw128(pa + kb * kPBlock + s * 32),
                       smem_desc_mn_sw128(vb + s * 16 * 128), idesc, (kb | s) ? 1u : 0u);
            mma_commit(&v_empty[st]);
          }
          mma_commit(&o_ready[half]);
        }
        // every MMA has completed before TMEM is released (bounded, also after an abort)
        mbar_drain(&o_ready[F::Halves - 1], 0u);
        // copies of other CTAs into this one's P have landed (bounded)
        if (C > 1 && !ok) mbar_drain(p_full, 0u);
      }
      mbar_drain(s_ready, 0u);
    }
    __syncwarp();
  } else {
    // ---------------- Q chunks (one thread)
    if (lane == 0 && nc > 0) {
      const uint32_t bytes = static_cast<uint32_t>(p.n_heads) * 128u;
      int issued = 0;
      for (int c = 0; c < kChunks; ++c) {
        const int qs = c % F::NQS;
        if (!mbar_wait(&q_empty[qs], ((c / F::NQS) & 1) ^ 1u, s_abort, err)) break;
        mbar_arrive_expect_tx(&q_full[qs], bytes);
        tma_load_2d(smem + F::OffQ + qs * kQBytes, &tmap_q, &q_full[qs], c * 64,
                    static_cast<int32_t>(t * p.n_heads));
        issued = c + 1;
      }
      for (int c = max(0, issued - F::NQS); c < issued; ++c)  // never exit with loads in flight
        mbar_drain(&q_full[c % F::NQS], (c / F::NQS) & 1);
    }
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

bool encode_q(CUtensorMap* m, const void* q, int64_t rows, int32_t box_rows) {
  std::call_once(g_enc_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult r{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      g_enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(kRowDims), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(kRowDims) * 2};
  cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1u, 1u};
  return g_enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(q), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int C>
int launch(const CUtensorMap& tq, const Params& p, int64_t T, void* stream) {
  if (cudaFuncSetAttribute(sparse_attn_q4_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<C>::Smem) != cudaSuccess) {
    cudaGetLastError();
    return DS4IDX_ERR_CUDA;
  }
  return launch_dependent(sparse_attn_q4_kernel<C>, static_cast<unsigned>(T * C), kThreads,
                          Cfg<C>::Smem, C, stream, tq, p);
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
  CUtensorMap tq;
  if (!encode_q(&tq, q, T * n_heads, n_heads)) return DS4IDX_ERR_CUDA;
  p.cache = cache;
  p.idx = idx;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.weights = weights;
  p.err = ds4a::sparse_attention_error_word();
  if (!p.err) return DS4IDX_ERR_CUDA;
  p.n_heads = n_heads;
  p.n_sel = n_sel;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  // The widest cluster whose CTAs still fit the 152 SMs at once (clusters of 8 pack two to a GPC).
  if (T <= 16) return launch<8>(tq, p, T, stream);
  if (T <= 32) return launch<4>(tq, p, T, stream);
  if (T <= 76) return launch<2>(tq, p, T, stream);
  return launch<1>(tq, p, T, stream);
}
