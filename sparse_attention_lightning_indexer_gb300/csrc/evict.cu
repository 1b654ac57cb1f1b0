// Eviction by accumulated attention weight, for sm_103a: the totals of the pool rows, the choice of
// the rows a sequence keeps, and the move of those rows.
//
// Totals are int64 in units of 2^-32. Integer adds commute, so the sum does not depend on the order
// in which the atomics of a chunk's tokens arrive; fp32 atomics would not give that.
//
// Choice. Of a sequence's rows between its sinks and its recent ones the need largest totals are
// kept, ties to the lower position. One CTA or a cluster of 8 owns a sequence, each CTA a contiguous
// part, each warp a contiguous segment, kept on chip up to 196608 totals. A radix select of 11 bits
// a pass: counts per digit in shared memory, each CTA sums a slice of the bins over the cluster, all
// scan the slice that holds the cut. The first digit is the leading bit's place and the five bits
// behind it, so the pass separates totals of any size; a pass ends the search when the whole digit
// is kept. Then one pass counts the kept rows per segment and one writes them in order. The bytes
// are few (8 a row, read once); bound by the instructions of the passes and the cluster's barriers.
//
// Move. Bound by HBM: each kept row is read and written once, in the widest units its size and
// addresses allow, by CTAs that take about 16 KB of one array each.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "launch.cuh"
#include "placement.cuh"
#include "ptx.cuh"

namespace ds4e {

using namespace ds4;

// ------------------------------------------------------------------------------ accumulation

constexpr int kAccThreads = 256;

__global__ void __launch_bounds__(kAccThreads)
    accumulate_kernel(unsigned long long* total, const float* weights, const int32_t* idx,
                      const __grid_constant__ Placement place, int32_t n_sel, int32_t per_token) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x / per_token;
  const int32_t j = static_cast<int32_t>(blockIdx.x % per_token) * kAccThreads + threadIdx.x;
  if (j >= n_sel) return;
  const int32_t s = idx[t * n_sel + j];
  const float w = weights[t * n_sel + j];
  const int64_t r = place_row(place, place_token(place, t), s);
  if (r < 0 || !(fabsf(w) < 1073741824.f)) return;
  const int64_t v = __float2ll_rn(w * 4294967296.f);  // the product is exact
  if (v != 0) atomicAdd(total + r, static_cast<unsigned long long>(v));
}

// ------------------------------------------------------------------------------ choice

constexpr int kMaxB = 64;
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kDigit = 11, kBins = 1 << kDigit;

struct SelectParams {
  const int64_t* total;
  int32_t* kept;
  int64_t width;
  int64_t sink, recent;
  int32_t cluster;
  int64_t start[kMaxB], len[kMaxB], keep[kMaxB];
};

__device__ __forceinline__ uint32_t peer_u32(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t ld_peer32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_u32(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// First digit of a total: 0 for negative ones, 1 for zero, else 32 bins per power of two by the five
// bits behind the leading one (of the truncating conversion to fp32, which keeps 23). Totals
// spread over many powers of two, so equal widths would put most of them into a few bins.
__device__ __forceinline__ uint32_t first_digit(uint64_t key) {
  const uint64_t t = key & ~(1ull << 63);
  const uint32_t f = __float_as_uint(__ull2float_rz(t)) >> 18;
  const uint32_t digit = t ? f - (127 * 32 - 2) : 1u;
  return key >> 63 ? digit : 0u;
}

constexpr int kOnChip = 24;  // keys of a thread in shared memory

// K = 4: a thread's keys (at most four) are in registers. K = 0: the first kOnChip are in shared
// memory, the rest (sequences past 24576 totals a CTA) are read again by every pass.
template <int K>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint32_t s_hist[2][kBins];
  __shared__ uint32_t s_sums[2][kBins / 2];  // this CTA's slice, summed over the cluster
  __shared__ uint32_t s_warp[kWarps];
  __shared__ uint32_t s_gt[kWarps], s_eq[kWarps];
  __shared__ uint32_t s_cut[3];       // digit, rows above it, rows in it
  __shared__ uint32_t s_slice[2];     // rows in this CTA's slice of the bins
  __shared__ uint32_t s_tot[2];       // this CTA's kept-for-sure and tied rows
  griddep_wait();
  griddep_launch_dependents();
  const int C = p.cluster;
  const int b = blockIdx.x / C;
  const uint32_t rank = blockIdx.x % C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = p.len[b], keep = p.keep[b];
  int32_t* out = p.kept + b * p.width;
  const int64_t cta_threads = static_cast<int64_t>(C) * kThreads;
  const int64_t me = static_cast<int64_t>(rank) * kThreads + tid;
  const int64_t count = keep < n ? keep : n;
  for (int64_t i = count + me; i < p.width; i += cta_threads) out[i] = -1;
  if (keep >= n) {  // the same for every CTA of the cluster
    for (int64_t i = me; i < n; i += cta_threads) out[i] = static_cast<int32_t>(i);
    return;
  }
  const int64_t sink = p.sink, recent = p.recent;
  for (int64_t i = me; i < sink; i += cta_threads) out[i] = static_cast<int32_t>(i);
  for (int64_t i = me; i < recent; i += cta_threads)
    out[keep - recent + i] = static_cast<int32_t>(n - recent + i);
  uint32_t need = static_cast<uint32_t>(keep - sink - recent);
  if (need == 0) return;  // the same for every CTA of the cluster

  const int64_t* mid = p.total + p.start[b] + sink;
  const int32_t m = static_cast<int32_t>(n - sink - recent);  // > need
  const int32_t per = (m + C - 1) / C;
  const int32_t c0 = min(m, static_cast<int32_t>(rank) * per), c1 = min(m, c0 + per);
  const int32_t seg = ((c1 - c0 + kWarps - 1) / kWarps + 31) & ~31;
  const int32_t w0 = min(c1, c0 + warp * seg), w1 = min(c1, w0 + seg);
  extern __shared__ uint64_t s_keys[];  // [kOnChip][kThreads]
  uint64_t keys[4];
  auto read = [&](int32_t i) { return i < w1 ? static_cast<uint64_t>(mid[i]) ^ (1ull << 63) : 0; };
  if constexpr (K == 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) keys[u] = read(w0 + u * 32 + lane);
  } else {
    // (asynchronous copies, all in flight together; the sign is turned when a key is used)
    for (int u = 0; u < kOnChip; ++u) {
      const int32_t i = w0 + u * 32 + lane;
      if (i < w1)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                         smem_u32(s_keys + u * kThreads + tid)),
                     "l"(mid + i)
                     : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // each thread reads only its own copies
  }
  // f(key, position, in): every key of this warp's segment, all lanes together
  auto each = [&](auto&& f) {
    if constexpr (K == 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (w0 + u * 32 >= w1) break;
        f(keys[u], w0 + u * 32 + lane, w0 + u * 32 + lane < w1);
      }
    } else {
      int32_t i0 = w0;
#pragma unroll 4
      for (int u = 0; u < kOnChip; ++u, i0 += 32) {
        if (i0 >= w1) break;
        f(s_keys[u * kThreads + tid] ^ (1ull << 63), i0 + lane, i0 + lane < w1);
      }
#pragma unroll 8
      for (; i0 < w1; i0 += 32) f(read(i0 + lane), i0 + lane, i0 + lane < w1);
    }
  };

  for (int i = tid; i < 2 * kBins; i += kThreads) (&s_hist[0][0])[i] = 0;
  for (int i = tid; i < kBins; i += kThreads) (&s_sums[0][0])[i] = 0;
  __syncthreads();
  int top = 64;          // undecided low bits of a key; 64: no pass done yet
  uint64_t lo = 0, hi = ~0ull;  // the keys that share the decided bits
  int buf = 0;
  bool whole = false;
  while (top > 0 && !whole) {
    const bool first = top == 64;
    const int d = min(kDigit, top), shift = top - d;
    uint32_t* hist = s_hist[buf];
    each([&](uint64_t key, int32_t, bool in) {
      in = in && key >= lo && key <= hi;
      const uint32_t act = __ballot_sync(0xffffffffu, in);
      if (!act) return;
      const uint32_t digit =
          first ? first_digit(key) : static_cast<uint32_t>(key >> shift) & ((1u << d) - 1);
      // many rows share one total (rows never attended): one add if the whole warp does
      const uint32_t d0 = __shfl_sync(0xffffffffu, digit, __ffs(act) - 1);
      if (__all_sync(0xffffffffu, !in || digit == d0)) {
        if (lane == 0) atomicAdd(hist + d0, __popc(act));
      } else if (in) {
        atomicAdd(hist + digit, 1u);
      }
    });
    // Sums over the cluster: CTA r adds up a slice of the bins (a peer's count a thread, so that
    // the loads' latencies overlap) and publishes the slice's total; then every CTA finds the slice
    // that holds the cut, and the digit in it.
    const int slice = kBins / C;
    uint32_t* sums = s_sums[buf];
    uint32_t base = 0;      // rows in the slices above the one that holds the cut
    int owner = 0;
    if (C == 1) {
      __syncthreads();
    } else {
      cluster_sync();
#pragma unroll
      for (int q = tid; q < kBins; q += kThreads) {
        const uint32_t v = ld_peer32(hist + rank * slice + q % slice, q / slice);
        if (v) atomicAdd(sums + q % slice, v);
      }
      __syncthreads();
      uint32_t sum = tid < slice ? sums[tid] : 0;  // slice <= 1024 = threads
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == 0) s_warp[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        sum = __reduce_add_sync(0xffffffffu, s_warp[lane]);
        if (lane == 0) s_slice[buf] = sum;
      }
      cluster_sync();
      // lane l: the slice C - 1 - l, so that a running sum counts the rows above
      const uint32_t t = lane < C ? ld_peer32(&s_slice[buf], C - 1 - lane) : 0;
      uint32_t inc = t;
      for (int o = 1; o < 16; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const int at = __ffs(__ballot_sync(0xffffffffu, lane < C && inc >= need)) - 1;
      base = __shfl_sync(0xffffffffu, inc - t, at);
      owner = C - 1 - at;
    }
    // the other buffers were last read before this pass's first barrier
    for (int i = tid; i < kBins; i += kThreads) s_hist[buf ^ 1][i] = 0;
    for (int i = tid; i < kBins / 2; i += kThreads) s_sums[buf ^ 1][i] = 0;
    // that slice's bins in falling order, two a thread at C = 1, else at most one or two
    const int per_thread = (slice + kThreads - 1) / kThreads;
    const int bin0 = owner * slice + slice - 1 - per_thread * tid;  // this thread's first bin
    uint32_t h0 = 0, h1 = 0;
    if (per_thread * tid < slice) {
      h0 = C > 1 ? ld_peer32(sums + bin0 - owner * slice, owner) : hist[bin0];
      if (per_thread == 2) h1 = hist[bin0 - 1];  // (C = 1)
    }
    uint32_t inc = h0 + h1;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();  // (s_warp is free again)
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    const uint32_t below = lane < warp ? s_warp[lane] : 0;
    const uint32_t ex = base + __reduce_add_sync(0xffffffffu, below) + inc - h0 - h1;
    if (ex < need && need <= ex + h0) {
      s_cut[0] = bin0;
      s_cut[1] = ex;
      s_cut[2] = h0;
    } else if (ex + h0 < need && need <= ex + h0 + h1) {
      s_cut[0] = bin0 - 1;
      s_cut[1] = ex + h0;
      s_cut[2] = h1;
    }
    __syncthreads();
    const uint32_t digit = s_cut[0];
    need -= s_cut[1];
    whole = need == s_cut[2];
    if (!first) {
      lo += static_cast<uint64_t>(digit) << shift;
      top = shift;
    } else if (digit == 0) {         // negative totals: bit 63 is decided
      top = 63;
    } else if (digit == 1) {         // zero
      lo = 1ull << 63;
      top = 0;
    } else {                         // leading bit e, then five bits (all of them if e < 5)
      const int e = (digit - 2) / 32;
      const uint32_t lead = 32 + (digit - 2) % 32;
      top = max(e - 5, 0);
      lo = (1ull << 63) | (e >= 5 ? static_cast<uint64_t>(lead) << top : lead >> (5 - e));
    }
    hi = lo + ((1ull << top) - 1);
    buf ^= 1;
  }
  // kept: above the cut, and of those at it the first `need` in position order
  uint32_t ng = 0, ne = 0;
  each([&](uint64_t key, int32_t, bool in) {
    ng += in && key > hi;
    ne += in && key >= lo && key <= hi;
  });
  ng = __reduce_add_sync(0xffffffffu, ng);
  ne = __reduce_add_sync(0xffffffffu, ne);
  if (lane == 0) {
    s_gt[warp] = ng;
    s_eq[warp] = ne;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t g = __reduce_add_sync(0xffffffffu, s_gt[lane]);
    const uint32_t e = __reduce_add_sync(0xffffffffu, s_eq[lane]);
    if (lane == 0) {
      s_tot[0] = g;
      s_tot[1] = e;
    }
  }
  if (C > 1) cluster_sync();
  uint32_t g = 0, e = 0;
  if (lane < rank) {
    g = ld_peer32(&s_tot[0], lane);
    e = ld_peer32(&s_tot[1], lane);
  }
  g += lane < warp ? s_gt[lane] : 0;
  e += lane < warp ? s_eq[lane] : 0;
  g = __reduce_add_sync(0xffffffffu, g);
  e = __reduce_add_sync(0xffffffffu, e);
  const uint32_t lt = (1u << lane) - 1;
  each([&](uint64_t key, int32_t i, bool in) {
    const bool is_g = in && key > hi, is_e = in && key >= lo && key <= hi;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_g), be = __ballot_sync(0xffffffffu, is_e);
    const uint32_t eb = e + __popc(be & lt);
    if (is_g || (is_e && eb < need))
      out[sink + g + __popc(bg & lt) + min(eb, need)] = static_cast<int32_t>(sink + i);
    g += __popc(bg);
    e += __popc(be);
  });
  if (C > 1) cluster_sync();  // no CTA leaves while another may still read its counts
}

// ------------------------------------------------------------------------------ move

constexpr int kMaxArrays = 8;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 1024;       // most rows of one CTA
constexpr int kMoveBytes = 16384;     // about what one CTA moves

struct Array {
  const uint8_t* src;
  uint8_t* dst;
  int32_t row_bytes, unit, units;  // unit: bytes a thread moves at once
  int32_t rows;                    // rows a CTA moves
  int64_t cta0;                    // first CTA of this array
};
struct MoveParams {
  Array a[kMaxArrays];
  const int32_t* kept;
  int64_t width, rows;
  int32_t n, B;
  int64_t first[kMaxB + 1];        // kept rows before sequence b
  int64_t src_start[kMaxB], src_len[kMaxB], dst_start[kMaxB];
};

template <typename U>
__device__ __forceinline__ void move_rows(const Array& a, const int64_t* s_src, const int64_t* s_dst,
                                          int rows) {
  constexpr int kFly = 4;
  const uint32_t units = a.units, all = units * rows;
  for (uint32_t u0 = threadIdx.x; u0 < all; u0 += kMoveThreads * kFly) {
    U v[kFly];
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      const uint32_t u = u0 + j * kMoveThreads, r = u / units;
      if (u < all && s_src[r] >= 0)
        v[j] = reinterpret_cast<const U*>(a.src + s_src[r] * a.row_bytes)[u - r * units];
    }
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      const uint32_t u = u0 + j * kMoveThreads, r = u / units;
      if (u < all && s_src[r] >= 0)
        reinterpret_cast<U*>(a.dst + s_dst[r] * a.row_bytes)[u - r * units] = v[j];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ MoveParams p) {
  __shared__ int64_t s_src[kMoveRows], s_dst[kMoveRows];
  griddep_wait();
  griddep_launch_dependents();
  int k = 0;
  while (k + 1 < p.n && blockIdx.x >= p.a[k + 1].cta0) ++k;
  const Array& a = p.a[k];
  const int64_t r0 = (blockIdx.x - a.cta0) * a.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), p.rows - r0));
  for (int i = threadIdx.x; i < rows; i += kMoveThreads) {
    int lo = 0, hi = p.B - 1;  // the last sequence that starts at or before this row
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (p.first[m] <= r0 + i) lo = m; else hi = m - 1;
    }
    const int64_t j = r0 + i - p.first[lo];
    const int32_t s = p.kept[lo * p.width + j];
    s_src[i] = s >= 0 && s < p.src_len[lo] ? p.src_start[lo] + s : -1;
    s_dst[i] = p.dst_start[lo] + j;
  }
  __syncthreads();
  switch (a.unit) {
    case 16: move_rows<uint4>(a, s_src, s_dst, rows); break;
    case 8: move_rows<uint2>(a, s_src, s_dst, rows); break;
    case 4: move_rows<uint32_t>(a, s_src, s_dst, rows); break;
    case 2: move_rows<uint16_t>(a, s_src, s_dst, rows); break;
    default: move_rows<uint8_t>(a, s_src, s_dst, rows); break;
  }
}

// A range of bytes that a move reads (a sequence's source rows) or writes.
struct Range {
  uintptr_t at, end;
  bool written;
};
// Whether a written range meets any other: sorted by their starts, a range that begins before the end
// of an earlier one meets it. Reads may share rows.
bool written_meets_another(Range* r, int n) {
  std::sort(r, r + n, [](const Range& a, const Range& b) { return a.at < b.at; });
  uintptr_t any_end = 0, written_end = 0;
  for (int i = 0; i < n; ++i) {
    if (r[i].at < (r[i].written ? any_end : written_end)) return true;
    any_end = std::max(any_end, r[i].end);
    if (r[i].written) written_end = std::max(written_end, r[i].end);
  }
  return false;
}

}  // namespace ds4e

extern "C" int ds4idx_evict_accumulate(int64_t* total, int64_t pool_rows, const float* weights,
                                       const int32_t* idx, const ds4idx_placement* where,
                                       int64_t T, int32_t n_sel, void* stream) {
  using namespace ds4e;
  if (T < 0 || n_sel < 1 || pool_rows < 1 || pool_rows > 0x7FFFFFFF) return DS4IDX_ERR_INVALID_ARG;
  if (T == 0) return DS4IDX_OK;
  const int64_t per_token = (static_cast<int64_t>(n_sel) + kAccThreads - 1) / kAccThreads;
  if (T > 0x7FFFFFFF / per_token) return DS4IDX_ERR_INVALID_ARG;
  Placement p;
  if (!total || !weights || !idx || !aligned_to(total, 8) || !aligned_to(weights, 4) ||
      !aligned_to(idx, 4) || !make_placement(where, pool_rows, T, &p))
    return DS4IDX_ERR_INVALID_ARG;
  return launch_dependent(accumulate_kernel, static_cast<unsigned>(T * per_token), kAccThreads, 0, 1,
                          stream, reinterpret_cast<unsigned long long*>(total), weights, idx, p,
                          n_sel, static_cast<int32_t>(per_token));
}

extern "C" int ds4idx_evict_select(const int64_t* total, int64_t pool_rows, int32_t B,
                                   const int64_t* starts, const int64_t* seq_lens,
                                   const int64_t* keep, int64_t n_sink, int64_t n_recent,
                                   int32_t* kept, int64_t width, void* stream) {
  using namespace ds4e;
  if (B < 1 || B > kMaxB || !starts || !seq_lens || !keep || n_sink < 0 || n_recent < 0 ||
      n_sink > 0x7FFFFFFF || n_recent > 0x7FFFFFFF || width < 0 || width > 0x7FFFFFFF ||
      pool_rows < 0)
    return DS4IDX_ERR_INVALID_ARG;
  SelectParams p{};
  int64_t longest = 0;
  for (int b = 0; b < B; ++b) {
    if (seq_lens[b] < 0 || seq_lens[b] > (1 << 30) || starts[b] < 0 ||
        starts[b] > pool_rows - seq_lens[b] || keep[b] < n_sink + n_recent ||
        std::min(keep[b], seq_lens[b]) > width)
      return DS4IDX_ERR_INVALID_ARG;
    p.start[b] = starts[b];
    p.len[b] = seq_lens[b];
    p.keep[b] = keep[b];
    if (keep[b] < seq_lens[b]) longest = std::max(longest, seq_lens[b]);
  }
  if (width == 0) return DS4IDX_OK;
  if (!kept || !aligned_to(kept, 4) || (longest > 0 && (!total || !aligned_to(total, 8))))
    return DS4IDX_ERR_INVALID_ARG;
  p.total = total;
  p.kept = kept;
  p.width = width;
  p.sink = n_sink;
  p.recent = n_recent;
  // One CTA up to four totals a thread (in registers: 9 us at 4096, of which a cluster would spend
  // more on its barriers); else a cluster of 8, the largest portable size. (Clusters of 16 hold
  // 262144 totals on chip, but only four of them run at once.)
  if (longest <= 4 * kThreads) {
    p.cluster = 1;
    return launch_dependent(select_kernel<4>, static_cast<unsigned>(B), kThreads, 0, 1, stream, p);
  }
  constexpr size_t kKeyBytes = kOnChip * kThreads * sizeof(uint64_t);
  static std::atomic<uint64_t> done{0};
  if (!allow_shared(select_kernel<0>, kKeyBytes, done)) return DS4IDX_ERR_CUDA;
  p.cluster = 8;
  return launch_dependent(select_kernel<0>, static_cast<unsigned>(B * 8), kThreads, kKeyBytes, 8,
                          stream, p);
}

extern "C" int ds4idx_evict_compact(const int32_t* kept, int64_t width, int32_t B,
                                    const int64_t* src_starts, const int64_t* src_lens,
                                    const int64_t* dst_starts, const int64_t* counts,
                                    int32_t n_arrays, const ds4idx_row_array* arrays,
                                    void* stream) {
  using namespace ds4e;
  if (B < 1 || B > kMaxB || n_arrays < 1 || n_arrays > kMaxArrays || !src_starts || !src_lens ||
      !dst_starts || !counts || !arrays || width < 0 || width > 0x7FFFFFFF)
    return DS4IDX_ERR_INVALID_ARG;
  MoveParams p{};
  p.kept = kept;
  p.width = width;
  p.n = n_arrays;
  p.B = B;
  for (int b = 0; b < B; ++b) {
    if (src_starts[b] < 0 || src_lens[b] < 0 || src_lens[b] > 0x7FFFFFFF || dst_starts[b] < 0 ||
        counts[b] < 0 || counts[b] > width || counts[b] > src_lens[b])
      return DS4IDX_ERR_INVALID_ARG;
    p.src_start[b] = src_starts[b];
    p.src_len[b] = src_lens[b];
    p.dst_start[b] = dst_starts[b];
    p.first[b + 1] = p.first[b] + counts[b];
  }
  p.rows = p.first[B];
  int64_t ctas = 0;
  Range ranges[kMaxArrays * 2 * kMaxB];
  int n_ranges = 0;
  for (int k = 0; k < n_arrays; ++k) {
    const ds4idx_row_array& d = arrays[k];
    if (d.row_bytes < 1 || d.row_bytes > 65536) return DS4IDX_ERR_INVALID_ARG;
    if (p.rows > 0 && (!d.src || !d.dst)) return DS4IDX_ERR_INVALID_ARG;
    const uint8_t* src = static_cast<const uint8_t*>(d.src);
    uint8_t* dst = static_cast<uint8_t*>(d.dst);
    for (int b = 0; b < B; ++b) {
      if (src_starts[b] > d.src_rows - src_lens[b] || dst_starts[b] > d.dst_rows - counts[b])
        return DS4IDX_ERR_INVALID_ARG;
      auto range = [&](const uint8_t* base, int64_t row, int64_t rows, bool written) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(base) + row * d.row_bytes;
        if (rows > 0) ranges[n_ranges++] = {at, at + rows * d.row_bytes, written};
      };
      range(src, src_starts[b], src_lens[b], false);
      range(dst, dst_starts[b], counts[b], true);
    }
    const uintptr_t bits = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) |
                           static_cast<uintptr_t>(d.row_bytes);
    Array& a = p.a[k];
    a.src = src;
    a.dst = dst;
    a.row_bytes = d.row_bytes;
    a.unit = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
    a.units = d.row_bytes / a.unit;
    a.rows = std::max(1, std::min(kMoveRows, kMoveBytes / d.row_bytes));
    a.cta0 = ctas;
    ctas += (p.rows + a.rows - 1) / a.rows;
  }
  if (p.rows == 0) return DS4IDX_OK;
  if (written_meets_another(ranges, n_ranges)) return DS4IDX_ERR_INVALID_ARG;
  if (!kept || !aligned_to(kept, 4) || ctas > 0x7FFFFFFF) return DS4IDX_ERR_INVALID_ARG;
  return launch_dependent(move_kernel, static_cast<unsigned>(ctas), kMoveThreads, 0, 1, stream, p);
}
