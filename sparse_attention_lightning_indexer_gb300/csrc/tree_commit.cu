// The rows of a drafted tree's accepted path to the end of their sequence, in place, in every per-row
// array of a pool: row len + j = row len + path[j], j < n_accepted, and the sequence's new length.
//
// A CTA takes one sequence and one slice of an array's rows: all rows of the path (at most 64) are read
// into shared memory before one is written, so a path may name any nodes in any order. Nothing but the
// accepted rows is moved; the time is the chain of three dependent reads (path, page table, rows).
// Measured on the device: one sequence 2.6 us, 64 paged ones of 64 nodes and five arrays 3.1.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "launch.cuh"
#include "placement.cuh"
#include "ptx.cuh"

namespace ds4tc {

using namespace ds4;

constexpr int kThreads = 256, kNodes = 64, kArrays = 8;
constexpr int kSlice = 640;  // bytes of a row that a CTA takes: 64 rows fit static shared memory

struct Array {
  uint8_t* at;
  int32_t row_bytes;
  int32_t unit;  // bytes of one access: 16, 8, 4, 2 or 1
};
struct Params {
  Array a[kArrays];
  int32_t slice0[kArrays + 1];  // the arrays' first slices in the grid
  const int32_t* lens;
  const int32_t* path;
  const int32_t* count;
  int32_t* new_lens;
  Placement place;
  int32_t n_arrays, n_nodes, slices;
};

template <typename T>
__device__ __forceinline__ void move(const Array& a, int byte0, int bytes, int n, const int64_t* src,
                                     const int64_t* dst, uint8_t* buf) {
  const int units = bytes / static_cast<int>(sizeof(T));
  T* s = reinterpret_cast<T*>(buf);
  for (int i = threadIdx.x; i < n * units; i += kThreads) {
    const int j = i / units, u = i - j * units;
    if (src[j] >= 0)
      s[i] = reinterpret_cast<const T*>(a.at + src[j] * a.row_bytes + byte0)[u];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * units; i += kThreads) {
    const int j = i / units, u = i - j * units;
    if (src[j] >= 0) reinterpret_cast<T*>(a.at + dst[j] * a.row_bytes + byte0)[u] = s[i];
  }
}

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) uint8_t buf[kNodes * kSlice];
  __shared__ int64_t src[kNodes], dst[kNodes];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
  const int64_t len = p.lens[b];
  const int n = min(max(p.count[b], 0), p.n_nodes);
  if (slice == 0 && threadIdx.x == 0)
    p.new_lens[b] = static_cast<int32_t>(min(len + n, static_cast<int64_t>(0x7FFFFFFF)));
  if (p.n_arrays == 0) return;
  if (threadIdx.x < n) {
    const int j = threadIdx.x;
    const int node = p.path[static_cast<int64_t>(b) * p.n_nodes + j];
    int64_t from = -1, to = -1;
    // (a node at its place already is left there)
    if (node >= 0 && node < p.n_nodes && node != j && len >= 0 && len <= 0x7FFFFFFF - kNodes) {
      const TokenPlace tp = place_token(p.place, b);
      from = place_row(p.place, tp, static_cast<int32_t>(len) + node);
      to = place_row(p.place, tp, static_cast<int32_t>(len) + j);
    }
    src[j] = to >= 0 ? from : -1;
    dst[j] = to;
  }
  __syncthreads();
  int k = 0;
  while (slice >= p.slice0[k + 1]) ++k;
  const Array a = p.a[k];
  const int byte0 = (slice - p.slice0[k]) * kSlice, bytes = min(kSlice, a.row_bytes - byte0);
  switch (a.unit) {
    case 16: move<uint4>(a, byte0, bytes, n, src, dst, buf); break;
    case 8: move<uint2>(a, byte0, bytes, n, src, dst, buf); break;
    case 4: move<uint32_t>(a, byte0, bytes, n, src, dst, buf); break;
    case 2: move<uint16_t>(a, byte0, bytes, n, src, dst, buf); break;
    default: move<uint8_t>(a, byte0, bytes, n, src, dst, buf);
  }
}

struct Bytes {
  uintptr_t low, high;
};
inline bool meet(const Bytes& a, const Bytes& b) { return a.low < b.high && b.low < a.high; }

}  // namespace ds4tc

extern "C" int ds4idx_tree_commit(const int32_t* kv_lens, const int32_t* path,
                                  const int32_t* n_accepted, int32_t* new_lens,
                                  const ds4idx_placement* where, int32_t B, int32_t n_nodes,
                                  int64_t rows, int32_t n_arrays, const ds4idx_row_array* arrays,
                                  void* stream) {
  using namespace ds4tc;
  if (B < 0 || n_nodes < 1 || n_nodes > kNodes || n_arrays < 0 || n_arrays > kArrays || rows < 1 ||
      rows > 0x7FFFFFFF || B > (1 << 20) || (n_arrays > 0 && !arrays))
    return DS4IDX_ERR_INVALID_ARG;
  if (B == 0) return DS4IDX_OK;
  Params p{};
  if (!kv_lens || !path || !n_accepted || !new_lens || !aligned_to(kv_lens, 4) ||
      !aligned_to(path, 4) || !aligned_to(n_accepted, 4) || !aligned_to(new_lens, 4) ||
      !make_placement(where, rows, B, &p.place))
    return DS4IDX_ERR_INVALID_ARG;
  auto span = [](const void* at, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(at);
    return Bytes{a, a + static_cast<uintptr_t>(bytes)};
  };
  // What a CTA reads while another may write: nothing of it may overlap what is written.
  Bytes read[6 + kArrays], written[1 + kArrays];
  int n_read = 0;
  read[n_read++] = span(kv_lens, 4ll * B);
  read[n_read++] = span(path, 4ll * B * n_nodes);
  read[n_read++] = span(n_accepted, 4ll * B);
  if (p.place.row0) read[n_read++] = span(p.place.row0, 8ll * B);
  if (p.place.table) read[n_read++] = span(p.place.table, 4ll * p.place.n_seqs * p.place.pages);
  if (p.place.seq) read[n_read++] = span(p.place.seq, 4ll * B);
  written[0] = span(new_lens, 4ll * B);
  for (int k = 0; k < n_arrays; ++k) {
    const ds4idx_row_array& a = arrays[k];
    if (!a.src || a.src != a.dst || a.src_rows != rows || a.dst_rows != rows || a.row_bytes < 1 ||
        a.row_bytes > 65536)
      return DS4IDX_ERR_INVALID_ARG;
    int unit = 16;
    while (unit > 1 && (a.row_bytes % unit || !aligned_to(a.src, unit))) unit >>= 1;
    p.a[k] = Array{static_cast<uint8_t*>(a.dst), a.row_bytes, unit};
    p.slice0[k + 1] = p.slice0[k] + (a.row_bytes + kSlice - 1) / kSlice;
    written[1 + k] = span(a.dst, rows * a.row_bytes);
  }
  for (int i = 0; i <= n_arrays; ++i) {
    for (int j = 0; j < n_read; ++j)
      if (meet(written[i], read[j])) return DS4IDX_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(written[i], written[j])) return DS4IDX_ERR_INVALID_ARG;
  }
  p.lens = kv_lens;
  p.path = path;
  p.count = n_accepted;
  p.new_lens = new_lens;
  p.n_arrays = n_arrays;
  p.n_nodes = n_nodes;
  p.slices = std::max(1, p.slice0[n_arrays]);
  if (static_cast<int64_t>(B) * p.slices > 0x7FFFFFFF) return DS4IDX_ERR_INVALID_ARG;
  return launch_dependent(tree_commit_kernel, static_cast<unsigned>(B) * p.slices, kThreads, 0, 1,
                          stream, p);
}
