// Where position s of a token's sequence lies in a pool of rows (ds4idx_placement on the device).
#pragma once
#include <cstdint>

#include "ds4idx.h"
#include "launch.cuh"

namespace ds4 {

struct Placement {
  const int64_t* row0;
  const int32_t* table;
  const int32_t* seq;
  int64_t n_seqs;
  int64_t rows;
  int32_t page, pages;
};

// The token's part of the look-up: the first row of a contiguous sequence, or its table row.
struct TokenPlace {
  int64_t row0;
  const int32_t* table;  // null: contiguous
  bool ok;
};
__device__ __forceinline__ TokenPlace place_token(const Placement& p, int64_t t) {
  if (!p.table) return {p.row0 ? p.row0[t] : 0, nullptr, true};
  const int64_t b = p.seq ? p.seq[t] : t;
  const bool ok = b >= 0 && b < p.n_seqs;
  return {0, p.table + (ok ? b * p.pages : 0), ok};
}
// Pool row of position s, or -1 if the entry is empty or the row lies outside the pool.
__device__ __forceinline__ int64_t place_row(const Placement& p, const TokenPlace& tp, int32_t s) {
  if (s < 0 || !tp.ok) return -1;
  int64_t r;
  if (tp.table) {
    const int32_t page = s / p.page;
    if (page >= p.pages) return -1;
    const int32_t id = tp.table[page];
    if (id < 0) return -1;
    r = static_cast<int64_t>(id) * p.page + (s - page * p.page);
  } else {
    r = tp.row0 + s;
  }
  return r >= 0 && r < p.rows ? r : -1;
}

// Checks the host struct; rows is the pool's size. T > 0.
inline bool make_placement(const ds4idx_placement* w, int64_t rows, int64_t T, Placement* p) {
  *p = Placement{};
  p->rows = rows;
  if (!w) return true;
  if (!w->page_table) {
    if (w->token_seq || (w->kv_row0 && !aligned_to(w->kv_row0, 8))) return false;
    p->row0 = w->kv_row0;
    return true;
  }
  if (w->kv_row0 || w->page_size < 1 || w->pages_per_seq < 1 || w->n_seqs < 1 ||
      !aligned_to(w->page_table, 4) || !aligned_to(w->token_seq, 4) ||
      (!w->token_seq && T > w->n_seqs))
    return false;
  p->table = w->page_table;
  p->seq = w->token_seq;
  p->n_seqs = w->n_seqs;
  p->page = w->page_size;
  p->pages = w->pages_per_seq;
  return true;
}

}  // namespace ds4
