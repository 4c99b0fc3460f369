// tern_cache.h -- the paged int8 cache as its kernels see it: where a
// sequence's rows and positions lie, checked against the buffers, so that no
// content of the caller's device arrays reaches past them.
#pragma once

#include "tern_device.h"

namespace tern {

// One sequence of a call: `n` new rows from `row0`, the first at position
// pos0 (negative where the length is shorter than the new rows: those rows
// have no place in the cache); `len` positions are held, at most as many as
// the table has pages for.
struct SeqView {
  int32_t row0, n;
  int64_t pos0, len;
};

__device__ __forceinline__ SeqView seq_view(const KvArgs& a, int s) {
  SeqView v;
  const int32_t r0 = load_g(a.start + s), r1 = load_g(a.start + s + 1);
  const bool ok = r0 >= 0 && r1 >= r0 && r1 <= a.rows;
  v.row0 = ok ? r0 : 0;
  v.n = ok ? r1 - r0 : 0;
  const int64_t len = max(load_g(a.len + s), 0);
  v.pos0 = len - v.n;
  v.len = min(len, (int64_t)a.ld_table << a.log_p);
  return v;
}

// Page `j` of a sequence as the table has it (-1 past the table), and that or -1
// where it is an id outside the cache.
__device__ __forceinline__ int32_t page_entry(const KvArgs& a, int s, int64_t j) {
  return j < 0 || j >= a.ld_table ? -1 : load_g(a.table + (int64_t)s * a.ld_table + j);
}
__device__ __forceinline__ int32_t valid_page(const KvArgs& a, int32_t id) { return id >= 0 && id < a.pages ? id : -1; }
__device__ __forceinline__ int32_t page_of(const KvArgs& a, int s, int64_t j) {
  return valid_page(a, page_entry(a, s, j));
}

}  // namespace tern
