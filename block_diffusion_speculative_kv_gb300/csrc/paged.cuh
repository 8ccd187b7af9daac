// Paged KV cache: addressing and argument checks shared by the append and the
// attention over pages (include/dflash.h, dflash_pages).
#pragma once

#include "common.cuh"

namespace dfl {

// Device view of a dflash_pages.
struct PagedView {
  void* k;
  void* v;
  const int32_t* table;
  int table_ld, n_pages, page_shift, n_kv;
};

inline int log2_int(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Page of a slot of request r, or -1 where there is none.
__device__ __forceinline__ int page_of(const PagedView& pv, int r, int slot) {
  const int i = slot >> pv.page_shift;
  if (slot < 0 || i >= pv.table_ld) return -1;
  const int page = __ldg(pv.table + (size_t)r * pv.table_ld + i);
  return static_cast<unsigned>(page) < static_cast<unsigned>(pv.n_pages) ? page : -1;
}

// Row of KV head g's slot inside a pool seen as [n_pages * n_kv * page_size] rows.
__device__ __forceinline__ long long pool_row(const PagedView& pv, int page, int g, int slot) {
  return ((((long long)page * pv.n_kv + g) << pv.page_shift) +
          (slot & ((1 << pv.page_shift) - 1)));
}

// The request of a global row: the number of requests that end at or before it
// (n_req when the row is past the last one).  All lanes of a warp call it with
// the same row; each round narrows the range 32-fold.
__device__ __forceinline__ int request_of(const int32_t* row_off, int n_req, int row, int lane) {
  int lo = 0, hi = n_req;   // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + step * (lane + 1) - 1;          // probe the last of each part
    const bool ended = i < hi && __ldg(row_off + i + 1) <= row;
    const int n = __popc(__ballot_sync(0xffffffffu, ended));
    lo += n * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// (n_req 0: a table of no rows, whose pointer may be null)
dflash_status check_pages(const dflash_pages* p, int n_req, const char* what, PagedView* out);

}  // namespace dfl
