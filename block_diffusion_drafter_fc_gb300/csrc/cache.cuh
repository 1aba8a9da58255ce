// Device helpers shared by the cache, rope and tree kernels.
#pragma once

#include "cache.h"
#include "common.cuh"

namespace dflash {

DF_DEVICE void set_status(unsigned* status, unsigned bit) { atomicOr(status, bit); }

// Sequence of entry s, -1 when out of range.
DF_DEVICE int entry_sequence(const RowView& r, int s, int max_seq) {
  const int q = r.seqs ? r.seqs[s] : s;
  return q >= 0 && q < max_seq ? q : -1;
}

// Rows lo .. lo + n - 1 of entry s; false when they are not within 0..T.
DF_DEVICE bool entry_rows(const RowView& r, int s, int& lo, int& n) {
  lo = r.row_start[s];
  const int hi = r.row_start[s + 1];
  n = hi - lo;
  return lo >= 0 && lo <= hi && hi <= r.T;
}

// Byte offset of slot row `at` of (page, layer, k|v, head).
DF_DEVICE size_t page_row(const CacheView& c, int page, int layer, int kv, int head, int at) {
  return ((((size_t)page * c.n_layer + layer) * 2 + kv) * c.n_head_kv + head) * ((size_t)c.ps * c.hd * c.el) +
         (size_t)at * c.hd * c.el;
}

// Whether sequence q of entry s is listed by an earlier entry (all threads of the block).
DF_DEVICE bool listed_before(const RowView& r, int s, int q) {
  int dup = 0;
  if (r.seqs)
    for (int i = threadIdx.x; i < s; i += blockDim.x) dup |= r.seqs[i] == q;
  return __syncthreads_or(dup) != 0;
}

}  // namespace dflash
