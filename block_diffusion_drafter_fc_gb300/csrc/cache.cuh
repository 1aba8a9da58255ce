// Device helpers shared by the cache, rope and tree kernels.
#pragma once

#include "cache.h"
#include "common.cuh"
#include "launch_shapes.h"

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

// y / d (launch_shapes.h: quotient_magic, and where it is exact)
DF_DEVICE int small_quotient(int y, uint32_t magic) { return magic ? (int)__umulhi((uint32_t)y, magic) : y; }

// A launch that may start while the kernel before it ends: every kernel here lets
// the next one be scheduled at once and waits for the one before it with
// griddepcontrol.wait before it touches global memory (a turn's small calls then
// cost no launch gaps).  One exception: verify_kernel reads its call's inputs ahead
// of its wait; row_stats_kernel, launched just before it, lets it start only behind
// its own wait, when everything that came earlier is done.  No launch may come
// between the two.
template <typename K, typename... A>
cudaError_t launch_dependent(K* kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dflash
