// Shared prefixes of a call's entries (the attention over them: tree_common.cuh).
//
// Sequences that were forked from one another hold the same pages for as long as their
// beginnings are full pages, so a group's common slots are found in the page table: no
// promise of the caller's is needed, and a wrong group only shares less.
#include "cache.cuh"

namespace dflash {

namespace {

constexpr int kPlanThreads = 1024;

// Fewest slots that sharing has to save, over all members, to be worth the rows' second part,
// for entries of one row (us of the attention shared, and with a plan of zeros): 4 members over
// 1024 slots 13.1, 14.8, over 512 12.9, 13.2; 32 members over 256 19.7, 25.6, over 64 20.6, 20.4.
// The rule does not know the rows.  32 members of 16: over 512 slots 35, 33, 1024 40.6, 40.6, 4096 62,
// 82; of 32: 4096 104, 93, 16384 260, 277; of 64 (x 4 heads: a tile of their own): 4096 182, 134.
constexpr int kWorthSlots = 2048;

// A block per group.  The group shares the full pages, below the least length, in which no
// member's row of the table differs from the first's.  Bound: latency, five dependent loads.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(CacheView c, RowView rows, int n_group,
                                                                   const int32_t* group_start, int32_t* plan) {
  __shared__ int s_pages;
  pdl_trigger();
  pdl_wait();
  const int g = blockIdx.x, tid = threadIdx.x, n = rows.n_seq;
  // group ranges that are none: nothing is shared
  int bad = 0;
  for (int i = tid; i < n_group; i += kPlanThreads) {
    const int a = group_start[i], b = group_start[i + 1];
    bad |= a < 0 || a > b || b > n;
  }
  if (tid == 0) s_pages = 0x7fffffff;
  if (__syncthreads_or(bad)) {
    if (g == 0) {
      for (int i = tid; i < n + n_group; i += kPlanThreads) plan[i] = 0;
      if (tid == 0) set_status(c.status, DEV_BAD_ROWS);
    }
    return;
  }
  const int e0 = group_start[g], e1 = group_start[g + 1], members = e1 - e0;
  // entries of no group
  if (g == 0)
    for (int i = tid; i < e0; i += kPlanThreads) plan[i] = 0;
  if (g == n_group - 1)
    for (int i = e1 + tid; i < n; i += kPlanThreads) plan[i] = 0;
  int pages = 0x7fffffff;
  for (int i = tid; i < members; i += kPlanThreads) {
    const int q = entry_sequence(rows, e0 + i, c.max_seq), len = q >= 0 ? c.length[q] : -1;
    pages = min(pages, len < 0 ? 0 : min(len >> c.ps_log2, c.max_pages));
  }
  atomicMin(&s_pages, pages);
  __syncthreads();
  pages = members > 1 ? s_pages : 0;
  __syncthreads();
  if (pages > 0) {
    const int32_t* first = c.table + (size_t)entry_sequence(rows, e0, c.max_seq) * c.max_pages;
    // (a warp a member, eight pages a lane at a time: 32 members of 256 pages in one round of
    // loads; page after page took 22 us)
    int same = pages;
    for (int i = 1 + (tid >> 5); i < members; i += kPlanThreads / 32) {
      const int32_t* mine = c.table + (size_t)entry_sequence(rows, e0 + i, c.max_seq) * c.max_pages;
      for (int p0 = tid & 31; p0 < same; p0 += 256) {
        int a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int p = min(p0 + 32 * k, pages - 1);
          a[k] = mine[p];
          b[k] = first[p];
        }
#pragma unroll
        for (int k = 7; k >= 0; --k)
          if (a[k] != b[k]) same = min(same, p0 + 32 * k);
      }
    }
    if (same < pages) atomicMin(&s_pages, same);
    __syncthreads();
    pages = s_pages;
  }
  const int slots = pages << c.ps_log2, shared = (long long)slots * (members - 1) < kWorthSlots ? 0 : slots;
  for (int i = tid; i < members; i += kPlanThreads) plan[e0 + i] = shared;
  if (tid == 0) plan[n + g] = shared;
}

}  // namespace

cudaError_t launch_prefix_plan(const CacheView& c, const RowView& rows, int n_group, const int32_t* group_start,
                               int32_t* plan, cudaStream_t st) {
  return launch_dependent(prefix_plan_kernel, dim3(n_group), kPlanThreads, 0, st, c, rows, n_group, group_start, plan);
}

}  // namespace dflash
