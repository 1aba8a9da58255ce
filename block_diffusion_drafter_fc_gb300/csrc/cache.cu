// Trees of drafted tokens (ancestor masks, greedy acceptance) and the pages of
// the cache (commit of an accepted path, reserve, fork, trim).
//
// All of these are small integer work, or copies that run at the memory's rate;
// every result is independent of the order in which blocks and atomics run
// (integer sums, minima, and ranks that come from scans).
#include "cache.cuh"

#include <limits.h>

namespace dflash {

namespace {

// ------------------------------------------------------------------ trees

// One block per entry.  M_i, the set of node i and its ancestors, by pointer
// doubling: with up_i the ancestor 2^r levels up, M_i |= M_{up_i} and up_i =
// up_{up_i}; after round r M_i covers 2^r levels, so a chain of n nodes takes
// log2 n rounds instead of n dependent steps.  Within a round a set may already
// hold another node's update: still only ancestors, and at least the levels the
// pointer read in this round skips.  Bound: latency, the rounds' barriers: masks
// and walk of 256 trees of 1..128 nodes take 6.4 us in a graph, of one of 26 4.4.
__global__ void tree_mask_kernel(RowView rows, const int32_t* parents, uint32_t* mask, int words,
                                 int32_t* depth, unsigned* status) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ uint32_t sm[];
  const int s = blockIdx.x;
  int lo, n;
  if (!entry_rows(rows, s, lo, n) || n > 32 * words) {
    if (threadIdx.x == 0) set_status(status, DEV_BAD_ROWS);
    return;
  }
  if (n == 0) return;
  const int nw = (n + 31) / 32;         // words that hold nodes
  int* up = reinterpret_cast<int*>(sm);
  uint32_t* m = sm + n;                 // [n][nw]
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int p = parents[lo + i];
    if (p < -1 || p >= i) {
      set_status(status, DEV_BAD_TREE);
      p = -1;
    }
    up[i] = p;
    for (int w = 0; w < nw; ++w) m[i * nw + w] = w == i / 32 ? 1u << (i & 31) : 0u;
  }
  __syncthreads();
  for (int span = 1; span < n; span *= 2) {
    // at most kTreeMax / blockDim nodes a thread: their new pointers wait in registers
    int next[kTreeMax / 128];
#pragma unroll
    for (int k = 0; k < kTreeMax / 128; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      next[k] = -1;
      if (i >= n || up[i] < 0) continue;
      const int a = up[i];
      next[k] = up[a];
      for (int w = 0; w < nw; ++w) m[i * nw + w] |= m[a * nw + w];
    }
    __syncthreads();
    int left = 0;
#pragma unroll
    for (int k = 0; k < kTreeMax / 128; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      if (i >= n) continue;
      up[i] = next[k];
      left |= next[k] >= 0;
    }
    if (!__syncthreads_or(left)) break;
  }
  for (int e = threadIdx.x; e < n * words; e += blockDim.x) {
    const int i = e / words, w = e - i * words;
    mask[(size_t)lo * words + e] = w < nw ? m[i * nw + w] : 0u;
  }
  if (depth)
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      int d = -1;
      for (int w = 0; w < nw; ++w) d += __popc(m[i * nw + w]);
      depth[lo + i] = d;
    }
}

// One block per entry: next[i] is node i's child of lowest index that carries
// the target's token (a minimum, whatever the order), then one thread walks the
// list from the anchor.
__global__ void tree_accept_kernel(RowView rows, const int32_t* parents, const int32_t* tokens,
                                   const int32_t* targets, int32_t* path, int max_path, int32_t* n_path,
                                   int32_t* id_last, unsigned* status) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ int next[];   // [kTreeMax], longer trees walk in pieces below
  __shared__ int s_len, s_cur;
  const int s = blockIdx.x;
  int lo, n;
  if (!entry_rows(rows, s, lo, n)) {
    if (threadIdx.x == 0) set_status(status, DEV_BAD_ROWS);
    n = 0;
  }
  int32_t* out = path + (size_t)s * max_path;
  if (threadIdx.x == 0) {
    s_len = 0;
    s_cur = n > 0 ? 0 : -1;
  }
  // pieces of kTreeMax parents: a walk that leaves the piece goes on in a later
  // one (children lie behind their parents)
  for (int base = 0; base < n; base += kTreeMax) {
    const int m = min(kTreeMax, n - base);
    for (int i = threadIdx.x; i < m; i += blockDim.x) next[i] = INT_MAX;
    __syncthreads();
    for (int i = max(base, 1) + threadIdx.x; i < n; i += blockDim.x) {
      const int p = parents[lo + i];
      if (p >= base && p < base + m && p < i && tokens[lo + i] == targets[lo + p]) atomicMin(&next[p - base], i);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int cur = s_cur, len = s_len;
      // s_cur: the next accepted node, or -1 once the walk has ended
      while (cur >= base && cur < base + m && len < max_path) {
        out[len++] = cur;
        const int to = next[cur - base];
        if (to == INT_MAX || len == max_path) {
          id_last[s] = targets[lo + cur];
          cur = -1;
        } else {
          cur = to;
        }
      }
      s_cur = cur;
      s_len = len;
    }
    __syncthreads();
  }
  __syncthreads();
  const int len = s_len;
  if (threadIdx.x == 0) n_path[s] = len;
  for (int j = len + threadIdx.x; j < max_path; j += blockDim.x) out[j] = -1;
}

// ------------------------------------------------------------------ commit

constexpr int kBatch = 8;   // tokens in flight per thread

// grid (blocks, entries).  A block first maps the path's slots to pages, then
// each thread owns 16-byte columns of (layer, k|v, head): it reads up to kBatch
// tokens of a column before it writes any of them, ascending, so a slot is read
// before it is overwritten (path[j] >= j, ascending; no other thread touches the
// column).  The last block of an entry to have read its length writes the new
// one.  Bound: memory: 92 MB (32 sequences, 32 layers, 12 slots) in 18 us from HBM =
// 5.1 TB/s, 14.6 us in a loop that finds them in L2.
__global__ void __launch_bounds__(256) commit_kernel(CacheView c, RowView rows, const int32_t* path,
                                                     int max_path, const int32_t* n_path, int* tickets) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ long long s_off[];   // [max_path] from, [max_path] to
  const int s = blockIdx.y;
  const int q = entry_sequence(rows, s, c.max_seq);
  const bool dup = listed_before(rows, s, q);
  const int n = n_path[s], len = q >= 0 ? c.length[q] : 0;
  unsigned bad = 0;
  if (q < 0 || dup)
    bad = DEV_BAD_SEQ;
  else if (n < 0 || len < 0 || (long long)len + n > (long long)c.max_pages * c.ps)
    bad = DEV_BAD_ROWS;
  else if (path && n > max_path)
    bad = DEV_BAD_TREE;
  if (!bad && path) {
    unsigned mine = 0;
    auto row_of = [&](int node) -> long long {
      const long long slot = (long long)len + node, idx = slot >> c.ps_log2;
      const int page = idx < c.max_pages ? c.table[(size_t)q * c.max_pages + idx] : -1;
      if (page < 0 || page >= c.n_pages || c.refs[page] > 1) {
        mine |= DEV_BAD_PAGE;
        return 0;
      }
      return (long long)page_row(c, page, 0, 0, 0, (int)(slot & (c.ps - 1)));
    };
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
      const int a = path[(size_t)s * max_path + j], before = j ? path[(size_t)s * max_path + j - 1] : -1;
      if (a <= before || a < j) {
        mine |= DEV_BAD_TREE;
        continue;
      }
      s_off[j] = row_of(a);
      s_off[max_path + j] = row_of(j);
    }
    bad = __syncthreads_or(mine & DEV_BAD_TREE) ? DEV_BAD_TREE : 0;
    if (__syncthreads_or(mine & DEV_BAD_PAGE)) bad |= DEV_BAD_PAGE;
  }
  if (!bad && !path && n > 0) {
    const int k1 = (int)(((long long)len + n - 1) >> c.ps_log2);
    int gone = 0;
    for (int k = (len >> c.ps_log2) + threadIdx.x; k <= k1; k += blockDim.x) {
      const int page = c.table[(size_t)q * c.max_pages + k];
      gone |= page < 0 || page >= c.n_pages || c.refs[page] > 1;   // (a shared one was not written for this sequence)
    }
    if (__syncthreads_or(gone)) bad = DEV_BAD_PAGE;
  }
  // every thread of the block has the length
  __syncthreads();
  if (threadIdx.x == 0) {
    if (bad && blockIdx.x == 0) set_status(c.status, bad);
    __threadfence();
    if (atomicAdd(&tickets[s], 1) == (int)gridDim.x - 1) {
      tickets[s] = 0;
      if (!bad) c.length[q] = len + n;
    }
  }
  if (bad || !path) return;
  int j0 = 0;   // the leading tokens that stay in place
  while (j0 < n && s_off[j0] == s_off[max_path + j0]) ++j0;
  if (j0 == n) return;
  const int chunks = c.hd * c.el / 16;
  const size_t head_bytes = (size_t)c.ps * c.hd * c.el;
  const long long cols = (long long)c.n_layer * 2 * c.n_head_kv * chunks;
  for (long long e = blockIdx.x * (long long)blockDim.x + threadIdx.x; e < cols;
       e += (long long)gridDim.x * blockDim.x) {
    const long long head = e / chunks;
    char* base = c.pages + head * head_bytes + (e - head * chunks) * 16;
    for (int j = j0; j < n; j += kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j + b < n) v[b] = *reinterpret_cast<const uint4*>(base + s_off[j + b]);
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j + b < n) *reinterpret_cast<uint4*>(base + s_off[max_path + j + b]) = v[b];
    }
  }
}

// ------------------------------------------------------------------ reserve

constexpr int kPlan = 1024;   // threads of the planning block

constexpr int kMany = 1 << 29;   // sums of the scan saturate here

// Exclusive sum over the block's threads (kPlan); total gets the sum.
DF_DEVICE int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = min(x + y, kMany);
  }
  __syncthreads();   // the previous scan's sums have been read
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w = min(w + y, kMany);
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return x - v + (warp ? before : 0);
}

// One block plans the call.  Entry s spans the table entries first .. first +
// span - 1 of its sequence; all spans together are one list, in the entries'
// order, and the entries of it that need a page are ranked by scans of the
// list; rank r gets the r-th free page.  Three passes over the list and one
// over refs (until enough free pages are found), each kPlan wide: nothing is
// changed before the totals are known.  Bound: latency, 9 us for 24 entries,
// cold; more blocks would have to agree on the pages' order.
__global__ void __launch_bounds__(kPlan) reserve_plan_kernel(CacheView c, RowView rows, const int32_t* count,
                                                             int32_t* free_list, int4* copies) {
  pdl_trigger();
  pdl_wait();
  __shared__ int s_warp[32];
  __shared__ int s_owner[4096];
  __shared__ int s_first[kCallSeq], s_end[kCallSeq], s_seq[kCallSeq], s_old[kCallSeq];
  const int s = threadIdx.x;
  for (int i = s; i < c.max_seq; i += kPlan) s_owner[i] = INT_MAX;
  __syncthreads();
  int q = -1, len = 0, cnt = 0;
  unsigned bad = 0;
  if (s < rows.n_seq) {
    q = entry_sequence(rows, s, c.max_seq);
    if (q >= 0) atomicMin(&s_owner[q], s);
    cnt = count[s];
  }
  __syncthreads();
  if (s < rows.n_seq) {
    if (q < 0 || s_owner[q] != s) {
      bad = DEV_BAD_SEQ;
      q = -1;
    } else {
      len = c.length[q];
      if (cnt < 0 || len < 0 || len > c.max_pages * c.ps) bad = DEV_BAD_ROWS;
    }
    if (bad) len = cnt = 0;   // (such an entry asks for nothing, and refuses nothing to the others)
  }
  const int first = len >> c.ps_log2;
  const long long last = cnt > 0 ? ((long long)len + cnt - 1) >> c.ps_log2 : first - 1;
  const bool fits = last < c.max_pages;
  const int span = fits ? min((int)(last - first + 1), kMany) : 0;
  // a part-filled page that others hold too: its earlier holders in the list
  // will have left it, so the last one of all its holders keeps it
  int old = -1;
  if (span > 0 && (len & (c.ps - 1))) {
    old = c.table[(size_t)q * c.max_pages + first];
    if (old >= c.n_pages || (old >= 0 && c.refs[old] <= 1)) old = -1;
  }
  s_old[s] = old;
  s_first[s] = first;
  s_seq[s] = q;
  int total;
  const int begin = block_scan(span, s_warp, total);
  s_end[s] = begin + span;
  const int list = total;
  bool copy = false;
  if (old >= 0) {
    int earlier = 0;
    for (int i = 0; i < s; ++i) earlier += s_old[i] == old;
    copy = c.refs[old] - earlier > 1;
  }
  if (bad) set_status(c.status, bad);
  if (__syncthreads_or(!fits) || list >= kMany) {
    if (s < rows.n_seq) copies[s] = make_int4(0, 0, 0, 0);
    if (s == 0) set_status(c.status, DEV_NO_PAGES);
    return;
  }
  __syncthreads();
  s_old[s] = copy ? old : -1;   // from here on: the page to copy
  __syncthreads();

  // list entry e -> its sequence entry, table index, and whether it needs a page
  auto look = [&](int e, int& i, int& idx) -> bool {
    int a = 0, b = rows.n_seq - 1;   // first entry whose list ends behind e
    while (a < b) {
      const int mid = (a + b) >> 1;
      if (s_end[mid] > e) b = mid; else a = mid + 1;
    }
    i = a;
    idx = s_first[a] + e - (a ? s_end[a - 1] : 0);
    if (idx == s_first[a] && s_old[a] >= 0) return true;
    return c.table[(size_t)s_seq[a] * c.max_pages + idx] < 0;
  };
  int need = 0;
  for (int e0 = 0; e0 < list; e0 += kPlan) {
    int i, idx, t;
    const bool want = e0 + s < list && look(e0 + s, i, idx);
    block_scan(want, s_warp, t);
    need += t;
  }
  // the first `need` free pages, in ascending order
  int found = 0;
  constexpr int kPer = 8;   // pages of a thread per round
  for (int p0 = 0; p0 < c.n_pages && found < need; p0 += kPlan * kPer) {
    const int p = p0 + s * kPer;
    int mine = 0;
    if (p + kPer <= c.n_pages) {
      const int4 a = *reinterpret_cast<const int4*>(c.refs + p), b = *reinterpret_cast<const int4*>(c.refs + p + 4);
      const int v[kPer] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < kPer; ++k) mine |= (v[k] == 0) << k;
    } else {
      for (int k = 0; k < kPer; ++k)
        if (p + k < c.n_pages) mine |= (c.refs[p + k] == 0) << k;
    }
    int t;
    int at = found + block_scan(__popc(mine), s_warp, t);
    for (; mine && at < need; mine &= mine - 1) free_list[at++] = p + __ffs(mine) - 1;
    found += t;
  }
  if (found < need) {
    if (s < rows.n_seq) copies[s] = make_int4(0, 0, 0, 0);
    if (s == 0) set_status(c.status, DEV_NO_PAGES);
    return;
  }
  __syncthreads();   // free_list is written
  if (s < rows.n_seq && !copy) copies[s] = make_int4(0, 0, 0, 0);
  int done = 0;
  for (int e0 = 0; e0 < list; e0 += kPlan) {
    int i = 0, idx = 0, t;
    const bool want = e0 + s < list && look(e0 + s, i, idx);
    const int r = done + block_scan(want, s_warp, t);
    done += t;
    if (!want) continue;
    const int page = free_list[r];
    c.refs[page] = 1;
    if (idx == s_first[i] && s_old[i] >= 0) {
      atomicSub(&c.refs[s_old[i]], 1);
      copies[i] = make_int4(s_old[i], page, c.length[s_seq[i]] & (c.ps - 1), 0);
    }
    c.table[(size_t)s_seq[i] * c.max_pages + idx] = page;
  }
}

// grid (blocks, entries): the slots an entry keeps of its part-filled page, for
// every (layer, k|v, head) a contiguous run; 74 MB in 13 us (5.7 TB/s).
__global__ void __launch_bounds__(256) reserve_copy_kernel(CacheView c, const int4* copies) {
  pdl_trigger();
  pdl_wait();
  const int4 w = copies[blockIdx.y];
  if (w.z <= 0) return;
  const size_t head_bytes = (size_t)c.ps * c.hd * c.el;
  const int heads = c.n_layer * 2 * c.n_head_kv;
  const int run = w.z * c.hd * c.el / 16;   // 16-byte vectors of one run
  const char* src = c.pages + (size_t)w.x * heads * head_bytes;
  char* dst = c.pages + (size_t)w.y * heads * head_bytes;
  const long long total = (long long)heads * run, step = (long long)gridDim.x * blockDim.x;
  constexpr int kU = 4;
  for (long long e = blockIdx.x * (long long)blockDim.x + threadIdx.x; e < total; e += kU * step) {
    uint4 v[kU];
    size_t off[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const long long x = e + u * step;
      if (x >= total) continue;
      const long long h = x / run;
      off[u] = (size_t)h * head_bytes + (size_t)(x - h * run) * 16;
      v[u] = *reinterpret_cast<const uint4*>(src + off[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (e + u * step < total) *reinterpret_cast<uint4*>(dst + off[u]) = v[u];
  }
}

// ------------------------------------------------------------------ fork, trim

// One block per entry.
__global__ void __launch_bounds__(256) fork_kernel(CacheView c, int n, const int32_t* src, const int32_t* dst) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x, a = src[i], b = dst[i];
  int bad = a < 0 || a >= c.max_seq || b < 0 || b >= c.max_seq;
  for (int j = threadIdx.x; j < n; j += blockDim.x) bad |= src[j] == b || (j < i && dst[j] == b);
  int32_t* to = c.table + (size_t)(bad ? 0 : b) * c.max_pages;
  // a sequence's pages are given out from its first on
  if (!bad && threadIdx.x == 0) bad = c.length[b] != 0 || to[0] >= 0;
  const int len = bad ? 0 : c.length[a];
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_status(c.status, DEV_BAD_SEQ);
    return;
  }
  const int held = (int)min((long long)c.max_pages, ((long long)max(len, 0) + c.ps - 1) >> c.ps_log2);
  const int32_t* from = c.table + (size_t)a * c.max_pages;
  for (int k = threadIdx.x; k < held; k += blockDim.x) {
    const int page = from[k];
    to[k] = page;
    if (page >= 0 && page < c.n_pages)
      atomicAdd(&c.refs[page], 1);
    else
      set_status(c.status, DEV_BAD_PAGE);
  }
  if (threadIdx.x == 0) c.length[b] = len;
}

// grid (blocks, entries): table entries from the first page that is not kept.
__global__ void __launch_bounds__(256) trim_kernel(CacheView c, RowView rows, const int32_t* new_len) {
  pdl_trigger();
  pdl_wait();
  const int s = blockIdx.y;
  const int q = entry_sequence(rows, s, c.max_seq);
  const bool dup = listed_before(rows, s, q);
  const int keep_len = new_len[s];
  const unsigned bad = q < 0 || dup ? DEV_BAD_SEQ : keep_len < 0 ? DEV_BAD_ROWS : 0u;
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(c.status, bad);
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && c.length[q] > keep_len) c.length[q] = keep_len;
  const long long keep = ((long long)keep_len + c.ps - 1) >> c.ps_log2;
  int32_t* t = c.table + (size_t)q * c.max_pages;
  for (long long k = keep + blockIdx.x * blockDim.x + threadIdx.x; k < c.max_pages; k += gridDim.x * blockDim.x) {
    const int page = t[k];
    if (page == -1) continue;
    t[k] = -1;
    if (page >= 0 && page < c.n_pages)
      atomicSub(&c.refs[page], 1);
    else
      set_status(c.status, DEV_BAD_PAGE);
  }
}

size_t mask_smem(int words) { return sizeof(uint32_t) * 32 * words * (1 + (size_t)words); }

}  // namespace

cudaError_t configure_tree() {
  return cudaFuncSetAttribute(tree_mask_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)mask_smem(kTreeMax / 32));
}

cudaError_t launch_tree_mask(const RowView& rows, const int32_t* parents, uint32_t* mask, int words,
                             int32_t* depth, unsigned* status, cudaStream_t st) {
  return launch_dependent(tree_mask_kernel, dim3(rows.n_seq), 128, mask_smem(words), st, rows, parents, mask, words,
                          depth, status);
}

cudaError_t launch_tree_accept(const RowView& rows, const int32_t* parents, const int32_t* tokens,
                               const int32_t* targets, int32_t* path, int max_path, int32_t* n_path,
                               int32_t* id_last, unsigned* status, cudaStream_t st) {
  return launch_dependent(tree_accept_kernel, dim3(rows.n_seq), 128, sizeof(int) * kTreeMax, st, rows, parents, tokens,
                          targets, path, max_path, n_path, id_last, status);
}

cudaError_t launch_commit(const CacheView& c, const RowView& rows, const int32_t* path, int max_path,
                          const int32_t* n_path, int* tickets, cudaStream_t st) {
  int gx = 1;
  if (path) {   // a column per thread, as long as that is at most four waves of blocks
    const long long cols = (long long)c.n_layer * 2 * c.n_head_kv * (c.hd * c.el / 16);
    const long long most = (4LL * 152 * 8 + rows.n_seq - 1) / rows.n_seq;
    const long long want = (cols + 255) / 256;
    gx = (int)(want < most ? want : most);
  }
  return launch_dependent(commit_kernel, dim3(gx, rows.n_seq), 256, path ? sizeof(long long) * 2 * max_path : 0, st, c,
                          rows, path, max_path, n_path, tickets);
}

cudaError_t launch_reserve(const CacheView& c, const RowView& rows, const int32_t* count,
                           int32_t* free_list, int4* copies, cudaStream_t st) {
  const cudaError_t e = launch_dependent(reserve_plan_kernel, dim3(1), kPlan, 0, st, c, rows, count, free_list, copies);
  if (e != cudaSuccess) return e;
  const long long vecs = (long long)c.n_layer * 2 * c.n_head_kv * c.ps * c.hd * c.el / 16;
  const long long most = (4LL * 152 * 8 + rows.n_seq - 1) / rows.n_seq, want = (vecs + 1023) / 1024;
  return launch_dependent(reserve_copy_kernel, dim3((int)(want < most ? want : most), rows.n_seq), 256, 0, st, c,
                          (const int4*)copies);
}

cudaError_t launch_fork(const CacheView& c, int n, const int32_t* src, const int32_t* dst, cudaStream_t st) {
  return launch_dependent(fork_kernel, dim3(n), 256, 0, st, c, n, src, dst);
}

cudaError_t launch_trim(const CacheView& c, const RowView& rows, const int32_t* new_len, cudaStream_t st) {
  const int gx = (c.max_pages + 1023) / 1024;   // four entries a thread
  return launch_dependent(trim_kernel, dim3(gx < 64 ? gx : 64, rows.n_seq), 256, 0, st, c, rows, new_len);
}

}  // namespace dflash
