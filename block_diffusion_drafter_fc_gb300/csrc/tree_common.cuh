// Shared parts of the tree-attention kernels: barriers and copies, the plan
// that cuts a call's work into equal ranges, and the join of tiles that ranges cut.
#pragma once

#include "cache.cuh"

#include <math_constants.h>

namespace dflash {
namespace tree {

constexpr long long kWait = 4000000000LL;   // ~2 s, then DFLASH_DEV_TIMEOUT
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

DF_DEVICE uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
DF_DEVICE void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n) : "memory");
}
DF_DEVICE void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes)
               : "memory");
}
DF_DEVICE void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
DF_DEVICE void bar_arrive_n(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(n) : "memory");
}
DF_DEVICE bool bar_try(uint64_t* b, uint32_t par) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(su32(b)), "r"(par)
      : "memory");
  return ok != 0;
}
// Bounded wait: false when it, or one of another thread, gave up; the block then
// runs to its end without waiting.
DF_DEVICE bool bar_wait(uint64_t* b, uint32_t par, volatile int* abort, unsigned* status) {
  if (bar_try(b, par)) return true;
  if (*abort) return false;
  const long long t0 = clock64();
  while (!bar_try(b, par)) {
    if (*abort) return false;
    if (clock64() - t0 > kWait) {
      *abort = 1;
      set_status(status, DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}
DF_DEVICE void tma3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(su32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(su32(b))
      : "memory");
}
DF_DEVICE float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Quotient of nonnegative numbers; the 64-bit division (some hundred clocks,
// which every block of a small call would wait for) only where it is needed.
DF_DEVICE long long quotient(long long a, long long b) {
  return ((unsigned long long)(a | b) >> 32) ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// An entry of the call.  Its rows (a row: one query head of a kv head's group,
// of one node) form tiles, its slots chunks; the work is the chunks of every
// tile of every kv head.
struct Entry {
  int lo, n, len, q;
};

// How a kernel cuts a call's rows and slots, and what the pieces cost: a chunk
// of a tile of more than `wide` rows `heavy` units, of others `light`, and every
// tile `extra` units for its start and end.  Without the weights a range of many
// short tiles took twice the time of a range within a long one.
struct Cutting {
  int tile, chunk, wide, heavy, light, extra;
  // chunks of w units that begin before unit x (divisions by constants, not by w)
  DF_DEVICE int chunks(long long x, int w) const;
};

DF_DEVICE int Cutting::chunks(long long x, int w) const {
  return (int)(w == light ? quotient(x + light - 1, light) : quotient(x + heavy - 1, heavy));
}

// The row blocks of one kv head of an entry and their cost.  Without a mask a
// tile sees no slot behind its last node: block i then has ceil((len + e_i) /
// chunk) chunks, e_i = tile (i + 1) / group nodes, summed in closed form (the
// tile holds whole nodes and one of tile / group and chunk divides the other);
// else every block has all chunks.
struct Blocks {
  Cutting c;
  int count, nch;          // row blocks; chunks of the last (longest) one
  int step;                // chain: nodes per block (0: not trimmed)
  int last;                // units of a chunk of the last block (the others are full)
  long long first;         // slots of block 0, + chunk - 1

  DF_DEVICE Blocks(const AttendParams& p, const Cutting& cut, const Entry& x) : c(cut), step(0), first(0) {
    const long long rows = (long long)x.n * p.grp;
    count = (int)quotient(rows + c.tile - 1, c.tile);
    nch = (int)quotient((long long)x.len + x.n + c.chunk - 1, c.chunk);
    last = rows - (long long)(count - 1) * c.tile > c.wide ? c.heavy : c.light;
    if (p.step && count > 1) {
      step = p.step;
      first = (long long)x.len + step + c.chunk - 1;
    }
  }
  DF_DEVICE int units(int i) const { return i == count - 1 ? last : c.heavy; }   // of a chunk of block i
  // chunks of blocks 0 .. i - 1, i <= count - 1
  DF_DEVICE long long chunks_before(int i) const {
    if (!step) return (long long)i * nch;
    if (step >= c.chunk)
      return (long long)i * quotient(first, c.chunk) + (long long)(step / c.chunk) * i * (i - 1) / 2;
    // sum of floor((first + j step) / chunk) = sum of a + floor((r + j) / 2^lq)
    // (step is a power of two: it divides the tile)
    const int ls = __ffs(step) - 1, lq = __ffs(c.chunk) - 1 - ls;
    const int a = (int)quotient(first, c.chunk), r = (int)(first - (long long)a * c.chunk) >> ls;
    auto tri = [&](long long x) {
      const long long t = x >> lq;
      return (t * (t - 1) / 2 << lq) + t * (x - (t << lq));
    };
    return (long long)i * a + tri(r + i) - tri(r);
  }
  // units of blocks 0 .. i - 1, i <= count
  DF_DEVICE long long before(int i) const {
    return chunks_before(min(i, count - 1)) * c.heavy + (i == count ? (long long)nch * last : 0) +
           (long long)i * c.extra;
  }
  DF_DEVICE int chunks(int i) const {
    return i == count - 1 ? nch : (int)(chunks_before(i + 1) - chunks_before(i));
  }
};

// Nodes of a tile, where Blocks may trim (see there).
inline int trim_step(const AttendParams& a, int tile, int chunk) {
  if (a.mask || tile % a.grp) return 0;
  const int per = tile / a.grp;
  return per % chunk == 0 || chunk % per == 0 ? per : 0;
}

// Entry s and its units (0: skipped; bad: why).
DF_DEVICE long long plan_entry(const AttendParams& p, const Cutting& cut, int s, Entry& x, unsigned& bad) {
  const CacheView& c = p.c;
  const int lo = p.rows.row_start[s], hi = p.rows.row_start[s + 1];   // (loads of one round trip)
  x.q = entry_sequence(p.rows, s, c.max_seq);
  x.len = x.q >= 0 ? c.length[x.q] : 0;
  x.lo = lo;
  x.n = hi - lo;
  bad = 0;
  if (lo < 0 || lo > hi || hi > p.rows.T || x.n > p.max_tree)
    bad = DEV_BAD_ROWS;
  else if (x.n > 0 && x.q < 0)
    bad = DEV_BAD_SEQ;
  else if (x.n > 0 && (x.len < 0 || (long long)x.len + x.n > (long long)c.max_pages * c.ps))
    bad = DEV_BAD_ROWS;
  if (bad) x.n = 0;
  if (x.n <= 0) return 0;
  const Blocks b(p, cut, x);
  return c.n_head_kv * b.before(b.count);
}

// plan_entries by one warp, of at most 32 entries: the block's other warps need not wait.
DF_DEVICE void plan_few(const AttendParams& p, const Cutting& cut, Entry* e, long long* end, bool report) {
  const int s = threadIdx.x & 31;
  Entry x;
  unsigned bad = 0;
  long long v = s < p.rows.n_seq ? plan_entry(p, cut, s, x, bad) : 0;
  if (bad && report) set_status(p.c.status, bad);
#pragma unroll 1
  for (int o = 1; o < p.rows.n_seq; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (s >= o) v += y;
  }
  if (s < p.rows.n_seq) {
    e[s] = x;
    end[s] = v;
  }
  __syncwarp();
}

// The call's work as one list of units, the entries' one after another: fills
// e[] and end[] (end[s]: units of entries 0..s; a skipped entry has none) with
// all `threads` threads of the block (a multiple of 32).  One block reports
// faults.  s_warp: a word per warp in shared memory.
DF_DEVICE void plan_entries(const AttendParams& p, const Cutting& cut, Entry* e, long long* end,
                            long long* s_warp, int threads, bool report) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long before = 0;
  for (int s0 = 0; s0 < p.rows.n_seq; s0 += threads) {
    const int s = s0 + threadIdx.x;
    long long units = 0;
    if (s < p.rows.n_seq) {
      Entry x;
      unsigned bad;
      units = plan_entry(p, cut, s, x, bad);
      if (bad && report) set_status(p.c.status, bad);
      e[s] = x;
    }
    long long v = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    long long base = before, all = 0;
    for (int w = 0; w < threads / 32; ++w) {
      if (w < warp) base += s_warp[w];
      all += s_warp[w];
    }
    if (s < p.rows.n_seq) end[s] = base + v;
    before += all;
    __syncthreads();
  }
}

// Vector of a lane's dims.
template <int N>
struct DimVec;
template <>
struct DimVec<1> { using T = float; };
template <>
struct DimVec<2> { using T = float2; };
template <>
struct DimVec<4> { using T = float4; };

// A run of chunks of one tile.
struct Segment {
  int s, kvh, row0;       // entry, kv head, first row of the tile
  int c0, c1, nch;        // chunks [c0, c1) of the tile's nch
  int w;                  // units of a chunk
  long long u0;           // the first unit of the tile's first chunk
};

// The segments of units [u, u1): call repeatedly; s carries the entry.
DF_DEVICE bool next_segment(const AttendParams& p, const Cutting& cut, const Entry* e,
                            const long long* end, long long& u, long long u1, int& s, Segment& g) {
  while (u < u1) {
    while (end[s] <= u) ++s;
    const Blocks b(p, cut, e[s]);
    const long long first = s ? end[s - 1] : 0, per = b.before(b.count), local = u - first;
    g.s = s;
    g.kvh = (int)quotient(local, per);
    const long long in = local - g.kvh * per;
    int i = 0;
    if (b.count > 1) {
      int hi = b.count - 1;   // the last block that begins at or before `in`
      while (i < hi) {
        const int mid = (i + hi + 1) >> 1;
        if (b.before(mid) <= in) i = mid; else hi = mid - 1;
      }
    }
    const long long start = b.before(i);
    g.row0 = i * cut.tile;
    g.nch = b.chunks(i);
    const int w = b.units(i);
    const long long from = in - start, to = min((long long)g.nch * w + cut.extra, from + (u1 - u));
    // a chunk belongs to the range that holds its first unit
    g.c0 = cut.chunks(max(from - cut.extra, 0LL), w);
    g.c1 = cut.chunks(max(to - cut.extra, 0LL), w);
    g.u0 = first + g.kvh * per + start + cut.extra;
    g.w = w;
    u += to - from;
    if (g.c1 > g.c0) return true;   // else the range holds no chunk of the tile
  }
  return false;
}

// First entry whose units end behind u.
DF_DEVICE int find_entry(const long long* end, int n, long long u) {
  int a = 0, b = n - 1;
  while (a < b) {
    const int m = (a + b) >> 1;
    if (end[m] > u) b = m; else a = m + 1;
  }
  return a;
}

// Blocks of a launch that take part: every range holds a chunk of each tile it
// lies in when it is as long as the dearest chunk.
DF_DEVICE int blocks_used(long long U, int launched, int least) {
  return (int)min((long long)launched, max(1LL, quotient(U, least)));
}

// Range of block b of G over U units, and the block that holds unit u.
DF_DEVICE long long range_begin(long long U, int G, int b) { return quotient(U * b, G); }
DF_DEVICE int block_of(long long U, int G, long long u) { return (int)quotient((u + 1) * G - 1, U); }

// ------------------------------------------------------------------ join

// Rows of tiles cut by ranges: grid (blocks of the attention launch, up to 16
// groups of four rows: 32 trees of 17..64 nodes took 91.6 us in all (88 now), 93.8 with
// 8 groups, 91.1 with 32, 93.0 with 64), a warp per row.  Part i of a tile that begins in block b0 is slot
// 2 i of the partial rows (b0 itself: the slot its description names).  Weights
// e^(m_i - max) are applied and summed in block order.
template <int EL, int HD>
__global__ void __launch_bounds__(128) attend_join_kernel(AttendParams p, const Cut* cuts, const float* part_o,
                                                          const float2* part_ml, int tile) {
  constexpr int VL = HD / 32;
  using V = typename DimVec<VL>::T;
  pdl_trigger();
  pdl_wait();
  const int b0 = blockIdx.x, lane = threadIdx.x & 31;
  const Cut d = cuts[b0];
  if (d.last < b0) return;
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < d.rows; r += 4 * gridDim.y) {
    float m = -CUDART_INF_F, sum = 0.f;
    alignas(16) float acc[VL] = {};
    for (int i0 = b0; i0 <= d.last; i0 += 32) {
      const int n = min(32, d.last - i0 + 1), i = i0 + lane;
      const int at = ((i == b0 ? d.slot : 2 * i) * tile + r);
      const float2 ml = lane < n ? part_ml[at] : make_float2(-CUDART_INF_F, 0.f);
      const float top = fmaxf(m, warp_max(ml.x)), use = top == -CUDART_INF_F ? 0.f : top;
      const float w = ex2(ml.x - use), fade = ex2(m - use);
      m = top;
      sum = sum * fade + warp_sum(w * ml.y);
#pragma unroll
      for (int v = 0; v < VL; ++v) acc[v] *= fade;
      for (int k = 0; k < n; k += 8) {
        V x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int a = __shfl_sync(0xffffffffu, at, min(k + q, n - 1));
          x[q] = *reinterpret_cast<const V*>(part_o + (size_t)a * HD + lane * VL);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float wk = k + q < n ? __shfl_sync(0xffffffffu, w, min(k + q, n - 1)) : 0.f;
#pragma unroll
          for (int v = 0; v < VL; ++v)
            if (k + q < n) acc[v] += wk * reinterpret_cast<const float*>(&x[q])[v];
        }
      }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int grp = p.grp, node = (d.row0 + r) / grp;
    const int h = d.kvh * grp + (d.row0 + r) - node * grp;
    char* dst = p.out + (size_t)(d.lo + node) * p.out_ld + (size_t)(h * HD + lane * VL) * EL;
#pragma unroll
    for (int v = 0; v < VL; ++v) acc[v] *= inv;
    if constexpr (EL == 4) {
      *reinterpret_cast<V*>(dst) = *reinterpret_cast<const V*>(acc);
    } else if constexpr (VL == 1) {
      *reinterpret_cast<uint16_t*>(dst) = f32_to_bf16_bits(acc[0]);
    } else {
#pragma unroll
      for (int v = 0; v < VL; v += 2) reinterpret_cast<uint32_t*>(dst)[v / 2] = pack_bf16x2(acc[v], acc[v + 1]);
    }
    if (p.lse && lane == 0)
      p.lse[(size_t)(d.lo + node) * p.c.n_head + h] = sum > 0.f ? (m + log2f(sum)) * kLn2 : -CUDART_INF_F;
  }
}

template <int EL, int HD>
cudaError_t launch_join(const AttendParams& p, const AttendWork& w, int tile, int blocks, cudaStream_t st) {
  const long long rows = (long long)p.max_tree * p.grp;
  const int most = rows < tile ? (int)rows : tile;
  return launch_dependent(attend_join_kernel<EL, HD>, dim3(blocks, most < 64 ? (most + 3) / 4 : 16), 128, 0, st, p,
                          (const Cut*)w.cuts, (const float*)w.part_o, (const float2*)w.part_ml, tile);
}

}  // namespace tree
}  // namespace dflash
