// Shared parts of the streaming attention kernels (bf16 heads of 32, f32): four
// warps that compute and a ring of K and V chunks that one warp refills.
#pragma once

#include "tree_common.cuh"

namespace dflash {
namespace tree {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * kConsumers;
constexpr int kMinUnits = 3;   // a block's least share of a call's units

template <int EL, int HD>
struct Geo {
  static constexpr int CS = EL == 2 ? 64 : 32;            // slots of a chunk
  static constexpr int WS = CS / kConsumers;              // slots of a warp
  static constexpr int kRowB = HD * EL;                   // bytes of a row
  static constexpr int kBoxB = kRowB < 128 ? kRowB : 128; // bytes of a row within a box
  static constexpr int kBoxes = kRowB / kBoxB;
  static constexpr int kHalf = CS * kRowB;                // bytes of a K or V chunk
};

// Offset of 16-byte piece `c` of row r in a block of `rows` rows as the copies
// lay it out: boxes of 128-byte (64-byte) rows, swizzled.
template <int RowB>
DF_DEVICE int swz(int rows, int r, int c) {
  if constexpr (RowB >= 128)
    return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  else
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// every chunk one unit, a tile two besides
template <int EL>
DF_DEVICE Cutting cutting(int tile) {
  return {tile, Geo<EL, 64>::CS, 0, 1, 1, 2};
}

struct StreamParams {
  CUtensorMap tm;     // pages as [rows of (page, layer, k|v, head)][page_size][hd]
  AttendParams a;
  float* part_o;      // [2 blocks][rows of a tile][hd]
  float2* part_ml;    // [2 blocks][rows of a tile] (maximum in powers of two, sum)
  Cut* cuts;          // [blocks]
  int stages, box_rows;
};

// The copies of a block's chunks, run ahead of their use by one warp: K, then V
// of every chunk of every segment.
template <int EL, int HD, typename E>
struct Copies {
  using G = Geo<EL, HD>;
  long long u;
  int s, it = 0, ch = 0, kv = 0;
  int base = 0, row = 0;    // lane i holds the tensor row of page base + i
  int off = 0;              // the entry's first slot
  bool more = false;
  Segment g;

  DF_DEVICE void open(const StreamParams& p, const E* e, const long long* end, long long u1, int tile) {
    more = next_segment(p.a, cutting<EL>(tile), e, end, u, u1, s, g);
    if (more) off = e[g.s].base();
    ch = g.c0;
    base = -64;
  }
  DF_DEVICE void issue(const StreamParams& p, uint8_t* sm, uint64_t* full, uint64_t* empty, const E* e,
                       const long long* end, long long u1, int tile, volatile int* abort) {
    if (!more) return;
    const CacheView& c = p.a.c;
    const int lane = threadIdx.x & 31, S = p.stages, st = it % S;
    const int none = c.n_pages * c.n_layer * 2 * c.n_head_kv;   // past the tensor: reads as zero
    if (kv == 0 && ((off + ch * G::CS + G::CS - 1) >> c.ps_log2) > base + 31) {
      const E x = e[g.s];
      base = (off + ch * G::CS) >> c.ps_log2;
      row = none;
      if (base + lane <= (x.len + x.nodes() - 1) >> c.ps_log2) {
        const int t = c.table[(size_t)x.q * c.max_pages + base + lane];
        if (t >= 0 && t < c.n_pages)
          row = (t * c.n_layer + p.a.layer) * 2 * c.n_head_kv + g.kvh;
        else
          set_status(c.status, DEV_BAD_PAGE);
      }
    }
    int stop = 0;
    if (lane == 0) {
      bar_wait(&empty[st], (uint32_t)((it / S) & 1) ^ 1, abort, c.status);
      stop = *abort;
      if (!stop) bar_expect(&full[st], G::kHalf);
    }
    if (__shfl_sync(0xffffffffu, stop, 0)) {
      more = false;
      return;
    }
    uint8_t* dst = sm + st * G::kHalf;
    for (int i = 0; i < G::CS; i += p.box_rows) {
      const int slot = off + ch * G::CS + i;
      const int r = __shfl_sync(0xffffffffu, row, ((slot >> c.ps_log2) - base) & 31);
      if (lane == 0)
#pragma unroll
        for (int x4 = 0; x4 < G::kBoxes; ++x4)
          tma3d(dst + x4 * G::CS * G::kBoxB + i * G::kBoxB, &p.tm, x4 * (G::kBoxB / EL), slot & (c.ps - 1),
                r == none ? none : r + kv * c.n_head_kv, &full[st]);
    }
    ++it;
    if (kv ^= 1) return;
    if (++ch == g.c1) open(p, e, end, u1, tile);
  }
  // no copy may still be landing when the block ends
  DF_DEVICE void drain(int S, uint64_t* full) {
    if ((threadIdx.x & 31) == 0)
      for (int j = max(0, it - S); j < it; ++j) {
        const long long t0 = clock64();
        while (!bar_try(&full[j % S], (uint32_t)((j / S) & 1)) && clock64() - t0 < kWait) {
        }
      }
  }
};

// Dynamic shared memory of a block, two blocks per SM: of its 228 KB each block takes 1 KB
// more than it asks for, and up to 128 bytes of static memory.  (512 bytes more fit one
// block only: a call of 215..236 entries with f32 heads of 128 took half as long again.)
constexpr size_t kSmemTwo = 113 * 1024 - 128;
constexpr int kStagesMost = 12;

// Parameters of a streaming launch whose blocks have tiles of `tile`
// rows and need `fixed` bytes of shared memory besides the ring.
template <int EL, int HD>
StreamParams stream_params(const AttendParams& a, const AttendWork& w, int tile, size_t fixed, size_t& smem) {
  using G = Geo<EL, HD>;
  StreamParams p;
  p.tm = *w.tm;
  p.a = a;
  p.a.step = trim_step(a, tile, G::CS);
  p.part_o = w.part_o;
  p.part_ml = w.part_ml;
  p.cuts = w.cuts;
  p.box_rows = a.c.ps < G::CS ? a.c.ps : G::CS;
  p.stages = (int)((kSmemTwo - fixed) / (G::kHalf + 16));
  if (p.stages > kStagesMost) p.stages = kStagesMost;
  smem = fixed + (size_t)p.stages * (G::kHalf + 16);
  return p;
}

}  // namespace tree
}  // namespace dflash
