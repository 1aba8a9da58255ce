// Arithmetic of launches that is the host's alone, or the same on both sides:
// plain C++, so that it can be checked without a GPU over every size.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define DF_BOTH __host__ __device__ __forceinline__
#else
#define DF_BOTH inline
#endif

namespace dflash {

// y / d of y <= 2^32 / d, magic = ceil(2^32 / d) (0: d = 1): the magic is off by less
// than one from 2^32 / d, the product by less than y
inline bool quotient_exact(long long y, long long d) { return y * d <= 1ll << 32; }
inline uint32_t quotient_magic(uint32_t d) {
  return d > 1 ? (uint32_t)((0x100000000ull + d - 1) / d) : 0;
}

// ------------------------------------------------------------------ rings

// `by` places on in a ring of S >= `by`, and the parity of the round that they are in: at
// most one round further.  A call of many entries leaves the attention a ring of 3, so its
// streams take 4 places in two steps.  (A step that allows for two rounds, on the path of
// tiles that go 2 on, cost a 2047-row prompt 2 us of 241.)
DF_BOTH void ring_step(int& pos, int& parity, int by, int S) {
  pos += by;
  if (pos >= S) {
    pos -= S;
    parity ^= 1;
  }
}

// ------------------------------------------------------------------ rope, append

namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxRows = 32;   // rows of one block
constexpr int kAppendRows = 16;

// A launch over T rows of `items` items each: `rows` rows a block, gx blocks of
// them; gy blocks share a row's items, `span` each.
struct Shape {
  int u, rows, gx, gy, span;
  size_t smem;
};

// What a block works on: rows [row0, row0 + n_rows) and items [it0, it1) of each.
struct Span {
  int row0, n_rows, it0, it1;
};
DF_BOTH Span block_span(int T, int rows_per_block, int items, int span, int bx, int by) {
  Span s;
  s.row0 = bx * rows_per_block;
  s.n_rows = rows_per_block < T - s.row0 ? rows_per_block : T - s.row0;
  s.it0 = by * span;
  s.it1 = items - s.it0 < span ? items : s.it0 + span;
  return s;
}

// Rows and items of a block: 4 items a thread once that still gives every SM
// a few blocks, else 1 (a small call is latency: as many blocks as there are).
inline Shape shape_of(int T, int items, int rd) {
  Shape s;
  s.u = (long long)T * items >= 152LL * 2 * 4 * kThreads ? 4 : 1;
  const int step = s.u * kThreads;
  s.rows = items >= step ? 1 : step / items;
  if (s.rows > kMaxRows) s.rows = kMaxRows;
  s.gx = (int)(((long long)T + s.rows - 1) / s.rows);
  s.gy = s.rows > 1 ? 1 : (items + step - 1) / step;
  s.span = s.rows > 1 ? items : step;
  s.smem = sizeof(float) * 2 * s.rows * (rd / 2);
  return s;
}

// The append's: its large calls (u = 4 becomes blocks that step through their items,
// 2 a thread) are one or more full waves of blocks (four per SM by their registers) of
// at most 16 rows each, every block with all items of its rows, also where it has one
// row only.  8192 rows of 48 heads: 39 us in blocks of 14 rows, 41 of 16, 50 of 27, 51
// of 11; 47 us with one pass of 4 items a thread, whose page look-ups nothing covered.
inline Shape append_shape(int T, int items, int rd) {
  Shape s = shape_of(T, items, rd);
  if (s.u == 1) return s;
  const long long wave = 4 * 152, waves = (T + wave * kAppendRows - 1) / (wave * kAppendRows);
  s.u = 2;
  s.rows = (int)((T + wave * waves - 1) / (wave * waves));
  // (thousands of heads: as many rows as the quotient by `items` is exact for)
  while (s.rows > 1 && !quotient_exact((long long)s.rows * items, items)) --s.rows;
  s.gx = (int)(((long long)T + s.rows - 1) / s.rows);
  s.gy = 1;
  s.span = items;
  s.smem = sizeof(float) * 2 * s.rows * (rd / 2);
  return s;
}
// The divisor of a block's item numbers (a block of one row needs none: one beyond them all).
inline uint32_t append_magic(const Shape& s, int items) { return quotient_magic(s.rows > 1 ? items : 1 << 30); }

}  // namespace rope

// ------------------------------------------------------------------ norms of heads

namespace norm {

constexpr int kThreads = 256;   // most threads of a block
constexpr int kMaxRows = 32;    // rows whose angles a block holds at once

// A block's threads own items of a row (its columns), `side` rows side by side where rows are
// short, and walk down rows: gx blocks of `rows` rows, gy of columns.  A head has two items or
// more, so a block has 64 threads or more: one for each row whose angles it holds.
struct Shape {
  int cols, side, threads, rows, gx, gy;
};
inline Shape columns_of(int items) {
  Shape s = {};
  s.gy = (items + kThreads - 1) / kThreads;
  s.cols = s.gy == 1 ? items : ((items + s.gy - 1) / s.gy + 31) / 32 * 32;
  s.side = s.cols < 256 ? 256 / s.cols : 1;
  if (s.side > kMaxRows) s.side = kMaxRows;
  s.threads = (s.cols * s.side + 31) / 32 * 32;
  return s;
}
constexpr int kSms = 152;
// Blocks that the GPU holds at once, `threads` threads an SM.
inline int wave_of(const Shape& s, int threads) { return kSms * (threads / s.threads > 1 ? threads / s.threads : 1); }
// Whole rounds of blocks of up to kRound rows (the append of 8192 rows of 48 heads: 39.4 us in
// blocks of 9 rows, 40.5 of 14, 40.7 of 27: the next round's look-ups run under a round's copies).
constexpr int kRound = 12;
inline Shape shape_of(int T, int items, int threads) {
  Shape s = columns_of(items);
  const int wave = wave_of(s, threads);
  const int most = kRound > s.side ? kRound / s.side * s.side : s.side;
  const long long per = (long long)T * s.gy, round = (long long)wave * most;
  const long long waves = (per + round - 1) / round;
  long long rows = (per + wave * waves - 1) / (wave * waves);
  rows = (rows + s.side - 1) / s.side * s.side;
  s.rows = (int)(rows < most ? rows : most);
  s.gx = (int)(((long long)T + s.rows - 1) / s.rows);
  return s;
}
// One round of blocks of any number of rows, at most `limit`.
inline Shape sum_shape_of(int T, int items, int threads, int limit) {
  Shape s = columns_of(items);
  const int most = wave_of(s, threads) < limit ? wave_of(s, threads) : limit;
  const long long least = ((long long)T + s.side - 1) / s.side, gx = most / s.gy > 1 ? most / s.gy : 1;
  s.gx = (int)(gx < least ? gx : least);
  const long long rows = ((long long)T + s.gx - 1) / s.gx;
  s.rows = (int)((rows + s.side - 1) / s.side * s.side);
  s.gx = (int)(((long long)T + s.rows - 1) / s.rows);
  return s;
}

}  // namespace norm
}  // namespace dflash
