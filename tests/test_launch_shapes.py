"""Launch arithmetic (csrc/launch_shapes.h, plain C++) over every size, without a GPU."""
import ctypes as C
import pathlib
import random
import subprocess

import pytest

CSRC = pathlib.Path(__file__).parents[1] / "block_diffusion_drafter_fc_gb300" / "csrc"

SOURCE = """
#include "launch_shapes.h"
using namespace dflash;

// 0: every item of every row belongs to exactly one block and is found by its number; else what does not hold
static int cover(const rope::Shape& s, int T, int items, int rd, bool append) {
  if (s.rows < 1 || s.rows > rope::kMaxRows || s.gx < 1 || s.gy < 1 || s.gy > 65535) return 1;
  if (s.smem < (size_t)8 * s.rows * (rd / 2) || s.smem > 48 * 1024) return 2;
  const rope::Span last = rope::block_span(T, s.rows, items, s.span, s.gx - 1, 0);
  if (last.n_rows < 1 || last.n_rows > s.rows || last.row0 + last.n_rows != T) return 3;
  if (append && s.u > 1 && (s.gy != 1 || s.span != items)) return 8;   // what its kernel goes by
  int at = 0;
  for (int y = 0; y < s.gy; ++y) {
    const rope::Span b = rope::block_span(T, s.rows, items, s.span, 0, y);
    if (b.it0 != at || b.it1 <= b.it0) return 4;
    at = b.it1;
    // (the kernels that take all items of a block at once: u a thread)
    const long long total = (long long)s.rows * (b.it1 - b.it0);
    if (!append && total > s.u * rope::kThreads) return 5;
    if (append) {
      const uint32_t magic = rope::append_magic(s, items);
      const int width = b.it1 - b.it0;
      for (int r = 0; r < s.rows; ++r)
        for (int e = 0; e < 2; ++e) {
          const uint32_t g = (uint32_t)(r * width + (e ? width - 1 : 0));
          const int row = magic ? (int)(((uint64_t)g * magic) >> 32) : (int)g;
          if (row != r) return 6;
        }
    }
  }
  return at == items ? 0 : 7;
}
extern "C" int rope_cover(int T, int items, int rd) { return cover(rope::shape_of(T, items, rd), T, items, rd, false); }
extern "C" int append_cover(int T, int items, int rd) {
  return cover(rope::append_shape(T, items, rd), T, items, rd, true);
}
// 0: positions and parities along a ring equal those of the copy's number
extern "C" int ring_walk(int S, int start, int steps, const int* by) {
  int pos = start % S, parity = start / S & 1;
  long long n = start;
  for (int i = 0; i < steps; ++i) {
    ring_step(pos, parity, by[i], S);
    n += by[i];
    if (pos != n % S || parity != (int)(n / S & 1)) return i + 1;
  }
  return 0;
}
extern "C" int append_rows(int T, int items) { return rope::append_shape(T, items, 128).rows; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("shapes")
    (d / "shapes.cc").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "shapes.cc"), "-o",
                    str(d / "shapes.so")], check=True)
    return C.CDLL(str(d / "shapes.so"))


def test_every_item_of_every_row_has_a_block(lib):
    """Rows from one to a long prompt's, heads from one to thousands, every head_dim and type."""
    rows = [*range(1, 1300), *range(9700, 9800), *range(19400, 19500), 65536, 1 << 20, (1 << 31) - 1]
    heads = {1, 2, 3, 5, 8, 12, 16, 24, 36, 40, 48, 80, 96, 160, 640, 1300, 2897, 5120, 6144, 12288}
    for items in sorted({h * hd * el // (2 * vec) for h in heads for hd in (32, 64, 128)
                         for el, vec in ((4, 16), (2, 16), (2, 8))}):
        for T in rows:
            assert lib.append_cover(T, items, 128) == 0, (T, items)
            assert lib.rope_cover(T, items, 128) == 0, (T, items)


@pytest.mark.parametrize("T,items", [(487, 640), (608, 640), (406, 768), (512, 768), (40, 49152), (1300, 49152)])
def test_large_appends_of_one_row_a_block(lib, T, items):
    """More items than a block takes in one step (512), and a block per row."""
    assert lib.append_rows(T, items) == 1 and lib.append_cover(T, items, 128) == 0


def test_ring_positions(lib):
    """Steps of 1 and 2 copies, as the streams of an attention tile take them (4 as two of 2),
    from rings of 2 stages on."""
    rng = random.Random(0)
    for S in range(2, 13):
        for start in range(3 * S):
            by = [rng.choice((1, 2)) for _ in range(200)]
            for steps in (by, [2] * 200, [1] * 200):
                assert lib.ring_walk(S, start, 200, (C.c_int * 200)(*steps)) == 0, (S, start)
