"""Launch arithmetic of the norms' kernels (csrc/launch_shapes.h, plain C++) over sizes, without a GPU."""
import ctypes as C
import subprocess

import pytest

from test_launch_shapes import CSRC

SOURCE = """
#include "launch_shapes.h"
using namespace dflash;

// 0: the blocks cover every item of every row once, within their limits; else what does not hold
static int cover(const norm::Shape& s, int T, int items, int ipr, long long limit) {
  if (s.threads < 2 * norm::kMaxRows || s.threads > norm::kThreads || s.threads % 32 || s.cols % ipr) return 1;
  if (s.cols * s.side > s.threads || s.side < 1 || s.side > norm::kMaxRows) return 2;
  if (s.rows < 1 || s.rows % s.side || s.gx < 1 || s.gy < 1 || s.gy > 65535) return 3;
  if ((long long)s.cols * s.gy < items || (long long)s.cols * (s.gy - 1) >= items) return 4;
  if ((long long)s.rows * s.gx < T || (long long)s.rows * (s.gx - 1) >= T) return 5;
  return limit && (long long)s.gx * s.gy > limit ? 6 : 0;
}
extern "C" int rows_cover(int T, int items, int ipr) {
  const norm::Shape s = norm::shape_of(T, items, 65536 / 80);
  return s.rows > norm::kMaxRows ? 7 : cover(s, T, items, ipr, 0);
}
extern "C" int grad_cover(int T, int items, int ipr) { return cover(norm::sum_shape_of(T, items, 65536 / 128, 608), T, items, ipr, 608); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("norm_shapes")
    (d / "shapes.cc").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "shapes.cc"), "-o",
                    str(d / "shapes.so")], check=True)
    return C.CDLL(str(d / "shapes.so"))


def test_every_item_of_every_row_has_a_thread(lib):
    """Rows from one to 2^31 - 1, heads from one to thousands, every number of lanes of a head."""
    rows = [*range(1, 700), *range(7290, 7310), 8191, 65536, 1 << 20, (1 << 31) - 1]
    heads = [1, 2, 3, 5, 6, 7, 8, 12, 16, 17, 24, 31, 32, 33, 40, 48, 63, 64, 80, 96, 129, 640, 1300, 2897, 5120, 8192]
    for ipr in (2, 4, 8, 16):
        for h in heads:
            for T in rows:
                assert lib.rows_cover(T, h * ipr, ipr) == 0, (T, h, ipr)
                assert lib.grad_cover(T, h * ipr, ipr) == 0, (T, h, ipr)
