"""Host check of the order of an expert's tiles in bands (bands.hpp ``band_tile``),
which the 8-bit products take: a small C++ driver runs the library's own header.

For 1 to 300 row tiles and several numbers of column tiles the order covers each
tile once; the bands' heights (runs of row tiles that a column is walked along) differ by at
most one, the higher ones first; and they are 6 to 11 where there are 6 row tiles or more.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_optimizer_step_owner_amd", "csrc")
GXX = shutil.which("g++")

DRIVER = r"""
#include <cstdio>
#include <vector>
#include "bands.hpp"

int fail(const char* what, int rows, int nq) {
  std::printf("%s: %d x %d\n", what, rows, nq);
  return 1;
}

int main() {
  for (int nq : {1, 2, 7, 56})
    for (int rows = 1; rows <= 300; ++rows) {
      std::vector<int> seen(rows * nq, 0), heights;
      int first = 0, at = 0;      // first row tile of the band, tiles before it
      for (int local = 0; local < rows * nq;) {
        // a band: its first column is as long as row tiles follow one another
        int h = 0;
        while (local + h < rows * nq) {
          const mfsdp::BandTile t = mfsdp::band_tile(rows, nq, 8, local + h);
          if (t.tj != 0 || t.ti != first + h) break;
          ++h;
        }
        // with one column tile the bands follow one another without a break
        if (nq == 1) { h = rows; }
        if (h == 0) return fail("a band does not start with its first tile", rows, nq);
        for (int j = 0; j < nq; ++j)
          for (int i = 0; i < h; ++i, ++local) {
            const mfsdp::BandTile t = mfsdp::band_tile(rows, nq, 8, local);
            if (t.ti != first + i || t.tj != j) return fail("order", rows, nq);
            ++seen[t.ti * nq + t.tj];
          }
        heights.push_back(h);
        first += h;
        at = local;
      }
      if (at != rows * nq || first != rows) return fail("rows", rows, nq);
      for (int v : seen)
        if (v != 1) return fail("not every tile once", rows, nq);
      if (nq == 1) continue;
      for (size_t b = 0; b < heights.size(); ++b) {
        if (b && heights[b] > heights[b - 1]) return fail("higher bands are not first", rows, nq);
        if (heights[0] - heights[b] > 1) return fail("heights differ by more than one", rows, nq);
        if (heights[b] > 11 || (rows >= 6 && heights[b] < 6)) return fail("height", rows, nq);
      }
    }
  std::printf("ok\n");
  return 0;
}
"""


@pytest.mark.skipif(GXX is None, reason="g++ not available")
def test_bands(tmp_path):
    src = tmp_path / "drv.cpp"
    src.write_text(DRIVER)
    exe = tmp_path / "drv"
    res = subprocess.run([GXX, "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr
