"""The 16-byte pieces in which the layer norm's gradient copies rows that are not whole
vectors: none is read past the array.  The rule of ``csrc/layernorm.cuh`` is compiled
for the host; no kernel runs."""
import os
import subprocess

import pytest

from linear_attention_lm_b200 import build as lab_build

PROGRAM = r"""
#include <cstdio>
#include "layernorm.cuh"
using namespace based;
int main() {
  long long past = 0, other = 0, looked = 0;
  // the pieces of a row: from the 16-byte boundary before it on, up to its end
  auto look = [&](long long row, int n, long long rows) {
    const long long begin = row * n, end = begin + n;
    const bool whole = n < 15 ? pieces_inside<true>(row, n, rows) : pieces_inside<false>(row, n, rows);
    if (n >= 15) other += whole != pieces_inside<true>(row, n, rows);
    for (long long at = begin - begin % 16; at < end; at += 16, ++looked) {
      const long long to = whole || at + 16 < end ? at + 16 : end;
      past += to > rows * n;
    }
    other += !whole && row + 16 < rows;  // far from the end they are copied whole
  };
  for (int size = 2; size <= 4; size += 2)
    for (int D = 1; D <= 70; ++D)
      for (long long rows = 1; rows <= 40; ++rows)
        for (long long row = 0; row < rows; ++row) look(row, D * size, rows);
  const long long many = (1LL << 33) + 1;  // an array of more than 2^32 bytes
  for (long long row = many - 20; row < many; ++row) look(row, 6, many);
  std::printf("%lld %lld %lld\n", past, other, looked);
}
"""


def test_pieces_stay_in_the_array(tmp_path):
    src, exe = tmp_path / "pieces.cu", tmp_path / "pieces"
    src.write_text(PROGRAM)
    try:
        nvcc = lab_build.nvcc_path()
    except RuntimeError:
        pytest.skip("no nvcc")
    res = subprocess.run([nvcc, *lab_build.ARCH_FLAGS, "-std=c++17", "-I", lab_build.CSRC, "-I",
                          lab_build.INCLUDE, "-o", str(exe), str(src)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    env = {k: v for k, v in os.environ.items() if not k.startswith("CUDA")}
    out = subprocess.run([str(exe)], capture_output=True, text=True, env=env)
    past, other, looked = map(int, out.stdout.split())
    assert looked > 100000
    assert (past, other) == (0, 0)
