"""Launches of more workgroups than a grid may have: in chunks that depend on the workgroup's size, as a grid's threads
are counted in 32 bits. The header has no HIP in it, so a host program checks it."""
import os
import shutil
import subprocess

import pytest

from linear_rnn_amd import build

PROGRAM = r"""
#include <initializer_list>
#include "launch_chunks.hpp"
int main() {
  const uint64_t sizes[] = {0, 1, (1u << 20) - 1, 1u << 20, (1u << 20) + 1, 1u << 21, 1u << 22, (1u << 22) + 5, 1u << 27, (1ull << 29) + 3};
  for (int threads : {64, 256, 512, 1024})
    for (uint64_t blocks : sizes) {
      uint64_t next = 0;
      bool fits = true, whole = true;
      const int e = rwkv7::in_chunks(blocks, threads, [&](uint32_t first, uint32_t n) {
        fits = fits && n > 0 && (uint64_t)n * threads < (1ull << 32);
        whole = whole && first == next;
        next += n;
        return 0;
      });
      if (e != 0 || !fits || !whole || next != blocks) return 1;
    }
  int calls = 0;  // the first refusal ends it
  const int e = rwkv7::in_chunks(1u << 24, 1024, [&](uint32_t, uint32_t) { return ++calls == 3 ? 7 : 0; });
  return e == 7 && calls == 3 ? 0 : 2;
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="no host compiler")
def test_chunks_fit_a_grid_whatever_the_workgroup(tmp_path):
    src, exe = tmp_path / "chunks.cpp", tmp_path / "chunks"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_the_gated_recurrence_launches_so():
    """All its kernels, of 256, 512 and 1024 threads, are launched by the one function that cuts into such chunks."""
    text = open(os.path.join(build.CSRC, "gscan.hip")).read()
    assert text.count("hipLaunchKernel(") == 1 and "in_chunks(blocks, threads," in text


def test_the_gated_unit_prepares_its_operands_so():
    """The one launch of the gated linear unit that may have more threads: weights of 2^34 elements, the most that is
    taken, are 2^31 threads of 8 each, and there are two; its tiles, of at least 64 x 128 for 256 threads, fit."""
    assert 2 * (1 << 34) // 8 >= 1 << 32
    # tiles: 2^28 rows of one column of tiles, or 2^34 elements in both directions
    assert (1 << 28) // 64 * 256 < 1 << 32 and (1 << 34) // (64 * 128) * 256 < 1 << 32
    text = open(os.path.join(build.CSRC, "glu.hip")).read()
    stage = text[text.index("struct Stage {"):]
    assert "in_chunks(blocks, 256," in stage[:stage.index("\n};")]
