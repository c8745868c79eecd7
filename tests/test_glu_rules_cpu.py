"""The gated linear unit's choice between its kernels, held to times measured of each, with weights in the last-level cache
and from memory: the chosen way is at most a quarter slower than the fastest with the former, at most 0.35 with the latter. The header with the rules has no HIP in it, so a host program asks it, for 256 compute units."""
import shutil
import subprocess

import pytest

from linear_rnn_amd import build

FEW, INSTRUCTIONS, TILES = range(3)

# us of a call in a graph: rows, channels, hidden channels, {way: us}
BF16 = [(1, 512, 256, 4.6, 10.2), (32, 1024, 4096, 9.6, 13.7), (1, 2048, 5504, 11.3, 18.6), (32, 2048, 256, 14.8, 14.5),
        (32, 2048, 16384, 24.2, 34.4), (1, 4096, 256, 17.5, 17.3), (1, 4096, 2048, 18.7, 19.0), (32, 4096, 512, 25.2, 20.2),
        (32, 4096, 2048, 26.2, 22.7), (32, 4096, 4096, 26.7, 28.8), (1, 4096, 10944, 27.5, 33.8), (1, 8192, 256, 32.3, 25.9),
        (32, 8192, 512, 46.0, 28.0), (32, 8192, 2048, 47.1, 36.6), (32, 8192, 4096, 48.3, 37.6), (1, 8192, 5504, 35.8, 37.8),
        (1, 8192, 8192, 43.9, 55.2), (32, 8192, 8192, 55.1, 61.6), (32, 8192, 10944, 90.3, 72.9), (1, 16384, 256, 61.9, 28.9),
        (16, 16384, 1024, 74.9, 34.9), (32, 16384, 256, 87.7, 32.5), (32, 16384, 512, 88.6, 32.3), (32, 16384, 4096, 100.4, 60.7)]
# the same with other weights from call to call, so that they come from memory
BF16_MEMORY = [(1, 2048, 5504, 17.1, 20.9), (32, 2048, 8192, 24.7, 33.0), (1, 4096, 512, 32.9, 18.8), (8, 4096, 2048, 36.0, 24.4),
               (16, 4096, 2048, 38.3, 23.1), (32, 4096, 2048, 42.5, 24.1), (32, 4096, 4096, 43.5, 32.4), (1, 8192, 1024, 64.6, 31.2),
               (16, 8192, 5504, 64.2, 44.4), (32, 8192, 5504, 72.7, 46.8), (32, 16384, 512, 155.6, 34.0), (32, 16384, 4096, 159.5, 68.8)]
# by the columns that a workgroup of few rows has, 32 and 64; by the float32 instructions; by pieces
F32 = [(1, 512, 256, 5.1, 7.0, 9.1, 17.8), (32, 512, 10944, 17.6, 15.1, 13.7, 49.3), (1, 2048, 5504, 17.8, 20.2, 32.1, 84.6),
       (32, 2048, 5504, 25.2, 38.0, 32.7, 87.6), (1, 2048, 8192, 21.7, 23.8, 32.2, 126.9), (32, 2048, 8192, 25.8, 38.0, 33.4, 129.4),
       (1, 2048, 10944, 32.1, 28.5, 34.2, 152.4), (32, 4096, 256, 38.0, 65.5, 53.0, 47.7), (32, 4096, 10944, 101.3, 82.3, 104.8, 347.2),
       (32, 8192, 256, 71.2, 134.7, 115.3, 55.0), (32, 8192, 512, 82.5, 135.4, 113.8, 58.8), (32, 8192, 1024, 82.6, 134.9, 113.2, 81.8),
       (1, 16384, 256, 75.5, 125.7, 225.9, 73.0), (16, 16384, 256, 86.5, 126.1, 226.5, 74.0), (32, 16384, 256, 161.0, 266.3, 227.3, 75.9),
       (32, 16384, 512, 160.9, 266.7, 225.2, 89.6), (32, 16384, 2048, 165.8, 268.3, 248.7, 257.6),
       (64, 512, 2048, 8.9, 13.0, 9.6, 29.9), (128, 1024, 2048, 13.6, 20.3, 16.1, 38.2), (256, 2048, 4096, 88.6, 73.8, 71.7, 90.8),
       (96, 2048, 8192, 72.0, 74.1, 56.1, 127.6)]

PROGRAM = r"""
#include <cstdio>
#include "glu_rules.hpp"
int main() {
  long M, D, F;
  int f32;
  while (std::scanf("%d %ld %ld %ld", &f32, &M, &D, &F) == 4) {
    const rwkv7::glu::Sizes z{M, D, F, f32 != 0};
    std::printf("%d %d\n", (int)rwkv7::glu::plan_forward(z, 256).way, rwkv7::glu::few_columns(z, 256));
  }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, str(d / "rules.cpp"), "-o", str(d / "rules")], check=True)

    def ask(sizes):
        text = "".join("%d %d %d %d\n" % s for s in sizes)
        r = subprocess.run([str(d / "rules")], input=text, capture_output=True, text=True, check=True)
        return [tuple(int(n) for n in line.split()) for line in r.stdout.splitlines()]

    return ask


def test_bfloat16(choose):
    for (M, D, F, few, tiles), (way, _) in zip(BF16, choose([(0,) + c[:3] for c in BF16])):
        assert {FEW: few, TILES: tiles}[way] <= 1.25 * min(few, tiles), (M, D, F, way)


def test_bfloat16_weights_from_memory(choose):
    for (M, D, F, few, tiles), (way, _) in zip(BF16_MEMORY, choose([(0,) + c[:3] for c in BF16_MEMORY])):
        assert {FEW: few, TILES: tiles}[way] <= 1.35 * min(few, tiles), (M, D, F, way)


def test_float32(choose):
    for (M, D, F, few32, few64, f32, pieces), (way, cols) in zip(F32, choose([(1,) + c[:3] for c in F32])):
        us = {FEW: few32 if cols == 32 else few64, INSTRUCTIONS: f32, TILES: pieces}
        assert us[way] <= 1.25 * min(few32, few64, f32, pieces), (M, D, F, way, cols)


def test_rows_that_begin_anywhere(choose):
    """A bfloat16 row of an odd width begins on two bytes: not for the kernel of few rows."""
    for M, D, F in ((1, 769, 2048), (32, 768, 2049), (100, 33, 21)):
        assert choose([(0, M, D, F)])[0][0] == TILES and choose([(1, M, D, F)])[0][0] != TILES


def test_few_rows_that_need_no_workspace(choose):
    """Up to 32 rows of up to 1024 channels, as the header says, whatever the hidden channels."""
    sizes = [(f32, M, D, F) for f32 in (0, 1) for M in (1, 16, 17, 32) for D in (2, 66, 512, 1000, 1024)
             for F in (2, 64, 1000, 8192, 8194, 100_000, 1 << 20)]
    assert all(way == FEW for way, _ in choose(sizes))
