"""What the library keeps for a stream is kept by a key in which hipStreamPerThread, one handle that names another
stream in every thread, differs from thread to thread, and every other handle does not. The header with the key has
no HIP in it, so a host program checks it."""
import os
import shutil
import subprocess

import pytest

from linear_rnn_amd import build

PROGRAM = r"""
#include <cstdio>
#include <set>
#include <thread>
#include <vector>
#include "stream_key.hpp"

int main() {
  const void* const per_thread = reinterpret_cast<const void*>(2);
  const void* const other = reinterpret_cast<const void*>(64);
  constexpr int kThreads = 8;
  std::vector<rwkv7::StreamKey> mine(kThreads), again(kThreads), shared(kThreads), null(kThreads);
  // one after the other, so that the system may give a thread the number of an ended one
  for (int i = 0; i < kThreads; ++i) {
    std::thread([&, i] {
      mine[i] = rwkv7::stream_key(0, per_thread, per_thread);
      again[i] = rwkv7::stream_key(0, per_thread, per_thread);
      shared[i] = rwkv7::stream_key(0, other, per_thread);
      null[i] = rwkv7::stream_key(0, nullptr, per_thread);
    }).join();
  }
  std::set<rwkv7::StreamKey> all(mine.begin(), mine.end());
  if (all.size() != kThreads) return 1;
  for (int i = 0; i < kThreads; ++i)
    if (mine[i] != again[i] || shared[i] != shared[0] || null[i] != null[0]) return 2;
  if (shared[0] == null[0] || rwkv7::stream_key(1, other, per_thread) == shared[0]) return 3;
  std::puts("ok");
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="no host compiler")
def test_keys_of_threads_and_streams(tmp_path):
    src, exe = tmp_path / "key.cpp", tmp_path / "key"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.returncode


def test_the_sources_keep_by_that_key():
    """No map of the library goes by the bare handle."""
    for src in build.sources():
        text = open(src).read()
        assert "std::map<std::pair<int, uintptr_t>" not in text and "std::map<std::tuple<int, uintptr_t" not in text, src
    kept = [os.path.basename(s) for s in build.sources() if "stream_key(dev, stream, hipStreamPerThread)" in open(s).read()]
    assert kept == ["wkv7_split.hip", "wkv7_stack.hip"]
