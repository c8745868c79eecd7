"""What a kernel asks of the runtime once on every device: on each device by itself, and again after a refusal. The
header has no HIP in it, so a host program checks it."""
import os
import shutil
import subprocess

import pytest

from linear_rnn_amd import build

PROGRAM = r"""
#include "once_per_device.hpp"
int main() {
  std::atomic<uint64_t> granted{0};
  int asked = 0, answer = 0;
  auto ask = [&] { ++asked; return answer; };
  answer = 7;  // refused: said so, and asked again
  if (rwkv7::once_per_device(granted, 0, ask) != 7 || asked != 1) return 1;
  answer = 0;
  if (rwkv7::once_per_device(granted, 0, ask) != 0 || asked != 2) return 2;
  answer = 7;  // granted: not asked again on this device, but on another
  if (rwkv7::once_per_device(granted, 0, ask) != 0 || asked != 2) return 3;
  if (rwkv7::once_per_device(granted, 1, ask) != 7 || asked != 3) return 4;
  answer = 0;
  if (rwkv7::once_per_device(granted, 63, ask) != 0 || rwkv7::once_per_device(granted, 63, ask) != 0 || asked != 4) return 5;
  for (int i = 0; i < 2; ++i)
    if (rwkv7::once_per_device(granted, 64, ask) != 0 || asked != 5 + i) return 6;
  return rwkv7::once_per_device(granted, -1, ask) != 0 || asked != 7 ? 7 : 0;
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="no host compiler")
def test_asked_on_every_device(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_linear_attention_asks_so():
    """No answer of one device, and no refusal, is kept for all calls."""
    for name in ("linattn_fwd.hip", "linattn_bwd.hip", "linattn_state.hip"):
        text = open(os.path.join(build.CSRC, name)).read()
        assert "static const hipError_t" not in text, name
