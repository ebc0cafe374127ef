"""The library's per-device numbers on the host: each device has its own, and a
failed query is not kept."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_fp8_expert_gb300", "csrc")

PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
int main() {
  moe::PerDevice known;
  int asked = 0;
  auto ask = [&](int device, int answer) { return known.get(device, [&] { ++asked; return answer; }); };
  const bool ok = ask(0, -1) == 0 && asked == 1 &&       // a failure: 0 this time, asked again
                  ask(0, 38) == 38 && asked == 2 && ask(0, 7) == 38 && asked == 2 &&
                  ask(1, 0) == 0 && asked == 3 && ask(1, 5) == 0 && asked == 3 &&  // 0 is an answer
                  ask(2, 76) == 76 && ask(0, 1) == 38 && asked == 4 &&
                  ask(-1, 9) == 0 && ask(1 << 20, 9) == 0 && asked == 4;
  std::puts(ok ? "ok" : "wrong");
  return ok ? 0 : 1;
}
"""


def test_each_device_answers_once_and_failures_are_not_kept(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "ok\n"
