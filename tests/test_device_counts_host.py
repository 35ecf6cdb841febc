"""Counts kept per device (csrc/device_counts.h): one device's answer is not another's, a failed query is asked again,
and a device that does not do what was asked is remembered.  Compiled for the host."""
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).parent.parent / "moe_expert_ffn_rms_gb300" / "csrc"

PROGRAM = r"""
#include <stdio.h>
#include <thread>
#include <vector>
#include "device_counts.h"
int main() {
  static moe::DeviceCounts<4> c;
  int asked = 0;
  auto answer = [&](int n) { return [&asked, n] { ++asked; return n; }; };
  auto check = [&](bool ok, const char* what) { if (!ok) { printf("%s\n", what); return 1; } return 0; };
  int bad = 0;
  bad |= check(c.get(0, 1, answer(7)) == 7 && c.get(0, 1, answer(9)) == 7 && asked == 1, "kept");
  bad |= check(c.get(1, 1, answer(5)) == 5 && c.get(0, 1, answer(9)) == 7, "each device has its own");
  bad |= check(c.get(0, 2, answer(3)) == 3 && c.get(0, 1, answer(9)) == 7, "each key has its own");
  asked = 0;
  bad |= check(c.get(0, 3, answer(-1)) == 0 && c.get(0, 3, answer(4)) == 4 && c.get(0, 3, answer(8)) == 4 && asked == 2,
               "a failed query is asked again");
  asked = 0;
  bad |= check(c.get(1, 3, answer(0)) == 0 && c.get(1, 3, answer(4)) == 0 && asked == 1, "none is an answer");
  bad |= check(c.get(-1, 0, answer(4)) == 0 && c.get(moe::kCountDevices, 0, answer(4)) == 0 && c.get(0, 4, answer(4)) == 0,
               "outside the table");
  std::vector<std::thread> threads;
  std::atomic<int> wrong{0};
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&wrong] {
      for (int d = 2; d < moe::kCountDevices; ++d)
        for (int k = 0; k < 4; ++k) wrong += c.get(d, k, [=] { return d * 4 + k; }) != d * 4 + k;
    });
  for (auto& t : threads) t.join();
  bad |= check(wrong == 0, "several threads");
  return bad;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_counts_are_kept_per_device(tmp_path):
    src, exe = tmp_path / "counts.cpp", tmp_path / "counts"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", str(CSRC), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_the_split_product_asks_per_device():
    src = (CSRC / "linear.cu").read_text()
    assert "f.clusters(device, s)" in src and "static DeviceCounts<kMaxSplit + 1> known;" in src
    assert "std::atomic" not in src  # no count of its own for the whole process
