"""The streaming norm kernels' CTAs all fit on an SM together with their stages (csrc/norm_stages.h), for every width and
type: one that does not runs a round of its own.  Compiled for the host."""
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).parent.parent / "moe_expert_ffn_rms_gb300" / "csrc"

PROGRAM = r"""
#include <stdio.h>
#include "norm_stages.h"
int main() {
  int bad = 0;
  auto check = [&](const char* what, int H, int ctas, int threads, long long bytes) {
    const int S = moe::norm_stages(ctas, bytes);
    // 228 KB of shared memory per SM, 227 for one CTA, 1 KB of each CTA's for the runtime; 2048 threads
    const long long cta = S * bytes + 512 + 1024;
    if (S < 2 || ctas < 1 || ctas * cta > 228 * 1024 || S * bytes > moe::kNormSmem || ctas * threads > 2048) {
      printf("%s H=%d: %d CTAs of %d stages of %lld bytes\n", what, H, ctas, S, bytes);
      bad = 1;
    }
  };
  for (int H = 8; H <= 16384; H += 8) {
    const int nv = H / 8;
    for (int x = 2; x <= 4; x += 2) {
      check("forward", H, moe::row_ctas(nv), moe::row_threads((nv + 1) / 2), (long long)H * x);
      for (int dy = 2; dy <= 4 && nv <= moe::kGradVpt * moe::kGradNw * 32; dy += 2)
        for (int res = 0; res < 2; ++res)
          check("backward", H, moe::grad_ctas(nv), moe::row_threads((nv + 1) / 2), (long long)H * (x * (1 + res) + dy));
    }
  }
  return bad;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_all_ctas_are_resident(tmp_path):
    src, exe = tmp_path / "stages.cpp", tmp_path / "stages"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", str(CSRC), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
