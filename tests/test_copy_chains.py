"""How long the chains are in which the copy of pages (csrc/gdn_kv_copy.cu) looks for conflicts, without a GPU: whatever
order the destinations have, a lookup meets about two links."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <vector>

#include "gdn_kv_copy.cu"

namespace gdn {
int sm_count() { return 152; }
}  // namespace gdn

int main() {
  const int n = 131072, step = 8 * 152;  // pairs, and blocks of the launch: a block has every step-th pair
  unsigned state = 1;
  for (int apart : {1, 2, 3, 16, 64, 256, 257, 1000, 4096, 0}) {
    std::vector<int> dst(n);
    for (int i = 0; i < n; i++) dst[i] = apart ? i * apart : (int)((state = state * 1664525u + 1013904223u) >> 6);
    double links = 0;  // that a warp's slowest lane meets, over blocks
    for (int b = 0; b < 8; b++) {
      std::vector<int> chain(gdn::kHeads);
      for (int i = b, k = 0; i < n && k < gdn::kOwn; i += step, k++) chain.at(gdn::chain_of(dst[i]))++;
      for (int w = 0; w < n / 32; w++) {
        int longest = 0;
        for (int l = 0; l < 32; l++) longest = std::max(longest, chain[gdn::chain_of(dst[w * 32 + l])]);
        links += longest / (n / 32. * 8);
      }
    }
    std::printf("%d: %.2f\n", apart, links);
    if (links > 4) return 1;
  }
  return 0;
}
"""


def test_chains_are_short(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "chains.cu", tmp_path / "chains"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
