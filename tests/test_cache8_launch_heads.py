"""What the entry of attention over an 8-bit cache hands to its launch where key/value heads are a multiple of eight, without
a GPU: the choices of a block for eight heads and of a warp for a unit are met, and their places for partial results lie within the workspace
that the query asks for."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build
from tests.test_cache8_launch_args import PROGRAM

MAIN = r"""int main() {
  int teams = 0, warps = 0, cut = 0, whole = 0;
  const int32_t *some = reinterpret_cast<const int32_t *>(addr(9));
  for (int d = 64; d <= 128; d += 64)
    for (int HKV = 8; HKV <= 24; HKV += 8)
      for (int G = 1; G <= 8; G *= 2)
        for (int n : {1, 3, 11, 24, 47, 48, 49, 96, 152, 304, 1000, 5000})
          for (int T = 1; T * G <= 40; T++)
            for (int max_pages = 1; max_pages < 600; max_pages *= 5) {
              const int H = HKV * G;
              const size_t ws = 1ull << 33;
              const size_t need = gdn_attn_paged_fp8_fwd_workspace_bytes(n, T, H, HKV, d, 0, 64, max_pages);
              const int before = gdn::launches;
              const gdn_status st = gdn_attn_paged_fp8_fwd(addr(0), addr(1), addr(2), (float *)addr(6), (float *)addr(7), some + 4096,
                  some + (1 << 24), addr(3), nullptr, nullptr, 0, n, T, H, HKV, d, H * d, 64, max_pages, 1000, 0.1f, GDN_BF16, nullptr, addr(5), ws, nullptr);
              if (st != GDN_OK || gdn::launches != before + 1) { std::printf("status %d\n", st); return 1; }
              const gdn::Attn8Launch &l = gdn::seen;
              char *f0 = nullptr, *f1 = nullptr, *m0 = nullptr, *m1 = nullptr;
              const bool f = l.has_few && l.few_launch.split, m = l.has_many && l.many_launch.split;
              bool ok = l.has_few != l.has_many && f == (l.few.part_o != nullptr) && m == (l.many.part_o != nullptr) && (f || m) == (need > 0);
              if (f) ok &= places(l.few, l.few_launch, d, f0, f1) && f0 >= addr(5) && f1 <= addr(5) + need;
              if (m) ok &= places(l.many, l.many_launch, d, m0, m1) && m0 >= addr(5) && m1 <= addr(5) + need;
              // the plan deals to blocks, or to eight warps of each
              if (l.teams || l.warps) ok &= l.has_few && T * G <= 8 && l.teams != l.warps && (!f || l.few_launch.blocks == (l.warps ? 8 : 1) * 2 * 152);
              if (l.teams) ok &= l.few_launch.rows == gdn::TeamShape8::kRows;
              // teams in place of warps, as where sequences are long, have places enough
              if (l.warps && f) ok &= (long)gdn::TeamShape8::kRows * l.few_launch.blocks / 8 <= (long)l.few_launch.rows * l.few_launch.blocks;
              if (!ok) { std::printf("d %d H %d HKV %d n %d T %d pages %d: need %zu\n", d, H, HKV, n, T, max_pages, need); return 1; }
              (f || m ? cut : whole)++;
              teams += l.teams && f;
              warps += l.warps && f;
            }
  if (cut < 100 || whole < 100 || teams < 100 || warps < 100) { std::printf("%d cut, %d whole, %d teams, %d warps\n", cut, whole, teams, warps); return 1; }
  std::printf("ok\n");
  return 0;
}
"""


def test_places_of_eight_heads_and_of_warps(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "heads.cu", tmp_path / "heads"
    src.write_text(PROGRAM[:PROGRAM.index("int main() {")] + MAIN)
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
