"""What the attention entries hand to a launch, without a GPU: the entries (csrc/gdn_attn_api.cu)
are compiled against stand-ins for the launchers.  Places for partial results are given exactly
when a call may cut units, and lie within the workspace."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build

PROGRAM = r"""
#include <cstdio>

#include "gdn_attn_api.cu"
#include "gdn_attn.cuh"

namespace gdn {
static AttnArgs seen;
static int launches = 0;
AttnLaunch attn_launch(AttnArgs &a, int, int dtype) {
  return dtype ? attn_plan_launch<TcShape>(a, 152) : attn_plan_launch<AttnShape<64, 64, 64, 2, 1, 2, 1, 16, 0, 1>>(a, 304);
}
cudaError_t launch_attn(const AttnArgs &a, int, int, const AttnLaunch &, cudaStream_t) {
  seen = a;
  launches++;
  return cudaSuccess;
}
cudaError_t launch_kv_append(const AppendArgs &, cudaStream_t) { return cudaSuccess; }
}  // namespace gdn

static char *addr(int i) { return reinterpret_cast<char *>((1ull << 40) + i * (1ull << 36)); }

int main() {
  int cut = 0, whole = 0;
  const int32_t *some = reinterpret_cast<const int32_t *>(addr(9));
  for (int dtype = 0; dtype < 2; dtype++)
    for (int d = 64; d <= 128; d += 64)
      for (int packed = 0; packed < 2; packed++)
        for (int T = 1; T < 40000; T = T * 3 + 1) {
          const int H = 8, HKV = 2, B = packed ? 1 : 3, n = packed ? 5 : 0;
          const int32_t *cu = packed ? some : nullptr;
          for (int paged = 0; paged < 2; paged++) {
            const size_t ws = 1ull << 33;
            const size_t need = paged ? gdn_attn_paged_fwd_workspace_bytes(B, T, H, HKV, d, n, 64, 40, dtype)
                                      : gdn_attn_fwd_workspace_bytes(B, T, H, HKV, d, n, dtype);
            const int before = gdn::launches;
            const gdn_status st =
                paged ? gdn_attn_paged_fwd(addr(0), addr(1), addr(2), some + 64, some + 4096, addr(3), nullptr, cu, n, B,
                                           T, H, HKV, d, H * d, 64, 40, 100, 0.1f, dtype, nullptr, addr(5), ws, nullptr)
                      : gdn_attn_fwd(addr(0), addr(1), addr(2), addr(3), nullptr, cu, n, B, T, H, HKV, d, H * d, HKV * d,
                                     HKV * d, 0.1f, dtype, nullptr, addr(5), ws, nullptr);
            if (st != GDN_OK || gdn::launches != before + 1) { std::printf("status %d\n", st); return 1; }
            const char *parts[3] = {(const char *)gdn::seen.part_o, (const char *)gdn::seen.part_ml,
                                    (const char *)gdn::seen.jobs};
            for (const char *p : parts)
              if ((p != nullptr) != (need > 0) || (p && (p < addr(5) || p >= addr(5) + need))) {
                std::printf("dtype %d d %d packed %d T %d paged %d: %p of %zu\n", dtype, d, packed, T, paged, p, need);
                return 1;
              }
            (need ? cut : whole)++;
          }
        }
  if (cut < 10 || whole < 10) { std::printf("%d cut, %d whole\n", cut, whole); return 1; }
  std::printf("ok\n");
  return 0;
}
"""


def test_places_for_partial_results(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "args.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "args"
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
