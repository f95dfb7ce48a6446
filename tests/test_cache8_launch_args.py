"""What the entry of attention over an 8-bit cache hands to its launch, without a GPU: the entry
(csrc/gdn_cache8_api.cu) is compiled with the host's decisions (csrc/gdn_attn8.cu) against a stand-in
for the tensor-core kernel's launch.  Places for partial results are given exactly when a kernel may
cut units, lie within the workspace that the query asks for, and those of the two kernels are apart."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from chunkwise_gated_delta_gdn_gb300 import build as cuda_build

PROGRAM = r"""
#include <cstdio>

#define launch_attn8 kernels_of_the_call
#include "gdn_attn8.cu"
#undef launch_attn8
namespace gdn {
cudaError_t launch_attn8(const Attn8Launch &l, int d, cudaStream_t stream);
}
#include "gdn_cache8_api.cu"

namespace gdn {
static Attn8Launch seen;
static int launches = 0;
int sm_count() { return 152; }
cudaError_t allow_smem(const void *, int, std::atomic<uint64_t> &) { return cudaSuccess; }
cudaError_t launch_attn8_tc(const AttnArgs &, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_attn8_merge(const AttnArgs &, int, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_attn8(const Attn8Launch &l, int, cudaStream_t) { seen = l; launches++; return cudaSuccess; }
cudaError_t launch_kv_append8(const Append8Args &, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_kv_copy_pages(const CopyPagesArgs &, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_rope(const RopeArgs &, int, bool, int, cudaStream_t) { return cudaSuccess; }
}  // namespace gdn

static char *addr(int i) { return reinterpret_cast<char *>((1ull << 40) + i * (1ull << 36)); }

// first and last byte of a kernel's places
static bool places(const gdn::AttnArgs &a, const gdn::AttnLaunch &l, int d, char *&from, char *&to) {
  from = reinterpret_cast<char *>(a.part_o);
  to = reinterpret_cast<char *>(a.jobs) + (size_t)l.blocks * gdn::kAttnJobBytes;
  const char *ml = reinterpret_cast<const char *>(a.part_ml);
  const size_t rows = (size_t)2 * l.blocks * l.rows;
  return ml == from + rows * d * 4 && reinterpret_cast<char *>(a.jobs) == ml + rows * 8;
}

int main() {
  int cut = 0, whole = 0, both = 0;
  const int32_t *some = reinterpret_cast<const int32_t *>(addr(9));
  for (int d = 64; d <= 128; d += 64)
    for (int H = 8; H <= 80; H += 24)
      for (int packed = 0; packed < 2; packed++)
        for (int n = 1; n < 900; n = n * 3 + 1)
          for (int T = 1; T < 3000; T = T * 3 + 1)
            for (int max_pages = 4; max_pages < 400; max_pages *= 8) {
              const int HKV = 2, B = packed ? 1 : n, seqs = packed ? n : 0;
              const int32_t *cu = packed ? some : nullptr;
              const size_t ws = 1ull << 33;
              const size_t need = gdn_attn_paged_fp8_fwd_workspace_bytes(B, T, H, HKV, d, seqs, 64, max_pages);
              const int before = gdn::launches;
              const gdn_status st = gdn_attn_paged_fp8_fwd(addr(0), addr(1), addr(2), (float *)addr(6), (float *)addr(7), some + 4096,
                  some + (1 << 24), addr(3), nullptr, cu, seqs, B, T, H, HKV, d, H * d, 64, max_pages, 1000, 0.1f, GDN_BF16, nullptr, addr(5), ws, nullptr);
              if (st != GDN_OK || gdn::launches != before + 1) { std::printf("status %d\n", st); return 1; }
              const gdn::Attn8Launch &l = gdn::seen;
              char *f0 = nullptr, *f1 = nullptr, *m0 = nullptr, *m1 = nullptr;
              const bool f = l.has_few && l.few_launch.split, m = l.has_many && l.many_launch.split;
              bool ok = (l.has_few || l.has_many) && f == (l.few.part_o != nullptr) && m == (l.many.part_o != nullptr) && (f || m) <= (need > 0);
              if (f) ok &= places(l.few, l.few_launch, d, f0, f1) && f0 >= addr(5) && f1 <= addr(5) + need;
              if (m) ok &= places(l.many, l.many_launch, d, m0, m1) && m0 >= addr(5) && m1 <= addr(5) + need && (size_t)m0 % 256 == 0;
              if (f && m) ok &= f1 <= m0;
              if (!ok) { std::printf("d %d H %d packed %d n %d T %d pages %d: need %zu\n", d, H, packed, n, T, max_pages, need); return 1; }
              (f || m ? cut : whole)++;
              both += f && m;
            }
  if (cut < 20 || whole < 20 || both < 20) { std::printf("%d cut, %d whole, %d both\n", cut, whole, both); return 1; }
  std::printf("ok\n");
  return 0;
}
"""


def test_places_for_partial_results(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "args.cu", tmp_path / "args"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, *cuda_build.ARCH, *cuda_build.NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
