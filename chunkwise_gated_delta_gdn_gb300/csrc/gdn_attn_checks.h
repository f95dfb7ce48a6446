// gdn_attn_checks.h -- argument checks that the entry points of attention, the paged
// cache and rotary positions share.  Each translation unit has its own.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "gdn.h"
#include "gdn_internal.h"

namespace {

using gdn::aligned_to;
using gdn::ranges_overlap;

// Sequences, heads and type; fills `n` (sequences) and `Ttot`.
inline gdn_status check_shape(int B, int T, int H, int HKV, int d, int n_seqs, bool packed, int dtype,
                              int &n, long &Ttot) {
  if (B <= 0 || T < 0 || H <= 0 || HKV <= 0 || d <= 0 || H % HKV != 0) return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (packed) {
    if (B != 1 || n_seqs <= 0) return GDN_ERR_INVALID_ARG;
    n = n_seqs;
  } else {
    if (n_seqs != 0 && n_seqs != B) return GDN_ERR_INVALID_ARG;
    n = B;
  }
  if (d != 64 && d != 128) return GDN_ERR_UNSUPPORTED;
  Ttot = (long)B * T;
  // rows and sequences are counted in 32 bits, with room for a tile past the last one
  if (Ttot > INT32_MAX - 1024 || n > INT32_MAX - 1024 || H > 65535) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

inline gdn_status check_cache(int page_size, int max_pages, int n_pages) {
  if (page_size <= 0 || max_pages <= 0 || n_pages <= 0) return GDN_ERR_INVALID_ARG;
  // positions, and 8-row groups of the whole cache, are counted in 32 bits
  if (page_size % 16 != 0 || (long)page_size * max_pages > INT32_MAX - 1024 ||
      (n_pages + 1L) * (page_size / 8) > INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

inline size_t part_bytes(const gdn::AttnLaunch &l, int d) {
  if (!l.split) return 0;
  const size_t rows = (size_t)2 * l.blocks * l.rows;
  return rows * d * sizeof(float) + rows * sizeof(float2) + (size_t)l.blocks * gdn::kAttnJobBytes;
}

// A token stride: at least the row, in 16-byte steps.
inline bool stride_ok(int64_t stride, int64_t row, size_t es) {
  return stride >= row && (stride * (int64_t)es) % 16 == 0 && stride <= INT32_MAX;
}
// Bytes from the first to the last element of a strided token array.
inline size_t span(long Ttot, int64_t stride, int64_t row, size_t es) {
  return Ttot ? ((size_t)(Ttot - 1) * stride + row) * es : 0;
}

struct Buf {
  const void *p;
  size_t n;
};
// No output may overlap an input or another output.
template <int NO, int NI>
bool disjoint(const Buf (&outs)[NO], const Buf (&ins)[NI]) {
  for (int i = 0; i < NO; i++) {
    for (int j = 0; j < NI; j++)
      if (ranges_overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return false;
    for (int j = 0; j < i; j++)
      if (ranges_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return false;
  }
  return true;
}

// Places of partial results in the workspace.
inline void place_parts(gdn::AttnArgs &a, int d, const gdn::AttnLaunch &l, void *workspace) {
  if (!l.split) return;
  const size_t rows = (size_t)2 * l.blocks * l.rows;
  a.part_o = static_cast<float4 *>(workspace);
  a.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + rows * d * sizeof(float));
  a.jobs = reinterpret_cast<gdn::AttnJob *>(a.part_ml + rows);
}

// What the plan goes by.
inline void fill_shape(gdn::AttnArgs &a, const int32_t *cu, int n, int T, long Ttot, int H, int HKV) {
  a.cu = cu;
  a.n_seqs = n;
  a.T = T;
  a.Ttot = (int)Ttot;
  a.H = H;
  a.HKV = HKV;
}
const int32_t kSomewhere[1] = {0};  // stands for device arrays in a workspace query: not read

}  // namespace
