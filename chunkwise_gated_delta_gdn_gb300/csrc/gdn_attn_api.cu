// gdn_attn_api.cu -- C entry points of softmax attention and the paged cache:
// argument validation, workspace sizing, launch.
#include "gdn_attn_checks.h"

namespace {

// Everything that both attention entries share once their own arguments are
// checked.
gdn_status launch(gdn::AttnArgs &a, int d, int dtype, float scale, const gdn::AttnLaunch &l,
                  void *workspace, gdn_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (a.flags && cudaMemsetAsync(a.flags, 0, sizeof(uint32_t), stream) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (a.Ttot == 0) return GDN_OK;
  a.scale_log2 = scale * 1.44269504088896340736f;
  place_parts(a, d, l, workspace);
  return gdn::launch_attn(a, d, dtype, l, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t gdn_attn_fwd_workspace_bytes(int B, int T, int H, int HKV, int d, int n_seqs, int dtype) {
  int n;
  long Ttot;
  const bool packed = B == 1 && n_seqs > 1;
  if (check_shape(B, T, H, HKV, d, n_seqs, packed, dtype, n, Ttot) != GDN_OK) return 0;
  // one sequence may come with or without cu_seqlens: the larger of the two
  size_t most = 0;
  for (int with_cu = packed || B == 1 ? 1 : 0; with_cu >= (packed ? 1 : 0); with_cu--) {
    gdn::AttnArgs a{};
    fill_shape(a, with_cu ? kSomewhere : nullptr, n, T, Ttot, H, HKV);
    const size_t bytes = part_bytes(gdn::attn_launch(a, d, dtype), d);
    if (bytes > most) most = bytes;
  }
  return most;
}

gdn_status gdn_attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                        const int32_t *cu_seqlens, int n_seqs, int B, int T, int H, int HKV, int d,
                        int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                        int dtype, uint32_t *flags, void *workspace, size_t workspace_bytes,
                        gdn_stream_t stream) {
  int n;
  long Ttot;
  const gdn_status st =
      check_shape(B, T, H, HKV, d, n_seqs, cu_seqlens != nullptr, dtype, n, Ttot);
  if (st != GDN_OK) return st;
  const size_t es = dtype == GDN_BF16 ? 2 : 4;
  const int64_t q_row = (int64_t)H * d, kv_row = (int64_t)HKV * d;
  if (!(std::isfinite(scale) && scale > 0.f)) return GDN_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, q_row, es) || !stride_ok(k_stride, kv_row, es) ||
      !stride_ok(v_stride, kv_row, es))
    return GDN_ERR_INVALID_ARG;
  if (Ttot > 0 && (!q || !k || !v || !o)) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(o, 16) ||
      !aligned_to(lse, 4) || !aligned_to(cu_seqlens, 4) || !aligned_to(flags, 4))
    return GDN_ERR_INVALID_ARG;
  gdn::AttnArgs a{};
  fill_shape(a, cu_seqlens, n, T, Ttot, H, HKV);
  const gdn::AttnLaunch l = gdn::attn_launch(a, d, dtype);
  if (l.blocks == 0) return GDN_ERR_UNSUPPORTED;
  const size_t ws = part_bytes(l, d);
  if (ws > 0 && (!workspace || workspace_bytes < ws)) return GDN_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return GDN_ERR_INVALID_ARG;
  const Buf outs[] = {{o, (size_t)Ttot * q_row * es}, {lse, (size_t)Ttot * H * 4}, {flags, 4},
                      {workspace, ws}};
  const Buf ins[] = {{q, span(Ttot, q_stride, q_row, es)}, {k, span(Ttot, k_stride, kv_row, es)},
                     {v, span(Ttot, v_stride, kv_row, es)},
                     {cu_seqlens, cu_seqlens ? ((size_t)n + 1) * 4 : 0}};
  if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.flags = flags;
  return launch(a, d, dtype, scale, l, workspace, stream);
}

size_t gdn_attn_paged_fwd_workspace_bytes(int B, int T, int H, int HKV, int d, int n_seqs,
                                          int page_size, int max_pages, int dtype) {
  int n;
  long Ttot;
  const bool packed = B == 1 && n_seqs > 1;
  if (check_shape(B, T, H, HKV, d, n_seqs, packed, dtype, n, Ttot) != GDN_OK) return 0;
  if (check_cache(page_size, max_pages, 1) != GDN_OK) return 0;
  size_t most = 0;
  for (int with_cu = packed || B == 1 ? 1 : 0; with_cu >= (packed ? 1 : 0); with_cu--) {
    gdn::AttnArgs a{};
    fill_shape(a, with_cu ? kSomewhere : nullptr, n, T, Ttot, H, HKV);
    a.kv_lens = kSomewhere;
    a.max_len = page_size * max_pages;
    const size_t bytes = part_bytes(gdn::attn_launch(a, d, dtype), d);
    if (bytes > most) most = bytes;
  }
  return most;
}

gdn_status gdn_attn_paged_fwd(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_table, const int32_t *kv_lens, void *o,
                              float *lse, const int32_t *cu_seqlens, int n_seqs, int B, int T,
                              int H, int HKV, int d, int64_t q_stride, int page_size,
                              int max_pages, int n_pages, float scale, int dtype, uint32_t *flags,
                              void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
  int n;
  long Ttot;
  gdn_status st = check_shape(B, T, H, HKV, d, n_seqs, cu_seqlens != nullptr, dtype, n, Ttot);
  if (st == GDN_OK) st = check_cache(page_size, max_pages, n_pages);
  if (st != GDN_OK) return st;
  const size_t es = dtype == GDN_BF16 ? 2 : 4;
  const int64_t q_row = (int64_t)H * d, kv_row = (int64_t)HKV * d;
  if (!(std::isfinite(scale) && scale > 0.f)) return GDN_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, q_row, es)) return GDN_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !block_table || !kv_lens) return GDN_ERR_INVALID_ARG;
  if (Ttot > 0 && (!q || !o)) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(o, 16) || !aligned_to(block_table, 4) || !aligned_to(kv_lens, 4) ||
      !aligned_to(lse, 4) || !aligned_to(cu_seqlens, 4) || !aligned_to(flags, 4))
    return GDN_ERR_INVALID_ARG;
  gdn::AttnArgs a{};
  fill_shape(a, cu_seqlens, n, T, Ttot, H, HKV);
  a.kv_lens = kv_lens;
  a.max_len = page_size * max_pages;
  const gdn::AttnLaunch l = gdn::attn_launch(a, d, dtype);
  if (l.blocks == 0) return GDN_ERR_UNSUPPORTED;
  const size_t ws = part_bytes(l, d);
  if (ws > 0 && (!workspace || workspace_bytes < ws)) return GDN_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return GDN_ERR_INVALID_ARG;
  const size_t cache = (size_t)n_pages * page_size * kv_row * es;
  const Buf outs[] = {{o, (size_t)Ttot * q_row * es}, {lse, (size_t)Ttot * H * 4}, {flags, 4},
                      {workspace, ws}};
  const Buf ins[] = {{q, span(Ttot, q_stride, q_row, es)}, {k_cache, cache}, {v_cache, cache},
                     {block_table, (size_t)n * max_pages * 4}, {kv_lens, (size_t)n * 4},
                     {cu_seqlens, cu_seqlens ? ((size_t)n + 1) * 4 : 0}};
  if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
  a.q = q; a.k = k_cache; a.v = v_cache; a.o = o; a.lse = lse; a.table = block_table;
  a.q_stride = q_stride;
  a.page_size = page_size; a.max_pages = max_pages; a.n_pages = n_pages;
  a.page_log = -1;
  for (int log = 4; log < 31; log++)
    if (page_size == 1 << log) a.page_log = log;
  a.flags = flags;
  return launch(a, d, dtype, scale, l, workspace, stream);
}

gdn_status gdn_kv_cache_append(const void *k, const void *v, void *k_cache, void *v_cache,
                               const int32_t *block_table, const int32_t *kv_lens,
                               const int32_t *cu_seqlens, int n_seqs, int B, int T, int HKV, int d,
                               int64_t k_stride, int64_t v_stride, int page_size, int max_pages,
                               int n_pages, int dtype, uint32_t *flags, gdn_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  int n;
  long Ttot;
  gdn_status st = check_shape(B, T, HKV, HKV, d, n_seqs, cu_seqlens != nullptr, dtype, n, Ttot);
  if (st == GDN_OK) st = check_cache(page_size, max_pages, n_pages);
  if (st != GDN_OK) return st;
  const size_t es = dtype == GDN_BF16 ? 2 : 4;
  const int64_t row = (int64_t)HKV * d;
  if (!stride_ok(k_stride, row, es) || !stride_ok(v_stride, row, es)) return GDN_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !block_table || !kv_lens) return GDN_ERR_INVALID_ARG;
  if (Ttot > 0 && (!k || !v)) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_cache, 16) ||
      !aligned_to(v_cache, 16) || !aligned_to(block_table, 4) || !aligned_to(kv_lens, 4) ||
      !aligned_to(cu_seqlens, 4) || !aligned_to(flags, 4))
    return GDN_ERR_INVALID_ARG;
  const size_t cache = (size_t)n_pages * page_size * row * es;
  const Buf outs[] = {{k_cache, cache}, {v_cache, cache}, {flags, 4}};
  const Buf ins[] = {{k, span(Ttot, k_stride, row, es)}, {v, span(Ttot, v_stride, row, es)},
                     {block_table, (size_t)n * max_pages * 4}, {kv_lens, (size_t)n * 4},
                     {cu_seqlens, cu_seqlens ? ((size_t)n + 1) * 4 : 0}};
  if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
  if (flags && cudaMemsetAsync(flags, 0, sizeof(uint32_t), stream) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (Ttot == 0) return GDN_OK;
  gdn::AppendArgs a{};
  a.k = k; a.v = v; a.k_cache = k_cache; a.v_cache = v_cache;
  a.cu = cu_seqlens; a.kv_lens = kv_lens; a.table = block_table;
  a.n_seqs = n; a.T = T; a.Ttot = (int)Ttot;
  a.k_stride = k_stride * (int64_t)es; a.v_stride = v_stride * (int64_t)es;
  a.row_bytes = (int)(row * es);
  a.page_size = page_size; a.max_pages = max_pages; a.n_pages = n_pages;
  a.max_len = page_size * max_pages;
  a.flags = flags;
  return gdn::launch_kv_append(a, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
