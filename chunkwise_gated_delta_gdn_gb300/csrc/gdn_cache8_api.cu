// gdn_cache8_api.cu -- C entry points of a cache in 8 bits (its write, attention over
// it), of page copies and of rotary positions: argument validation, workspace sizing,
// launch.
#include "gdn_attn_checks.h"

namespace {

// Bytes of a cache's scales.
size_t scale_bytes(int n_pages, int page_size, int HKV) {
  return (size_t)n_pages * (page_size / gdn::kScaleBlock) * HKV * sizeof(float);
}

// Partial results of the two kernels' plans, one behind the other.
size_t few_bytes(const gdn::Attn8Launch &l, int d) { return (part_bytes(l.few_launch, d) + 255) / 256 * 256; }
size_t parts8_bytes(const gdn::Attn8Launch &l, int d) {
  return few_bytes(l, d) + part_bytes(l.many_launch, d);
}

// Token arrays that may interleave: no element in common.
struct Rows {
  const void *p;
  int64_t stride, row;  // elements
};
bool apart(const Rows &a, const Rows &b, long Ttot, size_t es) {
  if (!ranges_overlap(a.p, span(Ttot, a.stride, a.row, es), b.p, span(Ttot, b.stride, b.row, es))) return true;
  if (a.stride != b.stride) return false;
  const int64_t step = a.stride * (int64_t)es;
  const int64_t gap = (int64_t)((intptr_t)b.p - (intptr_t)a.p) % step;
  const int64_t behind = gap < 0 ? gap + step : gap;  // b's row behind a's, within a step
  return behind >= a.row * (int64_t)es && behind + b.row * (int64_t)es <= step;
}

}  // namespace

extern "C" {

size_t gdn_attn_paged_fp8_fwd_workspace_bytes(int B, int T, int H, int HKV, int d, int n_seqs,
                                              int page_size, int max_pages) {
  int n;
  long Ttot;
  const bool packed = B == 1 && n_seqs > 1;
  if (check_shape(B, T, H, HKV, d, n_seqs, packed, GDN_BF16, n, Ttot) != GDN_OK) return 0;
  if (check_cache(page_size, max_pages, 1) != GDN_OK) return 0;
  size_t most = 0;
  for (int with_cu = packed || B == 1 ? 1 : 0; with_cu >= (packed ? 1 : 0); with_cu--) {
    gdn::AttnArgs a{};
    fill_shape(a, with_cu ? kSomewhere : nullptr, n, T, Ttot, H, HKV);
    a.kv_lens = kSomewhere;
    a.max_len = page_size * max_pages;
    gdn::Attn8Launch l;
    if (!gdn::attn8_launch(a, d, l)) continue;
    const size_t bytes = parts8_bytes(l, d);
    if (bytes > most) most = bytes;
  }
  return most;
}

gdn_status gdn_attn_paged_fp8_fwd(const void *q, const void *k_cache, const void *v_cache,
                                  const float *k_scale, const float *v_scale,
                                  const int32_t *block_table, const int32_t *kv_lens, void *o,
                                  float *lse, const int32_t *cu_seqlens, int n_seqs, int B, int T,
                                  int H, int HKV, int d, int64_t q_stride, int page_size,
                                  int max_pages, int n_pages, float scale, int dtype,
                                  uint32_t *flags, void *workspace, size_t workspace_bytes,
                                  gdn_stream_t stream) {
  int n;
  long Ttot;
  gdn_status st = check_shape(B, T, H, HKV, d, n_seqs, cu_seqlens != nullptr, dtype, n, Ttot);
  if (st == GDN_OK) st = check_cache(page_size, max_pages, n_pages);
  if (st != GDN_OK) return st;
  if (dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  const int64_t q_row = (int64_t)H * d, kv_row = (int64_t)HKV * d;
  if (!(std::isfinite(scale) && scale > 0.f)) return GDN_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, q_row, 2)) return GDN_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !kv_lens)
    return GDN_ERR_INVALID_ARG;
  if (Ttot > 0 && (!q || !o)) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) || !aligned_to(o, 16) ||
      !aligned_to(block_table, 4) || !aligned_to(kv_lens, 4) || !aligned_to(lse, 4) ||
      !aligned_to(cu_seqlens, 4) || !aligned_to(flags, 4))
    return GDN_ERR_INVALID_ARG;
  gdn::AttnArgs a{};
  fill_shape(a, cu_seqlens, n, T, Ttot, H, HKV);
  a.kv_lens = kv_lens;
  a.max_len = page_size * max_pages;
  a.q = q; a.k = k_cache; a.v = v_cache; a.o = o; a.lse = lse; a.table = block_table;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.q_stride = q_stride;
  a.page_size = page_size; a.max_pages = max_pages; a.n_pages = n_pages;
  a.page_log = -1;
  for (int log = 4; log < 31; log++)
    if (page_size == 1 << log) a.page_log = log;
  a.flags = flags;
  a.scale_log2 = scale * 1.44269504088896340736f;
  gdn::Attn8Launch l;
  if (!gdn::attn8_launch(a, d, l)) return GDN_ERR_UNSUPPORTED;
  const size_t ws = parts8_bytes(l, d);
  if (ws > 0 && (!workspace || workspace_bytes < ws)) return GDN_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return GDN_ERR_INVALID_ARG;
  const size_t cache = (size_t)n_pages * page_size * kv_row, scales = scale_bytes(n_pages, page_size, HKV);
  const Buf outs[] = {{o, (size_t)Ttot * q_row * 2}, {lse, (size_t)Ttot * H * 4}, {flags, 4},
                      {workspace, ws}};
  const Buf ins[] = {{q, span(Ttot, q_stride, q_row, 2)}, {k_cache, cache}, {v_cache, cache},
                     {k_scale, scales}, {v_scale, scales},
                     {block_table, (size_t)n * max_pages * 4}, {kv_lens, (size_t)n * 4},
                     {cu_seqlens, cu_seqlens ? ((size_t)n + 1) * 4 : 0}};
  if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.flags && cudaMemsetAsync(a.flags, 0, sizeof(uint32_t), s) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (a.Ttot == 0) return GDN_OK;
  place_parts(l.few, d, l.few_launch, workspace);
  place_parts(l.many, d, l.many_launch, static_cast<char *>(workspace) + few_bytes(l, d));
  return gdn::launch_attn8(l, d, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv_cache_append_fp8(const void *k, const void *v, void *k_cache, void *v_cache,
                                   float *k_scale, float *v_scale, const int32_t *block_table,
                                   const int32_t *kv_lens, const int32_t *cu_seqlens, int n_seqs,
                                   int B, int T, int HKV, int d, int64_t k_stride,
                                   int64_t v_stride, int page_size, int max_pages, int n_pages,
                                   int dtype, uint32_t *flags, gdn_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  int n;
  long Ttot;
  gdn_status st = check_shape(B, T, HKV, HKV, d, n_seqs, cu_seqlens != nullptr, dtype, n, Ttot);
  if (st == GDN_OK) st = check_cache(page_size, max_pages, n_pages);
  if (st != GDN_OK) return st;
  const size_t es = dtype == GDN_BF16 ? 2 : 4;
  const int64_t row = (int64_t)HKV * d;
  if (!stride_ok(k_stride, row, es) || !stride_ok(v_stride, row, es)) return GDN_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !kv_lens)
    return GDN_ERR_INVALID_ARG;
  if (Ttot > 0 && (!k || !v)) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_cache, 16) ||
      !aligned_to(v_cache, 16) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) ||
      !aligned_to(block_table, 4) || !aligned_to(kv_lens, 4) || !aligned_to(cu_seqlens, 4) ||
      !aligned_to(flags, 4))
    return GDN_ERR_INVALID_ARG;
  // blocks of 16 tokens, two more for each sequence, are counted in 32 bits
  if (Ttot / 16 + 2L * n > INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
  const size_t cache = (size_t)n_pages * page_size * row, scales = scale_bytes(n_pages, page_size, HKV);
  const Buf outs[] = {{k_cache, cache}, {v_cache, cache}, {k_scale, scales}, {v_scale, scales}, {flags, 4}};
  const Buf ins[] = {{k, span(Ttot, k_stride, row, es)}, {v, span(Ttot, v_stride, row, es)},
                     {block_table, (size_t)n * max_pages * 4}, {kv_lens, (size_t)n * 4},
                     {cu_seqlens, cu_seqlens ? ((size_t)n + 1) * 4 : 0}};
  if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
  if (flags && cudaMemsetAsync(flags, 0, sizeof(uint32_t), stream) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (Ttot == 0) return GDN_OK;
  gdn::Append8Args a{};
  a.k = k; a.v = v;
  a.k_cache = static_cast<uint8_t *>(k_cache); a.v_cache = static_cast<uint8_t *>(v_cache);
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.cu = cu_seqlens; a.kv_lens = kv_lens; a.table = block_table;
  a.n_seqs = n; a.T = T; a.Ttot = (int)Ttot;
  a.k_stride = k_stride; a.v_stride = v_stride;
  a.HKV = HKV;
  a.page_size = page_size; a.max_pages = max_pages; a.n_pages = n_pages;
  a.max_len = page_size * max_pages;
  a.flags = flags;
  return gdn::launch_kv_append8(a, d, dtype, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv_cache_copy_pages(void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                                   const int32_t *src, const int32_t *dst, int n_copies, int HKV,
                                   int d, int page_size, int n_pages, int dtype, uint32_t *flags,
                                   gdn_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (n_copies < 0 || HKV <= 0 || d <= 0) return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16 && dtype != GDN_E4M3) return GDN_ERR_INVALID_ARG;
  const gdn_status st = check_cache(page_size, 1, n_pages);
  if (st != GDN_OK) return st;
  if (d != 64 && d != 128) return GDN_ERR_UNSUPPORTED;
  // pairs are compared with one another: without a bound a call could take minutes
  if (HKV > 65535 || n_copies > gdn::kMaxCopies) return GDN_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || (n_copies > 0 && (!src || !dst))) return GDN_ERR_INVALID_ARG;
  // scales belong to a cache in 8 bits, and to no other
  if ((dtype == GDN_E4M3) != (k_scale != nullptr) || (dtype == GDN_E4M3) != (v_scale != nullptr))
    return GDN_ERR_INVALID_ARG;
  if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(k_scale, 4) ||
      !aligned_to(v_scale, 4) || !aligned_to(src, 4) || !aligned_to(dst, 4) || !aligned_to(flags, 4))
    return GDN_ERR_INVALID_ARG;
  const size_t page = (size_t)page_size * HKV * d * (dtype == GDN_E4M3 ? 1 : dtype == GDN_BF16 ? 2 : 4);
  const size_t scales = k_scale ? scale_bytes(n_pages, page_size, HKV) : 0;
  const Buf outs[] = {{k_cache, page * n_pages}, {v_cache, page * n_pages}, {k_scale, scales}, {v_scale, scales}, {flags, 4}};
  const Buf ins[] = {{src, (size_t)n_copies * 4}, {dst, (size_t)n_copies * 4}};
  if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
  if (flags && cudaMemsetAsync(flags, 0, sizeof(uint32_t), stream) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (n_copies == 0) return GDN_OK;
  gdn::CopyPagesArgs a{};
  void *const base[4] = {k_cache, v_cache, k_scale, v_scale};
  for (int i = 0; i < 4; i++) {
    a.base[i] = static_cast<char *>(base[i]);
    a.bytes[i] = (long long)(i < 2 ? page : scales / n_pages);
  }
  a.src = src; a.dst = dst;
  a.n = n_copies; a.n_pages = n_pages;
  a.flags = flags;
  return gdn::launch_kv_copy_pages(a, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

static gdn_status rope(const void *q, const void *k, void *q_out, void *k_out, const float *inv_freq,
                       int rot, int interleaved, float mscale, const int32_t *kv_lens,
                       const int32_t *cu_seqlens, int n_seqs, int B, int T, int H, int HKV, int d,
                       int64_t q_stride, int64_t k_stride, int64_t q_out_stride,
                       int64_t k_out_stride, int dtype, uint32_t *flags, gdn_stream_t stream_,
                       float sign) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  int n;
  long Ttot;
  if (HKV < 0 || rot <= 0 || rot > d || rot % 2 != 0) return GDN_ERR_INVALID_ARG;
  // no relation between H and HKV is asked for here; HKV = 0: queries only
  const gdn_status st = check_shape(B, T, H, H, d, n_seqs, cu_seqlens != nullptr, dtype, n, Ttot);
  if (st != GDN_OK) return st;
  if (rot % 16 != 0 || HKV > 65535) return GDN_ERR_UNSUPPORTED;
  if (!(interleaved == 0 || interleaved == 1) || !std::isfinite(mscale)) return GDN_ERR_INVALID_ARG;
  const size_t es = dtype == GDN_BF16 ? 2 : 4;
  const int64_t q_row = (int64_t)H * d, k_row = (int64_t)HKV * d;
  if (!stride_ok(q_stride, q_row, es) || !stride_ok(q_out_stride, q_row, es)) return GDN_ERR_INVALID_ARG;
  if (HKV > 0 && (!stride_ok(k_stride, k_row, es) || !stride_ok(k_out_stride, k_row, es)))
    return GDN_ERR_INVALID_ARG;
  if (!inv_freq || (Ttot > 0 && (!q || !q_out || (HKV > 0 && (!k || !k_out))))) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(q_out, 16) || !aligned_to(inv_freq, 4) ||
      !aligned_to(kv_lens, 4) || !aligned_to(cu_seqlens, 4) || !aligned_to(flags, 4) ||
      (HKV > 0 && (!aligned_to(k, 16) || !aligned_to(k_out, 16))))
    return GDN_ERR_INVALID_ARG;
  // An output is its own input, at the same stride, or has no element in common with
  // any other array; q and k may be slices of one.
  const Rows qi = {q, q_stride, q_row}, qo = {q_out, q_out_stride, q_row};
  const Rows ki = {k, k_stride, k_row}, ko = {k_out, k_out_stride, k_row};
  const bool q_ok = q_out == q ? q_out_stride == q_stride : apart(qo, qi, Ttot, es);
  if (!q_ok) return GDN_ERR_INVALID_ARG;
  if (HKV > 0) {
    const bool k_ok = k_out == k ? k_out_stride == k_stride : apart(ko, ki, Ttot, es);
    if (!k_ok || !apart(qo, ko, Ttot, es) || !apart(qo, ki, Ttot, es) || !apart(ko, qi, Ttot, es))
      return GDN_ERR_INVALID_ARG;
  }
  const size_t k_any = HKV > 0 ? 1 : 0;
  const Buf rows[] = {{q_out, span(Ttot, q_out_stride, q_row, es)}, {k_out, k_any * span(Ttot, k_out_stride, k_row, es)}};
  const Buf small[] = {{inv_freq, (size_t)rot * 2}, {kv_lens, kv_lens ? (size_t)n * 4 : 0},
                       {cu_seqlens, cu_seqlens ? ((size_t)n + 1) * 4 : 0}};
  const Buf word[] = {{flags, 4}};
  const Buf ins[] = {rows[0], rows[1], {q, span(Ttot, q_stride, q_row, es)}, {k, k_any * span(Ttot, k_stride, k_row, es)},
                     small[0], small[1], small[2]};
  for (const Buf &x : rows)
    for (const Buf &y : small)
      if (ranges_overlap(x.p, x.n, y.p, y.n)) return GDN_ERR_INVALID_ARG;
  if (!disjoint(word, ins)) return GDN_ERR_INVALID_ARG;
  if (flags && cudaMemsetAsync(flags, 0, sizeof(uint32_t), stream) != cudaSuccess) return GDN_ERR_CUDA;
  if (Ttot == 0) return GDN_OK;
  gdn::RopeArgs a{};
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.qo_stride = q_out_stride; a.ko_stride = k_out_stride;
  a.inv_freq = inv_freq;
  a.cu = cu_seqlens; a.kv_lens = kv_lens;
  a.n_seqs = n; a.T = T; a.Ttot = (int)Ttot;
  a.HQ = H; a.HK = HKV; a.rot = rot;
  a.mscale = mscale; a.sign = sign;
  a.flags = flags;
  return gdn::launch_rope(a, d, interleaved != 0, dtype, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_rope_fwd(const void *q, const void *k, void *q_out, void *k_out,
                        const float *inv_freq, int rot, int interleaved, float mscale,
                        const int32_t *kv_lens, const int32_t *cu_seqlens, int n_seqs, int B, int T,
                        int H, int HKV, int d, int64_t q_stride, int64_t k_stride,
                        int64_t q_out_stride, int64_t k_out_stride, int dtype, uint32_t *flags,
                        gdn_stream_t stream) {
  return rope(q, k, q_out, k_out, inv_freq, rot, interleaved, mscale, kv_lens, cu_seqlens, n_seqs, B,
              T, H, HKV, d, q_stride, k_stride, q_out_stride, k_out_stride, dtype, flags, stream, 1.f);
}

gdn_status gdn_rope_bwd(const void *dq, const void *dk, void *dq_in, void *dk_in,
                        const float *inv_freq, int rot, int interleaved, float mscale,
                        const int32_t *kv_lens, const int32_t *cu_seqlens, int n_seqs, int B, int T,
                        int H, int HKV, int d, int64_t dq_stride, int64_t dk_stride,
                        int64_t dq_in_stride, int64_t dk_in_stride, int dtype, uint32_t *flags,
                        gdn_stream_t stream) {
  return rope(dq, dk, dq_in, dk_in, inv_freq, rot, interleaved, mscale, kv_lens, cu_seqlens, n_seqs,
              B, T, H, HKV, d, dq_stride, dk_stride, dq_in_stride, dk_in_stride, dtype, flags, stream,
              -1.f);
}

}  // extern "C"
