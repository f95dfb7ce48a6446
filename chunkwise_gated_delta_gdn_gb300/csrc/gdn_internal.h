// gdn_internal.h -- declarations shared by the host API (gdn_api.cu) and the
// kernel translation units.  Not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gdn {

// Bytes at the start of the workspace reserved for the device status word.
constexpr size_t kWorkspaceHeader = 256;
// Width of one dv slice handled by a scan CTA (fp32 path / bf16 path).
constexpr int kScanSlice = 32;
constexpr int kScanTcSlice = 64;
// The bf16 path's per-(chunk, value head) operand image written by the prep
// kernel: 192 rows x 64 fp16, K-major with the 128-byte swizzle
// (rows 0..127 = P1 = Kt^T T, rows 128..191 = Aqk T).
constexpr int kPrepImageRows = 192;
constexpr int kPrepImageBytes = kPrepImageRows * 128;
// At chunk 32 (per-key gate) its columns beyond C are never read: the image is
// written as 160 rows x 32 fp16 instead (K-major with the 64-byte swizzle; rows
// 0..127 = P1, rows 128..159 = Aqk T) in the first 10 KB of the same record.
constexpr int kPrepImage32Rows = 160;
constexpr int kPrepImage32Bytes = kPrepImage32Rows * 64;
// The scalar-gate bf16 path's image (one-chunk lookahead): 256 rows x 64 fp16,
// K-major with the 128-byte swizzle: rows 0..127 = P1 of the chunk, rows
// 128..191 = E = K_next P1 (the next chunk's keys times this chunk's P1; zero
// for a sequence's last chunk), rows 192..255 = Aqk T.
constexpr int kLaImageRows = 256;
constexpr int kLaImageBytes = kLaImageRows * 128;
// The same path's key/query image of one (chunk, q/k head): the A operand
// [K_next; Q] of the scan's state product, 128 rows of fp16 (next chunk's keys
// at 0..C-1, zero for a sequence's last chunk; this chunk's queries at
// 64..64+C-1), dk/64 panels of 128 x 128 bytes, K-major, 128-byte swizzle.
__host__ __device__ constexpr int kq_image_bytes(int dk) { return (dk / 64) * 16384; }

// Where packed sequence n starts: cu_seqlens[n], or n*T for plain batches.
// Sequence n owns the chunk slots [floor(start_n / C) + n, ...): one slot per
// chunk, injective over all sequences, fewer than floor(Ttot / C) + n_seqs.
struct SeqInfo {
  const int32_t *cu;  // device, or nullptr for a plain batch
  int n_seqs;         // sequences (B for a plain batch)
  int T;              // tokens per batch row (plain batch only)
  int Ttot;           // packed token count
};

struct PrepArgs {
  const void *q, *k;
  const float *g, *beta;
  SeqInfo seq;
  int H, HV;
  float scale;
  float *tiles;      // [n_slots][HV][2][C][C]: T = (I+A)^-1, then Aqk
  uint32_t *flags;   // device status word
  int n_slots;
  unsigned char *kq_images;  // bf16 scalar gate: [K_next; Q] image per (slot, hq);
                             // bf16 per-key gate: gated [K~; Q~] image per (slot, hv)
  float *decays;             // bf16 per-key gate: e^{b_last} per (slot, hv, key channel)
};

struct ScanArgs {
  const void *q, *k, *v;
  const float *g, *beta, *h0;
  void *o;
  float *hT;
  SeqInfo seq;
  int H, HV, dv;
  float scale;
  const float *tiles;
  uint32_t *flags;
  const unsigned char *kq_images;  // as PrepArgs::kq_images (read by the scan)
  const float *decays;             // as PrepArgs::decays
};

// The token-serial form (gdn_recurrent.cu): state in registers, one token at
// a time; hT may be h0 itself.
struct RecurrentArgs {
  const void *q, *k, *v;
  const float *g, *beta, *h0;
  void *o;
  float *hT;
  SeqInfo seq;
  int H, HV, dv;
  float scale;
  uint32_t *flags;  // device status word, or nullptr
};

// The operations either side of the recurrence (gdn_prepost.cu).
struct ConvArgs {
  const void *x;
  const float *w, *bias, *h0;  // w [D][W]; bias [D] or nullptr; h0 [N][D][W-1] or nullptr
  void *y;
  float *hT;                   // [N][D][W-1] or nullptr; may be h0 itself
  SeqInfo seq;
  int D;
  uint32_t *flags;             // device status word, or nullptr
  int tile0 = 0;               // first token tile of this launch (set by the launcher)
};
struct RowNormArgs {
  const void *x, *z;           // z: gate rows (gated RMS norm only), or nullptr
  const float *weight;         // [dim] (gated RMS norm only)
  void *y;
  long rows;
  float eps;
};

// Composition of a segment's state transfer (gdn_transfer.cu):
// S_out = M S_in + S_seg per (state, value head); n_states = sequences x heads.
struct TransferArgs {
  const float *M, *S_in, *S_seg;
  float *S_out;
  long n_states;
  int dk, dv;
};

// Softmax attention (gdn_attn*.cu): causal over a whole prompt (kv_lens null:
// keys = new tokens, row-major with token strides) or over a paged cache.
struct AttnJob;
struct AttnArgs {
  const void *q, *k, *v;       // paged: k, v are the caches
  void *o;
  float *lse;                  // [Ttot][H] or nullptr
  const int32_t *cu;           // [n_seqs + 1] or nullptr (plain batch of T tokens)
  const int32_t *kv_lens;      // [n_seqs], paged only
  const int32_t *table;        // [n_seqs][max_pages], paged only
  int n_seqs, T, Ttot;
  int H, HKV;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  int page_size, max_pages, n_pages;
  int page_log;                // log2 of page_size, or -1
  int max_len;                 // longest length the table can hold
  float scale_log2;            // scale * log2(e)
  // the plan where the host can make it (gdn_attn.cuh): equal prompts;
  // plan_total = 0 otherwise
  uint32_t plan_total, plan_per, plan_seq;
  int plan_shift, plan_grains;
  int plan_whole;              // units are dealt whole
  int plan_coarse;             // log2 of the grain of equal shares
  int plan_least;              // log2 of the smallest other grain
  float4 *part_o;              // partial results (see gdn_attn.cuh); these three are
  float2 *part_ml;             // nullptr when nothing is cut
  AttnJob *jobs;               // [blocks] what is to be joined
  uint32_t *flags;             // device status word, or nullptr
};
// Writes the keys and values of new tokens into the pages of a cache.
struct AppendArgs {
  const void *k, *v;
  void *k_cache, *v_cache;
  const int32_t *cu, *kv_lens, *table;
  int n_seqs, T, Ttot;
  long long k_stride, v_stride;  // bytes between tokens
  int row_bytes;                 // HKV * d elements
  int page_size, max_pages, n_pages, max_len;
  uint32_t *flags;
};

// Status-word bits (same values as GDN_FLAG_* in include/gdn.h).
constexpr uint32_t kFlagPositiveGate = 1u << 0;
constexpr uint32_t kFlagNonfinite = 1u << 1;
constexpr uint32_t kFlagBadSeqlens = 1u << 2;
constexpr uint32_t kFlagTimeout = 1u << 3;
constexpr uint32_t kFlagLaunchConfig = 1u << 4;

// Host-side argument checks of the C entry points.
inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool ranges_overlap(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// Launchers; return cudaErrorInvalidValue for an uncompiled combination.
// dtype: 0 = fp32, 1 = bf16.  gate: 0 = scalar (GDN), 1 = per key (KDA).
cudaError_t launch_prep(const PrepArgs &a, int chunk, int dk, int dtype,
                        int gate, cudaStream_t stream);
cudaError_t launch_scan(const ScanArgs &a, int chunk, int dk, int dtype,
                        int gate, cudaStream_t stream);
// TMA descriptors of the bf16 path's scan: q, k as [Ttot][H][dk] and v as
// [Ttot][HV][dv], boxes of 64 columns x 1 head x C tokens, 128-byte swizzle.
struct ScanMaps {
  CUtensorMap q, k, v;
  CUtensorMap g;  // per-key gates (fp32 [Ttot][HV][dk], box 64 x 1 x chunk); zero otherwise
};
// Encode the maps (host); `g_per_key` null for the scalar gate.  False when
// the driver refuses.
bool make_scan_maps(ScanMaps &m, const void *q, const void *k, const void *v,
                    const float *g_per_key, int Ttot, int H, int HV, int dk, int dv, int chunk);

// bf16 per-key-gate path: prep writing fp16 operand images, tcgen05 scan
// consuming them
cudaError_t launch_prep_tc(const PrepArgs &a, int chunk, int dk, int gate,
                           cudaStream_t stream);
// bf16 per-key-gate prep at chunk 32 (gdn_prep_kda.cu): TMA tiles, the
// factored A / Aqk product on tcgen05; same outputs as launch_prep_tc
cudaError_t launch_prep_kda(const PrepArgs &a, const ScanMaps &maps, int dk, cudaStream_t stream);
cudaError_t launch_scan_tc(const ScanArgs &a, const ScanMaps &maps, int chunk, int dk,
                           int gate, cudaStream_t stream);
// bf16 scalar-gate path: prep on tensor memory writing the lookahead image,
// and the lookahead scan consuming it
// (n_slots >= 0: only the first n_slots chunk slots; ready != nullptr: each
// unit's flag in ready[slot * H + hq] is set once its images are complete)
cudaError_t launch_prep_tmem(const PrepArgs &a, const ScanMaps &maps, int chunk, int dk,
                             cudaStream_t stream, int n_slots = -1, int *ready = nullptr);
cudaError_t launch_scan_la(const ScanArgs &a, const ScanMaps &maps, int chunk, int dk,
                           cudaStream_t stream);
// the same two computations in one cooperative launch, the scan loading each
// prep image once the prep has set its (chunk slot, q/k head) flag in
// `ready` (n_slots x H ints, zeroed beforehand); the prep warpgroups take the
// units from slot `head_slots` on (the earlier ones come from a prep launch
// over the first head_slots slots, enqueued just before; head_slots < 0:
// chosen from the problem's shape);
// cudaErrorCooperativeLaunchTooLarge when the scan's blocks leave no SM for
// the prep
cudaError_t launch_lockstep(const PrepArgs &pa, const ScanArgs &sa, const ScanMaps &maps,
                            int *ready, int head_slots, int chunk, int dk, cudaStream_t stream);
// causal depthwise convolution (width 1..4, D a multiple of 8; activation 0 =
// none, 1 = SiLU) and the row norms (kind 0 = L2, 1 = gated RMS; dim 64, 128
// or 256)
cudaError_t launch_conv1d(const ConvArgs &a, int width, int activation, int dtype,
                          cudaStream_t stream);
cudaError_t launch_rownorm(const RowNormArgs &a, int dim, int kind, int dtype,
                           cudaStream_t stream);
// tensor map of a bf16 array (dims innermost first, strides in bytes from the
// second dimension on), 128-byte swizzle; false when the driver refuses
bool encode_bf16_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims,
                     const uint64_t *strides, const uint32_t *box);
// attention (bf16: tcgen05, gdn_attn_tc.cu; fp32: gdn_attn.cu).  A launch of
// `blocks` blocks; `split`: units may be cut between blocks, which takes the
// merge kernel and, in the workspace, 2 * blocks partial results of `rows`
// rows and a job for each block.
constexpr size_t kAttnJobBytes = 32;  // of an AttnJob
struct AttnLaunch {
  int blocks, rows;  // blocks = 0: more work than the plan can count
  bool split;
};
AttnLaunch attn_launch(AttnArgs &a, int d, int dtype);  // also fills the plan in `a`
cudaError_t launch_attn(const AttnArgs &a, int d, int dtype, const AttnLaunch &l, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnArgs &a, int d, int blocks, cudaStream_t stream);
int sm_count();  // of the current device
// Let `kernel` use `bytes` of dynamic shared memory, once per device (`done`
// has a bit for each of the first 64).
cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done);
cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t stream);
// S_out = M S_in + S_seg, per state
cudaError_t launch_state_combine(const TransferArgs &a, cudaStream_t stream);
// token-serial form; dv a multiple of 32
cudaError_t launch_recurrent(const RecurrentArgs &a, int dk, int dtype, int gate,
                             cudaStream_t stream);

}  // namespace gdn
