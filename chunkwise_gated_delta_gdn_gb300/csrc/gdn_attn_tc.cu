// gdn_attn_tc.cu -- bf16 causal softmax attention on the 5th-generation tensor
// cores, over a whole prompt or over a paged cache.
//
// One block per SM walks the units of its share of the plan (gdn_attn.cuh).
// Two score tiles X = 0, 1 of 128 rows x 128 keys are in flight: while the
// softmax of one runs, the tensor core does the products of the other.
//   S_X = Q_X K^T            both operands from shared memory
//   P_X = e^(scale S_X - m)  bf16, over the columns of S_X in tensor memory
//   O_X += P_X V             A from tensor memory, V key-major as it lies
// A unit of more than 128 rows is two row tiles over the same keys; a unit of
// at most 128 rows (a decode step, a short chunk) is one row tile whose even
// and odd key tiles go to X = 0 and X = 1, joined at its end.
//
// Warps 0-7 and 8-15: softmax of X = 0 and 1, half a row per thread (with a
// whole row per thread and half the warps, two warps to a scheduler did not
// cover one another's latencies: 2045 clocks for both tiles where this takes
// 1470, and the products of both take 2048).  Warp 16: TMA loads into a ring of
// key and value tiles.  Warps 17 and 19: the products of X = 0 and 1.  Warp 18:
// the plan, units published through a small ring.  The loader and the product
// warps go through the same sequence of tiles across units, so the ring stays
// full and the first scores of a unit are computed while the softmax warps write
// out the last one.
//
// What bounds it.  Prompts: the latency of the chain scores - softmax - weights
// - product of each X.  Two tiles of a wide unit take 3300 clocks: the products of
// both 2048 of them, a tile's softmax 1350 (the special functions, 32 results a
// clock, 512 of those), the way through the barriers the rest; a second pair of score tiles, which
// would hide it, does not fit tensor memory beside two outputs of 128 columns.  A
// unit's start and end take 10000 clocks beside its tiles, most of it for the
// 64 KB of its rows to leave the processor.  32768 tokens of 16 heads of 128:
// 2860 to 2990 us, 1470 to 1540 TFLOP/s; four of 2048 tokens, 32 heads: 126 us,
// 1090 TFLOP/s.
// One token per sequence: memory where heads are 128 wide (64 sequences over 8192
// keys 335 us, 6.4 TB/s), the chain of products and barriers, 2000 clocks a tile,
// where they are 64 wide (130 us for 32 sequences, 4.1 TB/s).  A call's start, plan
// and end take about 10 us.
//
// Over a cache in 8 bits (FP8; paged, more than 16 or 32 rows): four warps more turn
// loaded e4m3 tiles, and a unit's queries, into fp16 in place, and the softmax applies the
// scales of 16 keys each; see there.  512 tokens over 32768 keys, 32/8 heads: 264 us where
// keys differ in size, 1.04 PFLOP/s (286 over a bf16 cache of the same values), 252 where
// they do not (226).  What it costs more: turning tiles and fetching scales, as
// instructions beside the softmax and as reads and writes of shared memory, which the
// products read at full rate meanwhile; 16 keys' maxima and factors in the softmax (5 us
// of the 264); and rows that move their maximum, with keys of different sizes in a third of the
// tiles.
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "gdn_attn.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kThreads = 640;
constexpr int kThreads8 = 768;         // over a cache in 8 bits: four warps more
constexpr int kUnits = 4;              // unit ring
constexpr int kPanel = 128 * 128;      // bytes of 128 rows x 64 bf16
constexpr float kRescale = 8.f;        // log2 growth of a row maximum that is let stand
constexpr float kShift8 = 6.f;         // 8 bits: log2 of the weights' factor (fp16, below 2^15)
constexpr float kNone = -0x1p100f;     // 8 bits: a maximum before any visible key; finite

template <int D, bool FP8 = false>
struct Smem {
  static constexpr int kTileBytes = D / 64 * kPanel;  // 128 rows of D
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kRow = kRing + kStages * kTileBytes;  // [X][half][128] floats
  static constexpr int kUnit = kRow + 2 * 2 * 128 * 4;
  static constexpr int kBars = kUnit + kUnits * (int)sizeof(AttnUnit);
  // barriers, in order: Q full, Q empty, S full x2, P ready x2, O full x2,
  // swap x2, halves x8, turn x2, unit full x4, unit empty x4, tile full, tile
  // empty
  // (8 bits: and tile ready, Q ready, scales full)
  static constexpr int kScaleSlots = D == 128 ? 4 : 8;  // see the loads
  static constexpr int kBarCount = (20 + 2 * kUnits + (FP8 ? 3 * kStages + 1 + kScaleSlots : 2 * kStages) + 1) / 2 * 2;
  // tensor memory, abort, [X] stages that the scores free
  static constexpr int kSlot = kBars + kBarCount * 8;
  // 8 bits: scales of key tiles and the log2 of those of the values that go with them
  // [slot][16], Q's powers [two units][row tile][32 rows], and whether a stage has values
  static constexpr int kScale = kSlot + 16, kUp = kScale + kScaleSlots * 64;
  static constexpr int kKind = kUp + 64;
  static constexpr int kBytes = FP8 ? kKind + kStages * 4 : kScale;
  static_assert(kSlot % 16 == 0, "read at once");
};
static_assert(kStaged * sizeof(AttnStaged) + kThreads * sizeof(AttnChunk) <= Smem<128>::kStages * Smem<128>::kTileBytes,
              "staging in the ring");
static_assert(kStaged * sizeof(AttnStaged) + kThreads8 * sizeof(AttnChunk) <= Smem<128, true>::kStages * Smem<128, true>::kTileBytes,
              "staging in the ring");
static_assert(Smem<128, true>::kBytes <= 232448 && Smem<64, true>::kBytes <= 232448, "shared memory of one SM");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// kCols consecutive columns of this thread's lane (no wait)
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&y)[N]) {
  static_assert(N == 32 || N == 16, "");
  if constexpr (N == 32)
    tmem_ld32_nowait(at, reinterpret_cast<uint32_t(&)[32]>(y));
  else
    tmem_ld16_nowait(at, reinterpret_cast<uint32_t(&)[16]>(y));
}

__device__ __forceinline__ uint4 shared_uint4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

struct Maps {
  CUtensorMap q_pack, q, k, v;
};

__device__ __forceinline__ void store_uint4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// two e4m3 values (the low or high half of x) as two fp16
template <bool HIGH>
__device__ __forceinline__ uint32_t f16_of(uint32_t x) {
  uint32_t r;
  if constexpr (HIGH)
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(x));
  else
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// a whole number within 1 of x
__device__ __forceinline__ float whole(float x) { return __fadd_rn(__fadd_rn(x, 0x1.8p23f), -0x1.8p23f); }
// log2 of a scale: exact for powers of two; -191 for zero (of a bad page, whose values are
// zeros)
__device__ __forceinline__ float scale_log2_of(float x) {
  const bool small = x < 0x1p-100f;  // and maybe below the normal numbers
  const uint32_t b = __float_as_uint(small ? x * 0x1p64f : x);
  const float part = __uint_as_float((b & 0x7fffffu) | 0x3f800000u);
  return (float)((int)(b >> 23 & 255) - (small ? 191 : 127)) + (part == 1.f ? 0.f : __log2f(part));
}
__device__ __forceinline__ float two_to(int e) { return __int_as_float((127 + e) << 23); }
__device__ __forceinline__ int shared_int(uint32_t at) {
  int v;
  asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void store_int(uint32_t at, int v) { asm volatile("st.shared.s32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }
// TMA: a box at (x, y, z, w) of a 4-D map, with a policy for the lines in L2
__device__ __forceinline__ void tma_load_4d(uint32_t dst_saddr, const void *tmap, int x, int y, int z, int w, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst_saddr),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&p);
}

// The products, issued by one lane of a converged warp.  The operands' matrix
// descriptors differ between steps in the low word's address field only (16
// bytes a unit), so a step costs an addition: with the descriptors put together
// from scratch for each product the issue took longer than the product itself.
// high word: bytes from one 8-row group to the next
__host__ __device__ constexpr uint32_t desc_hi(int group_bytes) {
  return (uint32_t)(group_bytes >> 4) | (1u << 14) | (2u << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFF) | ((lbo >> 4) << 16);
}
// S = Q K^T over one 64-column panel of each (four K steps of 16)
template <bool FIRST>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi,
                                             uint32_t idesc, bool elected) {
  asm volatile(
      "{\n .reg .pred q, p;\n .reg .b64 da, db;\n .reg .b32 la, lb;\n setp.ne.b32 q, %6, 0;\n setp.ne.b32 p, %7, 0;\n"
      " mov.b64 da, {%1, %3};\n mov.b64 db, {%2, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n"
      " add.u32 la, %1, 2;\n add.u32 lb, %2, 2;\n mov.b64 da, {la, %3};\n mov.b64 db, {lb, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, 1;\n"
      " add.u32 la, %1, 4;\n add.u32 lb, %2, 4;\n mov.b64 da, {la, %3};\n mov.b64 db, {lb, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, 1;\n"
      " add.u32 la, %1, 6;\n add.u32 lb, %2, 6;\n mov.b64 da, {la, %3};\n mov.b64 db, {lb, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, 1;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(desc_hi(1024)), "r"(b_hi), "r"(idesc), "r"((int)elected), "r"(FIRST ? 0 : 1)
      : "memory");
}
// O (+)= P V over 64 keys (four K steps of 16, STEP bytes of V apart)
template <int STEP>
__device__ __forceinline__ void issue_output(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi,
                                             uint32_t idesc, bool accumulate, bool elected) {
  asm volatile(
      "{\n .reg .pred q, p;\n .reg .b64 db;\n .reg .b32 la, lb;\n setp.ne.b32 q, %5, 0;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 db, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n"
      " add.u32 la, %1, 8;\n add.u32 lb, %2, %7;\n mov.b64 db, {lb, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [la], db, %4, 1;\n"
      " add.u32 la, %1, 16;\n add.u32 lb, %2, %8;\n mov.b64 db, {lb, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [la], db, %4, 1;\n"
      " add.u32 la, %1, 24;\n add.u32 lb, %2, %9;\n mov.b64 db, {lb, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [la], db, %4, 1;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"((int)elected), "r"((int)accumulate), "n"(STEP >> 4),
      "n"(2 * STEP >> 4), "n"(3 * STEP >> 4)
      : "memory");
}

// A bounded wait by all lanes of a warp, converged afterwards.  After one that gave
// up (`abort`), the roles go on over whatever there is, within the same bounds, but
// nobody hands a place back to the loader any more, which so comes to its end: a
// place may not be filled while an earlier copy into it is on its way.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort) {
  const bool ok = mbar_wait(bar, parity, abort);
  __syncwarp();
  return ok;
}

struct Bars {
  uint32_t base;
  int stages;
  __device__ uint32_t at(int i) const { return base + i * 8; }
  __device__ uint32_t q_full() const { return at(0); }
  __device__ uint32_t q_empty() const { return at(1); }
  __device__ uint32_t s_full(int x) const { return at(2 + x); }
  __device__ uint32_t p_ready(int x) const { return at(4 + x); }
  __device__ uint32_t o_full(int x) const { return at(6 + x); }
  __device__ uint32_t swap(int i) const { return at(8 + i); }
  __device__ uint32_t halves(int i) const { return at(10 + i); }
  __device__ uint32_t turn(int x) const { return at(18 + x); }
  __device__ uint32_t unit_full(int i) const { return at(20 + i); }
  __device__ uint32_t unit_empty(int i) const { return at(20 + kUnits + i); }
  __device__ uint32_t kv_full(int i) const { return at(20 + 2 * kUnits + i); }
  __device__ uint32_t kv_empty(int i) const { return at(20 + 2 * kUnits + stages + i); }
  // 8 bits: what was loaded is there as fp16
  __device__ uint32_t kv_ready(int i) const { return at(20 + 2 * kUnits + 2 * stages + i); }
  __device__ uint32_t q_ready() const { return at(20 + 2 * kUnits + 3 * stages); }
  __device__ uint32_t scales(int i) const { return at(21 + 2 * kUnits + 3 * stages + i); }
};

// Position in a ring of N: index and how often it has gone round.
template <int N>
struct Ring {
  int i = 0;
  uint32_t round = 0;
  __device__ void step() {
    if (++i == N) {
      i = 0;
      round ^= 1;
    }
  }
};

// The same value in all lanes, known to be so by the compiler: what follows from
// it stays in uniform registers.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// A reader of the unit ring.
struct Units {
  const AttnUnit *ring;
  Bars bars;
  volatile int *abort;
  Ring<kUnits> at;
  // all lanes of a warp; false at the end of the block's work
  __device__ bool next(AttnUnit &u) {
    if (!__all_sync(0xffffffffu, mbar_wait(bars.unit_full(at.i), at.round, abort))) return false;
    u = ring[at.i];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bars.unit_empty(at.i));
    at.step();
    return u.seq >= 0;
  }
};

// N fp32 values of every lane's row as bf16 to columns [c, c + N) of its row
// `out`.  Written as they lie, a 16-byte piece per lane and instruction, every
// instruction touches 32 cache lines, one a clock: 4096 clocks for the 256 rows
// of a wide unit (`many`).  So N / 8 neighbouring lanes exchange pieces first,
// and each instruction writes 2 N byte stretches of rows (between two lanes
// only, packed prompts took 10% longer).  A narrow unit's few rows are written
// as they lie.
template <int N>
__device__ __forceinline__ void store_rows(const float (&y)[N], __nv_bfloat16 *out, bool valid,
                                           bool many, int c) {
  constexpr int kPieces = N / 8;  // 16-byte pieces of a row, and lanes that share them: 2 or 4
  const int lane = threadIdx.x & 31, me = lane & (kPieces - 1);
  uint4 p[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; i++)
    p[i] = make_uint4(pack2(y[8 * i], y[8 * i + 1]), pack2(y[8 * i + 2], y[8 * i + 3]),
                      pack2(y[8 * i + 4], y[8 * i + 5]), pack2(y[8 * i + 6], y[8 * i + 7]));
  if (!many) {
    if (valid)
#pragma unroll
      for (int i = 0; i < kPieces; i++) *reinterpret_cast<uint4 *>(out + c + 8 * i) = p[i];
    return;
  }
  auto swap = [](uint4 &keep, uint4 &give, bool upper, int mask) {
    // a lane keeps one of two pieces and gives the other to its partner
    const uint4 send = upper ? keep : give;
    uint4 got;
    got.x = __shfl_xor_sync(0xffffffffu, send.x, mask);
    got.y = __shfl_xor_sync(0xffffffffu, send.y, mask);
    got.z = __shfl_xor_sync(0xffffffffu, send.z, mask);
    got.w = __shfl_xor_sync(0xffffffffu, send.w, mask);
    if (upper) keep = got; else give = got;
  };
  // transposes the pieces of kPieces rows: afterwards p[i] is piece `me` of the
  // row of the group's lane i
#pragma unroll
  for (int step = 1; step < kPieces; step <<= 1)
#pragma unroll
    for (int i = 0; i < kPieces; i++)
      if (!(i & step)) swap(p[i], p[i | step], (me & step) != 0, step);
  const unsigned long long at = reinterpret_cast<unsigned long long>(out);
#pragma unroll
  for (int i = 0; i < kPieces; i++) {
    const int from = (lane & ~(kPieces - 1)) | i;
    const unsigned long long row = __shfl_sync(0xffffffffu, at, from);
    const bool ok = __shfl_sync(0xffffffffu, valid ? 1 : 0, from);
    if (ok) *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(row) + c + me * 8) = p[i];
  }
}

// FP8: over a cache in 8 bits, one that four warps more turn into fp16 on its way.
template <int D, bool PAGED, bool FP8 = false>
__global__ void __launch_bounds__(FP8 ? kThreads8 : kThreads, 1)
    gdn_attn_tc_kernel(const AttnArgs a, const __grid_constant__ Maps maps, const int box) {
  using SM = Smem<D, FP8>;
  using S = std::conditional_t<FP8, TcShape8, TcShape>;
  constexpr int THREADS = FP8 ? kThreads8 : kThreads;
  constexpr int kPanels = D / 64;
  // A key or value tile in shared memory, 8-row groups of 1024 bytes in the
  // 128-byte swizzle.  A prompt's: 64-column panels one after the other, each
  // one box of its tensor map.  A cache's: the panels of a group next to each
  // other, so that one box brings whole rows of a page (a page of 16 rows in
  // boxes of one panel held the loads at 4.3 TB/s).
  constexpr int kGroup = PAGED ? kPanels * 1024 : 1024;  // bytes from one 8-row group to the next
  constexpr int kPanelAt = PAGED ? 1024 : kPanel;        // and from one panel to the next
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_addr(sm) & 1023u) {
    if (tid == 0 && a.flags) atomicOr(a.flags, kFlagLaunchConfig);
    if (tid == 0 && a.jobs) a.jobs[blockIdx.x].rows = 0;  // the merge kernel reads it
    return;
  }
  const Bars bars{smem_addr(sm + SM::kBars), SM::kStages};
  uint32_t *slot = reinterpret_cast<uint32_t *>(sm + SM::kSlot);
  volatile int *abort = reinterpret_cast<volatile int *>(slot + 1);
  AttnUnit *unit_ring = reinterpret_cast<AttnUnit *>(sm + SM::kUnit);
  float *row_ex = reinterpret_cast<float *>(sm + SM::kRow);
  uint32_t *used = slot + 2;
  if (tid == 0) {
    *abort = 0;
    mbar_init(bars.q_full(), 1);
    mbar_init(bars.q_empty(), 2);
    for (int x = 0; x < 2; x++) {
      mbar_init(bars.s_full(x), 2);  // the products' commit, and the stages they free
      mbar_init(bars.p_ready(x), 8);
      mbar_init(bars.o_full(x), 1);
      mbar_init(bars.swap(x), 16);
      mbar_init(bars.turn(x), 1);
    }
    for (int i = 0; i < 8; i++) mbar_init(bars.halves(i), 2);
    for (int i = 0; i < kUnits; i++) {
      mbar_init(bars.unit_full(i), 1);
      mbar_init(bars.unit_empty(i), FP8 ? 23 : 19);  // loader, products x2, sixteen softmax warps (and those that turn)
    }
    for (int i = 0; i < SM::kStages; i++) {
      mbar_init(bars.kv_full(i), 1);
      if (FP8) mbar_init(bars.kv_ready(i), 4);
      if (FP8 && i == 0) mbar_init(bars.q_ready(), 4);
      if (FP8 && i < SM::kScaleSlots) mbar_init(bars.scales(i), 32);  // the loader's lanes
      mbar_init(bars.kv_empty(i), 2);  // one from each X, or two from the one that reads it
    }
    mbar_fence_init();
  }
  if (warp == 16 && lane < 4)
    prefetch_map(lane == 0 ? &maps.q : lane == 1 ? &maps.k : lane == 2 ? &maps.v : &maps.q_pack);
  if (warp == 17) tmem_alloc(smem_addr(slot), 512);
  AttnStaged *staged = reinterpret_cast<AttnStaged *>(sm + SM::kRing);  // until the first unit
  attn_stage<THREADS, S>(a, staged, blockIdx.x);
  fence_proxy_async();
  asm volatile("griddepcontrol.launch_dependents;");  // the merge kernel waits for this one's end
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *slot;
  const uint32_t sQ = smem_addr(sm + SM::kQ), sRing = smem_addr(sm + SM::kRing);
  const uint32_t tS = tmem, tO = tmem + 256;

  // 768 threads leave 80 registers each: the softmax takes of the others'
  if constexpr (FP8) {
    if (warp < 16) asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    else if (warp < 20) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  }
  if (warp < 16) {
    // ------------------------------------------------------------- softmax
    const int x = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)quarter << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t s_at = tS + x * 128 + half * 64 + lanes, p_at = tS + x * 128 + half * 32 + lanes;
    const uint32_t o_at = tO + x * D + lanes;
    float *own_ex = row_ex + (x * 2 + half) * 128 + r, *other_ex = row_ex + (x * 2 + (half ^ 1)) * 128 + r;
    const uint32_t halves = bars.halves(x * 4 + quarter);
    const float sl2 = a.scale_log2;
    const float grow = kRescale / sl2;
    Units units{unit_ring, bars, abort, {}};
    uint32_t s_phase = 0, o_phase = 0, half_phase = 0, swap_phase[2] = {0, 0};
    auto meet_half = [&] {  // the two warps of these 32 rows
      __syncwarp();
      if (lane == 0) mbar_arrive(halves);
      wait(halves, half_phase, abort);
      half_phase ^= 1;
    };
    auto meet_all = [&](int i) {  // all softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.swap(i));
      wait(bars.swap(i), swap_phase[i], abort);
      swap_phase[i] ^= 1;
    };
    AttnUnit u;
    [[maybe_unused]] int unit_parity = 1, tiles_before = 0;  // key tiles of the units before
    while (units.next(u)) {
      if constexpr (FP8) unit_parity ^= 1;
      const int t0 = uniform(u.t0), t1 = uniform(u.t1), rows = uniform(u.n_tok * u.gp);
      const bool narrow = rows <= 128;
      const bool both = narrow && t1 - t0 > 1;
      const int stride = narrow ? 2 : 1;
      const int row = narrow ? r : x * 128 + r;
      const int tok = row / u.gp;
      const int limit = u.pos0 + min(tok, u.n_tok - 1) - half * 64;  // last visible key, this half's columns
      const int all_see = __reduce_min_sync(0xffffffffu, limit);
      // 8 bits: m is the maximum of log2(weight times V's scale), a whole number, so that
      // the factor between two of them is exact in fp16.  A score is S times 2^-up and K's
      // scale of its block of 16 keys; weights have their block's scale of V in them, as a
      // summand of the exponent.  For l that is taken out again.  l has a maximum of its own,
      // lam, of the scores alone and of this half of the columns: a common one would be
      // one more number to exchange for each tile, so the halves' sums meet at the end.
      float m = FP8 ? kNone : -CUDART_INF_F, l = 0.f;
      [[maybe_unused]] float row_factor = 0.f, lam = kNone;
      const int first = narrow ? t0 + x : t0;
      const bool mine = first < t1;
      // rows past the unit's last one (most of a decode step's tile): their
      // weights are whatever the scores leave, and nobody reads their output
      const bool idle = narrow && quarter * 32 >= rows;
#pragma unroll 1
      for (int t = first; t < t1; t += stride) {
        wait(bars.s_full(x), s_phase, abort);
        s_phase ^= 1;
        fence_after_sync();
        if (half == 0 && quarter == 0 && lane == 0) {
          // These scores, and what this X was given before them, are done: hand
          // back their key tile and the value tile before.
          const uint4 now = shared_uint4(smem_addr(slot));
          if (now.y == 0) {  // or there may not have been scores yet
            const uint32_t stages = x == 0 ? now.z : now.w;
            const int key = stages & 255, value = (int)(stages >> 8) - 1;
            mbar_arrive(bars.kv_empty(key));
            if (value >= 0) mbar_arrive(bars.kv_empty(value));
            if (narrow) {
              mbar_arrive(bars.kv_empty(key));
              if (value >= 0) mbar_arrive(bars.kv_empty(value));
            }
          }
        }
        if (idle) {
          if (lane == 0) mbar_arrive(bars.p_ready(x));
          continue;
        }
        // The weights are e^(s - m) for a maximum m that is moved only when the
        // scores have outgrown it by 2^8: they then stay below 2^8, the sums in
        // fp32 far from overflow, and the output in tensor memory is rarely
        // touched.  So after a unit's first tile the weights are made from the m
        // at hand, while the halves of the rows exchange their maxima, and made
        // again in the rare case that m moves.
        if constexpr (FP8) {
          if (t == first) {
            const int up = shared_int(smem_addr(sm + SM::kUp) + (unit_parity * 8 + (row >> 5)) * 4);
            row_factor = sl2 * two_to(-(up / 2)) * two_to(up / 2 - up);
          }
        }
        // 8 bits: of this half's four blocks, K's scale times the row's factor and V's
        // log2; tile_max is that of the scores with V's scale then, own_max without
        [[maybe_unused]] float xs[4], vs[4], own_max;
        if constexpr (FP8) {
          const uint32_t at = smem_addr(sm + SM::kScale) + ((tiles_before + t - t0) & (SM::kScaleSlots - 1)) * 64 + half * 16;
          const uint4 ks = shared_uint4(at), lb = shared_uint4(at + 32);
          const uint32_t k4[4] = {ks.x, ks.y, ks.z, ks.w}, v4[4] = {lb.x, lb.y, lb.z, lb.w};
#pragma unroll
          for (int b = 0; b < 4; b++) {
            xs[b] = fmaxf(row_factor * __uint_as_float(k4[b]), 1e-37f);  // -inf times it stays that
            vs[b] = __uint_as_float(v4[b]);
          }
        }
        float s[64], tile_max;
        auto load_scores = [&] {
          uint32_t raw[2][32];
          tmem_ld32_nowait(s_at, raw[0]);
          tmem_ld32_nowait(s_at + 32, raw[1]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 64; c++) s[c] = __uint_as_float(raw[c >> 5][c & 31]);
          if (__builtin_expect(t * 128 + 63 > all_see, 0)) {
            const int lim = limit - t * 128;
#pragma unroll
            for (int c = 0; c < 64; c++)
              if (c > lim) s[c] = -CUDART_INF_F;
          }
          if constexpr (FP8) {
            float y[4];
#pragma unroll
            for (int b = 0; b < 4; b++) {
              float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
              for (int c = 0; c < 16; c += 4)
#pragma unroll
                for (int i = 0; i < 2; i++) top[i] = max3(top[i], s[16 * b + c + 2 * i], s[16 * b + c + 2 * i + 1]);
              y[b] = fmaxf(top[0], top[1]) * xs[b];
            }
            own_max = fmaxf(max3(y[0], y[1], y[2]), y[3]);
            tile_max = fmaxf(max3(y[0] + vs[0], y[1] + vs[1], y[2] + vs[2]), y[3] + vs[3]);
          } else {
            float top[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int c = 0; c < 64; c += 8)
#pragma unroll
              for (int i = 0; i < 4; i++) top[i] = max3(top[i], s[c + 2 * i], s[c + 2 * i + 1]);
            tile_max = fmaxf(max3(top[0], top[1], top[2]), top[3]);
          }
          *own_ex = tile_max;
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(halves);
        };
        auto other_half = [&] {
          // Both halves of the scores have been read: past this the weights may
          // be written over them.
          wait(halves, half_phase, abort);
          half_phase ^= 1;
          fence_after_sync();
          tile_max = fmaxf(tile_max, *other_ex);
        };
        if (!FP8 && t == first) {
          load_scores();
          other_half();
          m = tile_max;
          meet_half();  // read, before it is written again
        }
        uint32_t packed[32];
        uint64_t sum[2];
        float f = 1.f;       // 8 bits: of the output, where rows of the warp
        bool moved = false;  // have a new maximum
        while (true) {
          load_scores();
          // 8 bits: where this half of the row alone has outgrown m (in a unit's first tile
          // always), its own maximum is taken, and what that is off by after the exchange
          // is made good by a factor, not by a second pass: with keys of different sizes a
          // third of the tiles has a row that moves (512 tokens over 32768 keys 341 -> 308
          // us).
          float at_hand = m;
          if constexpr (FP8) {
            if (tile_max > m + kRescale) at_hand = whole(tile_max);
            const float next = own_max > lam + kRescale ? whole(own_max) : lam;
            l *= ex2(lam - next);
            lam = next;
            // Where a block's values are so much smaller than others' that its weights, with
            // V's scale, would vanish in 32 bits, they still count for l.  So a weight is
            // made at least 2^-40 of what it is without V's scale (2^-32 where lam lags):
            // zero in fp16, as with it.
#pragma unroll
            for (int b = 0; b < 4; b++) {
              const float off = fminf(at_hand - kShift8 - vs[b], lam + 40.f);
              const uint64_t scale2 = pair(xs[b], xs[b]), off2 = pair(-off, -off);
              uint64_t sums = 0;
#pragma unroll
              for (int c = 16 * b; c < 16 * b + 16; c += 2) {
                float p0, p1;
                unpair(fma2(pair(s[c], s[c + 1]), scale2, off2), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                sums = add2(sums, pair(p0, p1));
                packed[c >> 1] = pack_f16(p0, p1);
              }
              float l0, l1;
              unpair(sums, l0, l1);
              l = fmaf(l0 + l1, ex2(off - lam), l);
            }
          } else {
            const float off = m == -CUDART_INF_F ? 0.f : m * sl2;  // nothing visible yet: weights 0
            const uint64_t scale2 = pair(sl2, sl2), off2 = pair(-off, -off);
            sum[0] = sum[1] = 0;
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              float p0, p1;
              unpair(fma2(pair(s[c], s[c + 1]), scale2, off2), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pair(p0, p1));
              packed[c >> 1] = pack2(p0, p1);
            }
          }
          other_half();
          float top = tile_max;
          const bool move = top > m + (FP8 ? kRescale : grow);
          if constexpr (FP8) top = whole(top);
          if (__builtin_expect(!__any_sync(0xffffffffu, move), 1)) break;
          f = move ? ex2(FP8 ? m - top : (m - top) * sl2) : 1.f;
          if (move) m = top;
          if constexpr (!FP8) l *= f;
          if constexpr (FP8) {
            // a power of two; below 2^-24 in two steps: weights of up to 2^14 times 2^-38
            // still count
            const float e = at_hand == m ? 0.f : fmaxf(at_hand - m, -48.f);
            if (__any_sync(0xffffffffu, e != 0.f)) {
              auto scale_weights = [&](float by) {
                const float g = ex2(by);
                const uint32_t g2 = pack_f16(g, g);
#pragma unroll
                for (int c = 0; c < 32; c++) packed[c] = mul_f16(packed[c], g2);
              };
              scale_weights(fmaxf(e, -24.f));
              if (__any_sync(0xffffffffu, e < -24.f)) scale_weights(fminf(e + 24.f, 0.f));
            }
            moved = t != first;  // before, there is no output
            break;
          } else {
#pragma unroll 1
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
              uint32_t o[16];
              tmem_ld16_nowait(o_at + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16_nowait(o_at + c, o);
            }
            meet_half();
          }
        }
        tmem_st32_nowait(p_at, packed);
        if constexpr (FP8) {
          if (__builtin_expect(moved, 0)) {
#pragma unroll 1
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
              uint32_t o[32];
              tmem_ld32_nowait(o_at + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float y0, y1;
                unpair(mul2(pair(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), pair(f, f)), y0, y1);
                o[i] = __float_as_uint(y0);
                o[i + 1] = __float_as_uint(y1);
              }
              tmem_st32_nowait(o_at + c, o);
            }
          }
        }
        if constexpr (!FP8) {
          float l0, l1;
          unpair(add2(sum[0], sum[1]), l0, l1);
          l += l0 + l1;
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.p_ready(x));
      }
      // ---- the unit's output
      if (mine) {
        wait(bars.o_full(x), o_phase, abort);
        o_phase ^= 1;
        fence_after_sync();
      }
      if constexpr (FP8) {
        tiles_before += t1 - t0;
        // l of both halves relative to the larger lam
        if (mine && !idle) {
          *own_ex = lam;
          meet_half();
          const float top = fmaxf(lam, *other_ex);
          l *= ex2(lam - top);
          lam = top;
          meet_half();  // read, before it is written again
        }
      }
      // m_scaled: log2 of l's unit; `up`: of what the output's unit is more
      float m_scaled = FP8 ? (lam == kNone ? -CUDART_INF_F : lam) : m * sl2, f_own = 1.f, f_other = 0.f;
      [[maybe_unused]] const float up = FP8 ? (lam == kNone ? 0.f : m - kShift8 - lam) : 0.f;
      [[maybe_unused]] bool tiny = false;  // the output's factors are 2^64 too large: they could vanish
      if (both) {
        // Row sums and maxima of both X: the sum of the halves and the maximum
        // in the places of the two halves' tile maxima.  The meeting also says
        // that the other X's output is complete.
        float *place = row_ex + x * 256 + r, *other = row_ex + (x ^ 1) * 256 + r;
        if (!idle) {
          if (half == 1) *own_ex = l;
          meet_half();
          if (half == 0) {
            const float sum = l + *other_ex;
            place[0] = sum;
            place[128] = m_scaled;
          }
        }
        fence_before_sync();
        meet_all(0);
        fence_after_sync();
        const float top = fmaxf(m_scaled, other[128]);
        const float base = top == -CUDART_INF_F ? 0.f : top;
        f_own = ex2(m_scaled - base);
        f_other = ex2(other[128] - base);
        l = f_own * place[0] + f_other * other[0];
        if constexpr (FP8) {  // and the output's units
          meet_all(1);  // read, before it is written again
          if (half == 0 && !idle) place[0] = up;
          meet_all(0);
          const float own = m_scaled - base + up, others = other[128] - base + other[0];
          tiny = fmaxf(own, others) < -64.f;
          f_own = ex2(own + (tiny ? 64.f : 0.f));
          f_other = ex2(others + (tiny ? 64.f : 0.f));
        }
        m_scaled = top;
      } else if (mine && !idle) {
        *own_ex = l;
        meet_half();
        l += *other_ex;
        meet_half();  // read, before the next tile's maximum is written
        if constexpr (FP8) {
          tiny = up < -64.f;
          f_own = ex2(up + (tiny ? 64.f : 0.f));
        }
      }
      if (mine && !idle) {
        const bool valid = tok < u.n_tok;
        const bool part = u.slot >= 0;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const long long at = (long long)(u.row0 + tok) * a.H + u.head0 + row % u.gp;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.o) + at * D;
        bool finite = true;
        // each half writes half of the columns; of a joined output, each X half of those
        constexpr int kCols = D / 4;
        const int c0 = both ? (half * 2 + x) * kCols : half * 2 * kCols;
        const int c1 = both ? c0 + kCols : c0 + 2 * kCols;
#pragma unroll 1
        for (int c = c0; c < c1; c += kCols) {
          float y[kCols];
          tmem_ld<kCols>(o_at + c, y);
          tmem_wait_ld();
          if (both) {
            float other[kCols];
            tmem_ld<kCols>(tO + (x ^ 1) * D + lanes + c, other);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kCols; i++) y[i] = f_own * y[i] + f_other * other[i];
          } else if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < kCols; i++) y[i] *= f_own;
          }
          if (FP8 && tiny) {
#pragma unroll
            for (int i = 0; i < kCols; i++) y[i] *= 0x1p-64f;
          }
          if (valid && part) {
#pragma unroll
            for (int i = 0; i < kCols / 4; i++)
              a.part_o[((long long)u.slot * (D / 4) + (c >> 2) + i) * TcShape::kRows + row] =
                  make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
          if (!part) {
#pragma unroll
            for (int i = 0; i < kCols; i++) y[i] *= inv;
            if (a.flags && valid) {
#pragma unroll
              for (int i = 0; i < kCols; i++) finite &= fabsf(y[i]) < kBf16Inf;
            }
            store_rows<kCols>(y, out, valid, !narrow, c);
          }
          __syncwarp();
        }
        if (valid && half == 0 && (!both || x == 0)) {
          if (part)
            a.part_ml[(long long)u.slot * TcShape::kRows + row] = make_float2(m_scaled, l);
          else if (a.lse)
            a.lse[at] = l == 0.f ? -CUDART_INF_F : (m_scaled + __log2f(l)) * 0.69314718056f;
        }
        if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
      }
      if (both) {  // the other X's output and maxima have been read: they may be overwritten
        fence_before_sync();
        meet_all(1);
        fence_after_sync();
      }
    }
  } else {
    if (FP8 && warp >= 20) {
      // ------------------------------------------------------ 8 bits to fp16
      // Operands are fp16 here: an e4m3 value is exact in it, without its scale (the
      // softmax has those: relative to one for the whole tile, values of small blocks
      // lost bits beside larger ones, those of later tokens among them); 32 rows
      // of Q are scaled by a power of two into the middle of its range, which leaves a
      // score's error below 2^-39 of the largest one's products.  (bf16 takes more
      // instructions for two values.)
      // A warp has 32 rows of every tile, and turns them where they lie: they were
      // loaded into the second half of the place that they take as fp16, so eight rows
      // after the other never overwrite what all lanes have not read.  Lanes 0-7 have 8
      // rows of one 16-byte piece (16 columns), whose 16-byte pieces of fp16 lie in
      // different banks.
      constexpr int kRegion = SM::kTileBytes / 4, kPieces = D / 16;
      const int w = warp - 20, r = lane & 7, j0 = lane >> 3;
      Units units{unit_ring, bars, abort, {}};
      Ring<SM::kStages> ring;
      uint32_t n_keys = 0;  // tiles so far
      uint32_t q_phase = 0;
      int unit_parity = 1;
      AttnUnit u;
      while (units.next(u)) {
        const int tiles = uniform(2 * (u.t1 - u.t0));  // keys and values; the order is the loader's
        const int rows = uniform(u.n_tok * u.gp);
        unit_parity ^= 1;
        wait(bars.q_full(), q_phase, abort);
        q_phase ^= 1;
        // Q: this warp's 32 rows of each row tile, four at a time, 8 lanes to a row.  Rows of
        // the next sequence, and of tokens that see no key, do not count for the power.
        const int blind = uniform(min(max(-u.pos0, 0), u.n_tok) * u.gp);
        for (int r0 = w * 32; r0 < rows; r0 += 128) {
          const uint32_t at = sQ + (r0 >> 7) * SM::kTileBytes + (w * 32 + (lane >> 3)) * 128 + (lane & 7) * 16;
          const int steps = min((rows - r0 + 3) >> 2, 8);
          uint32_t top = 0;
          bool odd = false;  // something is not finite
          auto look = [&](bool all) {
            top = 0;
#pragma unroll 1
            for (int i = 0; i < steps; i++)
#pragma unroll
              for (int p = 0; p < kPanels; p++) {
                const uint4 x = shared_uint4(at + i * 512 + p * kPanel);
                const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                const uint32_t keep = (unsigned)(r0 + i * 4 + (lane >> 3) - blind) < (unsigned)(rows - blind) ? 0x7fffu : 0u;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                  const uint32_t lo = in[c] & keep, hi = in[c] >> 16 & keep;
                  top = max(top, max(all || lo < 0x7f80u ? lo : 0u, all || hi < 0x7f80u ? hi : 0u));
                }
              }
            top = __reduce_max_sync(0xffffffffu, top);
            odd = top >= 0x7f80u;
          };
          look(true);
          if (odd) look(false);  // a row's infinity is its own
          // 2^up brings the largest element to [2^14, 2^15)
          const int up = top == 0 ? 0 : 14 - ((int)(top >> 7) - 127);
          const float f1 = two_to(up / 2), f2 = two_to(up - up / 2);
#pragma unroll 1
          for (int i = 0; i < steps; i++)
#pragma unroll
            for (int p = 0; p < kPanels; p++) {
              const uint4 x = shared_uint4(at + i * 512 + p * kPanel);
              const uint32_t in[4] = {x.x, x.y, x.z, x.w};
              uint32_t out[4];
#pragma unroll
              for (int c = 0; c < 4; c++)
                out[c] = pack_f16(__uint_as_float(in[c] << 16) * f1 * f2, __uint_as_float(in[c] & 0xffff0000u) * f1 * f2);
              store_uint4(at + i * 512 + p * kPanel, out[0], out[1], out[2], out[3]);
            }
          if (lane == 0) store_int(smem_addr(sm + SM::kUp) + (unit_parity * 8 + (r0 >> 5)) * 4, up);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.q_ready());
        for (int i = 0; i < tiles; i++) {
          wait(bars.kv_full(ring.i), ring.round, abort);
          const uint32_t region = sRing + ring.i * SM::kTileBytes + w * kRegion, raw = region + kRegion / 2;
          if (w == 0 && shared_int(smem_addr(sm + SM::kKind) + ring.i * 4) == 0) {
            // keys: their scales, and those of the values that go with them as log2
            const int slot_i = n_keys & (SM::kScaleSlots - 1);
            const uint32_t at = smem_addr(sm + SM::kScale) + (slot_i * 16 + (lane & 15)) * 4;
            wait(bars.scales(slot_i), n_keys / SM::kScaleSlots & 1, abort);
            n_keys++;
            const float b = __int_as_float(shared_int(at));
            if (lane < 16) store_int(at, __float_as_int(lane < 8 ? b : scale_log2_of(b)));
            __syncwarp();
          }
          auto read = [&](int group, int j) {
            const int row = group * 8 + r;
            return shared_uint4(raw + row * D + ((D == 128 ? j ^ r : j ^ ((r >> 1) & 3)) << 4));
          };
          auto write = [&](int group, int j, const uint4 &x) {
            const uint32_t to = region + group * kGroup + (j >> 2) * 1024 + r * 128;
            const int c0 = (2 * j) & 7;
            store_uint4(to + ((c0 ^ r) << 4), f16_of<false>(x.x), f16_of<true>(x.x), f16_of<false>(x.y), f16_of<true>(x.y));
            store_uint4(to + (((c0 + 1) ^ r) << 4), f16_of<false>(x.z), f16_of<true>(x.z), f16_of<false>(x.w), f16_of<true>(x.w));
          };
          // one after the other: unrolled, with more reads on their way at once, these warps were
          // in the softmax's way (512 tokens over 32768 keys 277 us for 259)
#pragma unroll 1
          for (int g = 0; g < 4; g++) {
            uint4 x[kPieces / 4];
#pragma unroll
            for (int p = 0; p < kPieces / 4; p++) x[p] = read(g, p * 4 + j0);
            __syncwarp();
#pragma unroll
            for (int p = 0; p < kPieces / 4; p++) write(g, p * 4 + j0, x[p]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.kv_ready(ring.i));
          ring.step();
        }
      }
    } else if (warp == 18) {
      // -------------------------------------------------------------- plan
      AttnPlan<S> plan(a.H, a.HKV, a.plan_coarse, a.plan_least);
      const AttnStart st = attn_start(a, plan, staged, blockIdx.x, gridDim.x);
      fence_proxy_async();  // what was staged has been read: the ring may be filled
      __syncwarp();
      AttnWalk<S> walk(a, plan, st, blockIdx.x, gridDim.x);
      Ring<kUnits> at;
      AttnUnit u;
      bool more = true;
      if (a.jobs && lane == 0) a.jobs[blockIdx.x].rows = 0;
      while (more) {
        more = walk.next(u);
        if (more && u.slot >= 0 && !a.jobs) {  // a cut unit has no place: never by the plan
          if (lane == 0 && a.flags) atomicOr(a.flags, kFlagLaunchConfig);
          continue;
        }
        if (!more) u.seq = -1;
        else if (lane == 0 && u.slot == 2 * (int)blockIdx.x + 1) a.jobs[blockIdx.x] = attn_job(u);
        if (!__all_sync(0xffffffffu, mbar_wait(bars.unit_empty(at.i), at.round ^ 1, abort))) break;
        if (lane == 0) {
          unit_ring[at.i] = u;
          mbar_arrive(bars.unit_full(at.i));
        }
        __syncwarp();
        at.step();
      }
    } else if (warp == 16) {
      // ------------------------------------------------------------- loads
      // The order of the tiles is that of the products below; a unit's last
      // tiles go in the order of the keys.
      Units units{unit_ring, bars, abort, {}};
      Ring<SM::kStages> ring;
      uint32_t q_phase = 1;
      AttnUnit u, old;         // this unit, and the one whose last values are still to come
      int left[2] = {-1, -1};  // its last tiles
      bool shared = false;     // one value tile for both X
      bool lost = false;       // a wait of this lane gave up: it loads nothing any more
      auto place = [&](uint32_t bar, uint32_t parity) {
        lost |= !mbar_wait(bar, parity, abort);
        __syncwarp();
      };
      // Page numbers of 32 pages in a row, a lane each, for the key tiles and
      // for the value tiles that follow them: read once in 32 pages, not once
      // per tile, where their latency held the loads at 2700 clocks a tile.
      // A decode step reads a cache once: its keys and values make room for one
      // another in L2, not in place of what others need (this kernel's code for
      // the next call among it).
      const uint64_t once = l2_evict_first(), often = l2_evict_normal();
      struct Window {
        int seq, base, page;
      } win[2] = {{-1, 0, 0}, {-1, 0, 0}};
      const int groups = a.page_size >> 3, my_key = lane * box;  // 8-row groups of a page
      [[maybe_unused]] int scale_slot = 0;
      auto page_of = [&](int key) {
        return a.page_log >= 0 ? key >> a.page_log : key / a.page_size;
      };
      // one tile of keys (which = 0) or values (1) of unit w into the next stage
      auto load = [&](const AttnUnit &w, int tile, int which) {
        const CUtensorMap *map = which ? &maps.v : &maps.k;
        const uint32_t full = bars.kv_full(ring.i), dst = sRing + ring.i * SM::kTileBytes;
        const int key = tile * 128;
        if constexpr (PAGED) {
          // lane i takes the i-th box of `box` keys; boxes past the last key
          // are not loaded (what they leave in shared memory is masked)
          Window &pages = win[which];
          const int last = w.len - 1, k0 = min(key + my_key, last);
          const int lo = page_of(key), index = page_of(k0);
          if (key <= last && (pages.seq != w.seq || lo < pages.base || lo + 8 >= pages.base + 32)) {
            pages.seq = w.seq;
            pages.base = lo;
            pages.page = __ldg(a.table + (long long)w.seq * a.max_pages + min(lo + lane, page_of(last)));
          }
          const int held = __shfl_sync(0xffffffffu, pages.page, (index - pages.base) & 31);
          const bool mine = key + my_key <= last && my_key < 128;
          const bool good = (unsigned)held < (unsigned)a.n_pages;
          if (mine && !good && a.flags) atomicOr(a.flags, kFlagBadSeqlens);
          // a bad page reads as zeros: the box just past the cache
          const int group = (good ? held : a.n_pages) * groups + ((k0 - index * a.page_size) >> 3);
          const int n = min((last - key + box) / box, 128 / box);  // boxes; may be <= 0
          place(bars.kv_empty(ring.i), ring.round ^ 1);
          if constexpr (FP8) {
            if (lane == 0 && !lost) {
              store_int(smem_addr(sm + SM::kKind) + ring.i * 4, which);
              mbar_arrive_expect_tx(full, max(n, 0) * box * D);
            }
            __syncwarp();
            // into the second half of what 32 rows take as fp16
            if (mine && !lost)
              tma_load_4d(dst + (my_key >> 5) * (SM::kTileBytes / 4) + SM::kTileBytes / 8 + (my_key & 31) * D, map, 0, 0, group,
                          w.kvh, full, w.n_tok * w.gp <= 128 ? once : often);
            // With a key tile come its scales (lanes 0-7) and those of its values (8-15),
            // which follow in the same order: zero in a bad page and past the last key.  The
            // softmax has read a slot before its next filling: that is for a key tile at least
            // as many stages behind the values, whose products wait for their weights.
            if (which == 0) {
              const int k1 = min(key + (lane & 7) * kScaleBlock, last), page1 = page_of(max(k1, 0));
              const int from = __shfl_sync(0xffffffffu, pages.page, (page1 - pages.base) & 31);
              const bool there = key + (lane & 7) * kScaleBlock <= last && (unsigned)from < (unsigned)a.n_pages;
              if (lane < 16 && !lost)
                cp_async4(smem_addr(sm + SM::kScale) + (scale_slot * 16 + lane) * 4,
                          (lane >= 8 ? a.v_scale : a.k_scale) +
                              (there ? ((long long)from * (a.page_size / kScaleBlock) + (k1 - page1 * a.page_size) / kScaleBlock) * a.HKV + w.kvh : 0),
                          there ? 4 : 0);
              if (!lost) cp_async_arrive_noinc(bars.scales(scale_slot));
              scale_slot = (scale_slot + 1) % SM::kScaleSlots;
            }
            __syncwarp();
            ring.step();
            return;
          }
          if (lane == 0 && !lost) mbar_arrive_expect_tx(full, max(n, 0) * box * 128 * kPanels);
          __syncwarp();
          if (mine && !lost)
            tma_load_5d(dst + my_key * 128 * kPanels, map, 0, 0, 0, group, w.kvh, full,
                        w.n_tok * w.gp <= 128 ? once : often);
        } else {
          place(bars.kv_empty(ring.i), ring.round ^ 1);
          if (lane == 0 && !lost) {
            mbar_arrive_expect_tx(full, SM::kTileBytes);
            const int row = w.row0 - w.pos0 + key;  // a prompt's keys are its own tokens
#pragma unroll
            for (int p = 0; p < kPanels; p++)
              tma_load_3d(dst + p * kPanel, map, p * 64, w.kvh, row, full);
          }
          __syncwarp();
        }
        ring.step();
      };
      auto last_values = [&](int x) {
        if (left[x] >= 0 && !(shared && x == 1)) load(old, left[x], 1);
        left[x] = -1;
      };
      while (units.next(u)) {
        const bool narrow = u.n_tok * u.gp <= 128;
        if (left[1] < left[0]) last_values(1);
        last_values(0);
        place(bars.q_empty(), q_phase);
        q_phase ^= 1;
        if (lane == 0 && !lost) {
          const bool whole = u.gp == a.H / a.HKV;  // all heads of a key/value head
          const int toks = 128 / u.gp, tiles = narrow ? 1 : 2;
          mbar_arrive_expect_tx(bars.q_full(), tiles * kPanels * toks * u.gp * 128);
          for (int i = 0; i < tiles; i++)
#pragma unroll
            for (int p = 0; p < kPanels; p++)
              tma_load_3d(sQ + i * SM::kTileBytes + p * kPanel, whole ? &maps.q_pack : &maps.q, p * 64,
                          u.head0, u.row0 + i * toks, bars.q_full());
        }
        __syncwarp();
        load(u, u.t0, 0);
        last_values(1);
        if (narrow) {
          if (u.t0 + 1 < u.t1) load(u, u.t0 + 1, 0);
          for (int t = u.t0 + 2; t < u.t1; t++) {
            load(u, t - 2, 1);
            load(u, t, 0);
          }
          const int odd = (u.t1 - 1 - u.t0) & 1;  // which X has the last tile
          left[0] = u.t1 - 1 - odd;
          left[1] = u.t0 + 1 < u.t1 ? u.t1 - 2 + odd : -1;
        } else {
          for (int t = u.t0; t + 1 < u.t1; t++) {
            load(u, t, 1);
            load(u, t + 1, 0);
          }
          left[0] = left[1] = u.t1 - 1;
        }
        shared = !narrow;
        old = u;
      }
      if (left[1] < left[0]) last_values(1);
      last_values(0);
      last_values(1);
    } else {
      // ---------------------------------------------------------- products
      // A warp for each X: S(0), O(0), S(1), O(1), ...; scores overwrite weights,
      // so S(i + 1) is issued behind O(i), and the tensor core runs what it is
      // given in order.  Issuing blocks while the tensor core's queue is full,
      // which is short: one warp for both X left it idle for 270 clocks around
      // each product while it waited and prepared the next.  In a wide unit the
      // warps take turns, each ready to issue when its turn comes: without turns
      // the two X's products mix and their softmaxes fall together (a
      // 32768-token prompt 4.13 ms, with one warp 3.10 ms).
      const int x = warp == 17 ? 0 : 1;
      constexpr uint32_t kIdS = FP8 ? idesc_f16(128, 128, 0, 0) : idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t kIdO = FP8 ? idesc_f16(128, D, 0, 1) : idesc_bf16(128, D, 0, 1);
      Units units{unit_ring, bars, abort, {}};
      Ring<SM::kStages> ring;
      uint32_t q_phase = 0, p_phase = 0, turn = 0;
      AttnUnit u;
      // last tiles of the unit before, their values still to be used; `shared`:
      // one tile for both X
      int left0 = -1, left1 = -1, old_len = 0;
      bool shared = false, more = false;  // more: O has been written before
      // The next tile of the ring, once it is there.  Also the other X's tiles
      // are waited for: a wait tells two fillings of a stage apart by parity
      // only, and would take the one before last for the one it wants if the
      // last one had not arrived yet.
      auto next_tile = [&] {
        const int stage = ring.i;
        wait(FP8 ? bars.kv_ready(stage) : bars.kv_full(stage), ring.round, abort);
        ring.step();
        return stage;
      };
      auto clear_values = [&](int stage, int tile, int len) {
        // weights past the last key are zero, but 0 * NaN is not: clear the
        // value rows that belong to nobody (both X do, where they share a tile)
        const int rows = len - tile * 128;
        if (rows < 128) {
          unsigned char *tile_at = sm + SM::kRing + stage * SM::kTileBytes;
          for (int i = max(rows, 0) * 8 + lane; i < 128 * 8; i += 32) {
            const int row = i >> 3;
#pragma unroll
            for (int p = 0; p < kPanels; p++)
              *reinterpret_cast<uint4 *>(tile_at + (row >> 3) * kGroup + p * kPanelAt + (row & 7) * 128 +
                                         (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
        }
      };
      // S from key tile k; the softmax hands back k and value tile free_v (a
      // stage, or -1) when it sees the scores.  (A commit for each stage would
      // cost the tensor pipe 40 to 120 clocks: it does not start the next product
      // before the committed ones are through.)
      auto scores = [&](int k, int q_tile, int free_v) {
        const uint32_t q_lo = desc_lo(sQ + q_tile * SM::kTileBytes, 16);
        const uint32_t k_lo = desc_lo(sRing + k * SM::kTileBytes, 16);
        fence_after_sync();
        issue_scores<true>(tS + x * 128, q_lo, k_lo, desc_hi(kGroup), kIdS, lane == 0);
        if (D == 128)
          issue_scores<false>(tS + x * 128, q_lo + (kPanel >> 4), k_lo + (kPanelAt >> 4), desc_hi(kGroup),
                              kIdS, lane == 0);
        if (lane == 0) {
          mma_commit(bars.s_full(x));
          used[x] = k | (free_v + 1) << 8;
          mbar_arrive(bars.s_full(x));
        }
      };
      auto weights_ready = [&] {
        wait(bars.p_ready(x), p_phase, abort);
        p_phase ^= 1;
        fence_after_sync();
      };
      auto output = [&](int stage, bool accumulate) {
        const uint32_t v_lo = desc_lo(sRing + stage * SM::kTileBytes, kPanelAt);
        issue_output<2 * kGroup>(tO + x * D, tS + x * 128, v_lo, desc_hi(kGroup), kIdO, accumulate,
                                 lane == 0);
        issue_output<2 * kGroup>(tO + x * D, tS + x * 128 + 32, v_lo + (8 * kGroup >> 4), desc_hi(kGroup),
                                 kIdO, true, lane == 0);
      };
      auto last_output = [&](int v, int tile) {
        clear_values(v, tile, old_len);
        weights_ready();
        output(v, more);
        if (lane == 0) {
          if (!*abort) {
            mma_commit(bars.kv_empty(v));  // each stage waits for two arrivals
            if (!shared) mma_commit(bars.kv_empty(v));
          }
          mma_commit(bars.o_full(x));
        }
        __syncwarp();
      };
      // the last values up to those of X = 0, in the loader's order
      auto last_values = [&] {
        if (left1 >= 0 && left1 < left0) {
          const int v = next_tile();
          if (x == 1) last_output(v, left1);
          left1 = -1;
        }
        if (left0 >= 0) {
          const int v = next_tile();
          if (x == 0 || shared) last_output(v, left0);
          if (shared) left1 = -1;
          left0 = -1;
        }
      };
      auto last_values_1 = [&] {
        if (left1 < 0) return;
        const int v = next_tile();
        if (x == 1) last_output(v, left1);
        left1 = -1;
      };
      while (units.next(u)) {
        const int t0 = uniform(u.t0), t1 = uniform(u.t1), len = uniform(u.len);
        const bool narrow = uniform(u.n_tok * u.gp) <= 128;
        last_values();
        const int k = next_tile();
        wait(FP8 ? bars.q_ready() : bars.q_full(), q_phase, abort);
        q_phase ^= 1;
        if (x == 0) scores(k, 0, -1);
        last_values_1();
        if (narrow) {
          if (t0 + 1 < t1) {
            const int k1 = next_tile();
            if (x == 1) scores(k1, 0, -1);
          }
          for (int t = t0 + 2; t < t1; t++) {
            const int v = next_tile(), k_next = next_tile();
            if (((t - t0) & 1) != x) continue;
            clear_values(v, t - 2, len);
            weights_ready();
            output(v, t >= t0 + 4);
            scores(k_next, 0, v);
          }
          const int odd = (t1 - 1 - t0) & 1;  // which X has the last tile
          left0 = t1 - 1 - odd;
          left1 = t0 + 1 < t1 ? t1 - 2 + odd : -1;
          more = t0 + 2 + x < t1;
        } else {
          if (x == 1) scores(k, 1, -1);
          for (int t = t0; t + 1 < t1; t++) {
            const int v = next_tile(), k_next = next_tile();
            clear_values(v, t, len);
            weights_ready();
            wait(bars.turn(x), turn ^ (x == 0 ? 1 : 0), abort);
            turn ^= 1;
            output(v, t > t0);
            scores(k_next, x, v);
            if (lane == 0) mbar_arrive(bars.turn(x ^ 1));
          }
          left0 = left1 = t1 - 1;
          more = t0 + 1 < t1;
        }
        // behind the last scores: the queries may be replaced
        if (lane == 0 && !*abort) {
          if (x == 0 || !narrow || t0 + 1 < t1) mma_commit(bars.q_empty());
          else mbar_arrive(bars.q_empty());
        }
        __syncwarp();
        shared = !narrow;
        old_len = len;
      }
      last_values();
      last_values_1();
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (*abort) {
    // a wait gave up, and no warp issues anything any more: let copies and products
    // still in flight land before the shared and tensor memory are released
    // (bounded, about 10 ms)
    if (tid == 0 && a.flags) atomicOr(a.flags, kFlagTimeout);
    const long long t0 = clock64();
    while (clock64() - t0 < 20000000LL) {
    }
    __syncwarp();
  }
  if (warp == 17) tmem_dealloc(tmem, 512);
}

bool make_maps(Maps &m, const AttnArgs &a, int d, int box, bool fp8) {
  const AttnPlan<TcShape> plan(a.H, a.HKV, 0);
  const uint64_t D = d;
  const uint64_t q_dims[3] = {D, (uint64_t)a.H, (uint64_t)a.Ttot};
  const uint64_t q_strides[2] = {D * 2, (uint64_t)a.q_stride * 2};
  const uint32_t q_box[3] = {64, (uint32_t)plan.gp, (uint32_t)(128 / plan.gp)};
  if (!encode_bf16_map(&m.q, a.q, 3, q_dims, q_strides, q_box)) return false;
  m.q_pack = m.q;
  if (plan.G != plan.gp && plan.G <= 128) {
    const uint32_t pack_box[3] = {64, (uint32_t)plan.G, (uint32_t)(128 / plan.G)};
    if (!encode_bf16_map(&m.q_pack, a.q, 3, q_dims, q_strides, pack_box)) return false;
  }
  if (fp8) {  // [columns][8 rows][8-row group of all pages][head]
    const uint64_t row = (uint64_t)a.HKV * D;
    const uint64_t dims[4] = {D, 8, (uint64_t)a.n_pages * (a.page_size / 8), (uint64_t)a.HKV};
    const uint64_t strides[3] = {row, row * 8, D};
    const uint32_t kv_box[4] = {(uint32_t)D, 8, (uint32_t)box / 8, 1};
    return encode_byte_map(&m.k, a.k, 4, dims, strides, kv_box, d) && encode_byte_map(&m.v, a.v, 4, dims, strides, kv_box, d);
  }
  if (a.table) {  // [64 columns][8 rows][panel][8-row group of all pages][head]
    const uint64_t row = (uint64_t)a.HKV * D * 2;
    const uint64_t dims[5] = {64, 8, D / 64, (uint64_t)a.n_pages * (a.page_size / 8), (uint64_t)a.HKV};
    const uint64_t strides[4] = {row, 128, row * 8, D * 2};
    const uint32_t kv_box[5] = {64, 8, (uint32_t)(D / 64), (uint32_t)box / 8, 1};
    return encode_bf16_map(&m.k, a.k, 5, dims, strides, kv_box) &&
           encode_bf16_map(&m.v, a.v, 5, dims, strides, kv_box);
  }
  const uint32_t kv_box[3] = {64, 1, 128};
  const uint64_t dims[3] = {D, (uint64_t)a.HKV, (uint64_t)a.Ttot};
  const uint64_t ks[2] = {D * 2, (uint64_t)a.k_stride * 2}, vs[2] = {D * 2, (uint64_t)a.v_stride * 2};
  return encode_bf16_map(&m.k, a.k, 3, dims, ks, kv_box) &&
         encode_bf16_map(&m.v, a.v, 3, dims, vs, kv_box);
}

template <int D, bool PAGED, bool FP8>
std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use its shared memory

template <int D, bool PAGED, bool FP8 = false>
cudaError_t launch(const AttnArgs &a, const Maps &maps, int box, int blocks, cudaStream_t stream) {
  constexpr int kBytes = Smem<D, FP8>::kBytes;
  const cudaError_t e = allow_smem(reinterpret_cast<const void *>(&gdn_attn_tc_kernel<D, PAGED, FP8>), kBytes,
                                   allowed<D, PAGED, FP8>);
  if (e != cudaSuccess) return e;
  gdn_attn_tc_kernel<D, PAGED, FP8><<<blocks, FP8 ? kThreads8 : kThreads, kBytes, stream>>>(a, maps, box);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, int d, int blocks, cudaStream_t stream) {
  int box = 128;
  if (a.table && (a.page_size & -a.page_size) < box) box = a.page_size & -a.page_size;
  Maps maps;
  if (!make_maps(maps, a, d, box, false)) return cudaErrorInvalidValue;
  if (d == 64)
    return a.table ? launch<64, true>(a, maps, box, blocks, stream)
                   : launch<64, false>(a, maps, box, blocks, stream);
  return a.table ? launch<128, true>(a, maps, box, blocks, stream)
                 : launch<128, false>(a, maps, box, blocks, stream);
}

cudaError_t launch_attn8_tc(const AttnArgs &a, int d, int blocks, cudaStream_t stream) {
  // rows of one warp's share of a tile at most: they are turned to fp16 in place
  const int box = (a.page_size & -a.page_size) < 32 ? a.page_size & -a.page_size : 32;
  Maps maps;
  if (!make_maps(maps, a, d, box, true)) return cudaErrorInvalidValue;
  return d == 64 ? launch<64, true, true>(a, maps, box, blocks, stream) : launch<128, true, true>(a, maps, box, blocks, stream);
}

}  // namespace gdn
