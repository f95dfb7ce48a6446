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
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "gdn_attn.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kThreads = 640;
constexpr int kUnits = 4;              // unit ring
constexpr int kPanel = 128 * 128;      // bytes of 128 rows x 64 bf16
constexpr float kRescale = 8.f;        // log2 growth of a row maximum that is let stand

template <int D>
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
  static constexpr int kBarCount = 20 + 2 * kUnits + 2 * kStages;
  // tensor memory, abort, [X] stages that the scores free
  static constexpr int kSlot = kBars + kBarCount * 8;
  static constexpr int kBytes = kSlot + 16;
  static_assert(kSlot % 16 == 0, "read at once");
};
static_assert(kStaged * sizeof(AttnStaged) + kThreads * sizeof(AttnChunk) <= Smem<128>::kStages * Smem<128>::kTileBytes,
              "staging in the ring");
static_assert(Smem<128>::kBytes <= 232448 && Smem<64>::kBytes <= 232448, "shared memory of one SM");

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

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    gdn_attn_tc_kernel(const AttnArgs a, const __grid_constant__ Maps maps, const int box) {
  using SM = Smem<D>;
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
      mbar_init(bars.unit_empty(i), 19);  // loader, products x2, sixteen softmax warps
    }
    for (int i = 0; i < SM::kStages; i++) {
      mbar_init(bars.kv_full(i), 1);
      mbar_init(bars.kv_empty(i), 2);  // one from each X, or two from the one that reads it
    }
    mbar_fence_init();
  }
  if (warp == 16 && lane < 4)
    prefetch_map(lane == 0 ? &maps.q : lane == 1 ? &maps.k : lane == 2 ? &maps.v : &maps.q_pack);
  if (warp == 17) tmem_alloc(smem_addr(slot), 512);
  AttnStaged *staged = reinterpret_cast<AttnStaged *>(sm + SM::kRing);  // until the first unit
  attn_stage<kThreads>(a, staged, blockIdx.x);
  fence_proxy_async();
  asm volatile("griddepcontrol.launch_dependents;");  // the merge kernel waits for this one's end
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *slot;
  const uint32_t sQ = smem_addr(sm + SM::kQ), sRing = smem_addr(sm + SM::kRing);
  const uint32_t tS = tmem, tO = tmem + 256;

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
    while (units.next(u)) {
      const int t0 = uniform(u.t0), t1 = uniform(u.t1), rows = uniform(u.n_tok * u.gp);
      const bool narrow = rows <= 128;
      const bool both = narrow && t1 - t0 > 1;
      const int stride = narrow ? 2 : 1;
      const int row = narrow ? r : x * 128 + r;
      const int tok = row / u.gp;
      const int limit = u.pos0 + min(tok, u.n_tok - 1) - half * 64;  // last visible key, this half's columns
      const int all_see = __reduce_min_sync(0xffffffffu, limit);
      float m = -CUDART_INF_F, l = 0.f;
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
          float top[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int c = 0; c < 64; c += 8)
#pragma unroll
            for (int i = 0; i < 4; i++) top[i] = max3(top[i], s[c + 2 * i], s[c + 2 * i + 1]);
          tile_max = fmaxf(max3(top[0], top[1], top[2]), top[3]);
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
        if (t == first) {
          load_scores();
          other_half();
          m = tile_max;
          meet_half();  // read, before it is written again
        }
        uint32_t packed[32];
        uint64_t sum[2];
        while (true) {
          load_scores();
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
          other_half();
          const bool move = tile_max > m + grow;
          if (__builtin_expect(!__any_sync(0xffffffffu, move), 1)) break;
          const float f = move ? ex2((m - tile_max) * sl2) : 1.f;
          if (move) m = tile_max;
          l *= f;
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
        tmem_st32_nowait(p_at, packed);
        float l0, l1;
        unpair(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
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
      float m_scaled = m * sl2, f_own = 1.f, f_other = 0.f;
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
        m_scaled = top;
      } else if (mine && !idle) {
        *own_ex = l;
        meet_half();
        l += *other_ex;
        meet_half();  // read, before the next tile's maximum is written
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
    if (warp == 18) {
      // -------------------------------------------------------------- plan
      AttnPlan<TcShape> plan(a.H, a.HKV, a.plan_coarse, a.plan_least);
      const AttnStart st = attn_start(a, plan, staged, blockIdx.x, gridDim.x);
      fence_proxy_async();  // what was staged has been read: the ring may be filled
      __syncwarp();
      AttnWalk<TcShape> walk(a, plan, st, blockIdx.x, gridDim.x);
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
      constexpr uint32_t kIdS = idesc_bf16(128, 128, 0, 0), kIdO = idesc_bf16(128, D, 0, 1);
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
        wait(bars.kv_full(stage), ring.round, abort);
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
        wait(bars.q_full(), q_phase, abort);
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

bool make_maps(Maps &m, const AttnArgs &a, int d, int box) {
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

template <int D, bool PAGED>
std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use its shared memory

template <int D, bool PAGED>
cudaError_t launch(const AttnArgs &a, const Maps &maps, int box, int blocks, cudaStream_t stream) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void *>(&gdn_attn_tc_kernel<D, PAGED>),
                                   Smem<D>::kBytes, allowed<D, PAGED>);
  if (e != cudaSuccess) return e;
  gdn_attn_tc_kernel<D, PAGED><<<blocks, kThreads, Smem<D>::kBytes, stream>>>(a, maps, box);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, int d, int blocks, cudaStream_t stream) {
  int box = 128;
  if (a.table && (a.page_size & -a.page_size) < box) box = a.page_size & -a.page_size;
  Maps maps;
  if (!make_maps(maps, a, d, box)) return cudaErrorInvalidValue;
  if (d == 64)
    return a.table ? launch<64, true>(a, maps, box, blocks, stream)
                   : launch<64, false>(a, maps, box, blocks, stream);
  return a.table ? launch<128, true>(a, maps, box, blocks, stream)
                 : launch<128, false>(a, maps, box, blocks, stream);
}

}  // namespace gdn
