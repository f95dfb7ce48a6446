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
// Warps 0-3 and 4-7: softmax of X = 0 and 1, a row per thread.  Warp 8: TMA
// loads into a ring of key and value tiles.  Warp 9: the products.  Warp 10:
// the plan, units published through a small ring.  The loader and the product
// warp go through the same sequence of tiles across units, so the ring stays
// full and the first scores of a unit are computed while the softmax warps
// write out the last one.
#include <cuda_bf16.h>
#include <stdint.h>

#include "gdn_attn.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

using TcShape = AttnShape<256, 128, 128, 2>;
constexpr int kThreads = 384;
constexpr int kUnits = 4;              // unit ring
constexpr int kPanel = 128 * 128;      // bytes of 128 rows x 64 bf16
constexpr float kRescale = 8.f;        // log2 growth of a row maximum that is let stand

template <int D>
struct Smem {
  static constexpr int kTileBytes = D / 64 * kPanel;  // 128 rows of D
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kMl = kRing + kStages * kTileBytes;  // [2][128] float2
  static constexpr int kUnit = kMl + 2 * 128 * 8;
  static constexpr int kScratch = kUnit + kUnits * (int)sizeof(AttnUnit);
  static constexpr int kBars = (kScratch + (int)sizeof(AttnStartScratch<kThreads>) + 7) / 8 * 8;
  // barriers, in order: Q full, Q empty, S full x2, P ready x2, O full x2,
  // swap x2, unit full x4, unit empty x4, tile full, tile empty
  static constexpr int kBarCount = 10 + 2 * kUnits + 2 * kStages;
  static constexpr int kSlot = kBars + kBarCount * 8;
  static constexpr int kBytes = kSlot + 16;
};
static_assert(Smem<128>::kBytes <= 232448 && Smem<64>::kBytes <= 232448, "shared memory of one SM");

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

// A bounded wait by all lanes of a warp, converged afterwards.
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
  __device__ uint32_t unit_full(int i) const { return at(10 + i); }
  __device__ uint32_t unit_empty(int i) const { return at(10 + kUnits + i); }
  __device__ uint32_t kv_full(int i) const { return at(10 + 2 * kUnits + i); }
  __device__ uint32_t kv_empty(int i) const { return at(10 + 2 * kUnits + stages + i); }
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

// A step of a unit: one key tile for both row tiles (wide), or one key tile
// for each X (narrow).
struct Step {
  AttnUnit u;
  int step, steps;
  bool valid, narrow;
  __device__ void begin(Units &units) {
    valid = units.next(u);
    step = 0;
    narrow = u.n_tok * u.gp <= 128;
    steps = narrow ? (u.t1 - u.t0 + 1) / 2 : u.t1 - u.t0;
  }
  __device__ void advance(Units &units) {
    if (++step >= steps) begin(units);
  }
  __device__ int tile(int x) const { return narrow ? u.t0 + 2 * step + x : u.t0 + step; }
  __device__ bool active(int x) const { return valid && (!narrow || tile(x) < u.t1); }
  __device__ bool loads(int x) const { return active(x) && (narrow || x == 0); }
  __device__ bool frees(int x) const { return narrow || x == 1; }
  __device__ bool last(int x) const { return narrow ? tile(x) + 2 >= u.t1 : step == steps - 1; }
};

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    gdn_attn_tc_kernel(const AttnArgs a, const __grid_constant__ Maps maps, const int box) {
  using SM = Smem<D>;
  constexpr int kPanels = D / 64;
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_addr(sm) & 1023u) {
    if (tid == 0 && a.flags) atomicOr(a.flags, kFlagLaunchConfig);
    return;
  }
  const Bars bars{smem_addr(sm + SM::kBars), SM::kStages};
  uint32_t *slot = reinterpret_cast<uint32_t *>(sm + SM::kSlot);
  volatile int *abort = reinterpret_cast<volatile int *>(slot + 1);
  AttnUnit *unit_ring = reinterpret_cast<AttnUnit *>(sm + SM::kUnit);
  float2 *ml = reinterpret_cast<float2 *>(sm + SM::kMl);
  if (tid == 0) {
    *abort = 0;
    mbar_init(bars.q_full(), 1);
    mbar_init(bars.q_empty(), 1);
    for (int x = 0; x < 2; x++) {
      mbar_init(bars.s_full(x), 1);
      mbar_init(bars.p_ready(x), 4);
      mbar_init(bars.o_full(x), 1);
      mbar_init(bars.swap(x), 8);
    }
    for (int i = 0; i < kUnits; i++) {
      mbar_init(bars.unit_full(i), 1);
      mbar_init(bars.unit_empty(i), 10);  // loader, products, eight softmax warps
    }
    for (int i = 0; i < SM::kStages; i++) {
      mbar_init(bars.kv_full(i), 1);
      mbar_init(bars.kv_empty(i), 1);
    }
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(smem_addr(slot), 512);
  fence_before_sync();
  const AttnPlan<TcShape> plan(a.H, a.HKV);
  // synchronises the block twice: barriers and tensor memory are ready after it
  const AttnStart st = attn_start<TcShape, kThreads>(
      a, plan, blockIdx.x, gridDim.x, *reinterpret_cast<AttnStartScratch<kThreads> *>(sm + SM::kScratch));
  fence_after_sync();
  const uint32_t tmem = *slot;
  const uint32_t sQ = smem_addr(sm + SM::kQ), sRing = smem_addr(sm + SM::kRing);
  const uint32_t tS = tmem, tO = tmem + 256;

  if (warp < 8) {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t s_at = tS + x * 128 + lanes, o_at = tO + x * D + lanes;
    const float sl2 = a.scale_log2;
    const float grow = kRescale / sl2;
    Units units{unit_ring, bars, abort, {}};
    uint32_t s_phase = 0, o_phase = 0, swap_phase = 0;
    AttnUnit u;
    while (units.next(u)) {
      const bool narrow = u.n_tok * u.gp <= 128;
      const bool both = narrow && u.t1 - u.t0 > 1;
      const int stride = narrow ? 2 : 1;
      const int row = narrow ? r : x * 128 + r;
      const int tok = row / u.gp;
      const int limit = u.pos0 + min(tok, u.n_tok - 1);  // last visible key
      const int all_see = __reduce_min_sync(0xffffffffu, limit);
      float m = -CUDART_INF_F, l = 0.f;
      const int first = narrow ? u.t0 + x : u.t0;
      for (int t = first; t < u.t1; t += stride) {
        wait(bars.s_full(x), s_phase, abort);
        s_phase ^= 1;
        fence_after_sync();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; c++)
          tmem_ld32_nowait(s_at + c * 32, *reinterpret_cast<uint32_t(*)[32]>(s + c * 32));
        tmem_wait_ld();
        if (t * 128 + 127 > all_see) {
          const int lim = limit - t * 128;
#pragma unroll
          for (int c = 0; c < 128; c++)
            if (c > lim) s[c] = __float_as_uint(-CUDART_INF_F);
        }
        float top[4] = {__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]),
                        __uint_as_float(s[3])};
#pragma unroll
        for (int c = 4; c < 128; c++) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(s[c]));
        const float tile_max = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // The maximum is moved only when it has grown by a factor of 2^8: the
        // weights then stay below 2^8, the sums in fp32 far from overflow, and
        // the output in tensor memory is rarely touched.
        const bool move = tile_max > m + grow;
        if (t == first) {
          m = tile_max;
        } else if (__any_sync(0xffffffffu, move)) {
          const float f = move ? ex2((m - tile_max) * sl2) : 1.f;
          if (move) m = tile_max;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32_nowait(o_at + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32_nowait(o_at + c, o);
          }
        }
        const float off = m == -CUDART_INF_F ? 0.f : m * sl2;  // nothing visible yet: weights 0
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          const float p0 = ex2(fmaf(__uint_as_float(s[c]), sl2, -off));
          const float p1 = ex2(fmaf(__uint_as_float(s[c + 1]), sl2, -off));
          sum[(c >> 1) & 1] += p0;
          sum[2 + ((c >> 1) & 1)] += p1;
          s[c >> 1] = pack2(p0, p1);
        }
        tmem_st32_nowait(s_at, s);
        tmem_st32_nowait(s_at + 32, s + 32);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.p_ready(x));
      }
      // ---- the unit's output
      const bool mine = first < u.t1;
      if (mine) {
        wait(bars.o_full(x), o_phase, abort);
        o_phase ^= 1;
        fence_after_sync();
      }
      float m_scaled = m * sl2;
      float f_own = 1.f, f_other = 0.f;
      if (both) {
        ml[x * 128 + r] = make_float2(m_scaled, l);
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.swap(0));
        wait(bars.swap(0), swap_phase, abort);
        fence_after_sync();
        const float2 other = ml[(x ^ 1) * 128 + r];
        const float top = fmaxf(m_scaled, other.x);
        const float base = top == -CUDART_INF_F ? 0.f : top;
        f_own = ex2(m_scaled - base);
        f_other = ex2(other.x - base);
        l = f_own * l + f_other * other.y;
        m_scaled = top;
      }
      if (mine) {
        const bool valid = tok < u.n_tok;
        const float inv = u.slot >= 0 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
        const long long at = (long long)(u.row0 + tok) * a.H + u.head0 + row % u.gp;
        bool finite = true;
        // both: X = 0 writes the first half of the columns, X = 1 the second
        const int c0 = both ? x * (D / 2) : 0, c1 = both ? c0 + D / 2 : D;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t o[32], other[32];
          tmem_ld32_nowait(o_at + c, o);
          if (both) tmem_ld32_nowait(tO + (x ^ 1) * D + lanes + c, other);
          tmem_wait_ld();
          float y[32];
          if (both) {
#pragma unroll
            for (int i = 0; i < 32; i++)
              y[i] = f_own * __uint_as_float(o[i]) + f_other * __uint_as_float(other[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i++) y[i] = __uint_as_float(o[i]);
          }
          if (valid && u.slot >= 0) {
#pragma unroll
            for (int i = 0; i < 8; i++)
              a.part_o[((long long)u.slot * (D / 4) + (c >> 2) + i) * TcShape::kRows + row] =
                  make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          } else if (valid) {
            uint32_t out[16];
#pragma unroll
            for (int i = 0; i < 16; i++) {
              const float p = y[2 * i] * inv, q = y[2 * i + 1] * inv;
              finite &= isfinite(p) && isfinite(q);
              out[i] = pack2(p, q);
            }
            uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + c);
#pragma unroll
            for (int i = 0; i < 4; i++)
              to[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
          }
          __syncwarp();
        }
        if (valid && (!both || x == 0)) {
          if (u.slot >= 0)
            a.part_ml[(long long)u.slot * TcShape::kRows + row] = make_float2(m_scaled, l);
          else if (a.lse)
            a.lse[at] = l == 0.f ? -CUDART_INF_F : (m_scaled + log2f(l)) * 0.69314718056f;
        }
        if (!finite && a.flags) atomicOr(a.flags, kFlagNonfinite);
      }
      if (both) {  // the other output has been read: it may be overwritten
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.swap(1));
        wait(bars.swap(1), swap_phase, abort);
        fence_after_sync();
        swap_phase ^= 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 10) {
      // -------------------------------------------------------------- plan
      AttnWalk<TcShape> walk(a, plan, st, blockIdx.x);
      Ring<kUnits> at;
      AttnUnit u;
      bool more = true;
      while (more) {
        more = walk.next(u);
        if (!more) u.seq = -1;
        if (!__all_sync(0xffffffffu, mbar_wait(bars.unit_empty(at.i), at.round ^ 1, abort))) break;
        if (lane == 0) {
          unit_ring[at.i] = u;
          mbar_arrive(bars.unit_full(at.i));
        }
        __syncwarp();
        at.step();
      }
    } else if (warp == 8) {
      // ------------------------------------------------------------- loads
      Units units{unit_ring, bars, abort, {}};
      Ring<SM::kStages> ring;
      uint32_t q_phase = 1;
      Step cur, nxt;
      cur.valid = false;
      // one tile of keys or values of `s` into the next stage
      auto load = [&](const Step &s, int tile, const CUtensorMap *map) {
        const uint32_t full = bars.kv_full(ring.i), dst = sRing + ring.i * SM::kTileBytes;
        const int key = tile * 128;
        if constexpr (PAGED) {
          // lane i takes the i-th box of `box` keys; boxes past the last key
          // are not loaded (what they leave in shared memory is masked)
          const int left = s.u.len - key;
          const int n = left <= 0 ? 0 : min((left + box - 1) / box, 128 / box);
          int page = 0, first = 0;
          if (lane < n) {
            const int k0 = key + lane * box;
            page = __ldg(a.table + (long long)s.u.seq * a.max_pages + k0 / a.page_size);
            first = k0 % a.page_size;
            // an out-of-range page reads as zeros
            if ((page < 0 || page >= a.n_pages) && a.flags) atomicOr(a.flags, kFlagBadSeqlens);
          }
          wait(bars.kv_empty(ring.i), ring.round ^ 1, abort);
          if (lane == 0) mbar_arrive_expect_tx(full, n * box * 128 * kPanels);
          __syncwarp();
          if (lane < n)
#pragma unroll
            for (int p = 0; p < kPanels; p++)
              tma_load_4d(dst + p * kPanel + lane * box * 128, map, p * 64, s.u.kvh, first, page, full);
        } else {
          wait(bars.kv_empty(ring.i), ring.round ^ 1, abort);
          if (lane == 0) {
            mbar_arrive_expect_tx(full, SM::kTileBytes);
            const int row = s.u.row0 - s.u.pos0 + key;  // a prompt's keys are its own tokens
#pragma unroll
            for (int p = 0; p < kPanels; p++)
              tma_load_4d(dst + p * kPanel, map, p * 64, s.u.kvh, row, 0, full);
          }
          __syncwarp();
        }
        ring.step();
      };
      nxt.begin(units);
      while (true) {
#pragma unroll
        for (int x = 0; x < 2; x++) {
          if (cur.loads(x)) load(cur, cur.tile(x), &maps.v);
          if (nxt.valid && nxt.step == 0 && x == 0) {
            wait(bars.q_empty(), q_phase, abort);
            q_phase ^= 1;
            if (lane == 0) {
              const bool whole = nxt.u.gp == plan.G;  // all heads of a key/value head
              const int toks = 128 / nxt.u.gp, tiles = nxt.narrow ? 1 : 2;
              mbar_arrive_expect_tx(bars.q_full(), tiles * kPanels * toks * nxt.u.gp * 128);
              for (int i = 0; i < tiles; i++)
#pragma unroll
                for (int p = 0; p < kPanels; p++)
                  tma_load_3d(sQ + i * SM::kTileBytes + p * kPanel, whole ? &maps.q_pack : &maps.q,
                              p * 64, nxt.u.head0, nxt.u.row0 + i * toks, bars.q_full());
            }
            __syncwarp();
          }
          if (nxt.loads(x)) load(nxt, nxt.tile(x), &maps.k);
        }
        if (!nxt.valid) break;
        cur = nxt;
        nxt.advance(units);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- products
      constexpr uint32_t kIdS = idesc_bf16(128, 128, 0, 0), kIdO = idesc_bf16(128, D, 0, 1);
      Units units{unit_ring, bars, abort, {}};
      Ring<SM::kStages> ring;
      uint32_t q_phase = 0, p_phase[2] = {0, 0};
      int v_stage = 0, k_stage = 0;
      Step cur, nxt;
      cur.valid = false;
      nxt.begin(units);
      while (true) {
#pragma unroll
        for (int x = 0; x < 2; x++) {
          if (cur.active(x)) {
            if (cur.loads(x)) {
              v_stage = ring.i;
              wait(bars.kv_full(v_stage), ring.round, abort);
              ring.step();
              // weights past the last key are zero, but 0 * NaN is not: clear
              // the value rows that belong to nobody
              const int left = cur.u.len - cur.tile(x) * 128;
              if (left < 128) {
                const int from = left > 0 ? left : 0;
                for (int p = 0; p < kPanels; p++) {
                  uint4 *rows = reinterpret_cast<uint4 *>(sm + SM::kRing + v_stage * SM::kTileBytes +
                                                          p * kPanel);
                  for (int i = from * 8 + lane; i < 128 * 8; i += 32) rows[i] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
              }
            }
            wait(bars.p_ready(x), p_phase[x], abort);
            p_phase[x] ^= 1;
            fence_after_sync();
            if (lane == 0) {
              const uint32_t sV = sRing + v_stage * SM::kTileBytes;
#pragma unroll
              for (int k = 0; k < 8; k++)
                mma_f16_ta(tO + x * D, tS + x * 128 + k * 8, make_desc(sV + k * 2048, kPanel, 1024),
                           kIdO, cur.step > 0 || k > 0);
              if (cur.frees(x)) mma_commit(bars.kv_empty(v_stage));
              if (cur.last(x)) mma_commit(bars.o_full(x));
            }
            __syncwarp();
          }
          if (nxt.active(x)) {
            if (nxt.step == 0 && x == 0) {
              wait(bars.q_full(), q_phase, abort);
              q_phase ^= 1;
            }
            if (nxt.loads(x)) {
              k_stage = ring.i;
              wait(bars.kv_full(k_stage), ring.round, abort);
              ring.step();
            }
            fence_after_sync();
            if (lane == 0) {
              const uint32_t sK = sRing + k_stage * SM::kTileBytes;
              const uint32_t sA = sQ + (nxt.narrow ? 0 : x * SM::kTileBytes);
#pragma unroll
              for (int k = 0; k < D / 16; k++) {
                const uint32_t off = (k >> 2) * kPanel + (k & 3) * 32;
                mma_f16(tS + x * 128, make_desc(sA + off, 16, 1024), make_desc(sK + off, 16, 1024), kIdS,
                        k > 0);
              }
              mma_commit(bars.s_full(x));
              if (nxt.frees(x)) mma_commit(bars.kv_empty(k_stage));
              // the last scores of a unit: its queries may be replaced
              if (nxt.step == nxt.steps - 1 && (x == 1 || !nxt.active(1))) mma_commit(bars.q_empty());
            }
            __syncwarp();
          }
        }
        if (!nxt.valid) break;
        cur = nxt;
        nxt.advance(units);
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (tid == 0 && *abort && a.flags) atomicOr(a.flags, kFlagTimeout);
  if (warp == 9) tmem_dealloc(tmem, 512);
}

bool make_maps(Maps &m, const AttnArgs &a, int d, int box) {
  const AttnPlan<TcShape> plan(a.H, a.HKV);
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
  const uint32_t kv_box[4] = {64, 1, (uint32_t)box, 1};
  if (a.table) {
    const uint64_t row = (uint64_t)a.HKV * D * 2;
    const uint64_t dims[4] = {D, (uint64_t)a.HKV, (uint64_t)a.page_size, (uint64_t)a.n_pages};
    const uint64_t strides[3] = {D * 2, row, row * a.page_size};
    return encode_bf16_map(&m.k, a.k, 4, dims, strides, kv_box) &&
           encode_bf16_map(&m.v, a.v, 4, dims, strides, kv_box);
  }
  const uint64_t dims[4] = {D, (uint64_t)a.HKV, (uint64_t)a.Ttot, 1};
  const uint64_t ks[3] = {D * 2, (uint64_t)a.k_stride * 2, (uint64_t)a.k_stride * 2 * a.Ttot};
  const uint64_t vs[3] = {D * 2, (uint64_t)a.v_stride * 2, (uint64_t)a.v_stride * 2 * a.Ttot};
  return encode_bf16_map(&m.k, a.k, 4, dims, ks, kv_box) &&
         encode_bf16_map(&m.v, a.v, 4, dims, vs, kv_box);
}

template <int D, bool PAGED>
cudaError_t launch(const AttnArgs &a, const Maps &maps, int box, int blocks, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(
      gdn_attn_tc_kernel<D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  gdn_attn_tc_kernel<D, PAGED><<<blocks, kThreads, Smem<D>::kBytes, stream>>>(a, maps, box);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(AttnArgs a, int d, int blocks, cudaStream_t stream) {
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
