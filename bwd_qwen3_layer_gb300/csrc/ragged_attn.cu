// Attention of a ragged step over a paged key/value cache, on the 5th-generation
// tensor cores: request b feeds n_b = cu_rows[b+1] - cu_rows[b] new tokens (one
// when it decodes, a few drafted ones, a chunk of its prompt), and new token i
// attends to positions 0 .. ctx[b] + i of its request's pages:
//   o_i = sum_j softmax_j(q_i . k_j / sqrt(d)) v_j,  lse_i = log sum_j exp(q_i . k_j / sqrt(d)).
//
// Tiles. An item is (request, kv head, query tile). The G = Hq / Hkv query heads
// of a kv head read the same keys, so a query tile packs TQ = floor(128 / G)
// tokens x G heads into the 128 rows of one tcgen05 tile (row = token * G +
// head): each key and value tile is fetched once for all of them, and one shape
// of work covers decoding (G rows of 128 used: bound by HBM, the idle rows cost
// tensor-core time that the loads hide) and prompts (bound by the tensor cores).
//
// Work split. Lengths are on the device only, so the grid is one CTA per SM and
// every CTA finds its own work: the items' key tiles of 128 (plus four
// units for an item's start and end) laid end to end are W units, and CTA c takes units
// [c P, c P + P), P = ceil(W / CTAs). Every CTA thus streams the same number of
// key tiles whatever the lengths are. A CTA's first and last item may be cut; it
// leaves such a piece unnormalised (fp32 O, running max and sum per row) in the
// workspace and ragged_combine_kernel joins an item's pieces in CTA order, so
// results repeat bit for bit. The workspace holds two pieces per CTA and does
// not depend on the lengths.
//
// Roles (8 warps): warp 0 looks up the pages and copies the keys, warp 1 Q and
// the values, warp 2 issues the score products, warp 3 the P V products, warps
// 4..7 are the softmax (thread = query row = TMEM lane). A step's chain is
// scores -> softmax -> P V. S and P have two buffers each: S_(n+2) waits only for
// S_n to be read, P_n only for the product of step n - 2, so neither product's
// latency lies on the softmax warps' path. Each kind of product has a warp of
// its own because a warp's barrier probes queue up behind the products it has
// issued (measured: 514 cycles for 8 products of 64, 820 with three probes in
// between): one warp for both kept the tensor core waiting, 1850 cycles a step.
// Pages: with block_size a multiple of 8 a key tile is 128 / box TMA boxes of
// box = gcd(block_size, 128) rows, each found through the table; a box past the
// context, past its table row or whose table entry lies outside the pool starts
// past the tensor's last row and is filled with zeros by the copy. Other block
// sizes gather row by row with 16-byte cp.async. Slots behind the last position
// that a query tile sees may hold anything (NaN too): their scores are masked,
// and the last tile's value rows behind it are zeroed before the product reads them.
//
// Measured (64 / 8 heads, pages of 16): 64 requests of ~4096 keys 164-172 us, 0.92
// to 0.97 of the HBM copy rate; one of 32768 keys 30; 4096 rows over 12288 keys 1161-1180 us
// in a burst, 0.85 of the burst tensor rate, 1290-1344 back to back under the power cap. Pages
// of five, which go row by row: 321, 50 and 4053 us. The chunk's step is ~1440 cycles, of
// which the products take 1024 and shared memory's 160 KB (products' reads, copies'
// writes) 1250. Two warpgroups of softmax in turn (168 registers) gained 3 % there and
// lost 4 to 14 % everywhere else.
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "internal.h"
#include "kl_common.cuh"

namespace kl {
namespace {

constexpr int RA_D = 128;        // head dim
constexpr int RA_BQ = 128;       // rows of a query tile
constexpr int RA_BKV = 128;      // keys per tile
constexpr int RA_WARPS = 8;      // K copies, Q and V copies, score products, P V products, four of softmax
constexpr int RA_THREADS = 32 * RA_WARPS;
// A key or value tile (32 KB) is 16 groups of 8 keys, each group two swizzled
// blocks of 8 rows x 64 columns (1 KB): a page of 8 m tokens is then one TMA box
// of m groups x 2 column blocks x 8 rows, one copy instruction instead of two.
constexpr uint32_t RA_TILE = 128 * 128 * 2;
constexpr int RA_NST = 3;                     // stages of the K and of the V ring
constexpr uint32_t RA_OFF_Q = 0;
constexpr uint32_t RA_OFF_K = RA_OFF_Q + RA_TILE;
constexpr uint32_t RA_OFF_V = RA_OFF_K + RA_NST * RA_TILE;
constexpr uint32_t RA_OFF_BAR = RA_OFF_V + RA_NST * RA_TILE;
constexpr size_t RA_SMEM = 1024 + RA_OFF_BAR + 2048;
// Tensor memory: S of two steps, P of two steps (bf16 pairs), O: all 512 columns.
constexpr uint32_t RA_TM_P = 256, RA_TM_O = 384;
// Units that an item's start and end count for: its first scores, the last product
// and the epilogue take about four key tiles' time. Mixed batch of 20: with two,
// CTAs with two pieces ended at 51 us and those with eight at 61, 63 us in all;
// with four 60.4. A run may be as short as one unit: one request of 500 keys takes 8.8
// us, 11.2 with runs of at least five (100 keys: 8.3 and 7.9).
constexpr int RA_ITEM_UNITS = 4;
constexpr float RA_LOG2E = 1.4426950408889634f;
constexpr float RA_LN2 = 0.6931471805599453f;

// One request's rows and context, every value brought into range (no table row
// is as long as RA_MAX_CTX, so a context beyond it is past its table anyway).
constexpr int RA_MAX_CTX = 1 << 30;
struct RaReq {
  int r0, n, ctx;
};

// Where a CTA's run of units starts: the unit inside an item.
struct RaFound {
  int any;          // 0: no units left for this CTA
  int g, qt;
  RaReq q;
  long long off;
};
// The cut that a run's start makes, for the joining kernel: the item's pieces (0:
// nothing to join here), its rows, the first one's row of the step.
struct RaCut {
  int pieces, rows, row0, g;
  int first_slot;   // of the CTA before: 0 if this item was its first
};

struct RaParams {
  CUtensorMap tmQ, tmK, tmV;
  const __nv_bfloat16* kp;
  const __nv_bfloat16* vp;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* ctx;
  __nv_bfloat16* o;
  float* lse;            // [T, Hq] or null
  float* part_o;         // [CTA][2][32][128][4] unnormalised pieces: 4 columns of the 128 rows together
  float* part_ml;        // [CTA][2][128][2] (max in log2 units, sum)
  RaCut* cuts;           // [CTA]
  int B, T, Hq, Hkv, G, TQ;
  int bs, max_blocks, n_blocks;
  int box_log;           // log2 of the rows per TMA box (8 .. 128)
  float scale_log2;
  uint32_t* err;
};

__device__ __forceinline__ float ra_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Q, K-major (two 64-column swizzle blocks of 128 rows), k-step kk of 16 columns
__device__ __forceinline__ uint64_t ra_desc_q(uint32_t base, int kk) {
  return smem_desc_sw128(base + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024);
}
// Pairs of floats in one 64-bit register: one instruction for two elements.
__device__ __forceinline__ uint64_t ra_pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void ra_unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t ra_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t ra_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float ra_max3(float a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}
// K, K-major, in groups of 8 keys 2 KB apart
__device__ __forceinline__ uint64_t ra_desc_k(uint32_t base, int kk) {
  return smem_desc_sw128(base + (kk >> 2) * 1024 + (kk & 3) * 32, 16, 2048);
}
// V as the MN-major B operand: n = head dim in two 64-wide blocks 1 KB apart,
// k-step kk of 16 keys = two groups
__device__ __forceinline__ uint64_t ra_desc_v(uint32_t base, int kk) {
  return smem_desc_sw128(base + kk * 4096, 1024, 2048);
}
__device__ __forceinline__ void ra_tma_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void ra_tma_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// 32 bytes to a 32-byte aligned address
__device__ __forceinline__ void ra_st32(void* dst, const uint32_t (&x)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ void ra_cp16(uint32_t dst, const void* src, bool valid) {
  const int sz = valid ? 16 : 0;   // zero-fill
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(sz) : "memory");
}

// mbar_wait_warp for a copy warp, which is a ring ahead of the products: between
// probes it sleeps, so that its issue slots go to the softmax warp beside it.
__device__ __forceinline__ bool ra_wait_copy(uint32_t bar, uint32_t parity, uint32_t* err, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; !__all_sync(0xffffffffu, mbar_test_wait(bar, parity)); ++i) {
    __nanosleep(100);
    if ((i & 63u) == 63u) {
      const uint64_t t = global_timer_ns();
      if (i == 63u) t0 = t;
      const bool late = t - t0 > KL_WAIT_LIMIT_NS;
      if (late) record_error(err, KL_DEVERR_TIMEOUT);
      if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
    }
  }
  return true;
}

// What the walk reads of the parameters, handed over by value: a reference to
// kernel parameters makes every access of a called function a slow generic load.
struct RaLens {
  const int32_t* cu;
  const int32_t* ctx;
  int B, T, Hkv, TQ;
};
__device__ __forceinline__ RaReq ra_req(const RaLens& p, int b) {
  RaReq q;
  q.r0 = min(max(p.cu[b], 0), p.T);
  q.n = min(max(p.cu[b + 1], q.r0), p.T) - q.r0;
  q.ctx = min(max(p.ctx[b], 0), RA_MAX_CTX);
  return q;
}
// Key tiles of query tile qt (its last token's limit decides).
__device__ __forceinline__ int ra_tiles(const RaReq& q, int TQ, int qt) {
  return (q.ctx + min(q.n, (qt + 1) * TQ) - 1) / RA_BKV + 1;
}
// Units of query tiles 0 .. m-1, all but the request's last one:
//   sum_{k=1}^{m} (floor((ctx - 1 + k TQ) / 128) + 1 + RA_ITEM_UNITS).
// The quotients repeat with period 128 / gcd(TQ, 128) up to a constant step, so
// whole periods are summed in closed form.
__device__ __noinline__ long long ra_units_before(int ctx, int TQ, long long m) {
  const int sh = __ffs(TQ) - 1;                   // gcd(TQ, 128) = 2^sh, TQ <= 128
  const int period = RA_BKV >> sh, step = TQ >> sh;
  const long long a = static_cast<long long>(ctx) - 1;
  const long long c = m >> (7 - sh);
  const int r = static_cast<int>(m & (period - 1));
  long long full = 0, part = 0;
  for (int k = 1; k <= (c ? period : r); ++k) {
    const long long v = (a + static_cast<long long>(k) * TQ) >> 7;
    full += v;
    if (k <= r) part += v;
  }
  return m * (1 + RA_ITEM_UNITS) + (c ? c * full + static_cast<long long>(period) * step * (c * (c - 1) / 2) : 0) +
         part + static_cast<long long>(r) * step * c;
}
__device__ __forceinline__ long long ra_head_units(const RaReq& q, int TQ) {
  if (q.n <= 0) return 0;
  if (q.n <= TQ) return (q.ctx + q.n - 1) / RA_BKV + 1 + RA_ITEM_UNITS;
  const int QT = (q.n + TQ - 1) / TQ;
  return ra_units_before(q.ctx, TQ, QT - 1) + ra_tiles(q, TQ, QT - 1) + RA_ITEM_UNITS;
}

// Quotient of non-negative numbers; most fit 32 bits, whose division is several times faster.
__device__ __noinline__ long long ra_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// One piece of a CTA's run: the query tile and the range of its key tiles.
struct RaPiece {
  int b, g;                // request, kv head
  int row0, toks;          // the tile's first row of the step, its tokens
  int pos0, L;             // position of its first token; keys that its last one sees
  int ta, tb;              // key tiles; tb = 0: there is no such piece
  int flags;               // 1: all of the item's tiles; 2: the piece goes to slot 1
};
// The walk over a CTA's run. Every role's warp walks for itself, in shared
// memory: the softmax warps' registers are full of scores, and every one more
// costs their steps (with the walk in registers they spilled).
struct RaWalk {
  int b, g, qt;            // request (its lengths: q), kv head, query tile
  int idx;                 // items met so far: the first one's pieces take slot 0, a later one's slot 1
  RaReq q;
  long long off, left;     // unit inside the item, units left of the run
};
// The next piece with at least one key tile into c.
__device__ __forceinline__ void ra_step(const RaLens& p, RaWalk& w, RaPiece& c) {
  c.tb = 0;
  while (w.left > 0) {
    const int tiles = ra_tiles(w.q, p.TQ, w.qt);
    const int len = tiles + RA_ITEM_UNITS, off = static_cast<int>(w.off);
    const int e = static_cast<int>(min(w.left, static_cast<long long>(len - off))) + off;
    const int first = w.qt * p.TQ;
    c.ta = max(off - RA_ITEM_UNITS, 0);
    c.tb = max(e - RA_ITEM_UNITS, 0);
    c.b = w.b;
    c.g = w.g;
    c.row0 = w.q.r0 + first;
    c.toks = min(p.TQ, w.q.n - first);
    c.pos0 = w.q.ctx + first;
    c.L = c.pos0 + c.toks;
    c.flags = (c.ta == 0 && c.tb == tiles ? 1 : 0) | (w.idx > 0 ? 2 : 0);
    w.left -= e - off;
    ++w.idx;
    if (w.left > 0) {      // the item ends here: on to the next
      w.off = 0;
      if (first + p.TQ < w.q.n) {
        ++w.qt;
      } else {
        w.qt = 0;
        if (++w.g == p.Hkv) {
          w.g = 0;
          do {
            if (++w.b >= p.B) {      // cannot happen: the run lies inside the W units
              w.left = 0;
              break;
            }
            w.q = ra_req(p, w.b);
          } while (w.q.n <= 0);
        }
      }
    }
    if (c.tb > c.ta) break;
    c.tb = 0;
  }
}
// The same for a walk in shared memory, called by one lane: one copy of the code
// for all roles.
__device__ __noinline__ void ra_next(const RaLens p, const RaWalk& from, RaWalk& to, RaPiece& piece) {
  if (from.left <= 0) {
    piece.tb = 0;
    return;
  }
  RaWalk w = from;         // in registers: one read, one write each
  RaPiece c;
  ra_step(p, w, c);
  to = w;
  piece = c;
}

template <bool TMA>
__global__ void __launch_bounds__(RA_THREADS, 1) ragged_attn_kernel(const __grid_constant__ RaParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar = sb + RA_OFF_BAR;
  // barriers; those of a pair serve the steps of one parity each, so that a warp
  // which runs a step ahead of another cannot count for its phase
  const uint32_t q_full = bar + 0, drain = bar + 8;
  const uint32_t q_empty = bar + 16;                        // a piece's last S product is done with Q
  auto k_full = [&](int s) { return bar + 24 + 8 * s; };
  auto k_empty = [&](int s) { return bar + 48 + 8 * s; };
  auto v_full = [&](int s) { return bar + 72 + 8 * s; };
  auto v_empty = [&](int s) { return bar + 96 + 8 * s; };
  auto s_full = [&](int s) { return bar + 120 + 8 * s; };   // S_n computed
  auto s_free = [&](int s) { return bar + 136 + 8 * s; };   // S_n read
  auto p_full = [&](int s) { return bar + 152 + 8 * s; };   // P_n written (and V_n's tail cleared)
  auto p_done = [&](int s) { return bar + 168 + 8 * s; };   // O += P_n V_n computed
  const uint32_t drain_pv = bar + 184;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + RA_OFF_BAR + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + RA_OFF_BAR + 196);
  RaFound* found = reinterpret_cast<RaFound*>(smem + RA_OFF_BAR + 208);
  long long* wsum = reinterpret_cast<long long*>(smem + RA_OFF_BAR + 256);   // the warps' unit sums, then this CTA's units

  RaWalk* walks = reinterpret_cast<RaWalk*>(smem + RA_OFF_BAR + 336);        // the finder's, then one per warp
  RaPiece* pieces = reinterpret_cast<RaPiece*>(smem + RA_OFF_BAR + 848);     // the first one, then two per warp
  static_assert((RA_WARPS + 1) * sizeof(RaWalk) <= 512 && (RA_WARPS * 2 + 1) * sizeof(RaPiece) <= 1200, "shared-memory layout");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const RaLens lens = {p.cu, p.ctx, p.B, p.T, p.Hkv, p.TQ};

  if (warp == 3 && lane == 0) {      // not the first warps: they have the first requests to scan
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < RA_NST; ++s) {
      mbar_init(k_full(s), TMA ? 1 : 32);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), TMA ? 1 : 32);
      mbar_init(v_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(s_free(s), 4);
      mbar_init(p_full(s), 4);
      mbar_init(p_done(s), 1);
    }
    mbar_init(drain, 1);
    mbar_init(drain_pv, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }

  if (lane == 0 && warp >= 5 && (TMA || warp == 5))
    tma_prefetch_desc(warp == 5 ? &p.tmQ : warp == 6 ? &p.tmK : &p.tmV);

  // What is above reads nothing that an earlier kernel writes and runs while the last
  // one ends: this CTA's shared memory takes a whole SM, so nothing else is on it that
  // could want its tensor memory (every decoding case 0.2 us less).
  pdl_enter();

  // ---- this CTA's run: prefix sums of the requests' units, then the item at unit cta * P ----
  long long P;
  {
    const int per = (p.B + RA_THREADS - 1) / RA_THREADS;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    long long mine = 0, units = 0;
    RaReq q = {0, 0, 0};
    for (int b = b0; b < b1; ++b) {
      q = ra_req(lens, b);
      units = ra_head_units(q, p.TQ);
      mine += units * p.Hkv;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    long long before = 0, W = 0;
#pragma unroll
    for (int w = 0; w < RA_WARPS; ++w) {
      const long long v = wsum[w];
      if (w < warp) before += v;
      W += v;
    }
    P = max(ra_div(W + ctas - 1, ctas), 1LL);
    const long long u0 = cta * P;
    if (threadIdx.x == 0 && u0 >= W) {
      found->any = 0;
      pieces[0].tb = 0;
    }
    long long lo = before + incl - mine;      // units before this thread's requests
    if (mine > 0 && u0 >= lo && u0 < lo + mine) {
      int b = b0;
      if (per > 1) {                          // with one request a thread q and units are its own still
        for (;; ++b) {
          q = ra_req(lens, b);
          units = ra_head_units(q, p.TQ);
          if (u0 < lo + units * p.Hkv) break;
          lo += units * p.Hkv;
        }
      }
      const int g = static_cast<int>(ra_div(u0 - lo, units));
      const long long y = u0 - lo - g * units;
      int m0 = 0, m1 = q.n <= p.TQ ? 1 : (q.n + p.TQ - 1) / p.TQ;   // the query tile: units_before(m0) <= y < units_before(m1)
      while (m1 - m0 > 1) {
        const int m = (m0 + m1) >> 1;
        if (ra_units_before(q.ctx, p.TQ, m) <= y) m0 = m; else m1 = m;
      }
      const long long off = y - (m0 ? ra_units_before(q.ctx, p.TQ, m0) : 0);
      // the walk to the first piece, for every role at once
      RaWalk w = {b, g, m0, 0, q, off, min(P, W - u0)};
      RaPiece c;
      ra_step(lens, w, c);
      pieces[0] = c;
      walks[0] = w;
      *found = {1, g, m0, q, off};
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tmP = tmem + RA_TM_P, tmO = tmem + RA_TM_O;
  const int GT = p.G * p.TQ;            // rows of a full query tile

  // Piece 0 is shared (pieces[0]); from there each warp walks for itself.
  auto piece = [&](int k) -> RaPiece& { return pieces[k ? 1 + warp * 2 + (k & 1) : 0]; };
  // piece k of this CTA into its place; false if there is none
  auto find = [&](int k) -> bool {
    if (k > 0) {
      __syncwarp();                     // every lane is done with piece k - 2
      if (lane == 0) ra_next(lens, walks[k == 1 ? 0 : warp + 1], walks[warp + 1], piece(k));
      __syncwarp();
    }
    return piece(k).tb > 0;
  };

  if (warp < 2) {
    // ------- copies (warp 0: K, warp 1: Q and V; lane = page box of a tile) -------
    const bool is_k = warp == 0;
    const bool el = elect_one();
    const CUtensorMap* tm = is_k ? &p.tmK : &p.tmV;
    const __nv_bfloat16* pool = is_k ? p.kp : p.vp;
    const uint32_t ring = sb + (is_k ? RA_OFF_K : RA_OFF_V);
    const uint32_t full0 = is_k ? k_full(0) : v_full(0), empty0 = is_k ? k_empty(0) : v_empty(0);
    // rows of a box, boxes of a tile, tiles of a look-up, this lane's one
    const int box = 1 << p.box_log, nbox = RA_BKV >> p.box_log, per = box >> 2, my = lane >> (7 - p.box_log);
    const int no_row = p.n_blocks * p.bs;         // past the pool's last row: filled with zeros
    int issued_q = 0, issued = 0, s = 0, as = 0;  // s: the ring's stage; as: the next one to announce
    uint32_t ph = 1;                              // parity that an empty stage's wait passes with
    bool ok = true;
    // the pool row of a position at `at` of its page blk, or no_row
    auto pool_row = [&](int blk, int at) {
      if (blk >= 0 && blk < p.n_blocks) return blk * p.bs + at;
      record_error(p.err, KL_DEVERR_PAGE);
      return no_row;
    };
    auto page = [&](int b, int lb) { return lb < p.max_blocks ? p.table[static_cast<int64_t>(b) * p.max_blocks + lb] : -1; };
    // cp.async: the rows of one tile; row[k] of lane l is the pool row of key 32 k + l
    auto gather = [&](uint32_t dst, int g, const int (&row)[4]) {
      const int ch = lane & 15;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll 4
        for (int it = 0; it < 16; ++it) {
          const int key = 32 * k + 2 * it + (lane >> 4);
          const int src = __shfl_sync(0xffffffffu, row[k], 2 * it + (lane >> 4));
          const uint32_t off = (key >> 3) * 2048 + (ch >> 3) * 1024 + (key & 7) * 128 + (((ch & 7) ^ (key & 7)) << 4);
          const bool valid = src != no_row;
          ra_cp16(dst + off, pool + (static_cast<int64_t>(valid ? src : 0) * p.Hkv + g) * RA_D + ch * 8, valid);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // cp.async: once at most N copy groups are under way the oldest tile has
    // landed; made visible to the tensor core, then announced
    auto announce = [&](auto pending) {
      asm volatile("cp.async.wait_group %0;" ::"n"(decltype(pending)::value) : "memory");
      fence_async_shared();
      mbar_arrive(full0 + 8 * as);
      as = as == RA_NST - 1 ? 0 : as + 1;
    };
    for (int k = 0; ok && find(k); ++k) {
      const RaPiece w = piece(k);
      // TMA: one look at the table serves `per` tiles, a lane per box, and the
      // next tiles' pages are asked for before these are copied: a read of the table
      // takes 600 to 3000 cycles, which every tile of a run's start waited for.
      // cp.async: a lane for four of a tile's keys.
      int row[4], blk = 0, at = 0;
      const int keys = min(w.L, w.tb * RA_BKV);
      auto ask = [&](int j) {
        const int pos = j * RA_BKV + lane * box, lb = pos / p.bs;
        at = pos < keys ? pos - lb * p.bs : -1;
        if (at >= 0) blk = page(w.b, lb);
      };
      auto lookup = [&](int j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = j * RA_BKV + i * 32 + lane, lb = pos / p.bs;
          row[i] = pos < keys ? pool_row(page(w.b, lb), pos - lb * p.bs) : no_row;
        }
      };
      if (TMA) ask(w.ta); else lookup(w.ta);
      if (!is_k) {
        // Q: the buffer is free once the previous piece's last S product is done
        if (!ra_wait_copy(q_empty, (issued_q & 1) ^ 1u, p.err, abort_flag)) { ok = false; break; }
        if (el) {
          mbar_arrive_expect_tx(q_full, 2u * GT * 128u);
          ra_tma_3d(sb + RA_OFF_Q, &p.tmQ, 0, w.g * p.G, w.row0, q_full);
          ra_tma_3d(sb + RA_OFF_Q + 16384, &p.tmQ, 64, w.g * p.G, w.row0, q_full);
        }
        __syncwarp();
        ++issued_q;
      }
      for (int j = w.ta; j < w.tb; ++j) {
        const int nth = (j - w.ta) & (per - 1);
        if (TMA && nth == 0) {
          row[0] = at >= 0 ? pool_row(blk, at) : no_row;
          if (j + per < w.tb) ask(j + per);
        }
        if (!ra_wait_copy(empty0 + 8 * s, ph, p.err, abort_flag)) { ok = false; break; }
        const uint32_t dst = ring + s * RA_TILE;
        if (TMA) {
          if (el) mbar_arrive_expect_tx(full0 + 8 * s, RA_TILE);
          __syncwarp();
          if (my == nth) ra_tma_4d(dst + (lane & (nbox - 1)) * box * 256, tm, 0, 0, 2 * w.g, row[0] >> 3, full0 + 8 * s);
          __syncwarp();
        } else {
          gather(dst, w.g, row);
          if (j > w.ta) announce(std::integral_constant<int, 1>());   // the tile before
        }
        ++issued;
        if (++s == RA_NST) {
          s = 0;
          ph ^= 1u;
        }
        if (!TMA && j + 1 < w.tb) lookup(j + 1);
      }
      // the piece's last tile: its products free Q, which the next piece waits for
      if (!TMA && ok) announce(std::integral_constant<int, 0>());
    }
    if (!ok) *abort_flag = 1;
    // copies still in flight must land before exit
    if (issued_q > 0) mbar_wait(q_full, (issued_q - 1) & 1, p.err);
    if (TMA) {
      for (int j = max(0, issued - RA_NST); j < issued; ++j) mbar_wait(full0 + 8 * (j % RA_NST), (j / RA_NST) & 1, p.err);
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  } else if (warp == 2) {
    // ---------- S_n = Q K_n^T into S[n % 2] (whole warp; the elected lane issues) ----------
    const bool el = elect_one();
    const uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
    int n = 0, k = 0, ks = 0;                 // step, piece, K stage
    uint32_t kph = 0;
    bool ok = true;
    for (; ok && find(k); ++k) {
      const int tiles = piece(k).tb - piece(k).ta;
      if (!mbar_wait_warp(q_full, k & 1, p.err, abort_flag)) { ok = false; break; }
      for (int j = 0; j < tiles; ++j, ++n) {
        const int s = n & 1;
        if ((n >= 2 && !mbar_wait_warp(s_free(s), ((n >> 1) & 1) ^ 1u, p.err, abort_flag)) ||
            !mbar_wait_warp(k_full(ks), kph, p.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (el) {
          for (int kk = 0; kk < RA_D / 16; ++kk)
            umma_bf16(tmem + s * 128, ra_desc_q(sb + RA_OFF_Q, kk), ra_desc_k(sb + RA_OFF_K + ks * RA_TILE, kk), idesc, kk > 0);
          umma_commit(s_full(s));
          umma_commit(k_empty(ks));
          if (j == tiles - 1) umma_commit(q_empty);   // the piece's last use of Q
        }
        __syncwarp();
        if (++ks == RA_NST) {
          ks = 0;
          kph ^= 1u;
        }
      }
    }
    if (!ok) *abort_flag = 1;
    if (el) umma_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, p.err);
  } else if (warp == 3) {
    // ---------- O (+)= P_n V_n (whole warp; the elected lane issues) ----------
    const bool el = elect_one();
    const uint32_t idesc = idesc_bf16_f32(128, 128, 0, 1);
    int n = 0, vs = 0;                        // step, V stage
    uint32_t vph = 0;
    bool ok = true;
    for (int k = 0; ok && find(k); ++k) {
      const int tiles = piece(k).tb - piece(k).ta;
      for (int j = 0; j < tiles; ++j, ++n) {
        const int s = n & 1;
        if (!mbar_wait_warp(v_full(vs), vph, p.err, abort_flag) ||
            !mbar_wait_warp(p_full(s), (n >> 1) & 1, p.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (el) {
          for (int kk = 0; kk < RA_BKV / 16; ++kk)
            umma_bf16_ta(tmO, tmP + s * 64 + kk * 8, ra_desc_v(sb + RA_OFF_V + vs * RA_TILE, kk), idesc,
                         (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(p_done(s));
          umma_commit(v_empty(vs));
        }
        __syncwarp();
        if (++vs == RA_NST) {
          vs = 0;
          vph ^= 1u;
        }
      }
    }
    if (!ok) *abort_flag = 1;
    if (el) umma_commit(drain_pv);
    __syncwarp();
    mbar_wait(drain_pv, 0, p.err);
  } else {
    // ---------------- softmax / correction / epilogue ----------------
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;           // row within the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t oadr = tmO + lane_off, padr = tmP + lane_off;
    // The tile that holds the last key the query tile sees: its value rows behind it become zero
    // (each of the four warps its 32).
    auto clear_tail = [&](int end, int n) -> bool {
      if (end >= RA_BKV) return true;
      const int vs = n % RA_NST;
      if (!mbar_wait_warp(v_full(vs), (n / RA_NST) & 1, p.err, abort_flag)) return false;
      if (r >= end) {
        const uint32_t va = sb + RA_OFF_V + vs * RA_TILE + (r >> 3) * 2048 + (r & 7) * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          st_shared_v4(va + c * 16, 0u, 0u, 0u, 0u);
          st_shared_v4(va + 1024 + c * 16, 0u, 0u, 0u, 0u);
        }
      }
      fence_async_shared();
      return true;
    };
    // the cut at this CTA's start, by a warp that has nothing to do yet
    if (threadIdx.x == RA_THREADS - 1) {
      RaCut cut = {0, 0, 0, 0, 0};
      if (found->any) {
        const RaFound f = *found;
        // the first cut of its item with key tiles on both sides joins the pieces
        const long long len = ra_tiles(f.q, p.TQ, f.qt) + RA_ITEM_UNITS;
        if (f.off > RA_ITEM_UNITS && f.off - P <= RA_ITEM_UNITS) cut.pieces = 1 + static_cast<int>(ra_div(len - f.off + P - 1, P));
        cut.rows = min(p.TQ, f.q.n - f.qt * p.TQ) * p.G;
        cut.row0 = f.q.r0 + f.qt * p.TQ;
        cut.g = f.g;
        cut.first_slot = f.off - P >= 0 ? 0 : 1;
      }
      p.cuts[cta] = cut;
    }
    __syncwarp();
    bool ok = true;
    const float scale = p.scale_log2;
    int n = 0;
    float m = -INFINITY, l = 0.f;                  // the row's running max (log2 units) and sum
    int lim = 0, end = 0;                          // the row's last key and the end of the query tile's, from the tile's first key
    // One step of a warp with rows. CUT: some row of the tile ends inside its keys.
    // The whole tiles before have a body of their own, without what that takes
    // (tests and masks cost them ~180 cycles a step).
    auto step = [&](auto cut, bool first) -> bool {
      constexpr bool CUT = decltype(cut)::value;
      const int s = n & 1;
      if (CUT && TMA && !clear_tail(end, n)) return false;
      if (!mbar_wait_warp(s_full(s), (n >> 1) & 1, p.err, abort_flag)) return false;
      tc_fence_after();
      const uint32_t sadr = tmem + lane_off + s * 128;
      uint32_t sv[RA_BKV];
      tmem_ld_32x32b_x32(sadr, *reinterpret_cast<uint32_t(*)[32]>(sv));
      tmem_ld_32x32b_x32(sadr + 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32));
      tmem_ld_32x32b_x32(sadr + 64, *reinterpret_cast<uint32_t(*)[32]>(sv + 64));
      tmem_ld_32x32b_x32(sadr + 96, *reinterpret_cast<uint32_t(*)[32]>(sv + 96));
      // P's columns are free once the product of step n - 2 is done: probed here,
      // where the probe's latency costs nothing, and most likely it is
      const uint32_t done_ph = ((n >> 1) & 1) ^ 1u;
      const bool p_ready = n < 2 || mbar_test_wait(p_done(s), done_ph);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(s));       // S[s] may be overwritten from here on
      if (CUT) {                                   // keys 0 .. lim are kept
#pragma unroll
        for (int e = 0; e < RA_BKV; ++e)
          if (e > lim) sv[e] = __float_as_uint(-INFINITY);
      }
      float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
      for (int e = 0; e < RA_BKV; e += 8) {
        m0 = ra_max3(m0, sv[e], sv[e + 1]);
        m1 = ra_max3(m1, sv[e + 2], sv[e + 3]);
        m2 = ra_max3(m2, sv[e + 4], sv[e + 5]);
        m3 = ra_max3(m3, sv[e + 6], sv[e + 7]);
      }
      const float mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * scale;
      // The max is only raised when it grows by more than 2^8 (the final O / l
      // cancels a stale one). A row of a later piece's tile can be fully masked
      // (its token ends before these keys): mx = -inf, and m stays -inf.
      const bool raise = mx > m + 8.0f;
      if (__any_sync(0xffffffffu, raise)) {
        const float m_new = raise ? mx : m;
        const float alpha = raise ? ra_ex2(m - m_new) : 1.0f;
        m = m_new;
        l *= alpha;
        if (!first) {
          if (!mbar_wait_warp(p_done(s ^ 1), ((n - 1) >> 1) & 1, p.err, abort_flag)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(oadr + c * 16, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            tmem_st_32x32b_x16(oadr + c * 16, v);
          }
        }
      }
      const uint32_t neg = __float_as_uint(m > -INFINITY ? -m : 0.f), sc = __float_as_uint(scale);
      const uint64_t neg2 = ra_pair(neg, neg), sc2 = ra_pair(sc, sc);
      uint64_t r0 = 0, r1 = 0;
      uint32_t pk[64];
#pragma unroll
      for (int e = 0; e < RA_BKV; e += 4) {
        float p0, p1, p2, p3;
        ra_unpair(ra_fma2(ra_pair(sv[e], sv[e + 1]), sc2, neg2), p0, p1);
        ra_unpair(ra_fma2(ra_pair(sv[e + 2], sv[e + 3]), sc2, neg2), p2, p3);
        p0 = ra_ex2(p0);
        p1 = ra_ex2(p1);
        p2 = ra_ex2(p2);
        p3 = ra_ex2(p3);
        r0 = ra_add2(r0, ra_pair(__float_as_uint(p0), __float_as_uint(p1)));
        r1 = ra_add2(r1, ra_pair(__float_as_uint(p2), __float_as_uint(p3)));
        pk[e >> 1] = pack_bf16x2(p0, p1);          // P enters its product as bf16: half a step (2^-8 at most) per weight
        pk[(e >> 1) + 1] = pack_bf16x2(p2, p3);
      }
      float a0, a1, a2, a3;
      ra_unpair(r0, a0, a1);
      ra_unpair(r1, a2, a3);
      l += (a0 + a1) + (a2 + a3);
      if (!__all_sync(0xffffffffu, p_ready) && !mbar_wait_warp(p_done(s), done_ph, p.err, abort_flag)) return false;
      tc_fence_after();
      tmem_st_32x32b_x32(padr + s * 64, *reinterpret_cast<uint32_t(*)[32]>(pk));
      tmem_st_32x32b_x32(padr + s * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(pk + 32));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(s));
      lim -= RA_BKV;
      end -= RA_BKV;
      ++n;
      return true;
    };
    bool more = find(0);
    for (int k = 0; ok && more; ++k) {
      int left, whole;                             // tiles left; those that every row sees whole
      bool busy;
      {
        const RaPiece& c = piece(k);
        left = c.tb - c.ta;
        const int over = c.pos0 - c.ta * RA_BKV;   // the tile's first row's last key
        whole = min(left, (over + 1) >> 7);        // below zero: none
        lim = over + min(r / p.G, c.toks - 1);     // padding rows: the last real row's limit
        end = c.L - c.ta * RA_BKV;
        busy = quarter * 32 < c.toks * p.G;        // some row of this warp is real
      }
      m = -INFINITY;
      l = 0.f;
      if (busy) {
        bool first = true;
        for (int i = 0; ok && i < whole; ++i, first = false) ok = step(std::false_type(), first);
        for (int i = max(whole, 0); ok && i < left; ++i, first = false) ok = step(std::true_type(), first);
      } else {
        // no real row: P stays whatever it is, its O rows are never read. The product
        // of step n - 2 is waited for all the same: this warp must not count for
        // step n's phase while another still works on step n - 2.
        for (int i = 0; ok && i < left; ++i, ++n, end -= RA_BKV) {
          const int s = n & 1;
          ok = (!TMA || clear_tail(end, n)) && mbar_wait_warp(s_full(s), (n >> 1) & 1, p.err, abort_flag) &&
               (n < 2 || mbar_wait_warp(p_done(s), ((n >> 1) & 1) ^ 1u, p.err, abort_flag));
          __syncwarp();
          if (ok && lane == 0) {
            mbar_arrive(s_free(s));
            mbar_arrive(p_full(s));
          }
        }
      }
      if (!ok) break;
      more = find(k + 1);                          // while the piece's last P V product, step n - 1's, runs
      if (!mbar_wait_warp(p_done((n - 1) & 1), ((n - 1) >> 1) & 1, p.err, abort_flag)) { ok = false; break; }
      tc_fence_after();
      if (busy) {
        const RaPiece& c = piece(k);
        const bool whole = c.flags & 1;
        const int tok = r / p.G;
        const bool mine = r < c.toks * p.G;
        const int64_t orow = static_cast<int64_t>(c.row0 + tok) * p.Hq + c.g * p.G + (r - tok * p.G);
        const int64_t pslot = static_cast<int64_t>(cta) * 2 + (c.flags >> 1);
        const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(oadr + h * 32, v);
          tmem_ld_wait();
          if (mine && whole) {
            // whole 32-byte sectors: rows lie apart, and an SM writes ~0.7 sectors a
            // cycle whether they are full or not (16-byte stores took twice as long)
            __nv_bfloat16* orow_p = p.o + orow * RA_D + h * 32;
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                x[i] = pack_bf16x2(__uint_as_float(v[e + 2 * i]) * inv, __uint_as_float(v[e + 2 * i + 1]) * inv);
              ra_st32(orow_p + e, x);
            }
          } else if (mine) {
            float* po = p.part_o + (pslot * RA_D + h * 32) * RA_BQ + r * 4;      // lanes side by side
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(po + e * RA_BQ) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
          __syncwarp();                            // the next load is a whole warp's
        }
        if (mine) {
          if (whole) {
            if (p.lse) p.lse[orow] = (m + log2f(l)) * RA_LN2;
          } else {
            *reinterpret_cast<float2*>(p.part_ml + (pslot * RA_BQ + r) * 2) = make_float2(m, l);
          }
        }
      }
      // the next piece's first P V into O follows this warp's next arrival
      tc_fence_before();
      __syncwarp();
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Four CTAs per cut: the item that CTA c's run start cuts, if that is the item's
// first cut with key tiles on both sides, 32 columns each. A lane per row, a warp
// per 8 columns of 32 rows:
//   O = sum_s O_s 2^(m_s - M) / sum_s l_s 2^(m_s - M).
// Pieces lie in CTA order: CTA c - 1's (its last item), then c, c + 1, ... (each
// one's first). Bound by latency: the cut, then the pieces, five at a time (a
// request of 32768 keys has 19 per head, 77 KB: more than one SM fetches at once).
// Small CTAs, since most have no cut and only cost their start: 4 of 128 threads a
// cut; 4 of 256 lost 0.1 to 0.4 us on all but prompts of 200 rows (32.3 against
// 34.1), 1 of 256 was as fast without cuts but 72 against 63 us on the mixed batch.
constexpr int RC_THREADS = 128, RC_SPLIT = 4, RC_COLS = 8;
static_assert(RA_D / RC_SPLIT / RC_COLS == RC_THREADS / 32, "a warp per 8 of a CTA's columns");
__global__ void __launch_bounds__(RC_THREADS, 5) ragged_combine_kernel(const __grid_constant__ RaParams p) {
  pdl_enter();
  const int c = blockIdx.x / RC_SPLIT + 1;
  const RaCut st = p.cuts[c];
  if (st.pieces == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (blockIdx.x % RC_SPLIT) * (RA_D / RC_SPLIT) + warp * RC_COLS;
  auto slot = [&](int s) { return static_cast<int64_t>(c - 1 + s) * 2 + (s == 0 ? st.first_slot : 0); };
  for (int row0 = 0; row0 < st.rows; row0 += 32) {
    const int rows = st.rows - row0;
    // few rows (decoding): the lanes that have none take a share of the pieces
    const int R = rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
    const int r = row0 + (lane & (R - 1));
    // running max over the pieces, as within a piece
    float M = -INFINITY, l = 0.f, a[RC_COLS];
#pragma unroll
    for (int e = 0; e < RC_COLS; ++e) a[e] = 0.f;
    auto add = [&](float m2, float l2, const float (&v)[RC_COLS]) {
      // A piece whose keys this row does not see has the sum 0. Not the maximum: that of
      // scores which are all NaN is -inf too (max drops NaN), and their sum is NaN.
      if (l2 == 0.f) return;
      const float m_new = fmaxf(M, m2), f0 = exp2f(M - m_new), f = exp2f(m2 - m_new);
      M = m_new;
      l = fmaf(l2, f, l * f0);
#pragma unroll
      for (int e = 0; e < RC_COLS; ++e) a[e] = fmaf(v[e], f, a[e] * f0);
    };
    if (r < st.rows) {
      constexpr int U = 5;                         // pieces whose reads are under way together
      for (int s0 = lane / R; s0 < st.pieces; s0 += U * (32 / R)) {
        float2 ml[U];
        float v[U][RC_COLS];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int s = s0 + u * (32 / R);
          ml[u] = make_float2(-INFINITY, 0.f);
          if (s < st.pieces) {
            const int64_t at = slot(s);
            ml[u] = *reinterpret_cast<const float2*>(p.part_ml + (at * RA_BQ + r) * 2);
            const float* po = p.part_o + (at * RA_D + col) * RA_BQ + r * 4;
#pragma unroll
            for (int e = 0; e < RC_COLS / 4; ++e) {
              const float4 x = *reinterpret_cast<const float4*>(po + e * 4 * RA_BQ);
              v[u][4 * e] = x.x; v[u][4 * e + 1] = x.y; v[u][4 * e + 2] = x.z; v[u][4 * e + 3] = x.w;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) add(ml[u].x, ml[u].y, v[u]);
      }
    }
    for (int o = 16; o >= R; o >>= 1) {
      const float m2 = __shfl_down_sync(0xffffffffu, M, o), l2 = __shfl_down_sync(0xffffffffu, l, o);
      float v[RC_COLS];
#pragma unroll
      for (int e = 0; e < RC_COLS; ++e) v[e] = __shfl_down_sync(0xffffffffu, a[e], o);
      if (lane < o) add(m2, l2, v);
    }
    if (lane >= R || r >= st.rows) continue;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int tok = r / p.G;
    const int64_t orow = static_cast<int64_t>(st.row0 + tok) * p.Hq + st.g * p.G + (r - tok * p.G);
    *reinterpret_cast<uint4*>(p.o + orow * RA_D + col) =
        make_uint4(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv),
                   pack_bf16x2(a[4] * inv, a[5] * inv), pack_bf16x2(a[6] * inv, a[7] * inv));
    if (p.lse && col == 0) p.lse[orow] = (M + log2f(l)) * RA_LN2;
  }
}

kl_status ra_map(CUtensorMap* m, int rank, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
  auto fn = tensor_map_encoder();
  if (!fn) return set_error(KL_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(KL_ERR_INVALID_ARG, "ragged attention: tensor map encode failed (%d)", (int)r);
  return KL_OK;
}

struct RaWs {
  size_t o, ml, cuts, total;
};
RaWs ra_ws(int ctas) {
  RaWs w;
  w.o = 0;
  w.ml = w.o + static_cast<size_t>(ctas) * 2 * RA_BQ * RA_D * 4;
  w.cuts = w.ml + align_up(static_cast<size_t>(ctas) * 2 * RA_BQ * 2 * 4, 256);
  w.total = w.cuts + align_up(static_cast<size_t>(ctas) * sizeof(RaCut), 256);
  return w;
}

}  // namespace

size_t ragged_attention_ws() { return ra_ws(num_sms()).total; }

kl_status ragged_attention(const kl_ragged_cfg& rc, int Hq, int Hkv, const void* q, const void* kp, const void* vp,
                           const int32_t* table, const int32_t* cu, const int32_t* ctx, void* o, float* lse, void* ws,
                           size_t ws_bytes, cudaStream_t st) {
  const int ctas = num_sms();
  const RaWs lay = ra_ws(ctas);
  if (!ws || ws_bytes < lay.total || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return set_error(KL_ERR_NO_MEMORY, "ragged attention: workspace too small or not 256-byte aligned");
  RaParams p;
  memset(&p, 0, sizeof(p));
  p.G = Hq / Hkv;
  p.TQ = RA_BQ / p.G;
  const bool tma = rc.block_size % 8 == 0;
  p.box_log = 7;
  while (tma && rc.block_size & ((1 << p.box_log) - 1)) --p.box_log;    // gcd(block_size, 128)
  {
    const cuuint64_t dq[3] = {RA_D, static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(rc.T)};
    const cuuint64_t sq[2] = {RA_D * 2, static_cast<cuuint64_t>(Hq) * RA_D * 2};
    const cuuint32_t bq[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(p.TQ)};
    KL_TRY(ra_map(&p.tmQ, 3, q, dq, sq, bq));
  }
  if (tma) {
    // (64 columns, 8 rows, column blocks, groups of 8 rows)
    const cuuint64_t pitch = static_cast<cuuint64_t>(Hkv) * RA_D * 2;
    const cuuint64_t dk[4] = {64, 8, static_cast<cuuint64_t>(Hkv) * 2,
                              static_cast<cuuint64_t>(rc.n_blocks) * rc.block_size / 8};
    const cuuint64_t sk[3] = {pitch, 128, 8 * pitch};
    const cuuint32_t bk[4] = {64, 8, 2, 1u << (p.box_log - 3)};
    KL_TRY(ra_map(&p.tmK, 4, kp, dk, sk, bk));
    KL_TRY(ra_map(&p.tmV, 4, vp, dk, sk, bk));
  }
  p.kp = static_cast<const __nv_bfloat16*>(kp);
  p.vp = static_cast<const __nv_bfloat16*>(vp);
  p.table = table;
  p.cu = cu;
  p.ctx = ctx;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  uint8_t* wb = static_cast<uint8_t*>(ws);
  p.part_o = reinterpret_cast<float*>(wb + lay.o);
  p.part_ml = reinterpret_cast<float*>(wb + lay.ml);
  p.cuts = reinterpret_cast<RaCut*>(wb + lay.cuts);
  p.B = rc.B;
  p.T = rc.T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.bs = rc.block_size;
  p.max_blocks = rc.max_blocks;
  p.n_blocks = rc.n_blocks;
  p.scale_log2 = RA_LOG2E / sqrtf(static_cast<float>(RA_D));
  p.err = device_error_word();
  static uint64_t attr_done = 0;
  int dev = 0;
  KL_CUDA(cudaGetDevice(&dev));
  if (dev < 64 && !(attr_done >> dev & 1u)) {
    KL_CUDA(cudaFuncSetAttribute(ragged_attn_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(RA_SMEM)));
    KL_CUDA(cudaFuncSetAttribute(ragged_attn_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(RA_SMEM)));
    attr_done |= uint64_t(1) << dev;
  }
  {
    // the lengths are on the device: the rows' queries and outputs are what the host knows of the traffic
    ProfScope ps("ragged_attention", st, 0.0, 4.0 * rc.T * Hq * RA_D);
    if (tma)
      launch_pdl(ragged_attn_kernel<true>, ctas, RA_THREADS, RA_SMEM, st, p);
    else
      launch_pdl(ragged_attn_kernel<false>, ctas, RA_THREADS, RA_SMEM, st, p);
  }
  KL_CUDA(cudaGetLastError());
  if (ctas > 1) {
    ProfScope ps("ragged_combine", st, 0.0, 4.0 * ctas * RA_D);
    launch_pdl(ragged_combine_kernel, (ctas - 1) * RC_SPLIT, RC_THREADS, 0, st, p);
    KL_CUDA(cudaGetLastError());
  }
  return KL_OK;
}

}  // namespace kl
