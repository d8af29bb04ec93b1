// What the attention kernels of a ragged step share: how the step's work is cut into
// runs of key tiles, one a CTA, the walk over a run, and the join of items that were
// cut. (A query tile is floor(128 / G) tokens x G heads of one kv head, a key tile 128
// keys.)
#pragma once

#include <cudaTypedefs.h>
#include <math.h>

#include "internal.h"
#include "kl_common.cuh"

namespace kl {

constexpr int RA_D = 128;        // head dim
constexpr int RA_BQ = 128;       // rows of a query tile
constexpr int RA_BKV = 128;      // keys per tile
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

// Pieces of cut items, as the attention kernels leave them and the joining kernel reads them.
struct RaJoin {
  float* part_o;         // [CTA][2][32][128][4] unnormalised pieces: 4 columns of the 128 rows together
  float* part_ml;        // [CTA][2][128][2] (max in log2 units, sum)
  RaCut* cuts;           // [CTA]
  __nv_bfloat16* o;
  float* lse;            // [T, Hq] or null
  int Hq, G;
};
// Joins the pieces of a launch of `ctas` CTAs (ragged_attn.cu).
kl_status ragged_join(const RaJoin& j, int ctas, cudaStream_t st);

struct RaWs {
  size_t o, ml, cuts, total;
};
inline RaWs ra_ws(int ctas) {
  RaWs w;
  w.o = 0;
  w.ml = w.o + static_cast<size_t>(ctas) * 2 * RA_BQ * RA_D * 4;
  w.cuts = w.ml + align_up(static_cast<size_t>(ctas) * 2 * RA_BQ * 2 * 4, 256);
  w.total = w.cuts + align_up(static_cast<size_t>(ctas) * sizeof(RaCut), 256);
  return w;
}

inline kl_status ra_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box, CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  auto fn = tensor_map_encoder();
  if (!fn) return set_error(KL_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, type, rank, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(KL_ERR_INVALID_ARG, "ragged attention: tensor map encode failed (%d)", (int)r);
  return KL_OK;
}

__device__ __forceinline__ float ra_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
static __device__ __noinline__ long long ra_units_before(int ctx, int TQ, long long m) {
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
static __device__ __noinline__ long long ra_div(long long a, long long b) {
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
static __device__ __noinline__ void ra_next(const RaLens p, const RaWalk& from, RaWalk& to, RaPiece& piece) {
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

// This CTA's run, found by all its threads: prefix sums of the requests' units, then
// the item at unit cta * P, its place and the walk to the first piece. Returns P. The
// caller synchronises the block before it reads what was found.
template <int WARPS>
__device__ __forceinline__ long long ra_find_run(const RaLens& p, int cta, int ctas, long long* wsum, RaFound* found,
                                                 RaPiece* first, RaWalk* walk) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.B + 32 * WARPS - 1) / (32 * WARPS);
  const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
  long long mine = 0, units = 0;
  RaReq q = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    q = ra_req(p, b);
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
  for (int w = 0; w < WARPS; ++w) {
    const long long v = wsum[w];
    if (w < warp) before += v;
    W += v;
  }
  const long long P = max(ra_div(W + ctas - 1, ctas), 1LL);
  const long long u0 = cta * P;
  if (threadIdx.x == 0 && u0 >= W) {
    found->any = 0;
    first->tb = 0;
  }
  long long lo = before + incl - mine;      // units before this thread's requests
  if (mine > 0 && u0 >= lo && u0 < lo + mine) {
    int b = b0;
    if (per > 1) {                          // with one request a thread q and units are its own still
      for (;; ++b) {
        q = ra_req(p, b);
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
    ra_step(p, w, c);
    *first = c;
    *walk = w;
    *found = {1, g, m0, q, off};
  }
  return P;
}

}  // namespace kl
