// Attention of a ragged step over a paged cache of 8-bit codes with a scale for each
// page and head, on the 5th-generation tensor cores:
//   o_i = sum_j softmax_j(q_i . (a_j kc_j) / sqrt(d)) b_j vc_j,
// kc_j, vc_j the e4m3 codes of position j and a_j, b_j its page's scales.
//
// Exact products in 8 bits. Keys and values go to the tensor cores as they are cached,
// nothing is converted: half the bytes of a bf16 cache in HBM and in shared memory. The
// other operands are split. A bf16 query has 8 significant bits, which two e4m3
// numbers hold (row scaled by a power of two so that its largest element is in [128,
// 256); hi is the nearest e4m3, the rest has 4 bits: exact down to 2^-10 of the
// largest, off by 2^-17 of it below). e4m3 products run at twice the bf16 rate, so S =
// hi K^T + lo K^T takes the time of one bf16 product. Weights likewise: 4 bits by
// cutting, the rest rounded to 4, off by 2^-8 at most as a bf16 weight is.
//
// Scales. t_j = s_j a_j + log2 b_j is what the running maximum m is taken of, and P'_j =
// 2^(t_j - m + 6) = 2^(6 - m) p_j b_j goes into the product with the values' codes: its
// range does not depend on how the pages' scales differ. The row's sum adds P'_j / b_j.
// m is raised when t exceeds it by more than 2.5, so P' stays below 2^8.5 < 448. A
// weight below 2^-12 of the row's largest is off by 2^-16 of that one at most.
//
// Work split, walk and join are those of the bf16 kernel (ragged_walk.cuh): query tiles
// of floor(128 / G) tokens x G heads, runs of key tiles of 128 keys, one CTA per SM,
// pieces of cut items joined in CTA order: results repeat bit for bit.
//
// Roles (8 warps): warp 0 copies the keys, warp 1 the values and looks up the scales,
// warp 2 issues the score products and, between two of them, splits the next piece's
// queries, warp 3 issues the P V products, warps 4..11 are the softmax (thread = query row
// = TMEM lane and half of the tile's keys; idle at first, they split the first piece's
// queries). Two warps share an SM quarter's instruction issue, which one could not fill:
// with four softmax warps a step took 2900 cycles. They tell each other their row maxima.
// Barriers, stages and buffers as in the bf16
// kernel. A key tile of 16 KB is 16 groups of 8 keys x 128 bytes (one swizzle atom each);
// with block_size a multiple of 8 it is 128 / box TMA boxes, box = gcd(block_size, 128),
// and a scale serves whole groups; other block sizes go row by row with 16-byte cp.async
// and have a scale per key.
#include <string.h>

#include <type_traits>

#include "e4m3.cuh"
#include "ragged_walk.cuh"

namespace kl {
namespace {

constexpr int A8_WARPS = 12;
constexpr int A8_THREADS = 32 * A8_WARPS;
constexpr uint32_t A8_TILE = 128 * 128;       // a tile of keys, of values, of one part of the queries
constexpr int A8_NST = 4;                     // stages of the K and of the V ring
constexpr int A8_SCR = 4;                     // tiles in the ring of scales
constexpr uint32_t A8_OFF_Q = 0;              // two pieces' queries, high and low parts
constexpr uint32_t A8_OFF_K = A8_OFF_Q + 4 * A8_TILE;
constexpr uint32_t A8_OFF_V = A8_OFF_K + A8_NST * A8_TILE;
constexpr uint32_t A8_OFF_BAR = A8_OFF_V + A8_NST * A8_TILE;
constexpr uint32_t A8_OFF_QS = A8_OFF_BAR + 2560;           // the rows' factors, of four pieces
constexpr uint32_t A8_OFF_X = A8_OFF_QS + 4 * RA_BQ * 4;    // what the halves of a row tell each other
constexpr uint32_t A8_OFF_SC = A8_OFF_X + 4 * RA_BQ * 4;    // the ring of scales
constexpr size_t a8_smem(bool tma) { return 1024 + A8_OFF_SC + A8_SCR * 3 * (tma ? 16 : 128) * 4; }
// Tensor memory: S of two steps, P of two steps (high and low parts), O: all 512 columns.
constexpr uint32_t A8_TM_P = 256, A8_TM_O = 384;
constexpr float A8_LIFT = 6.0f;               // P' of the running maximum is 2^6 ...
constexpr float A8_LAG = 2.5f;                // ... to 2^8.5

struct A8Params {
  CUtensorMap tmK, tmV;
  const __nv_bfloat16* q;
  const uint8_t* kp;
  const uint8_t* vp;
  const float* ks;
  const float* vs;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* ctx;
  RaJoin j;              // o, lse and the pieces of cut items
  int B, T, Hq, Hkv, G, TQ;
  int bs, max_blocks, n_blocks;
  int box_log;           // log2 of the rows per TMA box (8 .. 128)
  float scale_log2;
  uint32_t* err;
};

// Queries and keys, K-major in groups of 8 rows 1 KB apart, k-step kk of 32 columns
__device__ __forceinline__ uint64_t a8_desc_k(uint32_t base, int kk) { return smem_desc_sw128(base + kk * 32, 16, 1024); }
// Values as the MN-major B operand: n = head dim, 128 bytes; k-step kk of 32 keys = four groups
__device__ __forceinline__ uint64_t a8_desc_v(uint32_t base, int kk) { return smem_desc_sw128(base + kk * 4096, 1024, 1024); }

__device__ __forceinline__ uint64_t a8_sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// max that a NaN survives
__device__ __forceinline__ float a8_max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float4 a8_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

template <bool TMA>
__global__ void __launch_bounds__(A8_THREADS, 1) ragged_attn8_kernel(const __grid_constant__ A8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar = sb + A8_OFF_BAR;
  auto q_full = [&](int k) { return bar + 0 + 8 * (k & 3); };      // piece k's queries: four, so that no
                                                                   // waiter is two phases behind
  auto q_empty = [&](int k) { return bar + 32 + 8 * (k & 1); };    // its last S product is done with them
  auto k_full = [&](int s) { return bar + 48 + 8 * s; };
  auto k_empty = [&](int s) { return bar + 80 + 8 * s; };
  auto v_full = [&](int s) { return bar + 112 + 8 * s; };
  auto v_empty = [&](int s) { return bar + 144 + 8 * s; };
  auto s_full = [&](int s) { return bar + 176 + 8 * s; };   // S_n computed
  auto s_free = [&](int s) { return bar + 192 + 8 * s; };   // S_n read
  auto p_full = [&](int s) { return bar + 208 + 8 * s; };   // P_n written (and V_n's tail cleared)
  auto p_done = [&](int s) { return bar + 224 + 8 * s; };   // O += P_n V_n computed
  auto sc_full = [&](int n) { return bar + 240 + 8 * (n & (A8_SCR - 1)); };    // the tile's scales written
  const uint32_t drain = bar + 272, drain_pv = bar + 280, q_first = bar + 288;   // the first piece's queries
  auto told = [&](int q, int x) { return bar + 296 + 16 * q + 8 * (x & 1); };   // both halves of quarter q's rows have spoken
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + A8_OFF_BAR + 360);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + A8_OFF_BAR + 364);
  RaFound* found = reinterpret_cast<RaFound*>(smem + A8_OFF_BAR + 368);
  long long* wsum = reinterpret_cast<long long*>(smem + A8_OFF_BAR + 432);
  RaWalk* walks = reinterpret_cast<RaWalk*>(smem + A8_OFF_BAR + 528);        // the finder's, then one per warp
  RaPiece* pieces = reinterpret_cast<RaPiece*>(smem + A8_OFF_BAR + 1152);    // the first one, then two per warp
  static_assert(sizeof(RaFound) <= 64 && A8_WARPS * 8 <= 96 && (A8_WARPS + 1) * sizeof(RaWalk) <= 624 && (A8_WARPS * 2 + 1) * sizeof(RaPiece) <= 1408,
                "shared-memory layout");
  float* qscale = reinterpret_cast<float*>(smem + A8_OFF_QS);
  constexpr int GRP = TMA ? 8 : 1;               // keys that share a scale
  constexpr int NG = RA_BKV / GRP;
  const uint32_t sc0 = sb + A8_OFF_SC;           // [tile][a, log2 b, 1 / b][group]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const RaLens lens = {p.cu, p.ctx, p.B, p.T, p.Hkv, p.TQ};

  if (warp == 3 && lane == 0) {
    for (int k = 0; k < 4; ++k) mbar_init(q_full(k), 1);
    mbar_init(q_first, 8);
    for (int k = 0; k < 8; ++k) mbar_init(told(k >> 1, k), 2);
    for (int k = 0; k < 2; ++k) mbar_init(q_empty(k), 1);
    for (int s = 0; s < A8_NST; ++s) {
      mbar_init(k_full(s), TMA ? 1 : 32);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), TMA ? 1 : 32);
      mbar_init(v_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(s_free(s), 8);
      mbar_init(p_full(s), 8);
      mbar_init(p_done(s), 1);
    }
    for (int n = 0; n < A8_SCR; ++n) mbar_init(sc_full(n), 1);
    mbar_init(drain, 1);
    mbar_init(drain_pv, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  if (TMA && lane == 0 && (warp == 6 || warp == 7)) tma_prefetch_desc(warp == 6 ? &p.tmK : &p.tmV);

  pdl_enter();      // nothing above reads what an earlier kernel writes

  const long long P = ra_find_run<A8_WARPS>(lens, cta, ctas, wsum, found, &pieces[0], &walks[0]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tmP = tmem + A8_TM_P, tmO = tmem + A8_TM_O;

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
  auto page = [&](int b, int lb) { return lb < p.max_blocks ? p.table[static_cast<int64_t>(b) * p.max_blocks + lb] : -1; };
  // Queries, two rows at a time, 16 lanes each: row r0 + (lane >> 4) of a piece with `rows` of them ...
  auto load_q = [&](const RaPiece& c, int rows, int r0) {
    const int r = r0 + (lane >> 4), tok = r / p.G;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows)
      x = *reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(c.row0 + tok) * p.Hq + c.g * p.G + (r - tok * p.G)) * RA_D + (lane & 15) * 8);
    return x;
  };
  // ... split into its two parts, and its factor, into piece k's places.
  auto split_q = [&](const uint4& x, int k, int rows, int r0) {
    const int r = r0 + (lane >> 4), j = lane & 15;
    const float2 f0 = unpack_bf16x2(x.x), f1 = unpack_bf16x2(x.y), f2 = unpack_bf16x2(x.z), f3 = unpack_bf16x2(x.w);
    // the largest size, as bits: an infinity or a NaN is above all numbers
    auto size = [](float a, float b) { return max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu); };
    uint32_t a = max(max(size(f0.x, f0.y), size(f1.x, f1.y)), max(size(f2.x, f2.y), size(f3.x, f3.y)));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    const int e = max(static_cast<int>(a >> 23) - 127, -110);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
    auto split = [&](const float2& s, const float2& t, uint32_t& hi4, uint32_t& lo4) {
      const float x0 = s.x * up, x1 = s.y * up, x2 = t.x * up, x3 = t.y * up;
      hi4 = e4m3x4(x0, x1, x2, x3);
      const float4 h = e4m3x4_to_f(hi4);
      lo4 = e4m3x4(x0 - h.x, x1 - h.y, x2 - h.z, x3 - h.w);
    };
    uint2 h, l;
    split(f0, f1, h.x, l.x);
    split(f2, f3, h.y, l.y);
    if (r < rows) {
      const uint32_t at = sb + A8_OFF_Q + (k & 1) * 2 * A8_TILE + r * 128 + (((j >> 1) ^ (r & 7)) << 4) + (j & 1) * 8;
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(h.x), "r"(h.y) : "memory");
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + A8_TILE), "r"(l.x), "r"(l.y) : "memory");
      if (j == 0) qscale[(k & 3) * RA_BQ + r] = a >= 0x7f800000u ? __int_as_float(0x7fffffff) : down * p.scale_log2;
    }
  };

  if (warp < 2) {
    // ------- copies (warp 0: K, warp 1: V; lane = page box of a tile) -------
    const bool is_k = warp == 0;
    const bool el = elect_one();
    const CUtensorMap* tm = is_k ? &p.tmK : &p.tmV;
    const uint8_t* pool = is_k ? p.kp : p.vp;
    const uint32_t ring = sb + (is_k ? A8_OFF_K : A8_OFF_V);
    const uint32_t full0 = is_k ? k_full(0) : v_full(0), empty0 = is_k ? k_empty(0) : v_empty(0);
    // rows of a box, boxes of a tile, tiles of a look-up, this lane's one
    const int box = 1 << p.box_log, nbox = RA_BKV >> p.box_log, per = box >> 2, my = lane >> (7 - p.box_log);
    const int no_row = p.n_blocks * p.bs;         // past the pool's last row: filled with zeros
    int issued = 0, s = 0, as = 0;                // s: the ring's stage; as: the next one to announce
    uint32_t ph = 1;                              // parity that an empty stage's wait passes with
    bool ok = true;
    // the pool row of a position at `at` of its page blk, or no_row
    auto pool_row = [&](int blk, int at) {
      if (blk >= 0 && blk < p.n_blocks) return blk * p.bs + at;
      record_error(p.err, KL_DEVERR_PAGE);
      return no_row;
    };
    // cp.async: the rows of one tile; row[k] of lane l is the pool row of key 32 k + l
    auto gather = [&](uint32_t dst, int g, const int (&row)[4]) {
      const int ch = lane & 7;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int key = 32 * k + 4 * it + (lane >> 3);
          const int src = __shfl_sync(0xffffffffu, row[k], 4 * it + (lane >> 3));
          const bool valid = src != no_row;
          ra_cp16(dst + key * 128 + ((ch ^ (key & 7)) << 4),
                  pool + (static_cast<int64_t>(valid ? src : 0) * p.Hkv + g) * RA_D + ch * 16, valid);
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
      as = as == A8_NST - 1 ? 0 : as + 1;
    };
    // Warp 1: the scales of the next tile in line, from a batch's lanes (TMA; `which` of its tiles) or a
    // lane's four keys, into the ring. Its entry is free: the copies wait for the product of four tiles before.
    float a[4] = {1.f, 1.f, 1.f, 1.f}, b[4] = {1.f, 1.f, 1.f, 1.f};
    int tile = 0;
    auto publish = [&](int which) {
      if (is_k) return;
      float* sc = reinterpret_cast<float*>(smem + A8_OFF_SC) + (tile & (A8_SCR - 1)) * 3 * NG;
      if (TMA) {
        if (my == which) {
          const float lb = log2f(b[0]), ib = 1.f / b[0];
          const int gs = box >> 3, g0 = (lane & (nbox - 1)) * gs;
          for (int g = g0; g < g0 + gs; ++g) {
            sc[g] = a[0];
            sc[NG + g] = lb;
            sc[2 * NG + g] = ib;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[(i * 32 + lane) % NG] = a[i];
          sc[NG + (i * 32 + lane) % NG] = log2f(b[i]);
          sc[2 * NG + (i * 32 + lane) % NG] = 1.f / b[i];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sc_full(tile));
      ++tile;
    };
    for (int k = 0; ok && find(k); ++k) {
      const RaPiece w = piece(k);
      // TMA: one look at the table serves `per` tiles, a lane per box, and the next
      // tiles' pages are asked for before these are copied. cp.async: a lane for four
      // of a tile's keys.
      int row[4], blk = 0, at = 0;
      const int keys = min(w.L, w.tb * RA_BKV);
      auto ask = [&](int j) {
        const int pos = j * RA_BKV + lane * box, lb = pos / p.bs;
        at = pos < keys ? pos - lb * p.bs : -1;
        if (at >= 0) blk = page(w.b, lb);
      };
      auto scales = [&](int i, int blk, bool there) {
        a[i] = b[i] = 1.f;                         // a page that is read as zero has none
        if (is_k || !there) return;
        const int64_t at = static_cast<int64_t>(blk) * p.Hkv + w.g;
        a[i] = p.ks[at];
        b[i] = p.vs[at];
      };
      auto lookup = [&](int j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = j * RA_BKV + i * 32 + lane, lb = pos / p.bs;
          const int pg = pos < keys ? page(w.b, lb) : 0;
          row[i] = pos < keys ? pool_row(pg, pos - lb * p.bs) : no_row;
          scales(i, pg, row[i] != no_row);
        }
      };
      if (TMA) ask(w.ta); else lookup(w.ta);
      for (int j = w.ta; j < w.tb; ++j) {
        const int nth = (j - w.ta) & (per - 1);
        if (TMA && nth == 0) {
          row[0] = at >= 0 ? pool_row(blk, at) : no_row;
          if (j > w.ta) publish(per - 1);          // the batch before is no longer at hand
          scales(0, blk, row[0] != no_row);
          if (j + per < w.tb) ask(j + per);
        }
        if (!ra_wait_copy(empty0 + 8 * s, ph, p.err, abort_flag)) { ok = false; break; }
        const uint32_t dst = ring + s * A8_TILE;
        if (TMA) {
          if (el) mbar_arrive_expect_tx(full0 + 8 * s, A8_TILE);
          __syncwarp();
          if (my == nth) ra_tma_3d(dst + (lane & (nbox - 1)) * box * 128, tm, 0, w.g, row[0], full0 + 8 * s);
          __syncwarp();
          if (nth > 0) publish(nth - 1);          // a tile later: the reads have had the time
        } else {
          gather(dst, w.g, row);
          publish(0);
          if (j > w.ta) announce(std::integral_constant<int, 1>());   // the tile before
        }
        ++issued;
        if (++s == A8_NST) {
          s = 0;
          ph ^= 1u;
        }
        if (!TMA && j + 1 < w.tb) lookup(j + 1);
      }
      if (TMA && ok) publish((w.tb - 1 - w.ta) & (per - 1));
      // the piece's last tile: its products free Q, which the next piece waits for
      if (!TMA && ok) announce(std::integral_constant<int, 0>());
    }
    if (!ok) *abort_flag = 1;
    // copies still in flight must land before exit
    if (TMA) {
      for (int j = max(0, issued - A8_NST); j < issued; ++j) mbar_wait(full0 + 8 * (j % A8_NST), (j / A8_NST) & 1, p.err);
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  } else if (warp == 2) {
    // ---------- S_n = hi K_n^T + lo K_n^T into S[n % 2] (whole warp; the elected lane issues) ----------
    const bool el = elect_one();
    const uint32_t idesc = idesc_e4m3_f32(128, 128, 0, 0);
    int n = 0, ks = 0;                        // step, K stage
    uint32_t kph = 0;
    bool ok = true, have = find(0);
    if (have && !mbar_wait_warp(q_first, 0, p.err, abort_flag)) ok = false;
    for (int k = 0; ok && have; ++k) {
      const int tiles = piece(k).tb - piece(k).ta;
      const uint32_t qb = sb + A8_OFF_Q + (k & 1) * 2 * A8_TILE;
      // The next piece's queries are split between this one's products, sixteen rows at a time; the
      // next sixteen are on their way meanwhile.
      have = find(k + 1);
      constexpr int U = 8;
      uint4 x[U];
      int at = 0, rows = 0;
      if (have) rows = piece(k + 1).toks * p.G;
      auto load = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (at + 2 * u < rows) x[u] = load_q(piece(k + 1), rows, at + 2 * u);
      };
      auto split = [&]() -> bool {
        // the buffer is free once the S products of the piece before this one are done
        if (at == 0 && k > 0 && !mbar_wait_warp(q_empty(k + 1), ((k - 1) >> 1) & 1, p.err, abort_flag)) return false;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (at + 2 * u < rows) split_q(x[u], k + 1, rows, at + 2 * u);
        at += 2 * U;
        load();
        return true;
      };
      load();
      for (int j = 0; j < tiles; ++j, ++n) {
        const int s = n & 1;
        if ((n >= 2 && !mbar_wait_warp(s_free(s), ((n >> 1) & 1) ^ 1u, p.err, abort_flag)) ||
            !mbar_wait_warp(k_full(ks), kph, p.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (el) {
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t kd = a8_desc_k(sb + A8_OFF_K + ks * A8_TILE, kk);
            umma_e4m3(tmem + s * 128, a8_desc_k(qb, kk), kd, idesc, kk > 0);
            umma_e4m3(tmem + s * 128, a8_desc_k(qb + A8_TILE, kk), kd, idesc, 1u);
          }
          umma_commit(s_full(s));
          umma_commit(k_empty(ks));
          if (j == tiles - 1) umma_commit(q_empty(k));   // the piece's last use of Q
        }
        __syncwarp();
        if (++ks == A8_NST) {
          ks = 0;
          kph ^= 1u;
        }
        if (at < rows && !split()) { ok = false; break; }
      }
      while (ok && at < rows) ok = split();
      if (ok && have) {
        for (int r = rows + lane; r < ((rows + 31) & ~31); r += 32) qscale[((k + 1) & 3) * RA_BQ + r] = 0.f;   // no rows: no factor
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full(k + 1));
      }
    }
    if (!ok) *abort_flag = 1;
    if (el) umma_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, p.err);
  } else if (warp == 3) {
    // ---------- O (+)= P_n V_n, both parts (whole warp; the elected lane issues) ----------
    const bool el = elect_one();
    const uint32_t idesc = idesc_e4m3_f32(128, 128, 0, 1);
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
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t vd = a8_desc_v(sb + A8_OFF_V + vs * A8_TILE, kk);
            umma_e4m3_ta(tmO, tmP + s * 64 + kk * 8, vd, idesc, (j > 0 || kk > 0) ? 1u : 0u);
            umma_e4m3_ta(tmO, tmP + s * 64 + 32 + kk * 8, vd, idesc, 1u);
          }
          umma_commit(p_done(s));
          umma_commit(v_empty(vs));
        }
        __syncwarp();
        if (++vs == A8_NST) {
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
    const int quarter = warp & 3, half = (warp >> 2) - 1;
    const int r = quarter * 32 + lane;           // row within the tile = TMEM lane
    constexpr int KEYS = RA_BKV / 2;             // keys 64 half .. 64 half + 63 of each tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t oadr = tmO + lane_off + half * 64, padr = tmP + lane_off + half * 16;
    float* said = reinterpret_cast<float*>(smem + A8_OFF_X);    // [exchange % 2][half][row]
    // The tile that holds the last key the query tile sees: its value rows behind it become zero
    // (each of the eight warps half of its 32).
    auto clear_tail = [&](int end, int n) -> bool {
      if (end >= RA_BKV) return true;
      const int vs = n % A8_NST;
      if (!mbar_wait_warp(v_full(vs), (n / A8_NST) & 1, p.err, abort_flag)) return false;
      if (r >= end) {
        const uint32_t va = sb + A8_OFF_V + vs * A8_TILE + r * 128 + half * 64;
#pragma unroll
        for (int c = 0; c < 4; ++c) st_shared_v4(va + c * 16, 0u, 0u, 0u, 0u);
      }
      fence_async_shared();
      return true;
    };
    bool more = find(0);
    if (more) {
      // the first piece's queries, each warp 16 rows
      const RaPiece& c = piece(0);
      const int r0 = quarter * 32 + half * 16, all = c.toks * p.G, rows = min(all, r0 + 16);
      for (int at = r0; at < rows; at += 8) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = load_q(c, rows, at + 2 * u);
#pragma unroll
        for (int u = 0; u < 4; ++u) split_q(x[u], 0, rows, at + 2 * u);
      }
      if (half == 0 && r >= all) qscale[r] = 0.f;  // no row: no factor
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_first);
    }
    // the cut at this CTA's start, by a warp that has little to do yet
    if (warp == 11 && lane == 31) {
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
      p.j.cuts[cta] = cut;
    }
    __syncwarp();
    bool ok = true;
    int n = 0, x = 0;                              // steps and exchanges so far
    float m = -INFINITY, l = 0.f;                  // the row's running max of t (log2 units), this half's sum of P' / b
    float rs = 0.f;                                // the row's factor: score in log2 units = S * rs * a
    int lim = 0, end = 0;                          // the row's last key, from this half's first; the end of the query tile's, from the tile's
    // v to the other half of the row, the other half's into v
    auto exchange = [&](float& v) -> bool {
      float* at = said + (x & 1) * 2 * RA_BQ + r;
      at[half * RA_BQ] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(told(quarter, x));
      if (!mbar_wait_warp(told(quarter, x), (x >> 1) & 1, p.err, abort_flag)) return false;
      v = at[(half ^ 1) * RA_BQ];
      ++x;
      return true;
    };
    // One step of a warp with rows. CUT: some row of the tile ends inside its keys.
    auto step = [&](auto cut, bool first) -> bool {
      constexpr bool CUT = decltype(cut)::value;
      const int s = n & 1;
      if (CUT && TMA && !clear_tail(end, n)) return false;
      if (!mbar_wait_warp(s_full(s), (n >> 1) & 1, p.err, abort_flag)) return false;
      tc_fence_after();
      const uint32_t sadr = tmem + lane_off + s * 128 + half * KEYS;
      uint32_t sv[KEYS];
      tmem_ld_32x32b_x32(sadr, *reinterpret_cast<uint32_t(*)[32]>(sv));
      tmem_ld_32x32b_x32(sadr + 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32));
      // P's columns are free once the product of step n - 2 is done: probed here,
      // where the probe's latency costs nothing, and most likely it is
      const uint32_t done_ph = ((n >> 1) & 1) ^ 1u;
      const bool p_ready = n < 2 || mbar_test_wait(p_done(s), done_ph);
      const bool sc_ok = mbar_wait_warp(sc_full(n), (n / A8_SCR) & 1, p.err, abort_flag);
      // this half's scales; what takes S of a group to the score (with keys cut off never zero, so
      // that their -inf stays)
      constexpr int HG = KEYS / GRP;
      const uint32_t sca = sc0 + (n & (A8_SCR - 1)) * 3 * NG * 4 + half * HG * 4;
      auto factor = [&](float a) { return CUT ? a8_max_nan(rs * a, 1.17549435e-38f) : rs * a; };
      float f[TMA ? HG : 1], lb[TMA ? HG : 1];
      if (TMA && sc_ok) {
#pragma unroll
        for (int g = 0; g < HG; g += 4) {
          const float4 a4 = a8_ld4(sca + g * 4), l4 = a8_ld4(sca + (NG + g) * 4);
          f[g % (TMA ? HG : 1)] = factor(a4.x);
          f[(g + 1) % (TMA ? HG : 1)] = factor(a4.y);
          f[(g + 2) % (TMA ? HG : 1)] = factor(a4.z);
          f[(g + 3) % (TMA ? HG : 1)] = factor(a4.w);
          lb[g % (TMA ? HG : 1)] = l4.x;
          lb[(g + 1) % (TMA ? HG : 1)] = l4.y;
          lb[(g + 2) % (TMA ? HG : 1)] = l4.z;
          lb[(g + 3) % (TMA ? HG : 1)] = l4.w;
        }
      }
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (!sc_ok) return false;
      if (lane == 0) mbar_arrive(s_free(s));       // S[s] may be overwritten from here on
      if (CUT) {                                   // keys 0 .. lim are kept
#pragma unroll
        for (int e = 0; e < KEYS; ++e)
          if (e > lim) sv[e] = __float_as_uint(-INFINITY);
      }
      float mx = -INFINITY;
      if (TMA) {
        float t[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const uint32_t* y = sv + g * 8;
          float v = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
          v = ra_max3(v, y[2], y[3]);
          v = ra_max3(v, y[4], y[5]);
          v = ra_max3(v, y[6], y[7]);
          t[g] = fmaf(v, f[g % (TMA ? HG : 1)], lb[g % (TMA ? HG : 1)]);
        }
#pragma unroll
        for (int g = 0; g < 8; g += 2) mx = ra_max3(mx, __float_as_uint(t[g]), __float_as_uint(t[g + 1]));
      } else {
        // t itself, in place of S
#pragma unroll
        for (int e = 0; e < KEYS; e += 4) {
          const float4 a4 = a8_ld4(sca + e * 4), l4 = a8_ld4(sca + (NG + e) * 4);
          float t[4] = {fmaf(__uint_as_float(sv[e]), factor(a4.x), l4.x), fmaf(__uint_as_float(sv[e + 1]), factor(a4.y), l4.y),
                        fmaf(__uint_as_float(sv[e + 2]), factor(a4.z), l4.z), fmaf(__uint_as_float(sv[e + 3]), factor(a4.w), l4.w)};
          mx = ra_max3(mx, __float_as_uint(t[0]), __float_as_uint(t[1]));
          mx = ra_max3(mx, __float_as_uint(t[2]), __float_as_uint(t[3]));
#pragma unroll
          for (int u = 0; u < 4; ++u) sv[e + u] = __float_as_uint(t[u]);
        }
      }
      {
        float other = mx;
        if (!exchange(other)) return false;
        mx = fmaxf(mx, other);
      }
      // A row of a later piece's tile can be fully masked (its token ends before these
      // keys): mx = -inf, and m stays -inf.
      const bool raise = mx > m + A8_LAG;
      if (__any_sync(0xffffffffu, raise)) {
        const float m_new = raise ? mx : m;
        const float alpha = raise ? ra_ex2(m - m_new) : 1.0f;
        m = m_new;
        l *= alpha;
        if (!first) {
          if (!mbar_wait_warp(p_done(s ^ 1), ((n - 1) >> 1) & 1, p.err, abort_flag)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {            // this half's columns of O
            uint32_t v[16];
            tmem_ld_32x32b_x16(oadr + c * 16, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            tmem_st_32x32b_x16(oadr + c * 16, v);
          }
        }
      }
      const float neg = m > -INFINITY ? A8_LIFT - m : 0.f;
      uint64_t r0 = 0, r1 = 0;
      uint32_t ph[16], pl[16];
      // four weights: their sum's halves, both parts
      auto weights = [&](int w, uint64_t x0, uint64_t x1, uint64_t& y0, uint64_t& y1) {
        float p0, p1, p2, p3;
        ra_unpair(x0, p0, p1);
        ra_unpair(x1, p2, p3);
        const uint32_t u0 = __float_as_uint(ra_ex2(p0)), u1 = __float_as_uint(ra_ex2(p1)), u2 = __float_as_uint(ra_ex2(p2)), u3 = __float_as_uint(ra_ex2(p3));
        y0 = ra_pair(u0, u1);
        y1 = ra_pair(u2, u3);
        // four bits kept, the rest rounded to four
        constexpr uint32_t KEEP = 0xfff00000u;
        ph[w] = e4m3x4(__uint_as_float(u0 & KEEP), __uint_as_float(u1 & KEEP), __uint_as_float(u2 & KEEP), __uint_as_float(u3 & KEEP));
        float d0, d1, d2, d3;
        ra_unpair(a8_sub2(y0, ra_pair(u0 & KEEP, u1 & KEEP)), d0, d1);
        ra_unpair(a8_sub2(y1, ra_pair(u2 & KEEP, u3 & KEEP)), d2, d3);
        pl[w] = e4m3x4(d0, d1, d2, d3);
      };
      if (TMA) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const uint32_t* v = sv + g * 8;
          float ib;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ib) : "r"(sca + (2 * NG + g) * 4));
          const uint32_t fu = __float_as_uint(f[g % (TMA ? HG : 1)]), cu = __float_as_uint(lb[g % (TMA ? HG : 1)] + neg), iu = __float_as_uint(ib);
          const uint64_t f2 = ra_pair(fu, fu), c2 = ra_pair(cu, cu), iv2 = ra_pair(iu, iu);
          uint64_t y0, y1, y2, y3;
          weights(2 * g, ra_fma2(ra_pair(v[0], v[1]), f2, c2), ra_fma2(ra_pair(v[2], v[3]), f2, c2), y0, y1);
          weights(2 * g + 1, ra_fma2(ra_pair(v[4], v[5]), f2, c2), ra_fma2(ra_pair(v[6], v[7]), f2, c2), y2, y3);
          r0 = ra_fma2(ra_add2(y0, y1), iv2, r0);
          r1 = ra_fma2(ra_add2(y2, y3), iv2, r1);
        }
      } else {
        const uint64_t neg2 = ra_pair(__float_as_uint(neg), __float_as_uint(neg));
#pragma unroll
        for (int e = 0; e < KEYS; e += 4) {
          const float4 ib = a8_ld4(sca + (2 * NG + e) * 4);
          uint64_t y0, y1;
          weights(e / 4, ra_add2(ra_pair(sv[e], sv[e + 1]), neg2), ra_add2(ra_pair(sv[e + 2], sv[e + 3]), neg2), y0, y1);
          r0 = ra_fma2(y0, ra_pair(__float_as_uint(ib.x), __float_as_uint(ib.y)), r0);
          r1 = ra_fma2(y1, ra_pair(__float_as_uint(ib.z), __float_as_uint(ib.w)), r1);
        }
      }
      float a0, a1, a2, a3;
      ra_unpair(r0, a0, a1);
      ra_unpair(r1, a2, a3);
      l += (a0 + a1) + (a2 + a3);
      if (!__all_sync(0xffffffffu, p_ready) && !mbar_wait_warp(p_done(s), done_ph, p.err, abort_flag)) return false;
      tc_fence_after();
      tmem_st_32x32b_x16(padr + s * 64, ph);
      tmem_st_32x32b_x16(padr + s * 64 + 32, pl);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(s));
      lim -= RA_BKV;
      end -= RA_BKV;
      ++n;
      return true;
    };
    for (int k = 0; ok && more; ++k) {
      int left, whole;                             // tiles left; those that every row sees whole
      bool busy;
      {
        const RaPiece& c = piece(k);
        left = c.tb - c.ta;
        const int over = c.pos0 - c.ta * RA_BKV;   // the tile's first row's last key
        whole = min(left, (over + 1) >> 7);        // below zero: none
        lim = over + min(r / p.G, c.toks - 1) - half * KEYS;     // padding rows: the last real row's limit
        end = c.L - c.ta * RA_BKV;
        busy = quarter * 32 < c.toks * p.G;        // some row of this warp is real
      }
      m = -INFINITY;
      l = 0.f;
      if (!mbar_wait_warp(k ? q_full(k) : q_first, k ? ((k - (k & 3 ? 0 : 4)) >> 2) & 1 : 0, p.err, abort_flag)) { ok = false; break; }
      rs = qscale[(k & 3) * RA_BQ + r];
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
        {
          float other = l;
          if (!exchange(other)) { ok = false; break; }
          l = half == 0 ? l + other : other + l;   // the same sum in both halves
        }
        const RaPiece& c = piece(k);
        const bool whole = c.flags & 1;
        const int tok = r / p.G;
        const bool mine = r < c.toks * p.G;
        const int64_t orow = static_cast<int64_t>(c.row0 + tok) * p.Hq + c.g * p.G + (r - tok * p.G);
        const int64_t pslot = static_cast<int64_t>(cta) * 2 + (c.flags >> 1);
        const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(oadr + h * 32, v);
          tmem_ld_wait();
          if (mine && whole) {
            __nv_bfloat16* orow_p = p.j.o + orow * RA_D + half * 64 + h * 32;
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[i] = pack_bf16x2(__uint_as_float(v[e + 2 * i]) * inv, __uint_as_float(v[e + 2 * i + 1]) * inv);
              ra_st32(orow_p + e, y);
            }
          } else if (mine) {
            float* po = p.j.part_o + (pslot * RA_D + half * 64 + h * 32) * RA_BQ + r * 4;      // lanes side by side
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(po + e * RA_BQ) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
          __syncwarp();                            // the next load is a whole warp's
        }
        if (mine && half == 0) {
          if (whole) {
            if (p.j.lse) p.j.lse[orow] = (m - A8_LIFT + log2f(l)) * RA_LN2;
          } else {
            *reinterpret_cast<float2*>(p.j.part_ml + (pslot * RA_BQ + r) * 2) = make_float2(m - A8_LIFT, l);
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

}  // namespace

size_t ragged_attention8_ws() { return ra_ws(num_sms()).total; }

kl_status ragged_attention8(const kl_ragged_cfg& rc, int Hq, int Hkv, const void* q, const void* kp, const void* vp,
                            const float* ks, const float* vs, const int32_t* table, const int32_t* cu,
                            const int32_t* ctx, void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t st) {
  const int ctas = num_sms();
  const RaWs lay = ra_ws(ctas);
  if (!ws || ws_bytes < lay.total || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return set_error(KL_ERR_NO_MEMORY, "ragged attention8: workspace too small or not 256-byte aligned");
  A8Params p;
  memset(&p, 0, sizeof(p));
  p.G = p.j.G = Hq / Hkv;
  p.TQ = RA_BQ / p.G;
  const bool tma = rc.block_size % 8 == 0;
  p.box_log = 7;
  while (tma && rc.block_size & ((1 << p.box_log) - 1)) --p.box_log;    // gcd(block_size, 128)
  if (tma) {
    // (128 columns, kv heads, rows)
    const cuuint64_t pitch = static_cast<cuuint64_t>(Hkv) * RA_D;
    const cuuint64_t dk[3] = {RA_D, static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(rc.n_blocks) * rc.block_size};
    const cuuint64_t sk[2] = {RA_D, pitch};
    const cuuint32_t bk[3] = {RA_D, 1, 1u << p.box_log};
    KL_TRY(ra_map(&p.tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, kp, dk, sk, bk));
    KL_TRY(ra_map(&p.tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, vp, dk, sk, bk));
  }
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kp = static_cast<const uint8_t*>(kp);
  p.vp = static_cast<const uint8_t*>(vp);
  p.ks = ks;
  p.vs = vs;
  p.table = table;
  p.cu = cu;
  p.ctx = ctx;
  p.j.o = static_cast<__nv_bfloat16*>(o);
  p.j.lse = lse;
  uint8_t* wb = static_cast<uint8_t*>(ws);
  p.j.part_o = reinterpret_cast<float*>(wb + lay.o);
  p.j.part_ml = reinterpret_cast<float*>(wb + lay.ml);
  p.j.cuts = reinterpret_cast<RaCut*>(wb + lay.cuts);
  p.B = rc.B;
  p.T = rc.T;
  p.Hq = p.j.Hq = Hq;
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
    KL_CUDA(cudaFuncSetAttribute(ragged_attn8_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(a8_smem(true))));
    KL_CUDA(cudaFuncSetAttribute(ragged_attn8_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(a8_smem(false))));
    attr_done |= uint64_t(1) << dev;
  }
  {
    // the lengths are on the device: the rows' queries and outputs are what the host knows of the traffic
    ProfScope ps("ragged_attention8", st, 0.0, 4.0 * rc.T * Hq * RA_D);
    if (tma)
      launch_pdl(ragged_attn8_kernel<true>, ctas, A8_THREADS, a8_smem(true), st, p);
    else
      launch_pdl(ragged_attn8_kernel<false>, ctas, A8_THREADS, a8_smem(false), st, p);
  }
  KL_CUDA(cudaGetLastError());
  return ragged_join(p.j, ctas, st);
}

}  // namespace kl
