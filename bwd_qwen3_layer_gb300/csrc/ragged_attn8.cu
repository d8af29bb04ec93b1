// Attention of a ragged step over a paged cache of 8-bit codes with a scale for each
// page and head, on the 5th-generation tensor cores:
//   o_i = sum_j softmax_j(q_i . (a_j kc_j) / sqrt(d)) b_j vc_j,
// kc_j, vc_j the e4m3 codes of position j and a_j, b_j its page's scales.
//
// Products in 8 bits. Keys and values go to the tensor cores as they are cached,
// nothing is converted: half the bytes of a bf16 cache in HBM and in shared memory. The
// other operands are split. A bf16 query has 8 significant bits, which two e4m3
// numbers hold (row scaled by a power of two so that its largest element is in [128,
// 256); hi is the nearest e4m3, the rest has 4 bits: exact down to 2^-10 of the
// largest, off by 2^-17 of it below). e4m3 products run at twice the bf16 rate, so S =
// hi K^T + lo K^T takes the time of one bf16 product. Weights are three e5m2 numbers:
// that type is the upper byte of an f16 number, so two cuts of three bits and one rounding take
// few instructions, and each weight is off by 2^-9 of itself and its f16's 2^-11.
//
// Range. Many small weights can outweigh a few large ones (a key at the start that takes half of the row,
// 32768 others the rest): what each of them loses adds up, so no weight may be cut off early.
// Here it is off by 2^-17 at most where the row's largest is 2^11 or more, 2^-28 of it. (Two e4m3 parts, 2^-14
// of it, lost half of the row in that example. On one GPU 64 x ~4096 keys took 98.7 us so and take 109, the chunk
// 1.75 and 2.0 ms: three products for two and three more instructions for four weights. Two e5m2 parts would be
// off by 2^-7.)
//
// Scales. t_j = s_j a_j + log2 b_j is what the running maximum m is taken of, and P'_j =
// 2^(t_j - m + 11) = 2^(11 - m) p_j b_j goes into the product with the values' codes: its
// range does not depend on how the pages' scales differ. The row's sum adds P'_j / b_j. m
// is raised when t exceeds it by more than 4.7 in some row of a warp, so P' stays below
// 2^15.7, which e5m2 and f16 hold (and then to the maximum of every row: O's columns are read and written once
// for all). (Raised at 2.5, a chunk's steps waited for the product before them a third of the time.)
//
// Work split, walk and join are those of the bf16 kernel (ragged_walk.cuh): query tiles
// of floor(128 / G) tokens x G heads, runs of key tiles of 128 keys, one CTA per SM,
// pieces of cut items joined in CTA order: results repeat bit for bit.
//
// Roles (16 warps): warp 0 copies the keys, warp 1 the values, warp 2 issues the score
// products, warp 3 the P V products. Warps 4..7 are the softmax of the even steps,
// 8..11 of the odd ones (thread = query row = TMEM lane): a step's chain of waits, loads,
// maxima, 128 exponentials and splits a row is longer than two steps' products, so two are
// under way. The running maximum passes from one group to the other through shared memory;
// O has one scale. Warp 12 looks up the scales, warps 13..15 split the next piece's queries
// (the first piece's: the softmax warps, idle at first): done by the copy warps in between,
// both held the copies up (124 us instead of 116 for 64 decoding requests).
// Scores stay in tensor memory and are read twice, for the maximum and for the weights, 32
// columns at a time, so that a step's code is a few small loops: unrolled over 128 keys (30
// KB a step, 170 KB in all) the instruction fetch took longer than the work, 3800 cycles a
// step. Keys cut off are marked in tensor memory beforehand for the same reason (6 % of a chunk). P takes the columns of S
// that have been read; three such buffers keep the score products two steps ahead.
//
// Few rows. A piece of at most 16 rows (decoding) would leave seven of eight TMEM lanes
// and all but one softmax warp idle, and its products, which read 128 rows of each part
// whatever they hold, would take more of shared memory's time than the copies. Both
// parts of its queries are rows of one tile instead, row r's at lanes r and 16 + r of
// each quarter of the lanes: half the products, and each quarter's warp, which takes 32 of
// the tile's keys (a lane 16), adds the parts. Weights likewise, in shared memory, from
// where the P V product reads them: up to ten rows' three parts at lanes r, 10 + r and 20 + r of O, added
// at the end. Of more rows the third parts are a tile with zeros, and a second product (64 requests of two tokens: 114
// us; as a tile of 128 rows 153).
//
// Measured (64 query heads, 8 kv heads, pages of 16): 64 requests of ~4096 keys 108-110 us, 0.73-0.74 of HBM's copy rate
// (128-byte pieces 1 KB apart, and a chain of waits from a tile's scores to its product); one of 32768 23-24 us; 4095 rows over
// 12288 keys 1.95 to 2.07 ms: a step takes ~2400 cycles, of which the products (two for the scores, three for the
// values) need 1280, the softmax warps' instructions for two warps a scheduler the rest.
//
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

constexpr int A8_WARPS = 16;
constexpr int A8_THREADS = 32 * A8_WARPS;
constexpr uint32_t A8_TILE = 128 * 128;       // a tile of keys, of values, of one part of the queries
constexpr int A8_NST = 4;                     // stages of the K and of the V ring
constexpr int A8_QR = 8;                      // pieces in the ring of the rows' factors
constexpr int a8_scr(bool tma) { return tma ? 8 : 4; }      // tiles in the ring of scales
constexpr int A8_QW = 3;                      // warps that split queries
constexpr int A8_SB = 3;                      // steps whose scores and weights are in tensor memory
constexpr int A8_FEW = 16;                    // rows at most of a piece that has the parts of its operands as rows of one tile
constexpr uint32_t A8_FEW_TILE = 2 * A8_FEW * 128;          // 32 rows: a quarter of the lanes
constexpr int A8_LEAST = 10;                  // rows whose three parts of weights are 32 rows, too
constexpr uint32_t A8_P_BYTES = 4 * A8_FEW_TILE;
constexpr uint32_t A8_OFF_Q = 0;              // two pieces' queries, high and low parts
constexpr uint32_t A8_OFF_P = A8_OFF_Q + 4 * A8_TILE;       // weights of few rows: three steps of 32 rows or two of 64
                                              // (the product reads 128: what lies behind gives rows that nobody reads)
constexpr uint32_t A8_OFF_K = A8_OFF_P + A8_P_BYTES;
constexpr uint32_t A8_OFF_V = A8_OFF_K + A8_NST * A8_TILE;
constexpr uint32_t A8_OFF_BAR = A8_OFF_V + A8_NST * A8_TILE;
constexpr uint32_t A8_OFF_QS = A8_OFF_BAR + 3 * 1024;       // the rows' factors, of eight pieces
constexpr uint32_t A8_OFF_MX = A8_OFF_QS + A8_QR * RA_BQ * 4;   // the rows' maxima, of four steps
constexpr uint32_t A8_OFF_L = A8_OFF_MX + 4 * RA_BQ * 4;    // the groups' sums, of two pieces
constexpr uint32_t A8_OFF_SC = A8_OFF_L + 4 * RA_BQ * 4;    // the ring of scales
constexpr size_t a8_smem(bool tma) { return 1024 + A8_OFF_SC + a8_scr(tma) * 3 * (tma ? 16 : 128) * 4; }
static_assert(a8_smem(false) <= 232448, "shared memory");
// Tensor memory: S of three steps, whose columns P takes as they are read, and O: all 512 columns.
constexpr uint32_t A8_TM_O = 384;
constexpr float A8_LIFT = 11.0f;              // P' of the running maximum is 2^11 ...
constexpr float A8_LAG = 4.7f;                // ... to 2^15.7

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
  int inv_g;             // ceil(2^16 / G): r / G = r inv_g >> 16 for r < 128
  int bs, max_blocks, n_blocks;
  int box_log;           // log2 of the rows per TMA box (8 .. 128)
  float scale_log2;
  uint32_t* err;
};

// Queries and keys, K-major in groups of 8 rows 1 KB apart, k-step kk of 32 columns
__device__ __forceinline__ uint64_t a8_desc_k(uint32_t base, int kk) { return smem_desc_sw128(base + kk * 32, 16, 1024); }
// Values as the MN-major B operand: n = head dim, 128 bytes; k-step kk of 32 keys = four groups
__device__ __forceinline__ uint64_t a8_desc_v(uint32_t base, int kk) { return smem_desc_sw128(base + kk * 4096, 1024, 1024); }

// Pairs of f16 in one register (the largest finite one for what is above), and four of them as e5m2: cut, which
// is their upper bytes, or rounded.
__device__ __forceinline__ uint32_t a8_f16x2(uint32_t lo, uint32_t hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  return d;
}
__device__ __forceinline__ uint32_t a8_e5m2x4_cut(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }
__device__ __forceinline__ uint32_t a8_sub_h(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t a8_e5m2x4_h(uint32_t a, uint32_t b) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo) : "r"(a));
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(hi) : "r"(b));
  uint32_t d;
  asm("mov.b32 %0, {%1, %2};" : "=r"(d) : "h"(lo), "h"(hi));
  return d;
}
// max that a NaN survives
__device__ __forceinline__ float a8_max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// 32 lanes x 8 consecutive 32-bit columns from registers into TMEM
__device__ __forceinline__ void a8_tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// mbar_wait_warp in few instructions (there are thirty of them in the kernel, whose hot loops have to fit
// the SM's instruction cache). A probe may sleep for a microsecond or so; their number has a limit.
static __device__ __noinline__ bool a8_give_up(uint32_t probes, uint32_t* err, volatile int* abort_flag) {
  const bool late = probes > 1u << 21;
  if (late) record_error(err, KL_DEVERR_TIMEOUT);
  return __any_sync(0xffffffffu, late || *abort_flag);
}
__device__ __forceinline__ bool a8_wait(uint32_t bar, uint32_t parity, uint32_t* err, volatile int* abort_flag) {
  for (uint32_t i = 0; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++i)
    if ((i & 63u) == 63u && a8_give_up(i, err, abort_flag)) return false;
  return true;
}

template <int N>
__device__ __forceinline__ void a8_ldv(uint32_t addr, float (&v)[4]) {
  if (N == 4)
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr));
  else
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(addr));
}

template <bool TMA>
__global__ void __launch_bounds__(A8_THREADS, 1) ragged_attn8_kernel(const __grid_constant__ A8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar = sb + A8_OFF_BAR;
  constexpr int A8_SCR = a8_scr(TMA);
  // A wait by parity is right only if the phase before the one it means has ended. What says so: for the stages' and
  // rings' producers and consumers (k_, v_, sc_, q_, p_full), that they wait for every phase in turn; for s_full(n) in the softmax,
  // that S of step n - 2 was waited for; for v_full(n) and p_done(n - 1) there, that S of step n was, which was issued after the
  // product of step n - 3; for told(t), that t - 1 was heard before; for sums and o_free, that every piece has one of each. Arrivals, too, count
  // for the phase that is open: sc_empty(n) comes before p_full(n), so that a warp without rows, which waits for S alone,
  // cannot arrive for a later tile of that place before the others have for this one.
  // piece k's queries: eight, since with pieces of one tile the score products run three pieces ahead of
  // the softmax and the queries two more, and no waiter may be two phases behind
  auto q_full = [&](int k) { return bar + 576 + 8 * (k & (A8_QR - 1)); };
  auto q_empty = [&](int k) { return bar + 0 + 8 * (k & 1); };    // its last S product is done with them
  auto k_full = [&](int s) { return bar + 48 + 8 * s; };
  auto k_empty = [&](int s) { return bar + 80 + 8 * s; };
  auto v_full = [&](int s) { return bar + 112 + 8 * s; };
  auto v_empty = [&](int s) { return bar + 144 + 8 * s; };
  auto s_full = [&](int n) { return bar + 176 + 8 * (n % A8_SB); };   // S_n computed
  auto p_full = [&](int n) { return bar + 200 + 8 * (n % A8_SB); };   // P_n written (and V_n's tail cleared)
  auto p_done = [&](int n) { return bar + 224 + 8 * (n % A8_SB); };   // O += P_n V_n computed
  auto phase = [&](int n) -> uint32_t { return (n / A8_SB) & 1; };    // their parity for step n
  auto sc_full = [&](int n) { return bar + 248 + 8 * (n & (A8_SCR - 1)); };    // the tile's scales written
  auto sc_empty = [&](int n) { return bar + 312 + 8 * (n & (A8_SCR - 1)); };   // and read
  const uint32_t drain = bar + 376, drain_pv = bar + 384;
  const uint32_t q_first = bar + 392;                              // the first piece's queries
  auto told = [&](int q, int t) { return bar + 400 + 32 * q + 8 * (t & 3); };   // the step's maxima of quarter q's rows
  auto told_few = [&](int t) { return bar + 528 + 8 * (t & 3); };  // those of all quarters
  const uint32_t sums = bar + 560;                                 // a piece's sums of both groups
  const uint32_t o_free = bar + 568;                               // a piece's O has been read
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + A8_OFF_BAR + 640);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + A8_OFF_BAR + 644);
  RaFound* found = reinterpret_cast<RaFound*>(smem + A8_OFF_BAR + 648);
  long long* wsum = reinterpret_cast<long long*>(smem + A8_OFF_BAR + 712);
  RaWalk* walks = reinterpret_cast<RaWalk*>(smem + A8_OFF_BAR + 840);        // the finder's, then one per warp
  RaPiece* pieces = reinterpret_cast<RaPiece*>(smem + A8_OFF_BAR + 1656);    // the first one, then two per warp
  static_assert(sizeof(RaFound) <= 64 && A8_WARPS * 8 <= 128 && (A8_WARPS + 1) * sizeof(RaWalk) <= 816 &&
                    (A8_WARPS * 2 + 1) * sizeof(RaPiece) <= 1416,
                "shared-memory layout");
  float* qscale = reinterpret_cast<float*>(smem + A8_OFF_QS);
  constexpr int GRP = TMA ? 8 : 1;               // keys that share a scale
  constexpr int NG = RA_BKV / GRP;
  const uint32_t sc0 = sb + A8_OFF_SC;           // [tile][a, log2 b, 1 / b][group]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const RaLens lens = {p.cu, p.ctx, p.B, p.T, p.Hkv, p.TQ};

  if (warp == 3 && lane == 0) {
    for (int k = 0; k < A8_QR; ++k) mbar_init(q_full(k), A8_QW);
    mbar_init(q_first, 8);
    for (int k = 0; k < 16; ++k) mbar_init(told(k >> 2, k), 1);
    for (int k = 0; k < 4; ++k) mbar_init(told_few(k), 4);
    mbar_init(sums, 8);
    mbar_init(o_free, 8);
    for (int k = 0; k < 2; ++k) mbar_init(q_empty(k), 1);
    for (int s = 0; s < A8_NST; ++s) {
      mbar_init(k_full(s), TMA ? 1 : 32);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), TMA ? 1 : 32);
      mbar_init(v_empty(s), 1);
    }
    for (int n = 0; n < A8_SB; ++n) {
      mbar_init(s_full(n), 1);
      mbar_init(p_full(n), 4);
      mbar_init(p_done(n), 1);
    }
    for (int n = 0; n < A8_SCR; ++n) {
      mbar_init(sc_full(n), 1);
      mbar_init(sc_empty(n), 4);
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
  if (TMA && lane == 0 && (warp == 6 || warp == 7)) tma_prefetch_desc(warp == 6 ? &p.tmK : &p.tmV);

  pdl_enter();      // nothing above reads what an earlier kernel writes

  const long long P = ra_find_run<A8_WARPS>(lens, cta, ctas, wsum, found, &pieces[0], &walks[0]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tmO = tmem + A8_TM_O;

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
  // the parity that piece k's queries' barrier is waited for with (q_full(0) serves from piece 8 on)
  auto q_phase = [&](int k) -> uint32_t { return k ? ((k - (k & (A8_QR - 1) ? 0 : A8_QR)) / A8_QR) & 1 : 0; };
  auto token_of = [&](int r) { return (r * p.inv_g) >> 16; };
  // where few rows' weights of step n are
  auto few_p = [&](bool least, int n) { return sb + A8_OFF_P + (least ? n % 3 : 2 * (n & 1)) * A8_FEW_TILE; };
  // Queries, four rows at a time, 8 lanes of 16 elements each: row r0 + (lane >> 3) of a piece with `rows` ...
  auto load_q = [&](const RaPiece& c, int rows, int r0, uint4 (&x)[2]) {
    const int r = r0 + (lane >> 3), tok = token_of(r);
    if (r >= rows) return;
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + (static_cast<int64_t>(c.row0 + tok) * p.Hq + c.g * p.G + (r - tok * p.G)) * RA_D + (lane & 7) * 16);
    x[0] = src[0];
    x[1] = src[1];
  };
  // ... split into its two parts, and its factor, into piece k's places (few rows: into every quarter's).
  auto split_q = [&](const uint4 (&x)[2], int k, int rows, int r0) {
    const int r = r0 + (lane >> 3), j = lane & 7;
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    // the largest size, as bits (two at a time): an infinity or a NaN is above all numbers
    uint32_t a2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a2 = __vmaxu2(a2, w[i] & 0x7fff7fffu);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) a2 = __vmaxu2(a2, __shfl_xor_sync(0xffffffffu, a2, o));
    const uint32_t a = max(a2 & 0xffffu, a2 >> 16);
    const int e = max(static_cast<int>(a >> 7) - 127, -110);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 s = unpack_bf16x2(w[2 * i]), t = unpack_bf16x2(w[2 * i + 1]);
      const float x0 = s.x * up, x1 = s.y * up, x2 = t.x * up, x3 = t.y * up;
      hi[i] = e4m3x4(x0, x1, x2, x3);
      const float4 h = e4m3x4_to_f(hi[i]);
      lo[i] = e4m3x4(x0 - h.x, x1 - h.y, x2 - h.z, x3 - h.w);
    }
    if (r < rows) {
      const bool few = rows <= A8_FEW;
      uint32_t at = sb + A8_OFF_Q + (k & 1) * 2 * A8_TILE + r * 128 + ((j ^ (r & 7)) << 4);
      float* f = qscale + (k & (A8_QR - 1)) * RA_BQ + r;
      const float v = a >= 0x7f80u ? __int_as_float(0x7fffffff) : down * p.scale_log2;
#pragma unroll 1
      for (int c = 0; c < (few ? 4 : 1); ++c, at += A8_FEW_TILE, f += 32) {
        st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(at + (few ? A8_FEW * 128 : A8_TILE), lo[0], lo[1], lo[2], lo[3]);
        if (j == 0) *f = v;
        if (j == 1 && few) f[A8_FEW] = v;
      }
    }
  };
  // no row: no factor (from place `from` on in steps of `by`)
  auto no_rows = [&](int k, int rows, int from, int by) {
#pragma unroll 1
    for (int r = from; r < RA_BQ; r += by)
      if ((rows <= A8_FEW ? r & (A8_FEW - 1) : r) >= rows) qscale[(k & (A8_QR - 1)) * RA_BQ + r] = 0.f;
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
    int row[4];
    int blk = 0, at = -1;                          // TMA: the next batch's page of this lane's box and the place in it
    auto ask = [&](const RaPiece& c, int j) {
      const int pos = j * RA_BKV + lane * box, lb = pos / p.bs;
      at = pos < min(c.L, c.tb * RA_BKV) ? pos - lb * p.bs : -1;
      if (at >= 0) blk = page(c.b, lb);
    };
    bool have = find(0);
    if (TMA && have) ask(piece(0), piece(0).ta);
    for (int k = 0; ok && have; ++k) {
      const RaPiece w = piece(k);
      have = find(k + 1);
      if (TMA) {
        // One look at the table serves a batch of `per` tiles, a lane per box; the next batch's pages (the
        // next piece's, at the end of this one) are asked for before this one's tiles are copied.
        for (int j = w.ta; j < w.tb; ++j) {
          const int nth = (j - w.ta) & (per - 1);
          if (nth == 0) {
            row[0] = at >= 0 ? pool_row(blk, at) : no_row;
            if (j + per < w.tb) ask(w, j + per);
            else if (have) ask(piece(k + 1), piece(k + 1).ta);
          }
          if (!a8_wait(empty0 + 8 * s, ph, p.err, abort_flag)) { ok = false; break; }
          if (el) mbar_arrive_expect_tx(full0 + 8 * s, A8_TILE);
          __syncwarp();
          if (my == nth) ra_tma_3d(ring + s * A8_TILE + (lane & (nbox - 1)) * box * 128, tm, 0, w.g, row[0], full0 + 8 * s);
          __syncwarp();
          ++issued;
          if (++s == A8_NST) {
            s = 0;
            ph ^= 1u;
          }
        }
      } else {
        // a lane for four of a tile's keys
        const int keys = min(w.L, w.tb * RA_BKV);
        auto lookup = [&](int j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = j * RA_BKV + i * 32 + lane, lb = pos / p.bs;
            row[i] = pos < keys ? pool_row(page(w.b, lb), pos - lb * p.bs) : no_row;
          }
        };
        lookup(w.ta);
        for (int j = w.ta; j < w.tb; ++j) {
          if (!a8_wait(empty0 + 8 * s, ph, p.err, abort_flag)) { ok = false; break; }
          gather(ring + s * A8_TILE, w.g, row);
          if (j > w.ta) announce(std::integral_constant<int, 1>());   // the tile before
          ++issued;
          if (++s == A8_NST) {
            s = 0;
            ph ^= 1u;
          }
          if (j + 1 < w.tb) lookup(j + 1);
        }
        // the piece's last tile: its products free Q, which the next piece waits for
        if (ok) announce(std::integral_constant<int, 0>());
      }
    }
    if (!ok) *abort_flag = 1;
    // copies still in flight must land before exit
    if (TMA) {
      for (int j = max(0, issued - A8_NST); j < issued; ++j) mbar_wait(full0 + 8 * (j % A8_NST), (j / A8_NST) & 1, p.err);
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  } else if (warp == 2) {
    // ---------- S_n = hi K_n^T + lo K_n^T into S[n % 3] (whole warp; the elected lane issues) ----------
    const bool el = elect_one();
    const uint32_t idesc = idesc_f8_f32(128, 128, 0, 0, 0);
    int n = 0, ks = 0;                        // step, K stage
    uint32_t kph = 0;
    bool ok = true;
    for (int k = 0; ok && find(k); ++k) {
      const int tiles = piece(k).tb - piece(k).ta;
      const bool few = piece(k).toks * p.G <= A8_FEW;
      const uint32_t qb = sb + A8_OFF_Q + (k & 1) * 2 * A8_TILE;
      if (!a8_wait(k ? q_full(k) : q_first, q_phase(k), p.err, abort_flag)) { ok = false; break; }
      for (int j = 0; j < tiles; ++j, ++n) {
        // the columns are free once the product of three steps before is done with its P
        if ((n >= A8_SB && !a8_wait(p_done(n), phase(n) ^ 1u, p.err, abort_flag)) ||
            !a8_wait(k_full(ks), kph, p.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (el) {
          const uint32_t kb = sb + A8_OFF_K + ks * A8_TILE;
#pragma unroll 1
          for (int kk = 0; kk < (few ? 4 : 8); ++kk)      // high parts, then low ones
            umma_f8(tmem + n % A8_SB * 128, a8_desc_k(qb + (kk >> 2) * A8_TILE, kk & 3), a8_desc_k(kb, kk & 3), idesc, kk > 0);
          umma_commit(s_full(n));
          umma_commit(k_empty(ks));
          if (j == tiles - 1) umma_commit(q_empty(k));   // the piece's last use of Q
        }
        __syncwarp();
        if (++ks == A8_NST) {
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
    // ---------- O (+)= P_n V_n, all parts (whole warp; the elected lane issues) ----------
    const bool el = elect_one();
    const uint32_t idesc = idesc_f8_f32(128, 128, 1, 0, 1);
    int n = 0, vs = 0;                        // step, V stage
    uint32_t vph = 0;
    bool ok = true;
    for (int k = 0; ok && find(k); ++k) {
      const int tiles = piece(k).tb - piece(k).ta;
      const int rows = piece(k).toks * p.G;
      const bool few = rows <= A8_FEW, least = rows <= A8_LEAST;
      if (k > 0 && !a8_wait(o_free, (k - 1) & 1, p.err, abort_flag)) { ok = false; break; }
      for (int j = 0; j < tiles; ++j, ++n) {
        if (!a8_wait(v_full(vs), vph, p.err, abort_flag) || !a8_wait(p_full(n), phase(n), p.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (el) {
          const uint32_t vb = sb + A8_OFF_V + vs * A8_TILE, pb = few_p(least, n);
          const uint32_t pt = tmem + n % A8_SB * 128;     // 24 columns for 32 keys: the three parts
#pragma unroll 1
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t v = a8_desc_v(vb, kk);
            const uint32_t acc = j > 0 || kk > 0;
            if (few) {                             // (more than A8_LEAST: two parts, then the third beside zeros)
              umma_f8(tmO, a8_desc_k(pb, kk), v, idesc, acc);
              if (!least) umma_f8(tmO, a8_desc_k(pb + A8_FEW_TILE, kk), v, idesc, 1);
            } else {
              umma_f8_ta(tmO, pt + kk * 24, v, idesc, acc);
              umma_f8_ta(tmO, pt + kk * 24 + 8, v, idesc, 1);
              umma_f8_ta(tmO, pt + kk * 24 + 16, v, idesc, 1);
            }
          }
          umma_commit(p_done(n));
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
  } else if (warp == 12) {
    // ---------- scales (TMA: lane = page box of a batch of tiles; else a lane for four of a tile's keys) ----------
    const int box = 1 << p.box_log, nbox = RA_BKV >> p.box_log, my = lane >> (7 - p.box_log);
    const int per = TMA ? box >> 2 : 1;            // tiles of a look-up
    constexpr int KS = TMA ? 1 : 4;
    // Pages are asked for two batches ahead (the next piece's too), scales one: a read takes 1000 to 3000
    // cycles while HBM is busy. The batches that have been asked for: this lane's pages (below zero: none) and
    // the kv head; the piece and tile of the next one.
    int blk[3][KS] = {}, head[3] = {}, queued = 0, ask_k = 0, ask_j = -1, n = 0;
    float a[2][KS], b[2][KS];                      // this batch's, the next one's
    bool asked = false;
    auto scales = [&](int i) {
#pragma unroll
      for (int e = 0; e < KS; ++e) {
        a[1][e] = b[1][e] = 1.f;                   // a page that is read as zero has none
        if (blk[i][e] < 0 || blk[i][e] >= p.n_blocks) continue;
        const int64_t sc = static_cast<int64_t>(blk[i][e]) * p.Hkv + head[i];
        a[1][e] = p.ks[sc];
        b[1][e] = p.vs[sc];
      }
    };
    bool ok = true, have = find(0);
    for (int k = 0; ok && have; ++k) {
      const RaPiece w = piece(k);
      have = find(k + 1);
      for (int j = w.ta; j < w.tb; ++j, ++n) {
        const int nth = (j - w.ta) & (per - 1);
        if (nth == 0) {
          while (queued < 3 && (ask_k < k + 1 || (ask_k == k + 1 && have))) {
            const RaPiece& c = piece(ask_k);
            if (ask_j < 0) ask_j = c.ta;
#pragma unroll
            for (int e = 0; e < KS; ++e) {
              const int pos = ask_j * RA_BKV + (TMA ? lane * box : e * 32 + lane);
              const int pg = pos < min(c.L, c.tb * RA_BKV) ? page(c.b, pos / p.bs) : -1;
#pragma unroll
              for (int i = 0; i < 3; ++i)
                if (queued == i) blk[i][e] = pg;
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
              if (queued == i) head[i] = c.g;
            ++queued;
            ask_j += per;
            if (ask_j >= c.tb) {
              ask_j = -1;
              ++ask_k;
            }
          }
          if (!asked) scales(0);
#pragma unroll
          for (int e = 0; e < KS; ++e) {
            a[0][e] = a[1][e];
            b[0][e] = b[1][e];
          }
          asked = queued > 1;
          if (asked) scales(1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            head[i] = head[i + 1];
#pragma unroll
            for (int e = 0; e < KS; ++e) blk[i][e] = blk[i + 1][e];
          }
          --queued;
        }
        if (n >= A8_SCR && !a8_wait(sc_empty(n), ((n / A8_SCR) & 1) ^ 1u, p.err, abort_flag)) { ok = false; break; }
        float* sc = reinterpret_cast<float*>(smem + A8_OFF_SC) + (n & (A8_SCR - 1)) * 3 * NG;
        if (TMA) {
          if (my == nth) {
            const float lb = log2f(b[0][0]), ib = 1.f / b[0][0];
            const int gs = box >> 3, g0 = (lane & (nbox - 1)) * gs;
            for (int g = g0; g < g0 + gs; ++g) {
              sc[g] = a[0][0];
              sc[NG + g] = lb;
              sc[2 * NG + g] = ib;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < KS; ++e) {
            sc[(e * 32 + lane) % NG] = a[0][e];
            sc[NG + (e * 32 + lane) % NG] = log2f(b[0][e]);
            sc[2 * NG + (e * 32 + lane) % NG] = 1.f / b[0][e];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_full(n));
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp > 12) {
    // ---------- queries of the pieces after the first, four rows at a time ----------
    bool ok = find(0);                             // a CTA without a run has no walk either
    for (int k = 1; ok && find(k); ++k) {
      const RaPiece& c = piece(k);
      const int rows = c.toks * p.G;
      uint4 x[2] = {}, y[2] = {};
      int at = 4 * (warp - 13);
      load_q(c, rows, at, x);
      // the buffer is free once the S products of the piece before the last are done
      if (k > 1 && !a8_wait(q_empty(k), ((k - 2) >> 1) & 1, p.err, abort_flag)) { ok = false; break; }
#pragma unroll 1
      for (; at < rows; at += 4 * A8_QW) {
        load_q(c, rows, at + 4 * A8_QW, y);        // the next ones are on their way
        split_q(x, k, rows, at);
        x[0] = y[0];
        x[1] = y[1];
      }
      no_rows(k, rows, lane + 32 * (warp - 13), 32 * A8_QW);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(k));
    }
    if (!ok && piece(0).tb > 0) *abort_flag = 1;
  } else {
    // ---------------- softmax / correction / epilogue ----------------
    const int quarter = warp & 3, grp = (warp >> 2) - 1;         // grp: the parity of its steps
    const int r = quarter * 32 + lane;           // TMEM lane: the row within the tile, or (few rows) a part of row lane & 15
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t oadr = tmO + lane_off;
    float* maxima = reinterpret_cast<float*>(smem + A8_OFF_MX);   // [step % 4][row]
    float* lsum = reinterpret_cast<float*>(smem + A8_OFF_L);      // [piece % 2][group][row]
    // The tile that holds the last key the query tile sees: its value rows behind it become zero
    // (each of the group's four warps its 32). Called once S of the step has been waited for, which was issued after the
    // product of the third step before: that one's values, and those of the step before it, whose stage this is, had
    // landed and been read, so that the wait by parity is for this step's. (Asked for before S, it passes while
    // the values of four steps before are still on their way, and zeroes those.) Nothing waits in a circle: the copy
    // needs the product of four steps before, no later one.
    auto clear_tail = [&](int end, int n) -> bool {
      if (end >= RA_BKV) return true;
      const int vs = n % A8_NST;
      if (!a8_wait(v_full(vs), (n / A8_NST) & 1, p.err, abort_flag)) return false;
      if (r >= end) {
        const uint32_t va = sb + A8_OFF_V + vs * A8_TILE + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) st_shared_v4(va + c * 16, 0u, 0u, 0u, 0u);
      }
      fence_async_shared();
      return true;
    };
    bool more = find(0);
    if (more) {
      // the first piece's queries, four rows a warp at a time
      const RaPiece& c = piece(0);
      const int rows = c.toks * p.G;
#pragma unroll 1
      for (int at = (warp - 4) * 4; at < rows; at += 32) {
        uint4 x[2] = {};
        load_q(c, rows, at, x);
        split_q(x, 0, rows, at);
      }
      no_rows(0, rows, threadIdx.x - 128, 256);
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
    int n0 = 0;                                    // the piece's first step
    int t_all = 0, t_few = 0;                      // steps before it whose maxima were told (of this quarter's rows; of few rows)
    float m = -INFINITY, l = 0.f;                  // the row's running max of t (log2 units) after this group's last step, its sum of P' / b
    float rs = 0.f;                                // the row's factor: score in log2 units = S * rs * a
    int lim = 0, end = 0;                          // from the piece's first key: the row's last key; the end of the query tile's
    bool real = false;                             // this lane's row is one of the piece's
    bool least = true;                             // (few rows) all parts of the weights are 32 rows ...
    int apart = A8_LEAST;                          // ... and so far apart
    // The maximum after one more step, which only moves when some row's would by more than A8_LAG (the
    // final O / l cancels a stale one). All warps that have these rows come to the same answer.
    auto raised = [&](float m, float mx) { return __any_sync(0xffffffffu, real && mx > m + A8_LAG) ? fmaxf(m, mx) : m; };
    // the rows' maxima of the piece's step j, told by all who have them
    auto heard = [&](auto few, int j, float& mx) -> bool {
      const int t = (decltype(few)::value ? t_few : t_all) + j;
      if (!a8_wait(decltype(few)::value ? told_few(t) : told(quarter, t), (t >> 2) & 1, p.err, abort_flag)) return false;
      const float* at = maxima + (t & 3) * RA_BQ;
      if (decltype(few)::value) {
        at += lane & 15;
        mx = fmaxf(fmaxf(fmaxf(at[0], at[16]), fmaxf(at[32], at[48])), fmaxf(fmaxf(at[64], at[80]), fmaxf(at[96], at[112])));
      } else {
        mx = at[r];
      }
      return true;
    };
    // Four weights' exponents -> their values (pairs), and three parts: as f16, of whose 11 bits three are kept,
    // of the rest three again, and what is left is rounded to three. (In fp32 the masks and differences took four
    // instructions more for four weights and two parts, and one warp 11.8 cycles a weight, 7.9 so.)
    auto weights = [&](uint64_t x0, uint64_t x1, uint64_t& y0, uint64_t& y1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
      float p0, p1, p2, p3;
      ra_unpair(x0, p0, p1);
      ra_unpair(x1, p2, p3);
      const uint32_t u0 = __float_as_uint(ra_ex2(p0)), u1 = __float_as_uint(ra_ex2(p1)), u2 = __float_as_uint(ra_ex2(p2)), u3 = __float_as_uint(ra_ex2(p3));
      y0 = ra_pair(u0, u1);
      y1 = ra_pair(u2, u3);
      constexpr uint32_t KEEP = 0xff00ff00u;
      uint32_t h0 = a8_f16x2(u0, u1), h1 = a8_f16x2(u2, u3);
      hi = a8_e5m2x4_cut(h0, h1);
      h0 = a8_sub_h(h0, h0 & KEEP);
      h1 = a8_sub_h(h1, h1 & KEEP);
      mid = a8_e5m2x4_cut(h0, h1);
      lo = a8_e5m2x4_h(a8_sub_h(h0, h0 & KEEP), a8_sub_h(h1, h1 & KEEP));
    };
    // What takes S to the score, S * factor(a); never zero, so that the -inf of keys cut off stays.
    auto factor = [&](float a) { return a8_max_nan(rs * a, 1.17549435e-38f); };
    // keys behind `last` of these do not count
    auto mask = [&](auto& sv, int last) {
      constexpr int N = sizeof(sv) / 4;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e > last) sv[e] = __float_as_uint(-INFINITY);
    };
    // The maximum of t over N keys, whose scales start at shared address sc (TMA: N / 8 of them, else N).
    auto max_t = [&](auto& sv, uint32_t sc) {
      constexpr int N = sizeof(sv) / 4, GV = N < 32 ? 2 : 4;
      float mx = -INFINITY;
      if (TMA) {
#pragma unroll
        for (int g = 0; g < N / 8; g += GV) {
          float a4[4], l4[4], t[4];
          a8_ldv<GV>(sc + g * 4, a4);
          a8_ldv<GV>(sc + (NG + g) * 4, l4);
#pragma unroll
          for (int u = 0; u < GV; ++u) {
            const uint32_t* y = sv + (g + u) * 8;
            float v = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
            v = ra_max3(v, y[2], y[3]);
            v = ra_max3(v, y[4], y[5]);
            v = ra_max3(v, y[6], y[7]);
            t[u] = fmaf(v, factor(a4[u]), l4[u]);
          }
#pragma unroll
          for (int u = 0; u < GV; u += 2) mx = ra_max3(mx, __float_as_uint(t[u]), __float_as_uint(t[u + 1]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          float a4[4], l4[4], t[4];
          a8_ldv<4>(sc + e * 4, a4);
          a8_ldv<4>(sc + (NG + e) * 4, l4);
#pragma unroll
          for (int u = 0; u < 4; ++u) t[u] = fmaf(__uint_as_float(sv[e + u]), factor(a4[u]), l4[u]);
          mx = ra_max3(mx, __float_as_uint(t[0]), __float_as_uint(t[1]));
          mx = ra_max3(mx, __float_as_uint(t[2]), __float_as_uint(t[3]));
        }
      }
      return mx;
    };
    // N keys' weights, four to a word of each of three parts; their sum goes into r0, r1.
    auto weigh = [&](auto& sv, uint32_t sc, float neg, auto& ph, auto& pm, auto& pl, uint64_t& r0, uint64_t& r1) {
      constexpr int N = sizeof(sv) / 4, GV = N < 32 ? 2 : 4;
      if (TMA) {
        float a4[4], l4[4], i4[4];
        a8_ldv<GV>(sc, a4);
        a8_ldv<GV>(sc + NG * 4, l4);
        a8_ldv<GV>(sc + 2 * NG * 4, i4);
#pragma unroll
        for (int g = 0; g < N / 8; ++g) {
          const uint32_t* v = sv + g * 8;
          const uint32_t fu = __float_as_uint(factor(a4[g])), cu = __float_as_uint(l4[g] + neg), iu = __float_as_uint(i4[g]);
          const uint64_t f2 = ra_pair(fu, fu), c2 = ra_pair(cu, cu), iv = ra_pair(iu, iu);
          uint64_t y0, y1, y2, y3;
          weights(ra_fma2(ra_pair(v[0], v[1]), f2, c2), ra_fma2(ra_pair(v[2], v[3]), f2, c2), y0, y1, ph[2 * g], pm[2 * g], pl[2 * g]);
          weights(ra_fma2(ra_pair(v[4], v[5]), f2, c2), ra_fma2(ra_pair(v[6], v[7]), f2, c2), y2, y3, ph[2 * g + 1], pm[2 * g + 1], pl[2 * g + 1]);
          r0 = ra_fma2(ra_add2(y0, y1), iv, r0);
          r1 = ra_fma2(ra_add2(y2, y3), iv, r1);
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          float a4[4], l4[4], i4[4];
          a8_ldv<4>(sc + e * 4, a4);
          a8_ldv<4>(sc + (NG + e) * 4, l4);
          a8_ldv<4>(sc + (2 * NG + e) * 4, i4);
          auto two = [&](float a, float b) { return ra_pair(__float_as_uint(a), __float_as_uint(b)); };
          uint64_t y0, y1;
          weights(ra_fma2(ra_pair(sv[e], sv[e + 1]), two(factor(a4[0]), factor(a4[1])), two(l4[0] + neg, l4[1] + neg)),
                  ra_fma2(ra_pair(sv[e + 2], sv[e + 3]), two(factor(a4[2]), factor(a4[3])), two(l4[2] + neg, l4[3] + neg)), y0, y1,
                  ph[e / 4], pm[e / 4], pl[e / 4]);
          r0 = ra_fma2(y0, two(i4[0], i4[1]), r0);
          r1 = ra_fma2(y1, two(i4[2], i4[3]), r1);
        }
      }
    };
    // What lies between a step's maximum and its weights. The maximum after the step before, which the other
    // group had, comes first; then this step's is told. (In this order: who hears step n knows that step n - 1 was
    // heard.) A row of a later piece's tile can be fully masked (its token ends before these keys): mx = -inf,
    // and m stays -inf.
    auto agree = [&](auto few, int j, float mx) -> bool {
      constexpr bool FEW = decltype(few)::value;
      float m1 = m;
      if (j > 0) {
        float before;
        if (!heard(few, j - 1, before)) return false;
        m1 = raised(m, before);
      }
      const int t = (FEW ? t_few : t_all) + j;
      maxima[(t & 3) * RA_BQ + r] = mx;
      __syncwarp();
      if (lane == 0) mbar_arrive(FEW ? told_few(t) : told(quarter, t));
      if (FEW && !heard(few, j, mx)) return false;
      const float m2 = raised(m1, mx);
      if (m2 > m) {
        l *= ra_ex2(m - m2);
        m = m2;
      }
      if (j > 0 && (!FEW || quarter == 0) && __any_sync(0xffffffffu, m2 > m1)) {
        // O at the new scale, after the product of the step before (its barrier is at no earlier phase: S_n was
        // computed after the product of step n - 3)
        float alpha = m2 > m1 ? ra_ex2(m1 - m2) : 1.0f;
        if (FEW) alpha = __shfl_sync(0xffffffffu, alpha, lane % apart);       // O's lane is a part of that row
        if (!a8_wait(p_done(n0 + j - 1), phase(n0 + j - 1), p.err, abort_flag)) return false;
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
      return true;
    };
    auto sum_up = [&](uint64_t r0, uint64_t r1) {
      float a0, a1, a2, a3;
      ra_unpair(r0, a0, a1);
      ra_unpair(r1, a2, a3);
      l += (a0 + a1) + (a2 + a3);
    };
    // Step j of the piece by a warp with rows. cut: some row of the tile ends inside its keys.
    auto step = [&](bool cut, int j) -> bool {
      const int n = n0 + j;
      if (!a8_wait(s_full(n), phase(n), p.err, abort_flag) || !a8_wait(sc_full(n), (n / A8_SCR) & 1, p.err, abort_flag)) return false;
      if (cut && TMA && !clear_tail(end - j * RA_BKV, n)) return false;
      tc_fence_after();
      const uint32_t sadr = tmem + lane_off + n % A8_SB * 128;
      const uint32_t sca = sc0 + (n & (A8_SCR - 1)) * 3 * NG * 4;
      if (cut) {
        // keys behind the row's last one: -inf, in place (masks in the loops below were in the way of their code)
#pragma unroll 1
        for (int c = 0; c < RA_BKV; c += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(sadr + c, v);
          tmem_ld_wait();
          mask(v, lim - j * RA_BKV - c);
          tmem_st_32x32b_x16(sadr + c, v);
        }
        tmem_st_wait();
      }
      float mx = -INFINITY;
      uint32_t sv[32];
      tmem_ld_32x32b_x32(sadr, sv);
#pragma unroll 1
      for (int c = 0; c < RA_BKV; c += 32) {
        tmem_ld_wait();
        mx = fmaxf(mx, max_t(sv, sca + c / GRP * 4));
        tmem_ld_32x32b_x32(sadr + ((c + 32) & (RA_BKV - 1)), sv);     // at the end the first ones again
      }
      if (!agree(std::false_type(), j, mx)) return false;
      const float neg = m > -INFINITY ? A8_LIFT - m : 0.f;
      uint64_t r0 = 0, r1 = 0;
      uint32_t ph[8], pm[8], pl[8];
#pragma unroll 1
      for (int c = 0; c < RA_BKV; c += 32) {       // P: 24 columns for 32 keys, the three parts, where S has been read
        tmem_ld_wait();
        weigh(sv, sca + c / GRP * 4, neg, ph, pm, pl, r0, r1);
        if (c < RA_BKV - 32) tmem_ld_32x32b_x32(sadr + c + 32, sv);
        const uint32_t at = sadr + c / 32 * 24;
        a8_tmem_st8(at, ph);
        a8_tmem_st8(at + 8, pm);
        a8_tmem_st8(at + 16, pl);
      }
      sum_up(r0, r1);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sc_empty(n));
        mbar_arrive(p_full(n));
      }
      return true;
    };
    // The same of a piece of few rows: this warp has 32 keys of the tile, a lane 16 of them.
    auto step_few = [&](bool cut, int j) -> bool {
      const int n = n0 + j;
      if (!a8_wait(s_full(n), phase(n), p.err, abort_flag) || !a8_wait(sc_full(n), (n / A8_SCR) & 1, p.err, abort_flag)) return false;
      if (cut && TMA && !clear_tail(end - j * RA_BKV, n)) return false;
      tc_fence_after();
      const int first = quarter * 32 + (lane & 16);      // this lane's first key of the tile
      const uint32_t sca = sc0 + ((n & (A8_SCR - 1)) * 3 * NG + first / GRP) * 4;
      uint32_t sw[32], sv[16];
      tmem_ld_32x32b_x32(tmem + lane_off + n % A8_SB * 128 + quarter * 32, sw);
      tmem_ld_wait();
      // lanes r and 16 + r: high and low part of row r over 32 keys; each takes 16 and adds the other's part
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t keep = lane & 16 ? sw[e + 16] : sw[e], give = lane & 16 ? sw[e] : sw[e + 16];
        sv[e] = __float_as_uint(__uint_as_float(keep) + __uint_as_float(__shfl_xor_sync(0xffffffffu, give, 16)));
      }
      if (cut) mask(sv, lim - j * RA_BKV - first);
      if (!agree(std::true_type(), j, max_t(sv, sca))) return false;
      const float neg = m > -INFINITY ? A8_LIFT - m : 0.f;
      uint64_t r0 = 0, r1 = 0;
      uint32_t ph[4], pm[4], pl[4];
      weigh(sv, sca, neg, ph, pm, pl, r0, r1);
      // with two buffers this step's is free once the product of two steps before is done (at no earlier phase: as in agree)
      if (!least && n >= 2 && !a8_wait(p_done(n - 2), phase(n - 2), p.err, abort_flag)) return false;
      // a row's three parts, `apart` rows from each other; 16 keys: one 16-byte chunk of a row's 128 bytes
      auto put = [&](int row, const uint32_t (&x)[4]) {
        st_shared_v4(few_p(least, n) + row * 128 + ((2 * quarter + (lane >> 4)) ^ (row & 7)) * 16, x[0], x[1], x[2], x[3]);
      };
      if ((lane & 15) < apart) {
        put(lane & 15, ph);
        put((lane & 15) + apart, pm);
        put((lane & 15) + 2 * apart, pl);
      }
      sum_up(r0, r1);
      fence_async_shared();
      tmem_st_wait();                              // O's, if the maximum was raised
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sc_empty(n));
        mbar_arrive(p_full(n));
      }
      return true;
    };
    for (int k = 0; ok && more; ++k) {
      int left, whole, rows;                       // tiles left; those that every row sees whole; rows
      {
        const RaPiece& c = piece(k);
        left = c.tb - c.ta;
        rows = c.toks * p.G;
        const int over = c.pos0 - c.ta * RA_BKV;   // the tile's first row's last key
        whole = min(left, (over + 1) >> 7);        // below zero: none
        lim = over + min(token_of(rows <= A8_FEW ? lane & 15 : r), c.toks - 1);     // padding rows: the last real row's limit
        end = c.L - c.ta * RA_BKV;
      }
      const bool few = rows <= A8_FEW;
      const bool busy = few || quarter * 32 < rows;      // some row of this warp is real
      real = (few ? lane & (A8_FEW - 1) : r) < rows;
      least = rows <= A8_LEAST;
      apart = least ? A8_LEAST : A8_FEW;
      // the zeros beside the third parts (nobody reads the buffers between two pieces)
      if (few && !least) st_shared_v4(few_p(false, grp) + A8_FEW_TILE + A8_FEW * 128 + r * 16, 0u, 0u, 0u, 0u);
      m = -INFINITY;
      l = 0.f;
      if (!a8_wait(k ? q_full(k) : q_first, q_phase(k), p.err, abort_flag)) { ok = false; break; }
      rs = qscale[(k & (A8_QR - 1)) * RA_BQ + r];
      int j = (n0 & 1) ^ grp;                      // this group's first step
      if (few) {
        for (; ok && j < left; j += 2) ok = step_few(j >= whole, j);
      } else if (busy) {
        for (; ok && j < left; j += 2) ok = step(j >= whole, j);
      } else {
        // no real row: P stays whatever it is, its O rows are never read
        for (; ok && j < left; j += 2) {
          const int n = n0 + j;
          ok = a8_wait(s_full(n), phase(n), p.err, abort_flag) && (!TMA || clear_tail(end - j * RA_BKV, n));
          __syncwarp();
          if (ok && lane == 0) {
            mbar_arrive(sc_empty(n));
            mbar_arrive(p_full(n));
          }
        }
      }
      if (!ok) break;
      // the last step's maximum, if the other group had it, and both groups' sums
      if (busy && j != left + 1) {
        float mx;
        if (!(few ? heard(std::true_type(), left - 1, mx) : heard(std::false_type(), left - 1, mx))) { ok = false; break; }
        const float m2 = raised(m, mx);
        if (m2 > m) {
          l *= ra_ex2(m - m2);
          m = m2;
        }
      }
      float* sum = lsum + (k & 1) * 2 * RA_BQ;
      sum[grp * RA_BQ + r] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(sums);
      n0 += left;
      if (few) t_few += left; else if (busy) t_all += left;
      const RaPiece c = piece(k);
      more = find(k + 1);                          // while the piece's last P V product, step n0 - 1's, runs
      // in this order: once both groups are through, the product of step n0 - 4 is done, and the barrier of
      // step n0 - 1's at no earlier phase
      if (!a8_wait(sums, k & 1, p.err, abort_flag) || !a8_wait(p_done(n0 - 1), phase(n0 - 1), p.err, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (few ? quarter == 0 : busy) {             // each group half of the columns
        if (few) {
          l = 0.f;
#pragma unroll 1
          for (int q = 0; q < 16; ++q) l += sum[q * 16 + (lane & 15)];
        } else {
          l = sum[r] + sum[RA_BQ + r];
        }
        const bool all = c.flags & 1;
        const int tok = token_of(r);
        const bool mine = r < rows;
        const int64_t orow = static_cast<int64_t>(c.row0 + tok) * p.Hq + c.g * p.G + (r - tok * p.G);
        const int64_t pslot = static_cast<int64_t>(cta) * 2 + (c.flags >> 1);
        const float inv = all ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(oadr + grp * 64 + h * 32, v);
          tmem_ld_wait();
          if (few) {                               // the other parts' share (more than A8_LEAST rows: one other lane's)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float b = __uint_as_float(__shfl_down_sync(0xffffffffu, v[e], apart));
              const float c = __uint_as_float(__shfl_down_sync(0xffffffffu, v[e], 2 * A8_LEAST));
              v[e] = __float_as_uint(__uint_as_float(v[e]) + (least ? b + c : b));
            }
          }
          if (mine && all) {
            __nv_bfloat16* orow_p = p.j.o + orow * RA_D + grp * 64 + h * 32;
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[i] = pack_bf16x2(__uint_as_float(v[e + 2 * i]) * inv, __uint_as_float(v[e + 2 * i + 1]) * inv);
              ra_st32(orow_p + e, y);
            }
          } else if (mine) {
            float* po = p.j.part_o + (pslot * RA_D + grp * 64 + h * 32) * RA_BQ + r * 4;      // lanes side by side
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(po + e * RA_BQ) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
          __syncwarp();                            // the next load is a whole warp's
        }
        if (mine && grp == 0) {
          if (all) {
            if (p.j.lse) p.j.lse[orow] = (m - A8_LIFT + log2f(l)) * RA_LN2;
          } else {
            *reinterpret_cast<float2*>(p.j.part_ml + (pslot * RA_BQ + r) * 2) = make_float2(m - A8_LIFT, l);
          }
        }
      }
      // O is read: the next piece's first P V may write it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
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
  p.inv_g = (65536 + p.G - 1) / p.G;
  const bool tma = rc.block_size % 8 == 0;
  p.box_log = 7;
  while (tma && rc.block_size & ((1 << p.box_log) - 1)) --p.box_log;    // gcd(block_size, 128)
  if (tma) {
    // (128 columns, kv heads, rows)
    const cuuint64_t pitch = static_cast<cuuint64_t>(Hkv) * RA_D;
    const cuuint64_t dk[3] = {RA_D, static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(rc.n_blocks) * rc.block_size};
    const cuuint64_t sk[2] = {RA_D, pitch};
    const cuuint32_t bk[3] = {RA_D, 1, 1u << p.box_log};
    // a row is 128 bytes, its neighbours are other heads': 256-byte fetches would bring those, too
    KL_TRY(ra_map(&p.tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, kp, dk, sk, bk, CU_TENSOR_MAP_L2_PROMOTION_L2_128B));
    KL_TRY(ra_map(&p.tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, vp, dk, sk, bk, CU_TENSOR_MAP_L2_PROMOTION_L2_128B));
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
