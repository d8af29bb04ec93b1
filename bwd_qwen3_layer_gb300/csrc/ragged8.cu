// The new tokens of a ragged step into pages of 8-bit codes: per-head norm and
// rotation of queries and keys, keys and values rounded to e4m3 with one scale for
// each page and head.
//
//   y = R(pos) (g * x / rms(x)),  a = max |y| over the page's new rows,
//   w = 2^max(e, -64), e least with a / 2^e <= 448,
//   scale = w for a page begun by this step, else max(scale, w),  code = e4m3(y / scale).
//
// A power of two costs no precision (e4m3 is a floating format: the scale only says
// where its range lies), and makes the rounding again of a growing page's older codes
// a change of exponent: whatever the order in which a page fills, its codes are those
// of the final scale but for subnormal ones.
//
// Bound by HBM and issue slots where there are many rows (9000 rows of nine prompts, 64
// and 8 heads, 16 slots: 62 us, 76 % of the copy rate, half of the issue slots; queries
// alone 50), by latency where there are few (64 decoding rows 6.9 us). CTAs of two
// kinds in one launch: the first look for the pages that rows of theirs begin in the step
// (a row whose predecessor is not the slot before), the others take some rows' queries.
// A CTA of the first kind takes the runs that begin in 16 rows, head by head, the rows of
// the next heads on their way: 16 rows from the first run's on, an eighth of one to a
// thread, its angles in registers, which meet for the runs' largest sizes. Where the runs
// have more rows these are read twice, 16 at a time (the prompts in blocks of 64: 84 us, and their angles formed twice for each head).
// Before, a CTA for each row and head, of which one of 16 found a run, formed the angles
// eight times over: 143 us (9000 decoding rows 348 against 71).
#include <float.h>

#include "e4m3.cuh"
#include "internal.h"
#include "kl_common.cuh"
#include "rope.cuh"

namespace kl {
namespace {

constexpr int R8_THREADS = 128;
constexpr int RQ_D = 128;
constexpr int RQ_LANES = 8;                      // threads per head: 8 planes (16 elements) each
constexpr int R8_UNITS = R8_THREADS / RQ_LANES;  // heads that a CTA has in flight at a time
constexpr int R8_TILE = 16;                      // rows whose runs a CTA takes
constexpr int R8_AHEAD = 4;                      // steps whose rows are on their way to a CTA of the first kind
constexpr int R8_MAX = 4;                        // query heads a thread has in flight
constexpr int R8_QROWS = 16;                     // rows of a query CTA at most

struct Rope8Params {
  const __nv_bfloat16* q_pre;
  const __nv_bfloat16* k_pre;
  const __nv_bfloat16* v;
  const __nv_bfloat16* gq;
  const __nv_bfloat16* gk;
  const int32_t* cu;
  const int32_t* pos;
  const int32_t* slots;
  __nv_bfloat16* q_out;
  uint8_t* k_pool;
  uint8_t* v_pool;
  float* k_scale;
  float* v_scale;
  float eps;
  int B, T, Hq, Hkv, inter, bs, pool_rows;
  int kv_parts, kv_ctas, q_rows;   // CTAs that share a tile's heads, CTAs of the first kind, rows of a query CTA
  uint32_t* err;
  RopeFreq f;
};

// rope_cos_sin in fewer instructions: the phase's upper bits give the quarter of a turn, exactly, and the rest is
// within an eighth, where the power series of sine and cosine are off by 2^-29 after five and six terms. 2^-23.3 in
// all, sincosf's precision; the hardware's functions (2^-21) left some codes and queries a step away.
__device__ __forceinline__ void r8_cos_sin(int pos, uint64_t turn, float* c, float* s) {
  const uint32_t t = static_cast<uint32_t>((static_cast<uint64_t>(pos) * turn) >> 32);   // turns mod 1, in 2^-32 units
  const uint32_t k = (t + 0x20000000u) >> 30;
  const float r = static_cast<float>(static_cast<int32_t>(t - (k << 30))) * 1.46291807926715968e-09f;   // 2 pi / 2^32
  const float x = r * r;
  const float sn = fmaf(r * x, fmaf(x, fmaf(x, fmaf(x, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), r);
  const float cs = fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float a = k & 1 ? -sn : cs, b = k & 1 ? cs : sn;
  *c = k & 2 ? -a : a;
  *s = k & 2 ? -b : b;
}
// The least power of two w >= 2^-64 with a / w <= 448 = 1.75 * 2^8, for finite a >= 0.
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -64) + 127) << 23);
}

// Pairs of floats, one instruction for two.
__device__ __forceinline__ uint64_t r8_two(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 r8_both(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t r8_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t r8_sub(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t r8_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// An eighth of a head as pairs of floats: (a[e], b[e]) is what plane 8 l + e turns. Loaded as words xa and xb,
// elements 8 l .. and 64 + 8 l .. (halves), or 16 l .. 16 l + 15 (pairs of neighbours).
struct R8Head {
  uint64_t a[4], b[4];
  __device__ __forceinline__ void unpack(const uint4& xa, const uint4& xb, bool neighbours) {
    const uint32_t w[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
    auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
    auto hi = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
    if (neighbours) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = r8_two(lo(w[2 * e]), lo(w[2 * e + 1]));
        b[e] = r8_two(hi(w[2 * e]), hi(w[2 * e + 1]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = r8_two(lo(w[e]), hi(w[e]));
        b[e] = r8_two(lo(w[4 + e]), hi(w[4 + e]));
      }
    }
  }
  // the 16 numbers in the words' order
  __device__ __forceinline__ void order(float (&x)[16], bool neighbours) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = r8_both(a[e]), v = r8_both(b[e]);
      if (neighbours) {
        x[4 * e] = u.x; x[4 * e + 1] = v.x; x[4 * e + 2] = u.y; x[4 * e + 3] = v.y;
      } else {
        x[2 * e] = u.x; x[2 * e + 1] = u.y; x[8 + 2 * e] = v.x; x[8 + 2 * e + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void pack(uint4& xa, uint4& xb, bool neighbours) const {
    float x[16];
    order(x, neighbours);
    xa = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    xb = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]), pack_bf16x2(x[14], x[15]));
  }
  // normed, if wanted, with the gains g, and turned by cosines c and sines s; called by whole warps
  __device__ __forceinline__ void turn(const R8Head& g, bool norm, float eps, const uint64_t (&c)[4], const uint64_t (&s)[4]) {
    if (norm) {
      uint64_t q = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) q = r8_fma(a[e], a[e], r8_fma(b[e], b[e], q));
      const float2 q2 = r8_both(q);
      float ss = q2.x + q2.y;
#pragma unroll
      for (int o = RQ_LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss / static_cast<float>(RQ_D) + eps);   // two ulp; the result is rounded to 8 bits at most
      const uint64_t r2 = r8_two(r, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = r8_mul(r8_mul(a[e], r2), g.a[e]);
        b[e] = r8_mul(r8_mul(b[e], r2), g.b[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t x = r8_sub(r8_mul(a[e], c[e]), r8_mul(b[e], s[e]));
      b[e] = r8_fma(a[e], s[e], r8_mul(b[e], c[e]));
      a[e] = x;
    }
  }
  // the largest size; NaN if there is one
  __device__ __forceinline__ float size() const {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = r8_both(a[e]), v = r8_both(b[e]);
      asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(u.x), "f"(u.y));
      asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v.x), "f"(v.y));
    }
    return m;
  }
  // the largest finite size
  __device__ __forceinline__ float finite_size() const {
    float x[16], m = 0.f;
    order(x, false);
#pragma unroll
    for (int e = 0; e < 16; ++e) m = fabsf(x[e]) <= FLT_MAX ? fmaxf(m, fabsf(x[e])) : m;
    return m;
  }
  // codes of the numbers times r, to their places; an infinity is held as NaN: the conversion alone would make it 448
  __device__ __forceinline__ void store(uint8_t* at, int ia, int ib, float r, bool neighbours, bool finite) const {
    R8Head h;
    const uint64_t r2 = r8_two(r, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h.a[e] = r8_mul(a[e], r2);
      h.b[e] = r8_mul(b[e], r2);
    }
    float x[16];
    h.order(x, neighbours);
    if (!finite) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (fabsf(x[e]) > FLT_MAX) x[e] = __int_as_float(0x7fffffff);
    }
    *reinterpret_cast<uint2*>(at + ia) = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
    *reinterpret_cast<uint2*>(at + ib) = make_uint2(e4m3x4(x[8], x[9], x[10], x[11]), e4m3x4(x[12], x[13], x[14], x[15]));
  }
};
// 16 codes at another scale.
__device__ __forceinline__ void r8_again(uint8_t* at, float ratio) {
  uint4 x = *reinterpret_cast<uint4*>(at);
  uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 f = e4m3x4_to_f(w[e]);
    w[e] = e4m3x4(f.x * ratio, f.y * ratio, f.z * ratio, f.w * ratio);
  }
  *reinterpret_cast<uint4*>(at) = x;
}
// Whether a row's slot begins a run of the step in its page. `before`: the slot of the row before (row > 0).
__device__ __forceinline__ bool r8_leads(const Rope8Params& p, int row, int slot, int before) {
  return slot >= 0 && slot < p.pool_rows && (row == 0 || slot % p.bs == 0 || before != slot - 1);
}
// The rows of a run that begins at `row`, counted by a warp.
__device__ __forceinline__ int r8_run(const Rope8Params& p, int row, int slot, int rows) {
  const int most = min(p.bs - slot % p.bs, rows - row), lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < most; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, i < most && p.slots[row + i] == slot + i);
    if (m != 0xffffffffu) return i0 + __ffs(~m) - 1;
  }
  return most;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src), "n"(BYTES) : "memory");
}

struct R8Angles {                                  // of a query CTA's rows
  float c[R8_QROWS][RQ_D / 2], s[R8_QROWS][RQ_D / 2];
};

// The queries of rows [row0, row0 + q_rows): R8_MAX heads a thread at a time, the first on their way before the
// angles are formed.
__device__ __forceinline__ void r8_queries(const Rope8Params& p, int row0, R8Angles& cs) {
  const int l = threadIdx.x % RQ_LANES, u0 = threadIdx.x / RQ_LANES;
  const int ia = p.inter ? 16 * l : 8 * l, ib = p.inter ? 16 * l + 8 : 64 + 8 * l;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  const bool norm = p.gq != nullptr;
  const int rows = min(p.q_rows, p.T - row0), units = rows * p.Hq;
  const __nv_bfloat16* q = p.q_pre + static_cast<int64_t>(row0) * p.Hq * RQ_D;
  __nv_bfloat16* y = p.q_out + static_cast<int64_t>(row0) * p.Hq * RQ_D;
  const uint4 ga = norm ? *reinterpret_cast<const uint4*>(p.gq + ia) : none, gb = norm ? *reinterpret_cast<const uint4*>(p.gq + ib) : none;
  const int last = min(p.cu[p.B], p.T) - row0;       // rows from here on are no request's
  for (int base = 0; base < units; base += R8_MAX * R8_UNITS) {
    uint4 xa[R8_MAX], xb[R8_MAX];
#pragma unroll
    for (int j = 0; j < R8_MAX; ++j) {
      const int u = base + j * R8_UNITS + u0;
      xa[j] = xb[j] = none;
      if (u < units) {
        xa[j] = *reinterpret_cast<const uint4*>(q + u * RQ_D + ia);
        xb[j] = *reinterpret_cast<const uint4*>(q + u * RQ_D + ib);
      }
    }
    if (base == 0) {
      for (int t = threadIdx.x; t < rows * (RQ_D / 2); t += R8_THREADS) {
        const int i = t / (RQ_D / 2), pl = t % (RQ_D / 2);
        r8_cos_sin(p.pos[row0 + i], p.f.turn[pl], &cs.c[i][pl], &cs.s[i][pl]);
      }
      __syncthreads();
    }
    R8Head g;
    g.unpack(ga, gb, p.inter);
#pragma unroll
    for (int j = 0; j < R8_MAX; ++j) {
      const int u = base + j * R8_UNITS + u0, i = u / p.Hq;
      uint64_t c[4], s[4];
      const ulonglong2* cp = reinterpret_cast<const ulonglong2*>(&cs.c[min(i, rows - 1)][8 * l]);
      const ulonglong2* sp = reinterpret_cast<const ulonglong2*>(&cs.s[min(i, rows - 1)][8 * l]);
      const ulonglong2 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
      c[0] = c0.x; c[1] = c0.y; c[2] = c1.x; c[3] = c1.y;
      s[0] = s0.x; s[1] = s0.y; s[2] = s1.x; s[3] = s1.y;
      R8Head x;
      x.unpack(xa[j], xb[j], p.inter);
      x.turn(g, norm, p.eps, c, s);
      x.pack(xa[j], xb[j], p.inter);
      if (u >= units || i >= last) continue;
      *reinterpret_cast<uint4*>(y + u * RQ_D + ia) = xa[j];
      *reinterpret_cast<uint4*>(y + u * RQ_D + ib) = xb[j];
    }
  }
}

__global__ void __launch_bounds__(R8_THREADS, 6) ragged_qkv8_kernel(const __grid_constant__ Rope8Params p) {
  pdl_enter();
  __shared__ union {
    R8Angles cs;
    struct {                                     // a thread's eighth of a row and its page's scale, for each step
      uint4 x[R8_AHEAD][2][R8_THREADS];
      float old[R8_AHEAD][R8_THREADS];
    } in;
  } sh;
  __shared__ int run_max[2][R8_TILE];            // the runs' largest sizes, at their first rows, as bits
  __shared__ float run_old[2][R8_TILE];          // and their pages' scales before the step, 0 for a page it begins
  __shared__ float ratio[R8_TILE];              // old scale to new one of runs whose page's scale grows, else 0
  if (static_cast<int>(blockIdx.x) >= p.kv_ctas) {
    r8_queries(p, (blockIdx.x - p.kv_ctas) * p.q_rows, sh.cs);
    return;
  }
  const int lane = threadIdx.x & 31, l = threadIdx.x % RQ_LANES, i = threadIdx.x / RQ_LANES;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  const bool norm = p.gk != nullptr;
  const int row0 = static_cast<int>(blockIdx.x) / p.kv_parts * R8_TILE, part = blockIdx.x % p.kv_parts;
  // the tile's runs, found by every warp: its lane k looks at row row0 + k
  const int slot_l = row0 + lane < p.T ? p.slots[row0 + lane] : -1, before = row0 > 0 ? p.slots[row0 - 1] : -1;
  if (threadIdx.x < 2 * R8_TILE) run_max[threadIdx.x / R8_TILE][threadIdx.x % R8_TILE] = 0;
  const int rows = min(p.cu[p.B], p.T), here = min(R8_TILE, rows - row0);
  if (here <= 0) return;
  const int above = __shfl_up_sync(0xffffffffu, slot_l, 1);
  uint32_t runs = __ballot_sync(0xffffffffu, lane < here && r8_leads(p, row0 + lane, slot_l, lane ? above : before));
  const uint32_t breaks = __ballot_sync(0xffffffffu, row0 + lane >= rows || slot_l != above + 1);
  if (part == 0 && threadIdx.x < here && slot_l >= p.pool_rows) record_error(p.err, KL_DEVERR_PAGE);
  const int w0 = part * (2 * p.Hkv) / p.kv_parts, w1 = (part + 1) * (2 * p.Hkv) / p.kv_parts;   // keys, then values
  // elements 8 l .. and 64 + 8 l .., or 16 l .. and 16 l + 8 ..
  const int ka = p.inter ? 16 * l : 8 * l, kb = p.inter ? 16 * l + 8 : 64 + 8 * l;
  R8Head g;
  g.unpack(norm ? *reinterpret_cast<const uint4*>(p.gk + ka) : none, norm ? *reinterpret_cast<const uint4*>(p.gk + kb) : none, p.inter);
  __syncthreads();                               // run_max is empty
  int buf = 0;                                   // of two in turn: one is emptied while the next head fills the other
  // runs that lie within R8_UNITS rows, or a longer one, at a time
  while (runs) {
    const int k0 = __ffs(runs) - 1;
    uint32_t lead = runs & (0xffffu << k0);
    int il = 31 - __clz(lead), end = 0;            // the last of them and its end
    auto last_run = [&] {
      const int slotl = __shfl_sync(0xffffffffu, slot_l, il);
      const uint32_t stop = breaks & (0xfffffffeu << il);
      end = min(il + p.bs - slotl % p.bs, stop ? __ffs(stop) - 1 : 32);
      if (end == 32) end = il + r8_run(p, row0 + il, slotl, rows);
    };
    last_run();
    if (end - k0 > R8_UNITS && il != k0) {
      lead &= ~(1u << il);
      il = 31 - __clz(lead);
      last_run();
    }
    runs &= ~lead;
    const int chunks = (end - k0 + R8_UNITS - 1) / R8_UNITS;
    // This thread's row of a chunk: row row0 + k, of the run that begins at row0 + i0 in slot slot0, place `at` of
    // its page; has: whether it is of one.
    struct Row {
      int k, i0, slot0, at;
      bool has;
    };
    auto row_of = [&](int chunk) {
      Row o;
      o.k = k0 + chunk * R8_UNITS + i;
      const uint32_t upto = 0xffffffffu >> (31 - min(o.k, 31));
      o.i0 = 31 - __clz(lead & upto);              // the last run that begins at or above it
      o.slot0 = __shfl_sync(0xffffffffu, slot_l, o.i0);
      o.at = o.slot0 % p.bs;
      o.has = o.i0 == il ? o.k < end : !(breaks & upto & (0xfffffffeu << o.i0)) && o.at + o.k - o.i0 < p.bs;
      return o;
    };
    auto first = [&](const Row& o) { return l == 0 && o.k == o.i0; };   // (such a row is of its run)
    Row me = row_of(0), ask = me;                  // of the step at hand, of the next to ask for
    // A step: the rows of a chunk for one head's keys or values; a head's steps are its chunks and, where they are
    // several, these once more.
    const int steps = chunks > 1 ? 2 * chunks : 1;
    int wi = w0, ti = 0, si = 0;                   // the next step to ask for, its place
    auto fetch = [&] {
      if (chunks > 1) ask = row_of(ti < chunks ? ti : ti - chunks);
      if (wi < w1 && ask.has) {
        const bool key = wi < p.Hkv;
        const int h = key ? wi : wi - p.Hkv;
        const __nv_bfloat16* x = (key ? p.k_pre : p.v) + (static_cast<int64_t>(row0 + ask.k) * p.Hkv + h) * RQ_D;
        cp_async<16>(&sh.in.x[si][0][threadIdx.x], x + (key ? ka : 16 * l));
        cp_async<16>(&sh.in.x[si][1][threadIdx.x], x + (key ? kb : 16 * l + 8));
        if (first(ask) && ti < chunks && ask.at > 0) cp_async<4>(&sh.in.old[si][threadIdx.x], (key ? p.k_scale : p.v_scale) + static_cast<int64_t>(ask.slot0 / p.bs) * p.Hkv + h);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      si = (si + 1) % R8_AHEAD;
      if (++ti == steps) {
        ti = 0;
        ++wi;
      }
    };
#pragma unroll 1
    for (int k = 0; k < R8_AHEAD - 1; ++k) fetch();
    uint64_t c[4], s[4];
    auto angles = [&] {
      const int pos = me.has ? p.pos[row0 + me.k] : 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float c0, s0, c1, s1;
        r8_cos_sin(pos, p.f.turn[8 * l + 2 * e], &c0, &s0);
        r8_cos_sin(pos, p.f.turn[8 * l + 2 * e + 1], &c1, &s1);
        c[e] = r8_two(c0, c1);
        s[e] = r8_two(s0, s1);
      }
    };
    if (w0 < p.Hkv && chunks == 1) angles();
    int so = 0;                                    // the step's place
#pragma unroll 1
    for (int w = w0; w < w1; ++w, buf ^= 1) {
      const bool key = w < p.Hkv;
      const int h = key ? w : w - p.Hkv;
      bool grows = false;
      float* scales = (key ? p.k_scale : p.v_scale) + h;
      uint8_t* pool = (key ? p.k_pool : p.v_pool) + h * RQ_D;
#pragma unroll 1
      for (int t = 0; t < steps; ++t) {
        fetch();
        if (chunks > 1) {
          me = row_of(t < chunks ? t : t - chunks);
          if (key) angles();
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(R8_AHEAD - 1) : "memory");
        R8Head x;
        x.unpack(sh.in.x[so][0][threadIdx.x], sh.in.x[so][1][threadIdx.x], key && p.inter);
        if (t < chunks && first(me)) run_old[buf][me.i0] = me.at > 0 ? sh.in.old[so][threadIdx.x] : 0.f;
        so = (so + 1) % R8_AHEAD;
        if (key) x.turn(g, norm, p.eps, c, s);
        const float size = x.size();
        const bool finite = size <= FLT_MAX;
        if (t < chunks) {
          float most = finite ? size : x.finite_size();
#pragma unroll
          for (int o = RQ_LANES / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          if (me.has && l == 0) atomicMax(&run_max[buf][me.i0], __float_as_int(most));     // sizes are not negative
        }
        if (t == chunks - 1) __syncthreads();
        if (chunks > 1 && t < chunks) continue;
        const float old = run_old[buf][me.i0], now = fmaxf(old, scale_for(__int_as_float(run_max[buf][me.i0]))), r = 1.f / now;
        if (first(me)) {
          scales[static_cast<int64_t>(me.slot0 / p.bs) * p.Hkv] = now;
          ratio[me.i0] = me.at > 0 && now > old ? old * r : 0.f;
          grows |= me.at > 0 && now > old;
        }
        if (me.has) x.store(pool + static_cast<int64_t>(me.slot0 + me.k - me.i0) * p.Hkv * RQ_D, key ? ka : 16 * l, key ? kb : 16 * l + 8, r, key && p.inter, finite);
      }
      const int any = __syncthreads_or(grows);
      if (threadIdx.x < R8_TILE) run_max[buf][threadIdx.x] = 0;
      // pages whose scale grows: their older codes again, by the whole CTA
      if (any)
        for (uint32_t m = lead; m; m &= m - 1) {
          const int k = __ffs(m) - 1, s0 = __shfl_sync(0xffffffffu, slot_l, k), older = s0 % p.bs;
          if (ratio[k] == 0.f) continue;
          for (int o = i; o < older; o += R8_UNITS) r8_again(pool + static_cast<int64_t>(s0 - older + o) * p.Hkv * RQ_D + 16 * l, ratio[k]);
        }
    }
  }
}

}  // namespace

kl_status ragged_qkv_rope8(const kl_ragged_cfg& rc, int Hq, int Hkv, const void* q_pre, const void* k_pre, const void* v,
                           const void* gq, const void* gk, float eps, float base, int inter, const int32_t* cu,
                           const int32_t* pos, const int32_t* slots, void* q_out, void* kp, void* vp, float* ks,
                           float* vs, cudaStream_t st) {
  Rope8Params p;
  p.q_pre = static_cast<const __nv_bfloat16*>(q_pre);
  p.k_pre = static_cast<const __nv_bfloat16*>(k_pre);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.gq = static_cast<const __nv_bfloat16*>(gq);
  p.gk = static_cast<const __nv_bfloat16*>(gk);
  p.cu = cu;
  p.pos = pos;
  p.slots = slots;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_pool = static_cast<uint8_t*>(kp);
  p.v_pool = static_cast<uint8_t*>(vp);
  p.k_scale = ks;
  p.v_scale = vs;
  p.eps = eps;
  p.B = rc.B;
  p.T = rc.T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.inter = inter;
  p.bs = rc.block_size;
  p.pool_rows = rc.n_blocks * rc.block_size;
  p.err = device_error_word();
  p.f = rope_freq(RQ_D, base);
  // Tiles are shared by CTAs, up to one for each head's keys or values, until there are four for each SM, of
  // tiles in which a page begins. Query CTAs: a thread's R8_MAX heads once, or one row where rows are few.
  const int tiles = (rc.T - 1) / R8_TILE + 1;
  const int64_t busy = min(tiles, max(rc.B, rc.T / max(rc.block_size, R8_TILE) + 1));
  int parts = 1;
  while (parts < 2 * Hkv && busy * parts < 4 * num_sms()) parts *= 2;
  p.kv_parts = min(parts, 2 * Hkv);
  p.q_rows = rc.T < 2 * num_sms() ? 1 : max(1, min(R8_MAX * R8_UNITS / Hq, R8_QROWS));
  const int64_t kv = static_cast<int64_t>(tiles) * p.kv_parts, grid = kv + (rc.T - 1) / p.q_rows + 1;    // below 2^31 for 2^24 rows
  p.kv_ctas = static_cast<int>(kv);
  ProfScope ps("ragged_qkv_rope8", st, 0.0, static_cast<double>(rc.T) * (4.0 * Hq + 6.0 * Hkv) * RQ_D);
  launch_pdl(ragged_qkv8_kernel, static_cast<int>(grid), R8_THREADS, 0, st, p);
  KL_CUDA(cudaGetLastError());
  return KL_OK;
}

}  // namespace kl
