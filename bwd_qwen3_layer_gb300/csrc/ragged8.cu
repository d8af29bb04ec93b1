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
// CTAs of two kinds in one launch. The first take a (row, kv head) each: if the row
// is its page's first one of the step, the CTA handles all the page's rows for that
// head (16 at a time, eight threads a row), since they share the scale. The others
// take a row's queries each.
#include <float.h>

#include "e4m3.cuh"
#include "ragged_rope.cuh"

namespace kl {
namespace {

constexpr int R8_THREADS = 128;
constexpr int R8_ROWS = R8_THREADS / RQ_LANES;   // rows of a page in flight
constexpr int R8_MAX = 4;                        // query heads a thread has in flight

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
  uint32_t* err;
  RopeFreq f;
};

// The least power of two w >= 2^-64 with a / w <= 448 = 1.75 * 2^8, for finite a >= 0.
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -64) + 127) << 23);
}

__global__ void __launch_bounds__(R8_THREADS, 6) ragged_qkv8_kernel(const __grid_constant__ Rope8Params p) {
  pdl_enter();
  __shared__ float2 cs[R8_ROWS][RQ_D / 2];
  __shared__ float red[2][R8_THREADS / 32];
  const int l = threadIdx.x % RQ_LANES, h0 = threadIdx.x / RQ_LANES, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ia = p.inter ? 16 * l : 8 * l, ib = p.inter ? 16 * l + 8 : 64 + 8 * l;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  const bool norm = p.gq != nullptr;
  const int rows = min(p.cu[p.B], p.T);
  const int kv_ctas = p.T * p.Hkv;

  if (static_cast<int>(blockIdx.x) < kv_ctas) {
    const int row = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
    if (row >= rows) return;
    const int slot = p.slots[row];
    if (slot < 0) return;
    if (slot >= p.pool_rows) {
      if (h == 0 && threadIdx.x == 0) record_error(p.err, KL_DEVERR_PAGE);
      return;
    }
    const int page = slot / p.bs, at = slot - page * p.bs;
    if (at > 0 && row > 0 && p.slots[row - 1] == slot - 1) return;      // an earlier row leads
    // the page's rows of this step
    const int most = min(p.bs - at, rows - row);
    int n = most;
    for (int i0 = 0; i0 < most; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, i < most && p.slots[row + i] == slot + i);
      if (m != 0xffffffffu) {
        n = i0 + __ffs(~m) - 1;
        break;
      }
    }
    const uint4 ga = norm ? *reinterpret_cast<const uint4*>(p.gk + ia) : none, gb = norm ? *reinterpret_cast<const uint4*>(p.gk + ib) : none;
    const int64_t sat = static_cast<int64_t>(page) * p.Hkv + h;
    const float k_old = at > 0 ? p.k_scale[sat] : 0.f, v_old = at > 0 ? p.v_scale[sat] : 0.f;
    float ka[8], kb[8], va[8], vb[8];
    // rows i0 .. i0 + 15: this thread's eighth of row i0 + h0 (zeros past the last)
    auto fetch = [&](int i0) {
      __syncthreads();                   // nobody reads the angles any more
      for (int t = threadIdx.x; t < R8_ROWS * (RQ_D / 2); t += R8_THREADS) {
        const int i = t / (RQ_D / 2), pl = t % (RQ_D / 2);
        if (i0 + i < n) {
          float c, sn;
          rope_cos_sin(p.pos[row + i0 + i], p.f.turn[pl], 1.0f, &c, &sn);
          cs[i][pl] = make_float2(c, sn);
        }
      }
      __syncthreads();
      uint4 xa = none, xb = none, ya = none, yb = none;
      const bool mine = i0 + h0 < n;
      if (mine) {
        const int64_t off = (static_cast<int64_t>(row + i0 + h0) * p.Hkv + h) * RQ_D;
        xa = *reinterpret_cast<const uint4*>(p.k_pre + off + ia);
        xb = *reinterpret_cast<const uint4*>(p.k_pre + off + ib);
        ya = *reinterpret_cast<const uint4*>(p.v + off + 16 * l);
        yb = *reinterpret_cast<const uint4*>(p.v + off + 16 * l + 8);
      }
      rq_unpack(xa, ka);
      rq_unpack(xb, kb);
      rq_unpack(ya, va);
      rq_unpack(yb, vb);
      rq_turn_f(ka, kb, ga, gb, norm, mine, p.inter, ia, p.eps, cs[h0]);
    };
    float km = 0.f, vm = 0.f;            // the largest finite sizes
    auto size = [](float m, float x) { return fabsf(x) <= FLT_MAX ? fmaxf(m, fabsf(x)) : m; };
    for (int i0 = 0; i0 < n; i0 += R8_ROWS) {
      fetch(i0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        km = size(size(km, ka[e]), kb[e]);
        vm = size(size(vm, va[e]), vb[e]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
      vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
    }
    if (lane == 0) {
      red[0][warp] = km;
      red[1][warp] = vm;
    }
    __syncthreads();                     // every thread has read the old scales, too
#pragma unroll
    for (int w = 0; w < R8_THREADS / 32; ++w) {
      km = fmaxf(km, red[0][w]);
      vm = fmaxf(vm, red[1][w]);
    }
    const float k_new = fmaxf(k_old, scale_for(km)), v_new = fmaxf(v_old, scale_for(vm));
    if (threadIdx.x == 0) {
      p.k_scale[sat] = k_new;
      p.v_scale[sat] = v_new;
    }
    // a page whose scale grows: its older codes again
    auto again = [&](uint8_t* pool, float ratio) {
      for (int t = threadIdx.x; t < at * 8; t += R8_THREADS) {
        uint4* c = reinterpret_cast<uint4*>(pool + ((static_cast<int64_t>(page) * p.bs + (t >> 3)) * p.Hkv + h) * RQ_D + (t & 7) * 16);
        uint4 x = *c;
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 f = e4m3x4_to_f(w[e]);
          w[e] = e4m3x4(f.x * ratio, f.y * ratio, f.z * ratio, f.w * ratio);
        }
        *c = x;
      }
    };
    if (at > 0 && k_new > k_old) again(p.k_pool, k_old / k_new);
    if (at > 0 && v_new > v_old) again(p.v_pool, v_old / v_new);
    const float kr = 1.f / k_new, vr = 1.f / v_new;
    // an infinity is held as NaN: the conversion alone would make it 448
    auto code = [](float x, float r) { return fabsf(x) <= FLT_MAX ? x * r : __int_as_float(0x7fffffff); };
    auto pack = [&](const float (&x)[8], float r) {
      return make_uint2(e4m3x4(code(x[0], r), code(x[1], r), code(x[2], r), code(x[3], r)),
                        e4m3x4(code(x[4], r), code(x[5], r), code(x[6], r), code(x[7], r)));
    };
    for (int i0 = 0; i0 < n; i0 += R8_ROWS) {
      if (n > R8_ROWS) fetch(i0);        // else they are at hand
      if (i0 + h0 < n) {
        const int64_t off = (static_cast<int64_t>(slot + i0 + h0) * p.Hkv + h) * RQ_D;
        *reinterpret_cast<uint2*>(p.k_pool + off + ia) = pack(ka, kr);
        *reinterpret_cast<uint2*>(p.k_pool + off + ib) = pack(kb, kr);
        const uint2 x = pack(va, vr), y = pack(vb, vr);
        *reinterpret_cast<uint4*>(p.v_pool + off + 16 * l) = make_uint4(x.x, x.y, y.x, y.y);
      }
    }
    return;
  }

  // ---- a row's queries ----
  const int row = blockIdx.x - kv_ctas;
  constexpr int STEP = R8_THREADS / RQ_LANES;
  const uint4 ga = norm ? *reinterpret_cast<const uint4*>(p.gq + ia) : none, gb = norm ? *reinterpret_cast<const uint4*>(p.gq + ib) : none;
  if (row >= rows) return;
  const int pos = p.pos[row];
  for (int base = 0; base < p.Hq; base += R8_MAX * STEP) {
    uint4 xa[R8_MAX], xb[R8_MAX];
#pragma unroll
    for (int j = 0; j < R8_MAX; ++j) {
      const int h = base + j * STEP + h0;
      xa[j] = xb[j] = none;
      if (h < p.Hq) {
        const __nv_bfloat16* x = p.q_pre + (static_cast<int64_t>(row) * p.Hq + h) * RQ_D;
        xa[j] = *reinterpret_cast<const uint4*>(x + ia);
        xb[j] = *reinterpret_cast<const uint4*>(x + ib);
      }
    }
    if (base == 0) {
      if (threadIdx.x < RQ_D / 2) {
        float c, sn;
        rope_cos_sin(pos, p.f.turn[threadIdx.x], 1.0f, &c, &sn);
        cs[0][threadIdx.x] = make_float2(c, sn);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < R8_MAX; ++j) {
      const int h = base + j * STEP + h0;
      rq_turn(xa[j], xb[j], ga, gb, norm, true, p.inter, ia, p.eps, cs[0]);
      if (h >= p.Hq) continue;
      __nv_bfloat16* y = p.q_out + (static_cast<int64_t>(row) * p.Hq + h) * RQ_D;
      *reinterpret_cast<uint4*>(y + ia) = xa[j];
      *reinterpret_cast<uint4*>(y + ib) = xb[j];
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
  const int64_t grid = static_cast<int64_t>(rc.T) * (Hkv + 1);
  if (grid > 2147483647LL) return set_error(KL_ERR_UNSUPPORTED, "ragged_qkv_rope8: %d rows of %d kv heads", rc.T, Hkv);
  ProfScope ps("ragged_qkv_rope8", st, 0.0, static_cast<double>(rc.T) * (4.0 * Hq + 6.0 * Hkv) * RQ_D);
  launch_pdl(ragged_qkv8_kernel, static_cast<int>(grid), R8_THREADS, 0, st, p);
  KL_CUDA(cudaGetLastError());
  return KL_OK;
}

}  // namespace kl
