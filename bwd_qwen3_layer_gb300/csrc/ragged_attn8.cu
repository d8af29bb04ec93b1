// Attention of a ragged step over a paged cache of 8-bit codes with a scale for each
// page and head:
//   o_i = sum_j softmax_j(q_i . (a_j kc_j) / sqrt(d)) b_j vc_j,
// a_j, b_j the scales of the page that position j lies in. One warp per row and
// query head, a running maximum and sum, four dims a lane.
#include <math.h>

#include "internal.h"
#include "kl_common.cuh"

namespace kl {
namespace {

constexpr int A8_D = 128;
constexpr int A8_MAX_CTX = 1 << 30;

struct A8Params {
  const __nv_bfloat16* q;
  const uint8_t* kp;
  const uint8_t* vp;
  const float* ks;
  const float* vs;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* ctx;
  __nv_bfloat16* o;
  float* lse;
  int B, T, Hq, Hkv, G, bs, max_blocks, n_blocks;
  float scale;
  uint32_t* err;
};

__device__ __forceinline__ float4 codes(uint32_t v) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(v)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(v >> 16)));
  float4 r;
  asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(r.x), "=f"(r.y) : "r"(lo));
  asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(r.z), "=f"(r.w) : "r"(hi));
  return r;
}

__global__ void __launch_bounds__(128) ragged_attn8_kernel(const __grid_constant__ A8Params p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int row = static_cast<int>(item / p.Hq), h = static_cast<int>(item % p.Hq);
  if (row >= min(p.cu[p.B], p.T)) return;
  int lo = 0, hi = p.B;                       // cu[lo] <= row < cu[hi]
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (p.cu[m] <= row) lo = m; else hi = m;
  }
  const int L = min(max(p.ctx[lo], 0), A8_MAX_CTX) + row - p.cu[lo] + 1;
  const int g = h / p.G;
  const uint2 qv = *reinterpret_cast<const uint2*>(p.q + item * A8_D + lane * 4);
  const float2 q0 = unpack_bf16x2(qv.x), q1 = unpack_bf16x2(qv.y);
  float m = -INFINITY, s = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < L; ++j) {
    const int lb = j / p.bs;
    const int blk = lb < p.max_blocks ? p.table[static_cast<int64_t>(lo) * p.max_blocks + lb] : -1;
    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
    float ks = 1.f, vs = 1.f;
    if (blk >= 0 && blk < p.n_blocks) {
      const int64_t at = ((static_cast<int64_t>(blk) * p.bs + (j - lb * p.bs)) * p.Hkv + g) * A8_D + lane * 4;
      k = codes(*reinterpret_cast<const uint32_t*>(p.kp + at));
      v = codes(*reinterpret_cast<const uint32_t*>(p.vp + at));
      ks = p.ks[static_cast<int64_t>(blk) * p.Hkv + g];
      vs = p.vs[static_cast<int64_t>(blk) * p.Hkv + g];
    } else if (lane == 0) {
      record_error(p.err, KL_DEVERR_PAGE);
    }
    float t = q0.x * k.x + q0.y * k.y + q1.x * k.z + q1.y * k.w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    t = vs == vs ? t * (ks * p.scale) : vs;   // a NaN scale of either kind makes the row NaN
    const float m2 = fmaxf(m, t), c = m2 > -INFINITY ? expf(m - m2) : 1.f, e = expf(t - m2);
    m = m2;
    s = s * c + e;
    const float w = e * vs;
    acc.x = acc.x * c + w * v.x;
    acc.y = acc.y * c + w * v.y;
    acc.z = acc.z * c + w * v.z;
    acc.w = acc.w * c + w * v.w;
  }
  *reinterpret_cast<uint2*>(p.o + item * A8_D + lane * 4) =
      make_uint2(pack_bf16x2(acc.x / s, acc.y / s), pack_bf16x2(acc.z / s, acc.w / s));
  if (p.lse && lane == 0) p.lse[item] = m + logf(s);
}

}  // namespace

size_t ragged_attention8_ws() { return 256; }

kl_status ragged_attention8(const kl_ragged_cfg& rc, int Hq, int Hkv, const void* q, const void* kp, const void* vp,
                            const float* ks, const float* vs, const int32_t* table, const int32_t* cu,
                            const int32_t* ctx, void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (!ws || ws_bytes < ragged_attention8_ws() || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return set_error(KL_ERR_NO_MEMORY, "ragged attention8: workspace too small or not 256-byte aligned");
  A8Params p = {static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(kp), static_cast<const uint8_t*>(vp), ks, vs,
                table, cu, ctx, static_cast<__nv_bfloat16*>(o), lse, rc.B, rc.T, Hq, Hkv, Hq / Hkv, rc.block_size,
                rc.max_blocks, rc.n_blocks, 1.f / sqrtf(static_cast<float>(A8_D)), device_error_word()};
  const int64_t items = static_cast<int64_t>(rc.T) * Hq;
  ProfScope ps("ragged_attention8", st, 0.0, 4.0 * rc.T * Hq * A8_D);
  launch_pdl(ragged_attn8_kernel, static_cast<unsigned>((items + 3) / 4), 128, 0, st, p);
  KL_CUDA(cudaGetLastError());
  return KL_OK;
}

}  // namespace kl
