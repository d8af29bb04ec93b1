// Norm and rotation of one head by eight threads, shared by the kernels that
// write a ragged step's keys and values into their pages.
#pragma once

#include "internal.h"
#include "kl_common.cuh"
#include "rope.cuh"

namespace kl {
namespace {

constexpr int RQ_D = 128;
constexpr int RQ_LANES = 8;        // threads per head: 8 planes (16 elements) each

__device__ __forceinline__ void rq_unpack(const uint4& a, float (&f)[8]) {
  const float2 x0 = unpack_bf16x2(a.x), x1 = unpack_bf16x2(a.y), x2 = unpack_bf16x2(a.z), x3 = unpack_bf16x2(a.w);
  f[0] = x0.x; f[1] = x0.y; f[2] = x1.x; f[3] = x1.y;
  f[4] = x2.x; f[5] = x2.y; f[6] = x3.x; f[7] = x3.y;
}
__device__ __forceinline__ uint4 rq_pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// One head's eighth: thread l of a head's eight holds planes 8 l .. 8 l + 7, that
// is elements 8 l .. and 64 + 8 l .. (planes (i, i + 64)), or 16 l .. 16 l + 15
// (planes (2i, 2i + 1)): offsets ia and ib. a, b: its elements, normed (gva,
// gvb: its gains) and turned by the row's (cos, sin). Called by whole
// warps; `turn` is off for values, which stay as they are.
__device__ __forceinline__ void rq_turn_f(float (&a)[8], float (&b)[8], const uint4& gva, const uint4& gvb, bool norm, bool turn,
                                          int inter, int ia, float eps, const float2* cs) {
  if (norm) {                                       // the same for all threads: the shuffles are convergent
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
    for (int o = RQ_LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (turn) {
      const float r = rsqrtf(ss / static_cast<float>(RQ_D) + eps);   // two ulp; the result is rounded to bf16
      float ga[8], gb[8];
      rq_unpack(gva, ga);
      rq_unpack(gvb, gb);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = a[e] * r * ga[e];
        b[e] = b[e] * r * gb[e];
      }
    }
  }
  if (!turn) return;
  const int l8 = inter ? ia >> 1 : ia;              // 8 l
  if (inter) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 c0 = cs[l8 + e], c1 = cs[l8 + 4 + e];
      const float x0 = a[2 * e], y0 = a[2 * e + 1], x1 = b[2 * e], y1 = b[2 * e + 1];
      a[2 * e] = x0 * c0.x - y0 * c0.y;
      a[2 * e + 1] = x0 * c0.y + y0 * c0.x;
      b[2 * e] = x1 * c1.x - y1 * c1.y;
      b[2 * e + 1] = x1 * c1.y + y1 * c1.x;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 c = cs[l8 + e];
      const float x = a[e], z = b[e];
      a[e] = x * c.x - z * c.y;
      b[e] = x * c.y + z * c.x;
    }
  }
}
// The same from and to bf16.
__device__ __forceinline__ void rq_turn(uint4& xa, uint4& xb, const uint4& gva, const uint4& gvb, bool norm, bool turn, int inter,
                                        int ia, float eps, const float2* cs) {
  float a[8], b[8];
  rq_unpack(xa, a);
  rq_unpack(xb, b);
  rq_turn_f(a, b, gva, gvb, norm, turn, inter, ia, eps, cs);
  if (!turn) return;
  xa = rq_pack(a);
  xb = rq_pack(b);
}

}  // namespace
}  // namespace kl
