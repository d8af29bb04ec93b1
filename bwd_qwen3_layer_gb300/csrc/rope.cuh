// Rotary angles, shared by the kernels that turn queries and keys.
#pragma once

#include <math.h>
#include <stdint.h>

namespace kl {

// ---------------------------------------------------------------------------
// RoPE. Plane i pairs element i with element i + d/2 and turns it by the
// angle s * base^(-2i/d). The angle is reduced exactly in fixed point, as a
// phase accumulator does: plane i's rate in turns per position,
// base^(-2i/d) / (2 pi), is formed on the host in fp64 and passed as a 64-bit
// binary fraction of a turn; on the device s times that rate, taken modulo
// 2^64 by the integer multiply, is the position's angle in turns modulo one,
// and its top 32 bits read as a signed integer give the remainder in
// [-pi, pi) for the fp32 sincosf. No fp64 arithmetic runs on the device; the
// angle error is ~1e-11 rad from the rate plus 2^-32 of a turn from the
// truncation, below the fp32 rounding of the remainder itself.
// ---------------------------------------------------------------------------
constexpr int ROPE_MAX_HALF = 128;
struct RopeFreq {
  uint64_t turn[ROPE_MAX_HALF];   // plane i's rate, turns per position, in units of 2^-64 turn
};

// The rates of a (d, base), formed once per host thread and kept until another
// pair is asked for: 64 pow() calls took ~3 us of a small launch's host time.
inline const RopeFreq& rope_freq(int d, float base) {
  static thread_local RopeFreq f;
  static thread_local int last_d = 0;
  static thread_local float last_base = 0.f;
  if (d != last_d || base != last_base) {
    for (int i = 0; i < ROPE_MAX_HALF; ++i) {
      const double rate = i < d / 2 ? pow(static_cast<double>(base), -2.0 * i / d) / 6.283185307179586 : 0.0;
      f.turn[i] = static_cast<uint64_t>(ldexp(rate, 64));   // rate < 1/(2 pi): fits in 64 bits
    }
    last_d = d;
    last_base = base;
  }
  return f;
}

__device__ __forceinline__ void rope_cos_sin(int s, uint64_t turn, float dir, float* c, float* sn) {
  const uint64_t phase = static_cast<uint64_t>(s) * turn;            // turns mod 1, in 2^-64 units
  const int32_t hi = static_cast<int32_t>(static_cast<uint32_t>(phase >> 32));
  const float r = static_cast<float>(hi) * 1.46291807926715968e-09f;  // 2 pi / 2^32
  float sf, cf;
  sincosf(r, &sf, &cf);
  *c = cf;
  *sn = dir * sf;
}

}  // namespace kl
