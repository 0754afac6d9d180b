// Angles of rotary positions, shared by the kernels that turn heads.
//
// The angle is reduced in turns, not radians: with f = freq / (2 pi) kept as an
// fp32 pair hi + lo and the position p < 2^24 exact in fp32, p * hi = t + e with
// one product and one fma (e exact), t - rint(t) is exact, and the fraction
// (t - rint(t)) + (e + p * lo) is off by a few 2^-26 turns at any position, where
// an fp32 product of radians would be off by p * 2^-24.  sincospif takes it from
// there.  It costs two fmas an angle, where 64-bit products would hold up the
// heads of small models (the fp64 pipe is 1/64 of the fp32 one).
#pragma once

#include "common.cuh"

namespace spec {
namespace rotary {

// A frequency (radians) in turns, hi + lo.
__device__ __forceinline__ float2 in_turns(double freq) {
  const double turns = freq * 0.15915494309189533577;  // 1 / (2 pi)
  const float hi = (float)turns;
  return make_float2(hi, (float)(turns - (double)hi));
}
// cos and sin, times the scale, of position x times the frequency.
__device__ __forceinline__ float2 cos_sin(float x, float2 turns, float scale) {
  const float m = x * turns.x, e = fmaf(x, turns.x, -m);
  const float frac = (m - rintf(m)) + fmaf(x, turns.y, e);
  float s, c;
  sincospif(2.f * frac, &s, &c);
  return make_float2(c * scale, s * scale);
}
__device__ __forceinline__ float2 cos_sin(float x, double freq, float scale) {
  return cos_sin(x, in_turns(freq), scale);
}

}  // namespace rotary
}  // namespace spec
