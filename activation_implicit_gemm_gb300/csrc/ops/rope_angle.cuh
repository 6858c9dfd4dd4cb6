// Positions and the sine and cosine of their angles, for the kernels that turn pairs.
//
// The angle in turns is position * inv_freq / (2 pi). The f32 product alone would be off by up
// to 2^-24 of its size (0.004 radians at an angle of 65536), so the products are kept with
// their exact remainders (one FMA each) until the whole turns are gone; what is left, within
// half a turn, is right to about 2^-24 turns at every position up to 2^23. Tokens with a longer
// position (integers past 2^24 are not f32 values any more) take the same steps in f64, right to
// that at every position up to 2^53.
#pragma once

#include <cstdint>

#include "ops_internal.h"

namespace fconv {
namespace ops {
namespace {

__device__ __forceinline__ void turn_of(float pos, float freq, float& sn, float& cs) {
  constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
  constexpr float kHi = (float)kTurn, kLo = (float)(kTurn - (double)kHi);
  const float p = pos * freq, e = fmaf(pos, freq, -p);  // p + e is the exact product
  const float t = p * kHi, f = fmaf(p, kHi, -t);        // t + f is p kHi exactly
  const float rest = fmaf(p, kLo, fmaf(e, kHi, f));
  sincospif(2.0f * ((t - rintf(t)) + rest), &sn, &cs);
}

// The same for a position that an f32 may not hold.
__device__ __noinline__ float2 turn_of_long(double pos, float freq) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
  const double p = pos * (double)freq, e = fma(pos, (double)freq, -p);
  const double t = p * kHi, f = fma(p, kHi, -t);
  const double rest = fma(p, kLo, fma(e, kHi, f));
  double turns = (t - rint(t)) + rest;
  turns -= rint(turns);
  float2 v;
  sincospif(2.0f * (float)turns, &v.x, &v.y);
  return v;
}

constexpr float kLongPosition = 8388608.0f;  // 2^23

__device__ __forceinline__ float position(const void* pos, int type, int64_t at) {
  if (type == FCONV_POS_I32) return (float)((const int32_t*)pos)[at];
  if (type == FCONV_POS_I64) return (float)((const int64_t*)pos)[at];
  return ((const float*)pos)[at];
}
__device__ __forceinline__ double long_position(const void* pos, int type, int64_t at) {
  if (type == FCONV_POS_I32) return (double)((const int32_t*)pos)[at];
  if (type == FCONV_POS_I64) return (double)((const int64_t*)pos)[at];
  return (double)((const float*)pos)[at];
}

}  // namespace
}  // namespace ops
}  // namespace fconv
