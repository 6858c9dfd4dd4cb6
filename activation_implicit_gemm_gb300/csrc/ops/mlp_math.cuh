// Activations of the gated feed-forward block with their slopes, and the layout in which the
// forward pass leaves its projections for the backward one.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ops_common.cuh"
#include "ops_internal.h"

namespace fconv {
namespace ops {
namespace {

// v, held within -most and most; NaN stays.
__device__ __forceinline__ float within(float v, float most) {
  float y;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(v), "f"(most));
  return y;
}
// Past it FastGelu is v or 0 and its slope 1 or 0 in f32 (from |v| = 6 and 12 on): held there, the
// powers of v that meet them stay finite.
constexpr float kFastGeluEnd = 32.0f;

// act(v) in f32, and with SLOPE its derivative.
template <int ACT, bool SLOPE>
__device__ __forceinline__ float act_exact(float alpha, float v, float& slope) {
  if (ACT == FCONV_ACT_RELU) {  // NaN goes through
    if (SLOPE) slope = v > 0.0f ? 1.0f : 0.0f;
    return v < 0.0f ? 0.0f : v;
  } else if (ACT == FCONV_ACT_SIGMOID) {
    const float p = 1.0f / (1.0f + expf(-v));
    if (SLOPE) slope = p * (1.0f / (1.0f + expf(v)));  // 1 - p loses its bits for large v
    return p;
  } else if (ACT == FCONV_ACT_QUICKGELU) {
    const float p = 1.0f / (1.0f + expf(-alpha * v));
    if (SLOPE) slope = p * (1.0f + alpha * v * (1.0f - p));
    return v * p;
  } else if (ACT == FCONV_ACT_GELU) {
    const float p = 0.5f * erfcf(v * -0.7071067811865476f);
    if (SLOPE) slope = p + v * 0.3989422804014327f * expf(-0.5f * v * v);
    return v * p;
  } else if (ACT == FCONV_ACT_FASTGELU) {
    // (1 + tanh z) / 2 is the logistic function of 2 z; 1 + tanh z itself would cancel for v < 0
    constexpr float k = 1.5957691216057308f, c = 0.044715f;  // sqrt(8 / pi)
    const float x = within(v, kFastGeluEnd), x2 = x * x, w = x * fmaf(k * c, x2, k);
    const float p = 1.0f / (1.0f + expf(-w));
    if (SLOPE) slope = p + x * fmaf(3.0f * k * c, x2, k) * p * (1.0f / (1.0f + expf(w)));
    return v * p;
  } else {
    if (SLOPE) slope = 1.0f;
    return v;
  }
}

// Calls M(ACT) with ACT the compile-time code of the activation, which is the same in all threads.
#define FCONV_GATE_SWITCH(act, M)                                  \
  switch (act) {                                                   \
    case FCONV_ACT_RELU: { M(FCONV_ACT_RELU); break; }             \
    case FCONV_ACT_SIGMOID: { M(FCONV_ACT_SIGMOID); break; }       \
    case FCONV_ACT_QUICKGELU: { M(FCONV_ACT_QUICKGELU); break; }   \
    case FCONV_ACT_GELU: { M(FCONV_ACT_GELU); break; }             \
    case FCONV_ACT_FASTGELU: { M(FCONV_ACT_FASTGELU); break; }     \
    default: { M(FCONV_ACT_NONE); break; }                         \
  }

template <bool SLOPE>
__device__ __forceinline__ float act_of(int act, float alpha, float v, float& slope) {
#define FCONV_M(ACT) return act_exact<ACT, SLOPE>(alpha, v, slope)
  FCONV_GATE_SWITCH(act, FCONV_M)
#undef FCONV_M
}

// The same with the special-function unit's exponential and reciprocal (each within 2 ulp of f32, the
// exponential of an argument x off by the rounding of x besides: |x| 2^-24 of the value), for values
// that are rounded to 16 bits right after: 5 to 20 instructions instead of 40 to 80,
// which set the time of the gradient's epilogue (8192 x 10240 values: 783 -> 485 us for the
// product and its epilogue). The activation is fixed at compile time: a branch outside the loops.
__device__ __forceinline__ float exp2_unit(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_unit(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + 2^-t): t = v log2 e gives the logistic function.
__device__ __forceinline__ float logistic2(float t) { return rcp_unit(1.0f + exp2_unit(-t)); }

template <int ACT, bool SLOPE>
__device__ __forceinline__ float act_fast(float alpha, float v, float& slope) {
  constexpr float kLog2e = 1.4426950408889634f;
  if (ACT == FCONV_ACT_RELU) {
    if (SLOPE) slope = v > 0.0f ? 1.0f : 0.0f;
    return v < 0.0f ? 0.0f : v;
  } else if (ACT == FCONV_ACT_SIGMOID) {
    const float p = logistic2(v * kLog2e);
    if (SLOPE) slope = p * logistic2(v * -kLog2e);
    return p;
  } else if (ACT == FCONV_ACT_QUICKGELU) {
    const float w = alpha * v, p = logistic2(w * kLog2e);
    if (SLOPE) slope = p * fmaf(w, 1.0f - p, 1.0f);
    return v * p;
  } else if (ACT == FCONV_ACT_GELU) {
    // Phi(v) from erfc(z), z = |v| / sqrt 2. For v < 0 it is all tail, so what counts is the error
    // relative to erfc: erfc(z) e^(z^2) is t P(t), t = 1 / (1 + 0.435 z), with the P of degree 5 whose
    // largest relative error over 0 <= z <= 9.3 is least, 3.7e-6 (a linear program over 4000 points). In
    // f32, with the exponential's argument rounded: 4.7e-6 of Phi down to v = -5, 1.9e-5 at -13, past
    // which Phi is no normal f32. The exponential is the slope's density too.
    const float z = fabsf(v) * 0.70710678118654752f;
    const float t = rcp_unit(fmaf(0.435f, z, 1.0f));
    float q = fmaf(-0.151734486f, t, 0.383800864f);
    q = fmaf(q, t, 0.0101330718f);
    q = fmaf(q, t, 0.274843603f);
    q = fmaf(q, t, 0.236997426f);
    q = fmaf(q, t, 0.24595587f);
    const float e = exp2_unit(-kLog2e * z * z);
    q *= t * e;
    const float p = v >= 0.0f ? fmaf(-0.5f, q, 1.0f) : 0.5f * q;
    if (SLOPE) slope = fmaf(v * 0.3989422804014327f, e, p);
    return v * p;
  } else if (ACT == FCONV_ACT_FASTGELU) {  // (1 + tanh z) / 2 is the logistic function of 2 z
    constexpr float k = 0.7978845608028654f, c = 0.044715f;
    const float x = within(v, kFastGeluEnd), x2 = x * x, z = x * fmaf(k * c, x2, k);
    const float p = logistic2(z * (2.0f * kLog2e));
    if (SLOPE) slope = p * fmaf(2.0f * x * (1.0f - p), fmaf(3.0f * k * c, x2, k), 1.0f);
    return v * p;
  } else {
    if (SLOPE) slope = 1.0f;
    return v;
  }
}

// The projections g and u of a training pass, f32: blocks of 32 rows by 4 columns, g's before
// u's, so that a warp with a row a lane (as accumulators come out of TMEM) moves 512 consecutive
// bytes with each 16-byte access.
__host__ __device__ __forceinline__ int64_t saved_index(int64_t row, int col, int64_t quads,
                                                        int which) {
  return (((row >> 5) * quads + (col >> 2)) * 2 + which) * 128 + (row & 31) * 4 + (col & 3);
}
inline int64_t saved_floats(int64_t rows, int64_t hidden) {
  return (rows + 31) / 32 * ((hidden + 3) / 4) * 256;
}

}  // namespace
}  // namespace ops
}  // namespace fconv
