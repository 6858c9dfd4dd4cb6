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

// act(v) in f32, and with SLOPE its derivative. The activation is the same in all threads.
template <bool SLOPE>
__device__ __forceinline__ float act_of(int act, float alpha, float v, float& slope) {
  switch (act) {
    case FCONV_ACT_RELU:  // NaN goes through
      if (SLOPE) slope = v > 0.0f ? 1.0f : 0.0f;
      return v < 0.0f ? 0.0f : v;
    case FCONV_ACT_SIGMOID: {
      const float p = 1.0f / (1.0f + expf(-v));
      if (SLOPE) slope = p * (1.0f / (1.0f + expf(v)));  // 1 - p loses its bits for large v
      return p;
    }
    case FCONV_ACT_QUICKGELU: {
      const float p = 1.0f / (1.0f + expf(-alpha * v));
      if (SLOPE) slope = p * (1.0f + alpha * v * (1.0f - p));
      return v * p;
    }
    case FCONV_ACT_GELU: {
      const float p = 0.5f * erfcf(v * -0.7071067811865476f);
      if (SLOPE) slope = p + v * 0.3989422804014327f * expf(-0.5f * v * v);
      return v * p;
    }
    case FCONV_ACT_FASTGELU: {
      constexpr float k = 0.7978845608028654f, c = 0.044715f;  // sqrt(2 / pi)
      const float th = tanhf(k * (v + c * v * v * v));
      if (SLOPE)
        slope = 0.5f * (1.0f + th) + 0.5f * v * (1.0f - th * th) * k * (1.0f + 3.0f * c * v * v);
      return 0.5f * v * (1.0f + th);
    }
    default:
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
