// f32 as the sum of three bf16 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace fconv {
namespace ops {
namespace {

// v = p[0] + p[1] + p[2], each what is left rounded to bf16: exact for values over 2^-110. Values
// that would round past bf16's largest keep that as p[0]; an infinity gives NaN as p[1].
__device__ __forceinline__ void split_bf16(float v, float (&p)[3]) {
  constexpr float kLargest = 3.3895313892515355e38f;  // (2 - 2^-7) 2^127
  float c;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(c) : "f"(v), "f"(kLargest));
  if (v != v) c = v;
  p[0] = __bfloat162float(__float2bfloat16_rn(c));
  const float rest = v - p[0];
  p[1] = __bfloat162float(__float2bfloat16_rn(rest));
  p[2] = __bfloat162float(__float2bfloat16_rn(rest - p[1]));
}

}  // namespace
}  // namespace ops
}  // namespace fconv
