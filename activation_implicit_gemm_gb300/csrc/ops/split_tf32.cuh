// f32 operands of the warp-level TF32 instructions as hi + lo.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace fconv {
namespace ops {
namespace {

// hi is v rounded to TF32 and lo = v - hi (exact, read as TF32): lo hi + hi lo + hi hi drops about
// 2^-23 of a product. Values past TF32's largest get that as hi and the rest as lo.
__device__ __forceinline__ void split_tf32(float v, uint32_t& hi, uint32_t& lo) {
  constexpr float kLargest = 3.4011621342146535e38f;  // (2 - 2^-10) 2^127
  float c;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(c) : "f"(v), "f"(kLargest));
  hi = (__float_as_uint(c) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(v - __uint_as_float(hi));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4],
                                         const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

}  // namespace
}  // namespace ops
}  // namespace fconv
