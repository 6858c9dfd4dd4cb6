// Operands of the gated block that TMA does not take as they are, written into rows of whole
// 16-byte units: 16-bit tensors copied, f32 ones split into three bf16 planes. Bound: HBM; one
// launch for all tensors of a call, a thread takes 8 columns of a row.
#include "ops_common.cuh"
#include "ops_internal.h"
#include "split_bf16.cuh"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kThreads = 256;

struct Prep {
  PrepArgs a;
  int64_t first[6];  // first unit of 8 columns of each tensor
};

__device__ __forceinline__ uint32_t word(uint16_t a, uint16_t b) { return a | (uint32_t)b << 16; }

template <typename T>
__global__ void __launch_bounds__(kThreads) mlp_prep(const __grid_constant__ Prep q) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  int i = 0;
  while (i < q.a.count && u >= q.first[i + 1]) ++i;
  if (i == q.a.count) return;
  u -= q.first[i];
  const PrepItem& m = q.a.m[i];
  const int64_t across = m.dst_row / 8, row = u / across, col = (u - row * across) * 8;
  const T* from = (const T*)m.src + row * m.src_row + col;
  T v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = col + e < m.cols ? from[e] : from_f<T>(0.0f);
  uint4* to = reinterpret_cast<uint4*>((uint16_t*)m.dst + row * m.dst_row + col);
  if constexpr (sizeof(T) == 2) {
    *to = *reinterpret_cast<const uint4*>(v);
  } else {
    uint16_t w[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float p[3];
      split_bf16(v[e], p);
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k][e] = __bfloat16_as_ushort(__float2bfloat16_rn(p[k]));
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      to[k * (m.plane / 8)] = make_uint4(word(w[k][0], w[k][1]), word(w[k][2], w[k][3]),
                                         word(w[k][4], w[k][5]), word(w[k][6], w[k][7]));
  }
}

}  // namespace

int launch_mlp_prep(int dtype, const PrepArgs& a, cudaStream_t s) {
  Prep q{};
  q.a = a;
  for (int i = 0; i < a.count; ++i) q.first[i + 1] = q.first[i] + a.m[i].rows * (a.m[i].dst_row / 8);
  const long long blocks = (q.first[a.count] + kThreads - 1) / kThreads;
  if (blocks == 0) return 0;
  if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
#define FCONV_M(T) return launch_pdl(mlp_prep<T>, dim3((unsigned)blocks), dim3(kThreads), 0, s, q)
  FCONV_OPS_TYPE(dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
