// What the attention kernels outside the tcgen05 route share: geometry, lengths, tiles in shared
// memory, delta.
#pragma once

#include <cmath>

#include "../fconv_internal.h"
#include "../ptx.cuh"
#include "ops_common.cuh"
#include "ops_internal.h"

namespace fconv {
namespace ops {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Geom {
  int64_t B, Lq, Lk;
  int Hq, Hk, G, D, Dp;  // Dp: D rounded up to a whole number of 8
  int64_t q[3], k[3], v[3], o[3], g[3], dq[3], dk[3], dv[3];
  float scale;
  int causal;
  const int32_t* q_lens;
  const int32_t* kv_lens;
};

struct Lens {
  int64_t q, k, shift;  // causal: query i sees keys j <= i + shift
};
__device__ __forceinline__ Lens lens_of(const Geom& g, int64_t b) {
  Lens l;
  l.q = g.q_lens ? __ldcg(g.q_lens + b) : g.Lq;
  l.k = g.kv_lens ? __ldcg(g.kv_lens + b) : g.Lk;
  l.q = l.q < 0 ? 0 : l.q > g.Lq ? g.Lq : l.q;
  l.k = l.k < 0 ? 0 : l.k > g.Lk ? g.Lk : l.k;
  l.shift = l.k - l.q;
  return l;
}

// BT rows of (row0..) of one head on their way into shared memory, as f32 with rows of Dp + 4;
// rows outside [lo, hi) become zeros, so what the tensors hold there never enters a product.
// Each of the block's WARPS warps takes every WARPS-th row. f32 rows of whole 16-byte units are
// copied asynchronously (VEC; complete after cp_async_wait and a barrier), others go through
// registers. Both read L2: attn_mma_dq loads its tiles before it waits for the launch before it,
// and nothing orders its SM's L1 after what wrote them.
template <typename T, int BT, int WARPS, bool VEC>
__device__ __forceinline__ void load_tile(float* dst, const T* src, int64_t row_stride,
                                          int64_t row0, int64_t lo, int64_t hi, const Geom& g) {
  const int pitch = g.Dp + 4, lane = threadIdx.x & 31;
#pragma unroll 8
  for (int n = 0; n < BT / WARPS; ++n) {
    const int r = n * WARPS + (threadIdx.x >> 5);
    const int64_t row = row0 + r;
    const bool ok = row >= lo && row < hi;
    const T* p = src + (ok ? row * row_stride : 0);
    if (VEC) {
      for (int d = lane * 4; d < g.Dp; d += 128)
        ptx::cp_async16_l2(ptx::smem_addr(dst + r * pitch + d), p + d, ok && d < g.D ? 16 : 0);
    } else {
      for (int d = lane; d < g.Dp; d += 32)
        dst[r * pitch + d] = ok && d < g.D ? to_f(__ldcg(p + d)) : 0.0f;
    }
  }
  ptx::cp_async_commit();
}

// delta = sum_d dout out, one warp per (b, h, i); rows past the length get 0.
template <typename T>
__global__ void __launch_bounds__(256)
    attn_delta(const T* __restrict__ o, const T* __restrict__ dout, float* delta,
               const Geom g) {
  ptx::pdl_wait();
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= g.B * g.Hq * g.Lq) return;
  const int64_t i = row % g.Lq, bh = row / g.Lq;
  const int h = (int)(bh % g.Hq);
  const int64_t b = bh / g.Hq;
  float s = 0.0f;
  if (i < lens_of(g, b).q)
    for (int d = threadIdx.x & 31; d < g.D; d += 32)
      s = fmaf(to_f(o[b * g.o[0] + i * g.o[1] + h * g.o[2] + d]),
               to_f(dout[b * g.g[0] + i * g.g[1] + h * g.g[2] + d]), s);
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) delta[row] = s;
}

inline Geom geom_of(const fconv_attn_desc& d, const AttnArgs& a) {
  Geom g{};
  g.B = d.batch;
  g.Lq = d.len_q;
  g.Lk = d.len_k;
  g.Hq = (int)d.heads_q;
  g.Hk = (int)d.heads_kv;
  g.G = g.Hq / g.Hk;
  g.D = (int)d.head_dim;
  g.Dp = (g.D + 7) / 8 * 8;
  for (int i = 0; i < 3; ++i) {
    g.q[i] = d.q_stride[i];
    g.k[i] = d.k_stride[i];
    g.v[i] = d.v_stride[i];
    g.o[i] = d.out_stride[i];
    g.g[i] = d.dout_stride[i];
    g.dq[i] = d.dq_stride[i];
    g.dk[i] = d.dk_stride[i];
    g.dv[i] = d.dv_stride[i];
  }
  g.scale = d.scale;
  g.causal = d.causal;
  g.q_lens = a.q_lens;
  g.kv_lens = a.kv_lens;
  return g;
}

// Whether every row starts and ends on a 16-byte unit.
inline bool whole_rows(const fconv_attn_desc& d, const AttnArgs& a) {
  int64_t units = d.head_dim;
  auto add = [&](const int64_t st[3], int64_t len, int64_t heads) {
    const int64_t ext[3] = {d.batch, len, heads};
    for (int i = 0; i < 3; ++i)
      if (ext[i] > 1) units |= st[i];
  };
  add(d.q_stride, d.len_q, d.heads_q);
  add(d.k_stride, d.len_k, d.heads_kv);
  add(d.v_stride, d.len_k, d.heads_kv);
  if (a.dout) add(d.dout_stride, d.len_q, d.heads_q);
  const uintptr_t addr = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.dout;
  return units % 4 == 0 && addr % 16 == 0;
}

}  // namespace
}  // namespace ops
}  // namespace fconv
