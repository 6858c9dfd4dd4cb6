// Layer norm forward and backward (include/fconv_ops.h), simple form.
//
// x is (outer, channels, inner). A block takes positions of one `outer` index; the mean comes
// first and the variance from the centred values (a one-pass sum of squares would cancel).
#include "ops_common.cuh"
#include "ops_internal.h"

namespace fconv {
namespace ops {
namespace {

constexpr int kX = 32, kY = 8;

// Sum over the kY threads that share a position.
__device__ __forceinline__ float slice_sum(float v, float (*red)[kX]) {
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kY; ++i) s += red[i][threadIdx.x];
  __syncthreads();
  return s;
}

// Position and channel walk of a thread: inner > 1 puts neighbouring positions on the lanes
// and splits the channels over threadIdx.y; inner = 1 gives a row to the whole block.
struct Walk {
  bool live;
  bool row;
  int64_t base, pos;
  int c0, dc;
  int64_t step;
};
__device__ __forceinline__ Walk walk_of(int64_t C, int64_t inner) {
  Walk w;
  w.row = inner == 1;
  if (w.row) {
    w.live = true;
    w.pos = blockIdx.x;
    w.base = w.pos * C;
    w.c0 = threadIdx.y * kX + threadIdx.x;
    w.dc = kX * kY;
  } else {
    const int64_t tiles = (inner + kX - 1) / kX;
    const int64_t n = blockIdx.x / tiles, i = (blockIdx.x - n * tiles) * kX + threadIdx.x;
    w.live = i < inner;
    w.pos = n * inner + i;
    w.base = n * C * inner + i;
    w.c0 = threadIdx.y;
    w.dc = kY;
  }
  w.step = inner;
  return w;
}
__device__ __forceinline__ float walk_sum(float v, const Walk& w, float (*red)[kX]) {
  if (w.row) v = warp_sum(v);
  return slice_sum(v, red);
}

template <typename T, typename P>
__global__ void __launch_bounds__(kX* kY)
    norm_forward_simple(const T* __restrict__ x, const P* __restrict__ w, const P* __restrict__ b,
                        T* y, float* mean, float* rstd, int64_t C, int64_t inner, float eps) {
  __shared__ float red[kY][kX];
  const Walk k = walk_of(C, inner);
  float s = 0.0f;
  if (k.live)
    for (int64_t c = k.c0; c < C; c += k.dc) s += to_f(x[k.base + c * k.step]);
  const float m = walk_sum(s, k, red) / (float)C;
  s = 0.0f;
  if (k.live)
    for (int64_t c = k.c0; c < C; c += k.dc) {
      const float d = to_f(x[k.base + c * k.step]) - m;
      s += d * d;
    }
  const float r = rsqrtf(walk_sum(s, k, red) / (float)C + eps);
  if (!k.live) return;
  if (k.row ? k.c0 == 0 : threadIdx.y == 0) {
    if (mean) mean[k.pos] = m;
    if (rstd) rstd[k.pos] = r;
  }
  for (int64_t c = k.c0; c < C; c += k.dc) {
    float v = (to_f(x[k.base + c * k.step]) - m) * r;
    if (w) v *= to_f(w[c]);
    if (b) v += to_f(b[c]);
    y[k.base + c * k.step] = from_f<T>(v);
  }
}

template <typename T, typename P>
__global__ void __launch_bounds__(kX* kY)
    norm_dx_simple(const T* dy, const T* __restrict__ x, const P* __restrict__ w,
                   const float* __restrict__ mean, const float* __restrict__ rstd, T* dx,
                   int64_t C, int64_t inner) {
  __shared__ float red[kY][kX];
  const Walk k = walk_of(C, inner);
  const float m = k.live ? mean[k.pos] : 0.0f, r = k.live ? rstd[k.pos] : 0.0f;
  float s = 0.0f, t = 0.0f;
  if (k.live)
    for (int64_t c = k.c0; c < C; c += k.dc) {
      const float g = to_f(dy[k.base + c * k.step]) * (w ? to_f(w[c]) : 1.0f);
      s += g;
      t += g * ((to_f(x[k.base + c * k.step]) - m) * r);
    }
  s = walk_sum(s, k, red) / (float)C;
  t = walk_sum(t, k, red) / (float)C;
  if (!k.live) return;
  for (int64_t c = k.c0; c < C; c += k.dc) {
    const float g = to_f(dy[k.base + c * k.step]) * (w ? to_f(w[c]) : 1.0f);
    const float h = (to_f(x[k.base + c * k.step]) - m) * r;
    dx[k.base + c * k.step] = from_f<T>(r * (g - s - h * t));
  }
}

// Partial sums of dw and db over a chunk of positions: part[chunk][0] = sum(dy * xhat),
// part[chunk][1] = sum(dy), each `C` floats.
template <typename T>
__global__ void __launch_bounds__(kX* kY)
    norm_dparam_simple(const T* __restrict__ dy, const T* __restrict__ x,
                       const float* __restrict__ mean, const float* __restrict__ rstd,
                       float* part, int64_t positions, int64_t C, int64_t inner, int64_t per) {
  __shared__ float red[kY][kX];
  const int64_t p0 = (int64_t)blockIdx.y * per;
  const int64_t p1 = p0 + per < positions ? p0 + per : positions;
  const int64_t c = (int64_t)blockIdx.x * kX + threadIdx.x;
  float s = 0.0f, t = 0.0f;
  if (c < C)
    for (int64_t p = p0 + threadIdx.y; p < p1; p += kY) {
      const int64_t n = p / inner, at = (n * C + c) * inner + (p - n * inner);
      const float g = to_f(dy[at]);
      s += g;
      t += g * ((to_f(x[at]) - mean[p]) * rstd[p]);
    }
  s = slice_sum(s, red);
  t = slice_sum(t, red);
  if (c < C && threadIdx.y == 0) {
    part[(2 * blockIdx.y) * C + c] = t;
    part[(2 * blockIdx.y + 1) * C + c] = s;
  }
}

// dw and db from the partial sums, added in order.
template <typename P>
__global__ void __launch_bounds__(256)
    norm_dparam_join(const float* __restrict__ part, P* dw, P* db, int64_t C, int chunks) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  float t = 0.0f, s = 0.0f;
  for (int i = 0; i < chunks; ++i) {
    t += part[(2 * (int64_t)i) * C + c];
    s += part[(2 * (int64_t)i + 1) * C + c];
  }
  if (dw) dw[c] = from_f<P>(t);
  if (db) db[c] = from_f<P>(s);
}

long long simple_blocks(const fconv_norm_desc& d) {
  return d.inner == 1 ? (long long)d.outer : (long long)d.outer * ((d.inner + kX - 1) / kX);
}
int64_t chunk_count(const fconv_norm_desc& d, int sms) {
  const int64_t positions = d.outer * d.inner;
  int64_t n = (positions + 255) / 256;
  if (n > sms) n = sms;
  return n < 1 ? 1 : n;
}

template <typename T, typename P>
int forward_t(const fconv_norm_desc& d, const NormArgs& a, cudaStream_t s) {
  const long long blocks = simple_blocks(d);
  if (blocks == 0) return 0;
  if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
  norm_forward_simple<T, P><<<(unsigned)blocks, dim3(kX, kY), 0, s>>>(
      (const T*)a.x, (const P*)a.w, (const P*)a.b, (T*)a.y, a.mean, a.rstd, d.channels, d.inner,
      d.eps);
  return (int)cudaGetLastError();
}

template <typename T, typename P>
int backward_t(const fconv_norm_desc& d, int sms, const NormArgs& a, cudaStream_t s) {
  const int64_t positions = d.outer * d.inner, C = d.channels;
  if (a.dw || a.db) {
    const int64_t chunks = chunk_count(d, sms);
    const int64_t per = (positions + chunks - 1) / chunks;
    norm_dparam_simple<T><<<dim3((unsigned)((C + kX - 1) / kX), (unsigned)chunks), dim3(kX, kY), 0,
                            s>>>((const T*)a.dy, (const T*)a.x, a.mean, a.rstd, a.ws, positions, C,
                                 d.inner, per);
    norm_dparam_join<P><<<(unsigned)((C + 255) / 256), 256, 0, s>>>(a.ws, (P*)a.dw, (P*)a.db, C,
                                                                    (int)chunks);
  }
  const long long blocks = simple_blocks(d);
  if (blocks > 0) {
    if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
    norm_dx_simple<T, P><<<(unsigned)blocks, dim3(kX, kY), 0, s>>>(
        (const T*)a.dy, (const T*)a.x, (const P*)a.w, a.mean, a.rstd, (T*)a.y, C, d.inner);
  }
  return (int)cudaGetLastError();
}

}  // namespace

size_t norm_workspace(const fconv_norm_desc& d, int sms) {
  return (size_t)chunk_count(d, sms) * 2 * (size_t)d.channels * sizeof(float);
}

int launch_norm_forward(const fconv_norm_desc& d, int sms, const NormArgs& a, cudaStream_t s) {
  (void)sms;
#define FCONV_M(T) \
  return d.param_dtype == FCONV_F32 ? forward_t<T, float>(d, a, s) : forward_t<T, T>(d, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

int launch_norm_backward(const fconv_norm_desc& d, int sms, const NormArgs& a, cudaStream_t s) {
#define FCONV_M(T)                                                          \
  return d.param_dtype == FCONV_F32 ? backward_t<T, float>(d, sms, a, s)    \
                                    : backward_t<T, T>(d, sms, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
