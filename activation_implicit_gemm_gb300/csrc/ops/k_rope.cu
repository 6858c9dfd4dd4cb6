// Rotary positions with one to three axes (include/fconv_ops.h), simple form: one thread per
// (token, pair) turns that pair in every head.
//
// The angle is position * inv_freq. Its f32 product p alone is off by up to p * 2^-24 radians,
// 0.004 at 65536; the exact remainder of the product (one FMA) is kept and added after p has
// been reduced by whole turns with 2 pi in two parts (Cody and Waite, "Software Manual for the
// Elementary Functions", 1980), so sine and cosine see an angle within about pi that is right
// to 2^-22 or so at every position up to 2^23.
#include "ops_common.cuh"
#include "ops_internal.h"

namespace fconv {
namespace ops {
namespace {

// p - k * kHi is exact: kHi is a multiple of 2^-21, so both terms are multiples of
// min(2^-21, ulp(p)) and the difference, at most 4, fits 24 bits. What kHi + kMid lack of
// 2 pi (1e-14) stays below 2e-8 for every k up to 2^21.
__device__ __forceinline__ void turn_of(float pos, float freq, float& sn, float& cs) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  constexpr float kHi = (float)kTwoPi;
  constexpr float kMid = (float)(kTwoPi - (double)kHi);
  constexpr float kInv = (float)(1.0 / kTwoPi);
  const float p = pos * freq;
  const float e = fmaf(pos, freq, -p);  // p + e is the exact product
  const float k = rintf(p * kInv);
  const float r = fmaf(-k, kHi, p);     // exact: |r| is small against p
  sincosf(fmaf(-k, kMid, r) + e, &sn, &cs);
}

__device__ __forceinline__ float position(const void* pos, int type, int64_t at) {
  if (type == FCONV_POS_I32) return (float)((const int32_t*)pos)[at];
  if (type == FCONV_POS_I64) return (float)((const int64_t*)pos)[at];
  return ((const float*)pos)[at];
}

struct RopeGeom {
  int64_t len, pos_batch, tokens;
  int heads_q, heads_k, head_dim, pairs, axes, sec0, sec1, pairing, pos_type, inverse;
  int64_t q_stride[3], k_stride[3], q_out_stride[3], k_out_stride[3];
};

template <typename T>
__device__ __forceinline__ void turn_head(const T* x, T* y, int lo, int hi, float cs, float sn) {
  const float u = to_f(x[lo]), v = to_f(x[hi]);
  y[lo] = from_f<T>(u * cs - v * sn);
  y[hi] = from_f<T>(v * cs + u * sn);
}

// Elements [0, pairs) of the walk are pairs; [pairs, head_dim - pairs) copy element
// pairs + index (the tail past the last pair).
template <typename T>
__global__ void __launch_bounds__(256)
    rope_simple(const T* q, const T* k, const void* pos, const float* __restrict__ inv_freq, T* qo,
                T* ko, const RopeGeom g) {
  const int work = g.head_dim - g.pairs;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t token = at / work;
  const int p = (int)(at - token * work);
  if (token >= g.tokens) return;
  const int64_t b = token / g.len, t = token - b * g.len;
  const T* qp = q + b * g.q_stride[0] + t * g.q_stride[1];
  T* qw = qo + b * g.q_out_stride[0] + t * g.q_out_stride[1];
  const T* kp = k + b * g.k_stride[0] + t * g.k_stride[1];
  T* kw = ko + b * g.k_out_stride[0] + t * g.k_out_stride[1];
  if (p >= g.pairs) {
    const int d = g.pairs + p;
    for (int h = 0; h < g.heads_q; ++h) qw[h * g.q_out_stride[2] + d] = qp[h * g.q_stride[2] + d];
    for (int h = 0; h < g.heads_k; ++h) kw[h * g.k_out_stride[2] + d] = kp[h * g.k_stride[2] + d];
    return;
  }
  const int axis = p < g.sec0 ? 0 : p < g.sec0 + g.sec1 ? 1 : 2;
  const int64_t pb = g.pos_batch == 1 ? 0 : b;
  float sn, cs;
  turn_of(position(pos, g.pos_type, (pb * g.len + t) * g.axes + axis), inv_freq[p], sn, cs);
  if (g.inverse) sn = -sn;
  int lo, hi;
  if (g.pairing == FCONV_ROPE_INTERLEAVED) {
    lo = 2 * p;
    hi = lo + 1;
  } else if (g.pairing == FCONV_ROPE_HALF) {
    lo = p;
    hi = p + g.pairs;
  } else {
    const int start = axis == 0 ? 0 : axis == 1 ? g.sec0 : g.sec0 + g.sec1;
    const int size = axis == 0 ? g.sec0 : axis == 1 ? g.sec1 : g.pairs - g.sec0 - g.sec1;
    lo = start + p;
    hi = lo + size;
  }
  for (int h = 0; h < g.heads_q; ++h)
    turn_head(qp + h * g.q_stride[2], qw + h * g.q_out_stride[2], lo, hi, cs, sn);
  for (int h = 0; h < g.heads_k; ++h)
    turn_head(kp + h * g.k_stride[2], kw + h * g.k_out_stride[2], lo, hi, cs, sn);
}

}  // namespace

int launch_rope(const fconv_rope_desc& d, int sms, const RopeArgs& a, cudaStream_t s) {
  (void)sms;
  RopeGeom g{};
  g.len = d.len;
  g.pos_batch = d.pos_batch;
  g.tokens = d.batch * d.len;
  g.heads_q = (int)d.heads_q;
  g.heads_k = (int)d.heads_k;
  g.head_dim = (int)d.head_dim;
  g.axes = d.axes;
  for (int i = 0; i < d.axes; ++i) g.pairs += (int)d.section[i];
  g.sec0 = (int)d.section[0];
  g.sec1 = d.axes > 1 ? (int)d.section[1] : 0;
  g.pairing = d.pairing;
  g.pos_type = d.pos_type;
  g.inverse = d.inverse;
  for (int i = 0; i < 3; ++i) {
    g.q_stride[i] = d.q_stride[i];
    g.k_stride[i] = d.k_stride[i];
    g.q_out_stride[i] = d.q_out_stride[i];
    g.k_out_stride[i] = d.k_out_stride[i];
  }
  const long long blocks = (long long)((g.tokens * (g.head_dim - g.pairs) + 255) / 256);
  if (blocks == 0) return 0;
  if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
#define FCONV_M(T)                                                                          \
  rope_simple<T><<<(unsigned)blocks, 256, 0, s>>>((const T*)a.q, (const T*)a.k, a.pos,      \
                                                  a.inv_freq, (T*)a.q_out, (T*)a.k_out, g)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
  return (int)cudaGetLastError();
}

}  // namespace ops
}  // namespace fconv
