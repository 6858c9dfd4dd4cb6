// RMS norm of every head of q and k with the position rotation in the same pass, forward and
// backward (include/fconv_ops.h).
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  z = n w,  y = turned z
//   g = dy turned back,  dw = sum g n,  a = g w,  dx = r a - x r^3 mean(a x)
// Bound: HBM; forward x in and y out, backward x and dy in and dx out, each element once.
//
// G lanes (a power of two, so that sums over a head are shuffles) own a token: each lane has the
// same VEC pairs of every head (two accesses of VEC elements, or one of 2 VEC where neighbours
// pair up), makes their sines and cosines once and goes through its share of the heads with the
// next one's values on their way. A block row (blockIdx.y) takes heads of q or of k only, so a
// thread keeps one weight in registers. In the backward pass blocks stay for many tokens and keep
// their part of dw in registers; the parts are joined in a fixed order by a second kernel.
#include "ops_common.cuh"
#include "ops_internal.h"
#include "rope_angle.cuh"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kThreads = 256;

struct Side {  // q or k
  const void* x;
  const void* dy;
  void* out;  // y, or dx
  const void* w;
  void* dw;
  int heads, per, groups;  // heads of a block row, block rows
  int64_t xs[3], ys[3], os[3];  // strides of x, dy and out
};
struct HeadGeom {
  Side side[2];
  const void* pos;
  const float* inv_freq;
  float* part;  // dw of every block, or null
  int64_t len, pos_batch, tokens;
  int D, pairs, pair_chunks, chunks, lanes, axes, sec0, sec1, pairing, pos_type, f32_params;
  float eps;
};

// Where a lane's chunk lies in a head and how its pairs turn.
template <int VEC>
struct Chunk {
  int lo, hi;       // first elements of its two accesses, hi < 0: no second one
  bool turns;
  float cs[VEC], sn[VEC];
};

template <int VEC, bool IL>
__device__ __forceinline__ void place(Chunk<VEC>& c, const HeadGeom& g, int chunk) {
  const int p0 = chunk * VEC;
  c.turns = chunk < g.pair_chunks;
  if (!c.turns) {
    c.lo = 2 * g.pairs + (chunk - g.pair_chunks) * 2 * VEC;
    c.hi = c.lo + VEC < g.D ? c.lo + VEC : -1;
  } else if (IL || g.pairing == FCONV_ROPE_INTERLEAVED) {
    c.lo = 2 * p0;
    c.hi = c.lo + VEC;  // without IL VEC is 1
  } else if (g.pairing == FCONV_ROPE_HALF) {
    c.lo = p0;
    c.hi = p0 + g.pairs;
  } else {
    const int s1 = g.sec0 + g.sec1;
    const int start = p0 < g.sec0 ? 0 : p0 < s1 ? g.sec0 : s1;
    c.lo = start + p0;
    c.hi = c.lo + (p0 < g.sec0 ? g.sec0 : p0 < s1 ? g.sec1 : g.pairs - s1);
  }
}

template <int VEC>
__device__ __forceinline__ void angles(Chunk<VEC>& c, const HeadGeom& g, int chunk, int64_t b,
                                       int64_t t) {
  const int p0 = chunk * VEC;
  const int64_t at = ((g.pos_batch == 1 ? 0 : b) * g.len + t) * g.axes;
  float pos[3];
#pragma unroll
  for (int a = 0; a < 3; ++a) pos[a] = a < g.axes ? position(g.pos, g.pos_type, at + a) : 0.0f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int p = p0 + i;
    const float x = p < g.sec0 ? pos[0] : p < g.sec0 + g.sec1 ? pos[1] : pos[2];
    if (fabsf(x) <= kLongPosition) {
      turn_of(x, g.inv_freq[p], c.sn[i], c.cs[i]);
    } else {
      const int a = p < g.sec0 ? 0 : p < g.sec0 + g.sec1 ? 1 : 2;
      const float2 v = turn_of_long(long_position(g.pos, g.pos_type, at + a), g.inv_freq[p]);
      c.sn[i] = v.x;
      c.cs[i] = v.y;
    }
  }
}

// A chunk's 2 VEC elements of one head as they lie in memory. Element e of them is member e / VEC
// of pair e % VEC, or with IL member e % 2 of pair e / 2.
template <typename T, int VEC, bool IL>
struct Raw {
  Vec<T, IL ? 2 * VEC : VEC> a, b;
  __device__ __forceinline__ void load(const T* p, const Chunk<VEC>& c) {
    a = *reinterpret_cast<const decltype(a)*>(p + c.lo);
    if (!IL && c.hi >= 0) b = *reinterpret_cast<const decltype(b)*>(p + c.hi);
  }
  __device__ __forceinline__ void store(T* p, const Chunk<VEC>& c) const {
    *reinterpret_cast<decltype(a)*>(p + c.lo) = a;
    if (!IL && c.hi >= 0) *reinterpret_cast<decltype(b)*>(p + c.hi) = b;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (IL ? 2 * VEC : VEC); ++i) a.v[i] = b.v[i] = from_f<T>(0.0f);
  }
  __device__ __forceinline__ T& at(int e) { return IL || e < VEC ? a.v[e] : b.v[e - VEC]; }
};
// Positions of a pair's members among the 2 VEC elements.
template <int VEC, bool IL>
__device__ __forceinline__ constexpr int first(int i) { return IL ? 2 * i : i; }
template <int VEC, bool IL>
__device__ __forceinline__ constexpr int second(int i) { return IL ? 2 * i + 1 : VEC + i; }

template <int VEC, bool IL>
__device__ __forceinline__ int element(const Chunk<VEC>& c, int e) {  // -1: there is none
  if (IL || e < VEC) return c.lo + e;
  return c.hi < 0 ? -1 : c.hi + e - VEC;
}

template <int VEC, bool IL>
__device__ __forceinline__ void load_weight(float (&w)[2 * VEC], const HeadGeom& g, const Side& s,
                                            const Chunk<VEC>& c, int dtype_f32, bool f16) {
#pragma unroll
  for (int e = 0; e < 2 * VEC; ++e) {
    const int at = element<VEC, IL>(c, e);
    w[e] = 1.0f;
    if (s.w && at >= 0)
      w[e] = dtype_f32 ? ((const float*)s.w)[at]
             : f16     ? to_f(((const __half*)s.w)[at])
                       : to_f(((const __nv_bfloat16*)s.w)[at]);
  }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
constexpr bool kIsHalf = false;
template <>
constexpr bool kIsHalf<__half> = true;

// R: chunks of a lane (more than one only where a head has more than 32).
template <typename T, int VEC, int R, bool IL>
__global__ void __launch_bounds__(kThreads, VEC * R > 8 ? 1 : 3)
    norm_rope_forward(const __grid_constant__ HeadGeom g) {
  using Row = Raw<T, VEC, IL>;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const bool is_k = (int)blockIdx.y >= g.side[0].groups;
  const Side& s = g.side[is_k];
  const int h0 = ((int)blockIdx.y - (is_k ? g.side[0].groups : 0)) * s.per;
  const int h1 = min(h0 + s.per, s.heads);
  const int lane = threadIdx.x & (g.lanes - 1);
  int64_t token = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / g.lanes;
  const bool here = token < g.tokens;  // all lanes take part in the sums
  if (!here) token = 0;
  const int64_t b = token / g.len, t = token - b * g.len;
  const T* xp = (const T*)s.x + b * s.xs[0] + t * s.xs[1];
  T* yp = (T*)s.out + b * s.os[0] + t * s.os[1];
  Chunk<VEC> c[R];
  bool on[R];
  Row row[R];
  float w[R][2 * VEC];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    on[r] = here && lane + r * g.lanes < g.chunks;
    row[r].zero();
    if (on[r]) {
      place<VEC, IL>(c[r], g, lane + r * g.lanes);
      row[r].load(xp + h0 * s.xs[2], c[r]);
      if (c[r].turns) angles<VEC>(c[r], g, lane + r * g.lanes, b, t);
      load_weight<VEC, IL>(w[r], g, s, c[r], g.f32_params, kIsHalf<T>);
    }
  }
  for (int h = h0; h < h1; ++h) {
    float x[R][2 * VEC], sum = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < 2 * VEC; ++e) {
        x[r][e] = to_f(row[r].at(e));
        sum = fmaf(x[r][e], x[r][e], sum);
      }
      if (on[r] && h + 1 < h1) row[r].load(xp + (h + 1) * s.xs[2], c[r]);
    }
    sum = lanes_sum(sum, g.lanes);
    const float scale = rsqrtf(sum / (float)g.D + g.eps);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!on[r]) continue;
      Row y;
      if (c[r].turns) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          constexpr auto F = first<VEC, IL>;
          constexpr auto S = second<VEC, IL>;
          const float u = x[r][F(i)] * scale * w[r][F(i)], v = x[r][S(i)] * scale * w[r][S(i)];
          y.at(F(i)) = from_f<T>(u * c[r].cs[i] - v * c[r].sn[i]);
          y.at(S(i)) = from_f<T>(v * c[r].cs[i] + u * c[r].sn[i]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) y.at(e) = from_f<T>(x[r][e] * scale * w[r][e]);
      }
      y.store(yp + h * s.os[2], c[r]);
    }
  }
}

template <typename T, int VEC, int R, bool IL>
__global__ void __launch_bounds__(kThreads, VEC * R > 8 ? 1 : 2)
    norm_rope_backward(const __grid_constant__ HeadGeom g) {
  using Row = Raw<T, VEC, IL>;
  extern __shared__ float sums[];  // a row of D for each warp
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const bool is_k = (int)blockIdx.y >= g.side[0].groups;
  const Side& s = g.side[is_k];
  const int h0 = ((int)blockIdx.y - (is_k ? g.side[0].groups : 0)) * s.per;
  const int h1 = min(h0 + s.per, s.heads);
  const int lane = threadIdx.x & (g.lanes - 1);
  const int64_t each = kThreads / g.lanes;  // tokens of a block at a time
  Chunk<VEC> c[R];
  float w[R][2 * VEC], dw[R][2 * VEC];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) dw[r][e] = 0.0f;
    if (lane + r * g.lanes < g.chunks) {
      place<VEC, IL>(c[r], g, lane + r * g.lanes);
      load_weight<VEC, IL>(w[r], g, s, c[r], g.f32_params, kIsHalf<T>);
    }
  }
  for (int64_t t0 = blockIdx.x * each; t0 < g.tokens; t0 += gridDim.x * each) {
    int64_t token = t0 + threadIdx.x / g.lanes;
    const bool here = token < g.tokens;
    if (!here) token = 0;
    const int64_t b = token / g.len, t = token - b * g.len;
    const T* xp = (const T*)s.x + b * s.xs[0] + t * s.xs[1];
    const T* yp = (const T*)s.dy + b * s.ys[0] + t * s.ys[1];
    T* op = (T*)s.out + b * s.os[0] + t * s.os[1];
    bool on[R];
    Row rx[R], ry[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      on[r] = here && lane + r * g.lanes < g.chunks;
      rx[r].zero();
      ry[r].zero();
      if (on[r]) {
        rx[r].load(xp + h0 * s.xs[2], c[r]);
        ry[r].load(yp + h0 * s.ys[2], c[r]);
        if (c[r].turns) angles<VEC>(c[r], g, lane + r * g.lanes, b, t);
      }
    }
    for (int h = h0; h < h1; ++h) {
      float x[R][2 * VEC], a[R][2 * VEC], sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) {
          x[r][e] = to_f(rx[r].at(e));
          a[r][e] = to_f(ry[r].at(e));
          sum = fmaf(x[r][e], x[r][e], sum);
        }
        if (!on[r]) continue;
        if (h + 1 < h1) {
          rx[r].load(xp + (h + 1) * s.xs[2], c[r]);
          ry[r].load(yp + (h + 1) * s.ys[2], c[r]);
        }
        if (c[r].turns) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            constexpr auto F = first<VEC, IL>;
            constexpr auto S = second<VEC, IL>;
            const float u = a[r][F(i)], v = a[r][S(i)];
            a[r][F(i)] = u * c[r].cs[i] + v * c[r].sn[i];
            a[r][S(i)] = v * c[r].cs[i] - u * c[r].sn[i];
          }
        }
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) dot = fmaf(a[r][e] * w[r][e], x[r][e], dot);
      }
      sum = lanes_sum(sum, g.lanes);
      dot = lanes_sum(dot, g.lanes);
      const float scale = rsqrtf(sum / (float)g.D + g.eps);
      const float along = dot / (float)g.D * scale * scale;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!on[r]) continue;
        Row o;
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) {
          dw[r][e] = fmaf(a[r][e], x[r][e] * scale, dw[r][e]);
          o.at(e) = from_f<T>(scale * (a[r][e] * w[r][e] - x[r][e] * along));
        }
        o.store(op + h * s.os[2], c[r]);
      }
    }
  }
  if (!g.part || !s.dw) return;
  // the block's part of dw: over the tokens of a warp by shuffles, over the warps in order
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e)
      for (int o = g.lanes; o < 32; o <<= 1)
        dw[r][e] += __shfl_xor_sync(0xffffffffu, dw[r][e], o);
    if ((threadIdx.x & 31) < g.lanes && lane + r * g.lanes < g.chunks) {
#pragma unroll
      for (int e = 0; e < 2 * VEC; ++e) {
        const int at = element<VEC, IL>(c[r], e);
        if (at >= 0) sums[(threadIdx.x >> 5) * g.D + at] = dw[r][e];
      }
    }
  }
  __syncthreads();
  float* part = g.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * g.D;
  for (int e = threadIdx.x; e < g.D; e += kThreads) {
    float v = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) v += sums[i * g.D + e];
    part[e] = v;
  }
}

// dw of q (blockIdx.y 0) or k: the parts of their blocks, 32 columns a block, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024)
    norm_rope_join(const __grid_constant__ HeadGeom g, int grid_x) {
  __shared__ float sums[32][33];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const Side& s = g.side[blockIdx.y];
  if (!s.dw) return;
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  const int64_t begin = blockIdx.y ? (int64_t)g.side[0].groups * grid_x : 0;
  const int64_t n = (int64_t)s.groups * grid_x;
  float v = 0.0f;
  if (col < g.D)
    for (int64_t i = row; i < n; i += 32) v += __ldcg(g.part + (begin + i) * g.D + col);
  sums[row][threadIdx.x & 31] = v;
  __syncthreads();
  if (row == 0 && col < g.D) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][threadIdx.x & 31];
    if (g.f32_params) ((float*)s.dw)[col] = v;
    else ((T*)s.dw)[col] = from_f<T>(v);
  }
}

// Elements of an access, as in the rotary kernel: as many as every pair's members allow, where
// the strides and addresses of all tensors of the call do too.
int width(const fconv_norm_rope_desc& d, const NormRopeArgs& a, int pairs, bool backward) {
  const int size = d.dtype == FCONV_F32 ? 4 : 2;
  int64_t units = d.head_dim - 2 * pairs;
  units |= d.pairing == FCONV_ROPE_INTERLEAVED ? 2 * pairs : pairs;
  if (d.pairing == FCONV_ROPE_HALF_PER_AXIS)
    for (int i = 0; i < d.axes; ++i) units |= d.section[i];
  const int64_t ext[3] = {d.batch, d.len, 0};
  for (int i = 0; i < 3; ++i) {
    if ((i < 2 ? ext[i] : d.heads_q) > 1)
      units |= d.q_stride[i] | d.q_out_stride[i] | (backward ? d.dq_stride[i] : 0);
    if (d.heads_k && (i < 2 ? ext[i] : d.heads_k) > 1)
      units |= d.k_stride[i] | d.k_out_stride[i] | (backward ? d.dk_stride[i] : 0);
  }
  const uintptr_t addr = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.q_out |
                         (uintptr_t)a.k_out | (uintptr_t)a.dq | (uintptr_t)a.dk;
  int n = 16 / size;
  while (n > 1 && (units % n != 0 || addr % (n * size) != 0)) n /= 2;
  return n;
}

struct Shape {
  dim3 grid;
  int vec, r;
  bool il;
};

// The variants: accesses of 16 bytes, of 8 (16-bit rows that allow no more), and of one element.
template <typename T, typename Run>
int by_shape(const Shape& v, Run run) {
  constexpr int kFull = 16 / sizeof(T);
  if (v.il) {
    if (v.r == 1) return run.template operator()<T, kFull / 2, 1, true>();
    return run.template operator()<T, kFull / 2, sizeof(T) == 4 ? 4 : 2, true>();
  }
  if (v.vec == kFull && v.r == 1) return run.template operator()<T, kFull, 1, false>();
  if (v.vec == 4) return run.template operator()<T, 4, 2, false>();
  return run.template operator()<T, 1, 8, false>();
}

struct RunForward {
  const HeadGeom& g;
  const Shape& v;
  cudaStream_t s;
  template <typename T, int VEC, int R, bool IL>
  int operator()() const {
    return launch_pdl(norm_rope_forward<T, VEC, R, IL>, v.grid, dim3(kThreads), 0, s, g);
  }
};
struct RunBackward {
  const HeadGeom& g;
  const Shape& v;
  cudaStream_t s;
  template <typename T, int VEC, int R, bool IL>
  int operator()() const {
    return launch_pdl(norm_rope_backward<T, VEC, R, IL>, v.grid, dim3(kThreads),
                      (size_t)(kThreads / 32) * g.D * sizeof(float), s, g);
  }
};

// Heads of a block row, at most `most` and as even as they go.
void share(Side& s, int most) {
  s.groups = s.heads ? (s.heads + most - 1) / most : 0;
  s.per = s.heads ? (s.heads + s.groups - 1) / s.groups : 0;
  s.groups = s.heads ? (s.heads + s.per - 1) / s.per : 0;
}

constexpr int kMostHeads = 8;  // of a block row in the backward pass
int backward_rows(const fconv_norm_rope_desc& d) {
  return (int)(d.heads_q + d.heads_k);  // at most
}
int backward_blocks(int sms) { return 4 * sms; }

HeadGeom geometry(const fconv_norm_rope_desc& d, const NormRopeArgs& a, bool backward, Shape& v) {
  HeadGeom g{};
  const void* x[2] = {a.q, a.k};
  const void* w[2] = {a.w, a.kw};
  const void* y[2] = {a.q_out, a.k_out};
  void* dx[2] = {a.dq, a.dk};
  void* dw[2] = {a.dw, a.dkw};
  for (int k = 0; k < 2; ++k) {
    Side& s = g.side[k];
    s.x = x[k];
    s.w = w[k];
    s.dy = backward ? y[k] : nullptr;
    s.out = backward ? dx[k] : const_cast<void*>(y[k]);
    s.dw = dw[k];
    s.heads = (int)(k ? d.heads_k : d.heads_q);
    for (int i = 0; i < 3; ++i) {
      s.xs[i] = k ? d.k_stride[i] : d.q_stride[i];
      s.ys[i] = k ? d.k_out_stride[i] : d.q_out_stride[i];
      s.os[i] = !backward ? s.ys[i] : k ? d.dk_stride[i] : d.dq_stride[i];
    }
  }
  g.pos = a.pos;
  g.inv_freq = a.inv_freq;
  g.part = a.ws;
  g.len = d.len;
  g.pos_batch = d.pos_batch;
  g.tokens = d.batch * d.len;
  g.D = (int)d.head_dim;
  g.axes = d.axes;
  for (int i = 0; i < d.axes; ++i) g.pairs += (int)d.section[i];
  g.sec0 = d.axes > 0 ? (int)d.section[0] : 0;
  g.sec1 = d.axes > 1 ? (int)d.section[1] : 0;
  g.pairing = d.pairing;
  g.pos_type = d.pos_type;
  g.f32_params = d.param_dtype == FCONV_F32;
  g.eps = d.eps;
  const int n = width(d, a, g.pairs, backward), full = d.dtype == FCONV_F32 ? 4 : 8;
  v.il = d.pairing == FCONV_ROPE_INTERLEAVED && g.pairs > 0 && n == full;
  v.vec = v.il ? full / 2 : d.pairing == FCONV_ROPE_INTERLEAVED && g.pairs > 0 ? 1 : n;
  if (v.vec != full && v.vec != 4 && !v.il) v.vec = 1;
  auto count = [&](int vec) {
    g.pair_chunks = g.pairs / vec;
    g.chunks = g.pair_chunks + (g.D - 2 * g.pairs + 2 * vec - 1) / (2 * vec);
  };
  count(v.vec);
  g.lanes = 1;
  while (g.lanes < g.chunks && g.lanes < 32) g.lanes *= 2;
  v.r = (g.chunks + g.lanes - 1) / g.lanes;
  return g;
}

}  // namespace

size_t norm_rope_workspace(const fconv_norm_rope_desc& d, int sms) {
  return (size_t)(backward_blocks(sms) + backward_rows(d)) * (size_t)d.head_dim * sizeof(float);
}

int launch_norm_rope_forward(const fconv_norm_rope_desc& d, int sms, const NormRopeArgs& a,
                             cudaStream_t s) {
  Shape v;
  HeadGeom g = geometry(d, a, false, v);
  const long long blocks = (g.tokens * g.lanes + kThreads - 1) / kThreads;
  if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
  // few tokens: the heads are shared out too, until there are about four blocks an SM
  const int heads = g.side[0].heads + g.side[1].heads;
  const long long want = (4LL * sms + blocks - 1) / blocks;
  const int shares = (int)(want < heads ? want : heads);
  const int per = (heads + shares - 1) / shares;
  share(g.side[0], per);
  share(g.side[1], per);
  v.grid = dim3((unsigned)blocks, (unsigned)(g.side[0].groups + g.side[1].groups));
  const RunForward run{g, v, s};
#define FCONV_M(T) return by_shape<T>(v, run)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

int launch_norm_rope_backward(const fconv_norm_rope_desc& d, int sms, const NormRopeArgs& a,
                              cudaStream_t s) {
  Shape v;
  HeadGeom g = geometry(d, a, true, v);
  const int each = kThreads / g.lanes;
  const long long all = (g.tokens + each - 1) / each;  // blocks with one round of tokens
  const int most = backward_blocks(sms);
  int per = kMostHeads;  // fewer where the tokens alone do not fill the GPU
  for (;;) {
    share(g.side[0], per);
    share(g.side[1], per);
    if (per == 1 || all * (g.side[0].groups + g.side[1].groups) >= most) break;
    per /= 2;
  }
  const int rows = g.side[0].groups + g.side[1].groups;
  long long bx = most / rows;  // at most what the workspace holds
  if (bx < 1) bx = 1;
  if (bx > all) bx = all;
  int e = 0;
  if (bx > 0) {
    v.grid = dim3((unsigned)bx, (unsigned)rows);
    const RunBackward run{g, v, s};
#define FCONV_M(T) e = by_shape<T>(v, run)
    FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
  }
  if (e || (!a.dw && !a.dkw)) return e;
  const dim3 grid((unsigned)((g.D + 31) / 32), 2);
#define FCONV_M(T) return launch_pdl(norm_rope_join<T>, grid, dim3(1024), 0, s, g, (int)bx)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
