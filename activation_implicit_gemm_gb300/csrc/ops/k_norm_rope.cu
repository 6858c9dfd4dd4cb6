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
// next one's values on their way. Blocks take heads of q or of k only, so a thread
// keeps one weight in registers. In the backward pass blocks stay for many tokens and keep
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
  int heads, per, groups;  // heads of a group, groups
  int blocks;              // backward: of a group
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

template <typename T>
constexpr bool kBf16 = false;
template <>
constexpr bool kBf16<__nv_bfloat16> = true;

// Where a lane's chunk lies in a head.
struct Chunk {
  int lo, hi;  // first elements of its two accesses, hi < 0: no second one
  bool turns;
};

template <int VEC, bool IL>
__device__ __forceinline__ void place(Chunk& c, const HeadGeom& g, int chunk) {
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

// The sine and cosine of a chunk's pairs.
template <int VEC>
__device__ __forceinline__ void angles(float (&sn)[VEC], float (&cs)[VEC], const HeadGeom& g,
                                       int chunk, int64_t b, int64_t t) {
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
      turn_of(x, g.inv_freq[p], sn[i], cs[i]);
    } else {
      const int a = p < g.sec0 ? 0 : p < g.sec0 + g.sec1 ? 1 : 2;
      const float2 v = turn_of_long(long_position(g.pos, g.pos_type, at + a), g.inv_freq[p]);
      sn[i] = v.x;
      cs[i] = v.y;
    }
  }
}

// A chunk's 2 VEC elements of one head, worked on as VEC packed pairs of f32: with both members
// of a pair in one (kMembers: neighbours that turn with each other, or a chunk of one pair), else
// VEC / 2 packed pairs of first members and as many of second ones.
template <typename T, int VEC, bool IL>
struct Raw {
  static constexpr bool kMembers = IL || VEC == 1;
  Vec<T, IL ? 2 * VEC : VEC> a, b;
  __device__ __forceinline__ void load(const T* p, const Chunk& c) {
    a = *reinterpret_cast<const decltype(a)*>(p + c.lo);
    if (!IL && c.hi >= 0) b = *reinterpret_cast<const decltype(b)*>(p + c.hi);
  }
  __device__ __forceinline__ void store(T* p, const Chunk& c) const {
    *reinterpret_cast<decltype(a)*>(p + c.lo) = a;
    if (!IL && c.hi >= 0) *reinterpret_cast<decltype(b)*>(p + c.hi) = b;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (IL ? 2 * VEC : VEC); ++i) a.v[i] = b.v[i] = from_f<T>(0.0f);
  }
  __device__ __forceinline__ T& at(int e) { return IL || e < VEC ? a.v[e] : b.v[e - VEC]; }
  __device__ __forceinline__ uint64_t get(int i) {
    if constexpr (sizeof(T) == 4) {
      return pair((float)at(2 * i), (float)at(2 * i + 1));
    } else if constexpr (VEC == 1) {
      return pair(to_f(a.v[0]), to_f(b.v[0]));
    } else if constexpr (kBf16<T>) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(&at(2 * i));
      return pair(w << 16, w & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&at(2 * i)));
      return pair(f.x, f.y);
    }
  }
  __device__ __forceinline__ void set(int i, uint64_t v) {
    if constexpr (sizeof(T) == 4) {
      at(2 * i) = low(v);
      at(2 * i + 1) = high(v);
    } else if constexpr (VEC == 1) {
      a.v[0] = from_f<T>(low(v));
      b.v[0] = from_f<T>(high(v));
    } else if constexpr (kBf16<T>) {
      *reinterpret_cast<__nv_bfloat162*>(&at(2 * i)) = __floats2bfloat162_rn(low(v), high(v));
    } else {
      *reinterpret_cast<__half2*>(&at(2 * i)) = __floats2half2_rn(low(v), high(v));
    }
  }
};
__device__ __forceinline__ uint64_t swapped(uint64_t v) { return pair(high(v), low(v)); }

template <int VEC, bool IL>
__device__ __forceinline__ int element(const Chunk& c, int e) {  // -1: there is none
  if (IL || e < VEC) return c.lo + e;
  return c.hi < 0 ? -1 : c.hi + e - VEC;
}

// A chunk's weights in the order of its elements.
template <typename T, int VEC, bool IL>
__device__ __forceinline__ void load_weight(float (&w)[2 * VEC], const HeadGeom& g, const Side& s,
                                            const Chunk& c) {
#pragma unroll
  for (int e = 0; e < 2 * VEC; ++e) {
    const int at = element<VEC, IL>(c, e);
    w[e] = 1.0f;
    if (s.w && at >= 0) w[e] = g.f32_params ? ((const float*)s.w)[at] : to_f(((const T*)s.w)[at]);
  }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Heads whose values are on their way while one is worked on: `bytes` of them a thread.
template <typename T, int VEC, int R>
__host__ __device__ constexpr int ahead(int bytes) {
  const int each = 2 * VEC * R * (int)sizeof(T);
  return R > 2 || each > bytes ? 1 : bytes / each;
}

// R: chunks of a lane (more than one only where a head has more than 32).
template <typename T, int VEC, int R, bool IL>
__global__ void __launch_bounds__(kThreads, R > 2 ? 1 : R == 2 ? 2 : 3)
    norm_rope_forward(const __grid_constant__ HeadGeom g) {
  using Row = Raw<T, VEC, IL>;
  constexpr int A = ahead<T, VEC, R>(VEC == 8 ? 32 : 64);
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
  Chunk c[R];
  bool on[R];
  Row row[A][R];
  // The turn and the weights in one: y = r (x m + x' m'), x' the pairs' other members.
  uint64_t m[R][VEC], mx[R][VEC];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    on[r] = here && lane + r * g.lanes < g.chunks;
    if (on[r]) place<VEC, IL>(c[r], g, lane + r * g.lanes);
#pragma unroll
    for (int i = 0; i < A; ++i) {
      row[i][r].zero();
      if (on[r] && h0 + i < h1) row[i][r].load(xp + (h0 + i) * s.xs[2], c[r]);
    }
    if (on[r]) {
      float sn[VEC], cs[VEC], w[2 * VEC];
      load_weight<T, VEC, IL>(w, g, s, c[r]);
      if (c[r].turns) {
        angles<VEC>(sn, cs, g, lane + r * g.lanes, b, t);
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) sn[k] = 0.0f, cs[k] = 1.0f;
      }
      if (Row::kMembers) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          m[r][k] = pair(w[2 * k] * cs[k], w[2 * k + 1] * cs[k]);
          mx[r][k] = pair(-w[2 * k + 1] * sn[k], w[2 * k] * sn[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          const int e = 2 * k, f = VEC + 2 * k;
          m[r][k] = pair(w[e] * cs[e], w[e + 1] * cs[e + 1]);
          mx[r][k] = pair(-w[f] * sn[e], -w[f + 1] * sn[e + 1]);
          m[r][VEC / 2 + k] = pair(w[f] * cs[e], w[f + 1] * cs[e + 1]);
          mx[r][VEC / 2 + k] = pair(w[e] * sn[e], w[e + 1] * sn[e + 1]);
        }
      }
    }
  }
  const float inv = 1.0f / (float)g.D;
  const T* ahead_p = xp + (h0 + A) * s.xs[2];
  yp += h0 * s.os[2];
  for (int h = h0; h < h1; h += A) {
#pragma unroll
    for (int i = 0; i < A; ++i) {
      if (h + i >= h1) break;
      uint64_t x[R][VEC], sums = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          x[r][k] = row[i][r].get(k);
          sums = fma2(x[r][k], x[r][k], sums);
        }
        if (on[r] && h + i + A < h1) row[i][r].load(ahead_p, c[r]);
      }
      ahead_p += s.xs[2];
      const float sum = lanes_sum(low(sums) + high(sums), g.lanes);
      const float scale = rsqrtf(fmaf(sum, inv, g.eps));
      const uint64_t both = pair(scale, scale);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!on[r]) continue;
        Row out;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          uint64_t y = mul2(x[r][k], m[r][k]);
          if (c[r].turns) {
            const uint64_t other = Row::kMembers ? swapped(x[r][k])
                                                 : x[r][k < VEC / 2 ? k + VEC / 2 : k - VEC / 2];
            y = fma2(other, mx[r][k], y);
          }
          out.set(k, mul2(y, both));
        }
        out.store(yp, c[r]);
      }
      yp += s.os[2];
    }
  }
}

template <typename T, int VEC, int R, bool IL>
__global__ void __launch_bounds__(kThreads, R > 2 ? 1 : 2)
    norm_rope_backward(const __grid_constant__ HeadGeom g) {
  using Row = Raw<T, VEC, IL>;
  constexpr int A = ahead<T, VEC, R>(32);
  extern __shared__ float sums[];  // a row of D for each warp
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int of_q = g.side[0].groups * g.side[0].blocks;
  const bool is_k = (int)blockIdx.x >= of_q;
  const Side& s = g.side[is_k];
  const int block = (int)blockIdx.x - (is_k ? of_q : 0);
  const int h0 = block / s.blocks * s.per;
  const int h1 = min(h0 + s.per, s.heads);
  const int lane = threadIdx.x & (g.lanes - 1);
  const int64_t each = kThreads / g.lanes;  // tokens of a block at a time
  const float inv = 1.0f / (float)g.D;
  Chunk c[R];
  uint64_t w[R][VEC], dw[R][VEC];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (lane + r * g.lanes < g.chunks) {
      float v[2 * VEC];
      place<VEC, IL>(c[r], g, lane + r * g.lanes);
      load_weight<T, VEC, IL>(v, g, s, c[r]);
#pragma unroll
      for (int k = 0; k < VEC; ++k) w[r][k] = pair(v[2 * k], v[2 * k + 1]);
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) dw[r][k] = 0;
  }
  for (int64_t t0 = block % s.blocks * each; t0 < g.tokens; t0 += s.blocks * each) {
    int64_t token = t0 + threadIdx.x / g.lanes;
    const bool here = token < g.tokens;
    if (!here) token = 0;
    const int64_t b = token / g.len, t = token - b * g.len;
    const T* xp = (const T*)s.x + b * s.xs[0] + t * s.xs[1] + h0 * s.xs[2];
    const T* yp = (const T*)s.dy + b * s.ys[0] + t * s.ys[1] + h0 * s.ys[2];
    T* op = (T*)s.out + b * s.os[0] + t * s.os[1] + h0 * s.os[2];
    bool on[R];
    Row rx[A][R], ry[A][R];
    float sn[R][VEC], cs[R][VEC];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      on[r] = here && lane + r * g.lanes < g.chunks;
#pragma unroll
      for (int i = 0; i < A; ++i) {
        rx[i][r].zero();
        ry[i][r].zero();
        if (on[r] && h0 + i < h1) {
          rx[i][r].load(xp + i * s.xs[2], c[r]);
          ry[i][r].load(yp + i * s.ys[2], c[r]);
        }
      }
      if (on[r] && c[r].turns) angles<VEC>(sn[r], cs[r], g, lane + r * g.lanes, b, t);
    }
    xp += A * s.xs[2];
    yp += A * s.ys[2];
    for (int h = h0; h < h1; h += A) {
#pragma unroll
      for (int i = 0; i < A; ++i) {
        if (h + i >= h1) break;
        uint64_t x[R][VEC], g2[R][VEC], squares = 0, dots = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            x[r][k] = rx[i][r].get(k);
            g2[r][k] = ry[i][r].get(k);
            squares = fma2(x[r][k], x[r][k], squares);
          }
          if (!on[r]) continue;
          if (h + i + A < h1) {
            rx[i][r].load(xp, c[r]);
            ry[i][r].load(yp, c[r]);
          }
          if (c[r].turns) {  // back
            if (Row::kMembers) {
#pragma unroll
              for (int k = 0; k < VEC; ++k)
                g2[r][k] = fma2(swapped(g2[r][k]), pair(sn[r][k], -sn[r][k]),
                                mul2(g2[r][k], pair(cs[r][k], cs[r][k])));
            } else {
#pragma unroll
              for (int k = 0; k < VEC / 2; ++k) {
                const uint64_t cc = pair(cs[r][2 * k], cs[r][2 * k + 1]);
                const uint64_t ss = pair(sn[r][2 * k], sn[r][2 * k + 1]);
                const uint64_t u = g2[r][k], v = g2[r][VEC / 2 + k];
                g2[r][k] = fma2(v, ss, mul2(u, cc));
                const uint64_t vc = mul2(v, cc);
                g2[r][VEC / 2 + k] = pair(fmaf(-low(u), sn[r][2 * k], low(vc)),
                                          fmaf(-high(u), sn[r][2 * k + 1], high(vc)));
              }
            }
          }
#pragma unroll
          for (int k = 0; k < VEC; ++k) dots = fma2(mul2(g2[r][k], w[r][k]), x[r][k], dots);
        }
        xp += s.xs[2];
        yp += s.ys[2];
        const float sum = lanes_sum(low(squares) + high(squares), g.lanes);
        const float dot = lanes_sum(low(dots) + high(dots), g.lanes);
        const float scale = rsqrtf(fmaf(sum, inv, g.eps));
        const float along = -(dot * inv) * scale * scale;
        const uint64_t scales = pair(scale, scale), alongs = pair(along, along);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (!on[r]) continue;
          Row out;
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            dw[r][k] = fma2(g2[r][k], mul2(x[r][k], scales), dw[r][k]);
            out.set(k, mul2(fma2(x[r][k], alongs, mul2(g2[r][k], w[r][k])), scales));
          }
          out.store(op, c[r]);
        }
        op += s.os[2];
      }
    }
  }
  if (!g.part || !s.dw) return;
  // the block's part of dw: over the tokens of a warp by shuffles, over the warps in order
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) {
      float v = e & 1 ? high(dw[r][e / 2]) : low(dw[r][e / 2]);
      for (int o = g.lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if ((threadIdx.x & 31) < g.lanes && lane + r * g.lanes < g.chunks) {
        const int at = element<VEC, IL>(c[r], e);
        if (at >= 0) sums[(threadIdx.x >> 5) * g.D + at] = v;
      }
    }
  }
  __syncthreads();
  float* part = g.part + (int64_t)blockIdx.x * g.D;
  for (int e = threadIdx.x; e < g.D; e += kThreads) {
    float v = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) v += sums[i * g.D + e];
    part[e] = v;
  }
}

// dw of q (blockIdx.y 0) or k: the parts of their blocks, 32 columns a block, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024)
    norm_rope_join(const __grid_constant__ HeadGeom g) {
  __shared__ float sums[32][33];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const Side& s = g.side[blockIdx.y];
  if (!s.dw) return;
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  const int64_t begin = blockIdx.y ? (int64_t)g.side[0].groups * g.side[0].blocks : 0;
  const int64_t n = (int64_t)s.groups * s.blocks;
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

// The variants: accesses of 16 bytes, of 8 (16-bit rows that allow no more), of one element, and
// more chunks a lane for heads that 32 lanes do not hold.
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

// Groups of heads, at most `most` in each and as even as they go.
void share(Side& s, int most) {
  s.groups = s.heads ? (s.heads + most - 1) / most : 0;
  s.per = s.heads ? (s.heads + s.groups - 1) / s.groups : 0;
  s.groups = s.heads ? (s.heads + s.per - 1) / s.per : 0;
}

// Blocks of the backward pass: two an SM, shared out by the heads of a group, one a group at least.
int backward_blocks(int sms) { return 2 * sms; }

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
  // il: 16 bytes hold whole pairs of neighbours
  const int n = width(d, a, g.pairs, backward), full = d.dtype == FCONV_F32 ? 4 : 8;
  const bool neighbours = d.pairing == FCONV_ROPE_INTERLEAVED && g.pairs > 0;
  v.il = neighbours && n == full;
  v.vec = v.il ? full / 2 : neighbours || n < 4 ? 1 : n;
  g.pair_chunks = g.pairs / v.vec;
  g.chunks = g.pair_chunks + (g.D - 2 * g.pairs + 2 * v.vec - 1) / (2 * v.vec);
  g.lanes = 1;
  while (g.lanes < g.chunks && g.lanes < 32) g.lanes *= 2;
  v.r = (g.chunks + g.lanes - 1) / g.lanes;
  return g;
}

}  // namespace

size_t norm_rope_workspace(const fconv_norm_rope_desc& d, int sms) {
  // groups * per stays under twice the heads, and a group has one block at least
  const size_t most = 2 * (size_t)backward_blocks(sms) + (size_t)(d.heads_q + d.heads_k);
  return most * (size_t)d.head_dim * sizeof(float);
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
  const long long most = backward_blocks(sms);
  int per = g.side[0].heads;  // fewer where the tokens alone do not fill the GPU
  if (per < g.side[1].heads) per = g.side[1].heads;
  for (;; per = (per + 1) / 2) {
    share(g.side[0], per);
    share(g.side[1], per);
    if (per == 1 || all * (g.side[0].groups + g.side[1].groups) >= most) break;
  }
  const int heads = g.side[0].heads + g.side[1].heads;
  long long total = 0;
  for (Side& side : g.side) {
    long long n = most * side.per / heads;
    if (n > all) n = all;
    if (n < 1) n = 1;
    side.blocks = (int)n;
    total += n * side.groups;
  }
  int e = 0;
  if (all > 0) {
    v.grid = dim3((unsigned)total);
    const RunBackward run{g, v, s};
#define FCONV_M(T) e = by_shape<T>(v, run)
    FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
  } else {
    g.side[0].groups = g.side[1].groups = 0;  // no parts: zero
  }
  if (e || (!a.dw && !a.dkw)) return e;
  const dim3 grid((unsigned)((g.D + 31) / 32), 2);
#define FCONV_M(T) return launch_pdl(norm_rope_join<T>, grid, dim3(1024), 0, s, g)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
