// Rotary positions with one to three axes (include/fconv_ops.h).
//
//   angle = position[axis(p)] * inv_freq[p],  (u, v) -> (u cos - v sin, v cos + u sin)
// A thread owns VEC neighbouring pairs of one token, makes their sines and cosines once and
// turns them in every head of q and k (or of its share of the heads when there are few tokens).
// Bound: HBM, q and k in and out; 36864 tokens of 40 heads of 128 in bf16 move 1.51 GB.
#include "ops_common.cuh"
#include "ops_internal.h"
#include "rope_angle.cuh"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

struct RopeGeom {
  const void* q;
  const void* k;
  const void* pos;
  const float* inv_freq;
  void* q_out;
  void* k_out;
  int64_t len, pos_batch, tokens;
  int heads_q, heads, per;  // heads: of q and k together; per: heads of a block row
  int pairs, chunks, axes, sec0, sec1, pairing, pos_type, inverse;
  int64_t q_stride[3], k_stride[3], q_out_stride[3], k_out_stride[3];
};

// VEC: pairs a thread, one access of VEC elements each for the first and the second members
// of a head; interleaved pairs are one access of 2 VEC elements (IL). Chunks past the last pair
// copy the elements that no pair covers. One head at a time and as many threads as registers
// allow (64 a thread with two accesses, 32 with one) beat more heads in flight in fewer threads:
// at the size above 244 and 253 us (6.2 and 6.0 TB/s) against 340 and 382 us with two.
template <typename T, int VEC, bool IL>
__global__ void __launch_bounds__(256, IL ? 8 : 4) rope_kernel(const RopeGeom g) {
  constexpr int N = IL ? 2 * VEC : VEC;  // elements of an access
  using V = Vec<T, N>;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t token = at / g.chunks;
  const int chunk = (int)(at - token * g.chunks);
  if (token >= g.tokens) return;
  const int64_t b = token / g.len, t = token - b * g.len;
  const int p0 = chunk * VEC;
  const bool copy = p0 >= g.pairs;
  float cs[VEC], sn[VEC];
  int lo = 2 * g.pairs + (chunk - g.pairs / VEC) * N, hi = lo;
  if (!copy) {
    const int64_t pt = ((g.pos_batch == 1 ? 0 : b) * g.len + t) * g.axes;
    float pos[3];
#pragma unroll
    for (int a = 0; a < 3; ++a) pos[a] = a < g.axes ? position(g.pos, g.pos_type, pt + a) : 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int p = p0 + i;
      const float x = p < g.sec0 ? pos[0] : p < g.sec0 + g.sec1 ? pos[1] : pos[2];
      if (fabsf(x) <= kLongPosition) {
        turn_of(x, g.inv_freq[p], sn[i], cs[i]);
      } else {
        const int a = p < g.sec0 ? 0 : p < g.sec0 + g.sec1 ? 1 : 2;
        const float2 v = turn_of_long(long_position(g.pos, g.pos_type, pt + a), g.inv_freq[p]);
        sn[i] = v.x;
        cs[i] = v.y;
      }
      if (g.inverse) sn[i] = -sn[i];
    }
    if (IL) {
      lo = 2 * p0;
    } else if (g.pairing == FCONV_ROPE_INTERLEAVED) {
      lo = 2 * p0;  // VEC is 1
      hi = lo + 1;
    } else if (g.pairing == FCONV_ROPE_HALF) {
      lo = p0;
      hi = p0 + g.pairs;
    } else {
      const int s1 = g.sec0 + g.sec1;
      const int start = p0 < g.sec0 ? 0 : p0 < s1 ? g.sec0 : s1;
      const int size = p0 < g.sec0 ? g.sec0 : p0 < s1 ? g.sec1 : g.pairs - s1;
      lo = start + p0;
      hi = lo + size;
    }
  }
  const T* qp = (const T*)g.q + b * g.q_stride[0] + t * g.q_stride[1];
  const T* kp = (const T*)g.k + b * g.k_stride[0] + t * g.k_stride[1];
  T* qw = (T*)g.q_out + b * g.q_out_stride[0] + t * g.q_out_stride[1];
  T* kw = (T*)g.k_out + b * g.k_out_stride[0] + t * g.k_out_stride[1];
  const int h0 = blockIdx.y * g.per, h1 = min(h0 + g.per, g.heads);
  for (int h = h0; h < h1; ++h) {
    const bool is_q = h < g.heads_q;
    const T* p = is_q ? qp + h * g.q_stride[2] : kp + (h - g.heads_q) * g.k_stride[2];
    T* w = is_q ? qw + h * g.q_out_stride[2] : kw + (h - g.heads_q) * g.k_out_stride[2];
    V x = *reinterpret_cast<const V*>(p + lo), y;
    if (!copy) {
      if (!IL) y = *reinterpret_cast<const V*>(p + hi);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        T& u = IL ? x.v[2 * e] : x.v[e];
        T& v = IL ? x.v[2 * e + 1] : y.v[e];
        const float a = to_f(u), c = to_f(v);
        u = from_f<T>(a * cs[e] - c * sn[e]);
        v = from_f<T>(c * cs[e] + a * sn[e]);
      }
      if (!IL) *reinterpret_cast<V*>(w + hi) = y;
    }
    *reinterpret_cast<V*>(w + lo) = x;
  }
}

// Elements of an access: as many as every pair's members allow. Sections (or all pairs) and the
// tail are whole chunks, and every row and tensor starts at a multiple of it.
int width(const fconv_rope_desc& d, const RopeArgs& a, int pairs) {
  const int size = d.dtype == FCONV_F32 ? 4 : 2;
  int64_t units = d.head_dim - 2 * pairs;
  units |= d.pairing == FCONV_ROPE_INTERLEAVED ? 2 * pairs : pairs;
  if (d.pairing == FCONV_ROPE_HALF_PER_AXIS)
    for (int i = 0; i < d.axes; ++i) units |= d.section[i];
  const int64_t ext[3] = {d.batch, d.len, d.heads_q};
  for (int i = 0; i < 3; ++i) {
    if (ext[i] > 1) units |= d.q_stride[i] | d.q_out_stride[i];
    if (d.heads_k && (i < 2 ? ext[i] : d.heads_k) > 1) units |= d.k_stride[i] | d.k_out_stride[i];
  }
  const uintptr_t addr = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.q_out | (uintptr_t)a.k_out;
  int n = 16 / size;
  while (n > 1 && (units % n != 0 || addr % (n * size) != 0)) n /= 2;
  return n;
}

// Interleaved pairs that no access holds whole (odd strides) take two accesses of one element.
template <typename T, int N>
int start(const RopeGeom& g, dim3 grid, cudaStream_t s) {
  if constexpr (N > 1) {
    if (g.pairing == FCONV_ROPE_INTERLEAVED)
      return launch_pdl(rope_kernel<T, N / 2, true>, grid, dim3(256), 0, s, g);
  }
  return launch_pdl(rope_kernel<T, N, false>, grid, dim3(256), 0, s, g);
}

template <typename T>
int start_t(const RopeGeom& g, int n, dim3 grid, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (n == 8) return start<T, 8>(g, grid, s);
  }
  if (n == 4) return start<T, 4>(g, grid, s);
  if (n == 2) return start<T, 2>(g, grid, s);
  return start<T, 1>(g, grid, s);
}

}  // namespace

int launch_rope(const fconv_rope_desc& d, int sms, const RopeArgs& a, cudaStream_t s) {
  RopeGeom g{};
  g.q = a.q;
  g.k = a.k;
  g.pos = a.pos;
  g.inv_freq = a.inv_freq;
  g.q_out = a.q_out;
  g.k_out = a.k_out;
  g.len = d.len;
  g.pos_batch = d.pos_batch;
  g.tokens = d.batch * d.len;
  g.heads_q = (int)d.heads_q;
  g.heads = (int)(d.heads_q + d.heads_k);
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
  const int n = width(d, a, g.pairs);
  const bool whole = d.pairing == FCONV_ROPE_INTERLEAVED && n > 1;  // an access holds both members
  g.chunks = (whole ? (int)d.head_dim : (int)d.head_dim - g.pairs) / n;
  const long long blocks = (g.tokens * g.chunks + 255) / 256;
  if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
  // few tokens: the heads are shared out too, until there are about four blocks an SM
  const long long want = (4LL * sms + blocks - 1) / blocks;
  const int shares = (int)(want < g.heads ? want : g.heads);
  g.per = (g.heads + shares - 1) / shares;
  const dim3 grid((unsigned)blocks, (unsigned)((g.heads + g.per - 1) / g.per));
#define FCONV_M(T) return start_t<T>(g, n, grid, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
