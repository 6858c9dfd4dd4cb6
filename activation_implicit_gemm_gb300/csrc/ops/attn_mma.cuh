// Attention forward and backward with f32 operands on the warp-level tensor instructions
// (include/fconv_ops.h): f32, and f16 and bf16 calls that the tcgen05 route does not take (head
// lengths over 128 or odd, other strides or addresses).
//
//   s = scale q k^T,  p = softmax(s),  out = p v,  lse = log sum exp s
//   p = exp(s - lse),  ds = p (dout v^T - delta),  dv = p^T dout,  dq = scale ds k,
//   dk = scale ds^T q
// An f32 value is the sum of hi, rounded to TF32, and lo = v - hi (exact, read as TF32); a
// product is lo hi + hi lo + hi hi in three m16n8k8 TF32 instructions. What is dropped is about
// 2^-23 of a product either way (hi cut off instead of rounded: 2^-21, always the same way). The
// instructions' own f32 sums round towards zero, so they run over 16 products only and are then
// added to the accumulator in plain f32. Against 64 bits the outputs are as near as those of
// f32 FMAs in sequence (3e-7 to 5e-7 of their norm at the size below; 4e-6 with hi cut off and
// one accumulator throughout, at 0.94 of the time). p and ds are split the same way: nothing is
// rounded to fewer bits, but that values under 2^-113 lose what of lo lies under TF32's smallest
// step, 2^-136.
//
// A block owns 64 rows (of queries, or of keys for dk and dv), a warp 16 of them and the columns
// of a score tile in registers: all of them for dk and dv, half in the other kernels, whose
// accumulators leave room for twice the warps (the halves are joined at the end; 528 -> 434 us a
// training pass of the size below when that was made). The score accumulator is the next
// product's A operand as it is: its column pair (2t, 2t + 1) of a lane takes the places of k = t
// and k = t + 4, and the B operand is read with rows 2t and 2t + 1 to match. Tiles lie in shared
// memory as f32 with rows of Dp + 4 floats, Dp a multiple of 8: both ways of reading a B operand
// (along a row, and down two rows) then touch all 32 banks. The next tile is on its way while the
// current one's products run. As in the other routes every gradient has one writer and no
// atomics. dq needs nothing of dk and dv: its kernel is launched after theirs but takes the SMs as
// their blocks leave them (it reads what the delta pass wrote, which theirs has waited for, from
// L2) and waits for them only before it ends: 461 -> 383 us a training pass of the size below when
// that was made.
//
// Bound: latency. 3 x 333 queries x 777 keys, 16 heads of 72, f32 (one sequence without keys,
// one cut short): 408 us for the pass; forward 101, delta 9, dk and dv 258 and dq 166 where each
// is alone under the profiler, the last two overlapping in the pass. A scheduler has four warps (two for dk and dv, whose two accumulators fill the
// registers) to cover the time of the products and of the shared-memory reads that feed them (a
// 4-byte operand a lane for 1.5 instructions). Head lengths over 128, one block of eight warps an
// SM: 4 x 1024 tokens of 8 heads of 256, f32, forward 0.83 ms (41 TFLOP/s), backward 3.5 ms (24
// counted; each half's warps of the dk, dv kernel make the scores for themselves).
#pragma once

#include "attn_geom.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kRows = 64;
constexpr float kLargestTf32 = 3.4011621342146535e38f;  // (2 - 2^-10) 2^127

struct Split4 {
  uint32_t hi[4], lo[4];
};
// Values that would round past TF32's largest, and infinities, get the largest as hi: lo is then
// what is missing, an infinity where v is one, and a product with it comes out infinite once
// instead of as inf - inf (383 -> 408 us a training pass of the size above; the conversion
// instruction that saturates took 499).
__device__ __forceinline__ void split(float v, uint32_t& hi, uint32_t& lo) {
  float c;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(c) : "f"(v), "f"(kLargestTf32));
  hi = (__float_as_uint(c) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(v - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}
// x[n] = a b[n], or x[n] += a b[n], for N sums, one kind of product after the other: a sum is
// used again only N instructions later.
template <bool FIRST, int N>
__device__ __forceinline__ void mma3(float (&x)[N][4], const Split4& a, const float (&b)[N][2]) {
  uint32_t h[N][2], l[N][2];
  const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int n = 0; n < N; ++n) {
    split(b[n][0], h[n][0], l[n][0]);
    split(b[n][1], h[n][1], l[n][1]);
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (FIRST) mma_tf32(x[n], a.lo, h[n][0], h[n][1], zero);
    else mma_tf32(x[n], a.lo, h[n][0], h[n][1], x[n]);
  }
#pragma unroll
  for (int n = 0; n < N; ++n) mma_tf32(x[n], a.hi, l[n][0], l[n][1], x[n]);
#pragma unroll
  for (int n = 0; n < N; ++n) mma_tf32(x[n], a.hi, h[n][0], h[n][1], x[n]);
}
template <int N>
__device__ __forceinline__ void add_to(float (*d)[4], const float (&x)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const uint64_t v = add2(pair(d[n][e], d[n][e + 1]), pair(x[n][e], x[n][e + 1]));
      d[n][e] = low(v);
      d[n][e + 1] = high(v);
    }
}

// s = a b^T over d for 16 rows of a (this warp's) and 8 N rows of b.
template <int N>
__device__ __forceinline__ void scores(float (&s)[N][4], const float* a, const float* b, int nd,
                                       int pitch, int gr, int t) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
  constexpr int GS = N < 4 ? N : 4;
  const float* ap = a + gr * pitch + t;
  const float* bp = b + gr * pitch + t;
  auto rows = [&](Split4& x, int k) {
    split(ap[k * 8], x.hi[0], x.lo[0]);
    split(ap[8 * pitch + k * 8], x.hi[1], x.lo[1]);
    split(ap[k * 8 + 4], x.hi[2], x.lo[2]);
    split(ap[8 * pitch + k * 8 + 4], x.hi[3], x.lo[3]);
  };
  auto cols = [&](float (&y)[GS][2], int n, int k) {
#pragma unroll
    for (int i = 0; i < GS; ++i) {
      y[i][0] = bp[(n + i) * 8 * pitch + k * 8];
      y[i][1] = bp[(n + i) * 8 * pitch + k * 8 + 4];
    }
  };
  int k = 0;
  for (; k + 1 < nd; k += 2) {
    Split4 x[2];
    rows(x[0], k);
    rows(x[1], k + 1);
#pragma unroll
    for (int n = 0; n < N; n += GS) {
      float y[GS][2], z[GS][4];
      cols(y, n, k);
      mma3<true>(z, x[0], y);
      cols(y, n, k + 1);
      mma3<false>(z, x[1], y);
      add_to(s + n, z);
    }
  }
  if (k < nd) {
    Split4 x;
    rows(x, k);
#pragma unroll
    for (int n = 0; n < N; n += GS) {
      float y[GS][2], z[GS][4];
      cols(y, n, k);
      mma3<true>(z, x, y);
      add_to(s + n, z);
    }
  }
}

// acc += p b: p the 16 x 8 N accumulator of scores(), b's 8 N rows of head_dim.
template <int NT, int N>
__device__ __forceinline__ void mix(float (&acc)[NT][4], const float (&p)[N][4], const float* b,
                                    int nd, int pitch, int gr, int t) {
  constexpr int GS = NT % 3 == 0 ? 3 : 4;
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    Split4 x[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      split(p[k + w][0], x[w].hi[0], x[w].lo[0]);
      split(p[k + w][2], x[w].hi[1], x[w].lo[1]);
      split(p[k + w][1], x[w].hi[2], x[w].lo[2]);
      split(p[k + w][3], x[w].hi[3], x[w].lo[3]);
    }
    const float* bp = b + (k * 8 + 2 * t) * pitch + gr;
#pragma unroll
    for (int n = 0; n < NT; n += GS) {
      if (n >= nd) break;
      float z[GS][4];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float y[GS][2];
#pragma unroll
        for (int i = 0; i < GS; ++i) {
          // past the row's end: its own first columns, into accumulators that no one reads
          const int at = w * 8 * pitch + (n + i < nd ? (n + i) * 8 : 0);
          y[i][0] = bp[at];
          y[i][1] = bp[pitch + at];
        }
        if (w == 0) mma3<true>(z, x[0], y);
        else mma3<false>(z, x[1], y);
      }
      add_to(acc + n, z);
    }
  }
}

template <typename T, int NT>
__device__ __forceinline__ void store_rows(T* dst, int64_t row_stride, int64_t row0, int64_t rows,
                                           const float (&acc)[NT][4], const float (&mul)[2], int D,
                                           int gr, int t) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = row0 + gr + 8 * h;
    if (row >= rows) continue;
    T* p = dst + row * row_stride;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int d = n * 8 + 2 * t;
      if (d < D) p[d] = from_f<T>(acc[n][2 * h] * mul[h]);
      if (d + 1 < D) p[d + 1] = from_f<T>(acc[n][2 * h + 1] * mul[h]);
    }
  }
}
template <int NT>
__device__ __forceinline__ void clear(float (&acc)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
}

// Columns of a tile in the gradient kernels. With 64 the four tiles of a head length of 128 leave
// room for one block an SM, with 32 for two (4 x 1024 tokens of 8 heads of 128, f32, backward:
// 2022 -> 1338 us when that was made, 1438 now); over 128 they would not fit at all.
template <int NT>
constexpr int kColsOf = NT > 12 ? 32 : 64;

// lse in log2 as the gradients subtract it. A row whose scores are all -inf has lse -inf and
// probabilities of 0, not 2^(-inf + inf).
__device__ __forceinline__ float lse_log2(float lse) {
  return lse == -INFINITY ? INFINITY : lse * kLog2e;
}

// Keys [0, end) that the query rows [i0, i0 + kRows) need.
__device__ __forceinline__ int64_t key_end(const Geom& g, const Lens& L, int64_t i0) {
  if (i0 >= L.q) return 0;
  if (!g.causal) return L.k;
  const int64_t last = (i0 + kRows < L.q ? i0 + kRows : L.q) + L.shift;
  return last < L.k ? last : L.k;
}

template <typename T, int NT, bool VEC>
__global__ void __launch_bounds__(256, NT > 16 ? 1 : 2)
    attn_mma_forward(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                     T* __restrict__ o, float* __restrict__ lse, const Geom g) {
  constexpr int kCols = 64;
  extern __shared__ float4 smem4[];
  const int pitch = g.Dp + 4, nd = g.Dp / 8;
  float* qs = reinterpret_cast<float*>(smem4);
  float* ks = qs + kRows * pitch;
  float* vs = ks + kCols * pitch;
  const int64_t tiles = (g.Lq + kRows - 1) / kRows;
  int64_t u = blockIdx.x;
  const int64_t i0 = u % tiles * kRows;
  u /= tiles;
  const int h = (int)(u % g.Hq);
  const int64_t b = u / g.Hq;
  const Lens L = lens_of(g, b);
  const int warp = (threadIdx.x >> 5) & 3, half = threadIdx.x >> 7;
  const int gr = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const int64_t nk = key_end(g, L, i0);
  const T* kp = k + b * g.k[0] + (h / g.G) * g.k[2];
  const T* vp = v + b * g.v[0] + (h / g.G) * g.v[2];
  load_tile<T, kRows, 8, VEC>(qs, q + b * g.q[0] + h * g.q[2], g.q[1], i0, 0, L.q, g);
  load_tile<T, kCols, 8, VEC>(ks, kp, g.k[1], 0, 0, L.k, g);
  load_tile<T, kCols, 8, VEC>(vs, vp, g.v[1], 0, 0, L.k, g);
  float acc[NT][4];
  clear(acc);
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  const float c = g.scale * kLog2e;
  for (int64_t j0 = 0; j0 < nk; j0 += kCols) {
    ptx::cp_async_wait<1>();  // all but the values
    __syncthreads();
    float s[kCols / 16][4];
    scores(s, qs + warp * 16 * pitch, ks + half * (kCols / 2) * pitch, nd, pitch, gr, t);
    __syncthreads();
    load_tile<T, kCols, 8, VEC>(ks, kp, g.k[1], j0 + kCols, 0, L.k, g);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t i = i0 + warp * 16 + gr + 8 * r;
      const int64_t end = i < L.q ? (g.causal && i + L.shift + 1 < L.k ? i + L.shift + 1 : L.k) : 0;
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < kCols / 16; ++n)
#pragma unroll
        for (int e = 2 * r; e < 2 * r + 2; ++e) {
          const int64_t j = j0 + half * (kCols / 2) + n * 8 + 2 * t + (e & 1);
          s[n][e] = j < end ? s[n][e] * c : -INFINITY;
          top = fmaxf(top, s[n][e]);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float mn = fmaxf(m[r], top);
      const float ref = mn == -INFINITY ? 0.0f : mn;  // a row without keys so far
      const float shrink = exp2f(m[r] - ref);
      float sum = 0.0f;
#pragma unroll
      for (int n = 0; n < kCols / 16; ++n)
#pragma unroll
        for (int e = 2 * r; e < 2 * r + 2; ++e) {
          s[n][e] = exp2f(s[n][e] - ref);
          sum += s[n][e];
        }
      l[r] = l[r] * shrink + sum;  // the lane's columns only, joined at the end
      m[r] = mn;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[n][2 * r] *= shrink;
        acc[n][2 * r + 1] *= shrink;
      }
    }
    ptx::cp_async_wait<1>();  // all but the next keys
    __syncthreads();
    mix(acc, s, vs + half * (kCols / 2) * pitch, nd, pitch, gr, t);
    __syncthreads();
    load_tile<T, kCols, 8, VEC>(vs, vp, g.v[1], j0 + kCols, 0, L.k, g);
  }
  ptx::cp_async_wait<0>();
  __syncthreads();
  // the second half of the columns' warps hand theirs over
  float* box = reinterpret_cast<float*>(smem4) + (threadIdx.x & 127);
  if (half) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      box[r * 128] = m[r];
      box[(2 + r) * 128] = l[r];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (n < nd)
#pragma unroll
        for (int e = 0; e < 4; ++e) box[(4 + n * 4 + e) * 128] = acc[n][e];
  }
  __syncthreads();
  if (half) return;
  float mul[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float mo = box[r * 128], mn = fmaxf(m[r], mo), ref = mn == -INFINITY ? 0.0f : mn;
    const float f = exp2f(m[r] - ref), fo = exp2f(mo - ref);
    l[r] = l[r] * f + box[(2 + r) * 128] * fo;
    m[r] = mn;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (n < nd)
#pragma unroll
        for (int e = 2 * r; e < 2 * r + 2; ++e)
          acc[n][e] = acc[n][e] * f + box[(4 + n * 4 + e) * 128] * fo;
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    mul[r] = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
    const int64_t i = i0 + warp * 16 + gr + 8 * r;
    if (lse && t == 0 && i < g.Lq)
      lse[(b * g.Hq + h) * g.Lq + i] = l[r] == 0.0f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
  }
  store_rows<T, NT>(o + b * g.o[0] + h * g.o[2], g.o[1], i0 + warp * 16, g.Lq, acc, mul, g.D, gr,
                    t);
}

template <typename T, int NT, bool VEC>
__global__ void __launch_bounds__(256, NT > 16 ? 1 : 2)
    attn_mma_dq(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                const T* __restrict__ dout, const float* __restrict__ lse,
                const float* __restrict__ delta, T* __restrict__ dq, const Geom g) {
  constexpr int kCols = kColsOf<NT>;
  extern __shared__ float4 smem4[];
  const int pitch = g.Dp + 4, nd = g.Dp / 8;
  float* qs = reinterpret_cast<float*>(smem4);
  float* gs = qs + kRows * pitch;
  float* ks = gs + kRows * pitch;
  float* vs = ks + kCols * pitch;
  const int64_t tiles = (g.Lq + kRows - 1) / kRows;
  int64_t u = blockIdx.x;
  const int64_t i0 = u % tiles * kRows;
  u /= tiles;
  const int h = (int)(u % g.Hq);
  const int64_t b = u / g.Hq;
  const Lens L = lens_of(g, b);
  const int warp = (threadIdx.x >> 5) & 3, half = threadIdx.x >> 7;
  const int gr = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const int64_t nk = key_end(g, L, i0);
  const T* kp = k + b * g.k[0] + (h / g.G) * g.k[2];
  const T* vp = v + b * g.v[0] + (h / g.G) * g.v[2];
  load_tile<T, kRows, 8, VEC>(qs, q + b * g.q[0] + h * g.q[2], g.q[1], i0, 0, L.q, g);
  load_tile<T, kRows, 8, VEC>(gs, dout + b * g.g[0] + h * g.g[2], g.g[1], i0, 0, L.q, g);
  load_tile<T, kCols, 8, VEC>(ks, kp, g.k[1], 0, 0, L.k, g);
  load_tile<T, kCols, 8, VEC>(vs, vp, g.v[1], 0, 0, L.k, g);
  float acc[NT][4];
  clear(acc);
  const float c = g.scale * kLog2e;
  float ls[2], del[2];
  int64_t end[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t i = i0 + warp * 16 + gr + 8 * r, at = (b * g.Hq + h) * g.Lq + i;
    const bool in = i < L.q;
    ls[r] = in ? lse_log2(__ldcg(lse + at)) : 0.0f;
    del[r] = in ? __ldcg(delta + at) : 0.0f;
    end[r] = in ? (g.causal && i + L.shift + 1 < L.k ? i + L.shift + 1 : L.k) : 0;
  }
  for (int64_t j0 = 0; j0 < nk; j0 += kCols) {
    ptx::cp_async_wait<0>();
    __syncthreads();
    float s[kCols / 16][4], dp[kCols / 16][4];
    scores(s, qs + warp * 16 * pitch, ks + half * (kCols / 2) * pitch, nd, pitch, gr, t);
    scores(dp, gs + warp * 16 * pitch, vs + half * (kCols / 2) * pitch, nd, pitch, gr, t);
    __syncthreads();
    load_tile<T, kCols, 8, VEC>(vs, vp, g.v[1], j0 + kCols, 0, L.k, g);
#pragma unroll
    for (int n = 0; n < kCols / 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = e >> 1;
        const bool ok = j0 + half * (kCols / 2) + n * 8 + 2 * t + (e & 1) < end[r];
        const float p = ok ? exp2f(s[n][e] * c - ls[r]) : 0.0f;
        dp[n][e] = p == 0.0f ? 0.0f : p * (dp[n][e] - del[r]);  // dp may not be finite there
      }
    mix(acc, dp, ks + half * (kCols / 2) * pitch, nd, pitch, gr, t);
    __syncthreads();
    load_tile<T, kCols, 8, VEC>(ks, kp, g.k[1], j0 + kCols, 0, L.k, g);
  }
  ptx::cp_async_wait<0>();
  __syncthreads();
  float* box = reinterpret_cast<float*>(smem4) + (threadIdx.x & 127);
#pragma unroll
  for (int n = 0; n < NT; ++n)
    if (n < nd && half)
#pragma unroll
      for (int e = 0; e < 4; ++e) box[(n * 4 + e) * 128] = acc[n][e];
  __syncthreads();
  if (half) return;
#pragma unroll
  for (int n = 0; n < NT; ++n)
    if (n < nd)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] += box[(n * 4 + e) * 128];
  const float mul[2] = {g.scale, g.scale};
  store_rows<T, NT>(dq + b * g.dq[0] + h * g.dq[2], g.dq[1], i0 + warp * 16, g.Lq, acc, mul, g.D,
                    gr, t);
  ptx::pdl_wait();  // attn_mma_dkv: what follows this kernel follows both
}

// DH: head_dim halves of NT column tiles, each with four warps of its own that make the scores
// over the whole length and keep dk and dv of their half.
template <typename T, int NT, int DH, bool VEC>
__global__ void __launch_bounds__(128 * DH)
    attn_mma_dkv(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                 const T* __restrict__ dout, const float* __restrict__ lse,
                 const float* __restrict__ delta, T* __restrict__ dk, T* __restrict__ dv,
                 const Geom g) {
  ptx::pdl_wait();
  ptx::pdl_trigger();  // attn_mma_dq's blocks fill the SMs as this kernel's leave them
  constexpr int kCols = kColsOf<NT * DH>, WARPS = 4 * DH;
  extern __shared__ float4 smem4[];
  __shared__ float ls[kCols], del[kCols];  // lse (log2) and delta of the tile's queries
  const int pitch = g.Dp + 4, nd = g.Dp / 8;
  float* ks = reinterpret_cast<float*>(smem4);
  float* vs = ks + kRows * pitch;
  float* qs = vs + kRows * pitch;
  float* gs = qs + kCols * pitch;
  const int64_t tiles = (g.Lk + kRows - 1) / kRows;
  int64_t u = blockIdx.x;
  const int64_t j0 = u % tiles * kRows;
  u /= tiles;
  const int hk = (int)(u % g.Hk);
  const int64_t b = u / g.Hk;
  const Lens L = lens_of(g, b);
  const int warp = (threadIdx.x >> 5) & 3, gr = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const int c0 = DH > 1 ? threadIdx.x >> 7 : 0, d0 = c0 * NT * 8;  // this half's columns
  const int nh = min(nd - c0 * NT, NT);
  load_tile<T, kRows, WARPS, VEC>(ks, k + b * g.k[0] + hk * g.k[2], g.k[1], j0, 0, L.k, g);
  load_tile<T, kRows, WARPS, VEC>(vs, v + b * g.v[0] + hk * g.v[2], g.v[1], j0, 0, L.k, g);
  int64_t first = g.causal ? j0 - L.shift : 0;  // first query that sees key j0
  if (first < 0) first = 0;
  // queries that see no key at all take no part either (their scores are all hidden)
  const int64_t lead = g.causal && L.shift < 0 ? -L.shift : 0;
  const int64_t end = j0 < L.k ? L.q : 0;
  // the walk: query tiles of every head that shares the keys
  const int64_t start = first / kCols * kCols;
  const int64_t steps = end > start ? (end - start + kCols - 1) / kCols : 0, all = steps * g.G;
  auto head_of = [&](int64_t n) { return hk * g.G + (int)(n / steps); };
  auto row_of = [&](int64_t n) { return start + n % steps * kCols; };
  auto load_q = [&](int64_t n) {
    if (n < all)
      load_tile<T, kCols, WARPS, VEC>(qs, q + b * g.q[0] + head_of(n) * g.q[2], g.q[1], row_of(n),
                                       lead, L.q, g);
  };
  auto load_g = [&](int64_t n) {
    if (n < all)
      load_tile<T, kCols, WARPS, VEC>(gs, dout + b * g.g[0] + head_of(n) * g.g[2], g.g[1],
                                       row_of(n), lead, L.q, g);
  };
  load_q(0);
  load_g(0);
  float ak[NT][4], av[NT][4];
  clear(ak);
  clear(av);
  const float c = g.scale * kLog2e;
  for (int64_t n = 0; n < all; ++n) {
    const int64_t i0 = row_of(n);
    if (threadIdx.x < kCols) {
      const int64_t i = i0 + threadIdx.x, at = (b * g.Hq + head_of(n)) * g.Lq + i;
      ls[threadIdx.x] = i < L.q ? lse_log2(lse[at]) : 0.0f;
      del[threadIdx.x] = i < L.q ? delta[at] : 0.0f;
    }
    ptx::cp_async_wait<0>();
    __syncthreads();
    float s[kCols / 8][4];
    scores(s, ks + warp * 16 * pitch, qs, nd, pitch, gr, t);
#pragma unroll
    for (int x = 0; x < kCols / 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = x * 8 + 2 * t + (e & 1);
        const int64_t i = i0 + col, j = j0 + warp * 16 + gr + 8 * (e >> 1);
        const bool ok = i < L.q && j < L.k && (!g.causal || j <= i + L.shift);
        s[x][e] = ok ? exp2f(s[x][e] * c - ls[col]) : 0.0f;
      }
    mix(av, s, gs + d0, nh, pitch, gr, t);
    float dp[kCols / 8][4];
    scores(dp, vs + warp * 16 * pitch, gs, nd, pitch, gr, t);
#pragma unroll
    for (int x = 0; x < kCols / 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = x * 8 + 2 * t + (e & 1);
        dp[x][e] = s[x][e] == 0.0f ? 0.0f : s[x][e] * (dp[x][e] - del[col]);
      }
    __syncthreads();
    load_g(n + 1);
    mix(ak, dp, qs + d0, nh, pitch, gr, t);
    __syncthreads();
    load_q(n + 1);
  }
  ptx::cp_async_wait<0>();
  const float one[2] = {1.0f, 1.0f}, mul[2] = {g.scale, g.scale};
  store_rows<T, NT>(dk + b * g.dk[0] + hk * g.dk[2] + d0, g.dk[1], j0 + warp * 16, g.Lk, ak, mul,
                    g.D - d0, gr, t);
  store_rows<T, NT>(dv + b * g.dv[0] + hk * g.dv[2] + d0, g.dv[1], j0 + warp * 16, g.Lk, av, one,
                    g.D - d0, gr, t);
}

size_t tile_bytes(const Geom& g, int rows) {
  return sizeof(float) * (size_t)rows * (g.Dp + 4);
}

template <typename T, int NT, bool VEC>
int forward_t(const Geom& g, const AttnArgs& a, cudaStream_t s) {
  const long long blocks = g.B * g.Hq * ((g.Lq + kRows - 1) / kRows);
  if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
  const size_t smem = tile_bytes(g, kRows + 2 * 64);
  auto kern = attn_mma_forward<T, NT, VEC>;
  const int e = allow_smem((const void*)kern, smem);
  if (e) return e;
  kern<<<(unsigned)blocks, 256, smem, s>>>((const T*)a.q, (const T*)a.k, (const T*)a.v,
                                                   (T*)a.o, a.lse, g);
  return (int)cudaGetLastError();
}

template <typename T, int NT, bool VEC>
int backward_t(const Geom& g, const AttnArgs& a, cudaStream_t s) {
  const long long rows = g.B * g.Hq * g.Lq;
  const long long bq = g.B * g.Hq * ((g.Lq + kRows - 1) / kRows);
  const long long bk = g.B * g.Hk * ((g.Lk + kRows - 1) / kRows);
  float* delta = (float*)a.ws;
  const size_t smem = tile_bytes(g, 2 * kRows + 2 * kColsOf<NT>);
  int e = 0;
  if ((rows > 0 && (!grid_ok((rows + 7) / 8) || !grid_ok(bq))) || (bk > 0 && !grid_ok(bk)))
    return (int)cudaErrorInvalidValue;
  if (rows > 0)
    e = launch_pdl(attn_delta<T>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s,
                   (const T*)a.out, (const T*)a.dout, delta, g);
  if (!e && bk > 0) {
    constexpr int DH = NT > 16 ? 2 : 1;
    auto kern = attn_mma_dkv<T, NT / DH, DH, VEC>;
    e = allow_smem((const void*)kern, smem);
    if (!e)
      e = launch_pdl(kern, dim3((unsigned)bk), dim3(128 * DH), smem, s, (const T*)a.q,
                     (const T*)a.k, (const T*)a.v, (const T*)a.dout, (const float*)a.lse,
                     (const float*)delta, (T*)a.dk, (T*)a.dv, g);
  }
  if (!e && rows > 0) {
    auto kern = attn_mma_dq<T, NT, VEC>;
    e = allow_smem((const void*)kern, smem);
    if (!e)
      e = launch_pdl(kern, dim3((unsigned)bq), dim3(256), smem, s, (const T*)a.q, (const T*)a.k,
                     (const T*)a.v, (const T*)a.dout, (const float*)a.lse, (const float*)delta,
                     (T*)a.dq, g);
  }
  return e;
}

}  // namespace
}  // namespace ops
}  // namespace fconv
