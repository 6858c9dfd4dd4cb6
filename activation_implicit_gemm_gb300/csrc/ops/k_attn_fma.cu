// Attention forward and backward on CUDA cores (include/fconv_ops.h): every type and stride,
// for head lengths from 129 to 256, whose gradients of a key tile no longer fit the registers of
// the kernels in k_attn_mma.cu.
//
//   s = scale q k^T,  p = softmax(s),  out = p v,  lse = log sum exp s
// Forward: a block owns BT query rows of one head and walks the keys in tiles of BT with the
// running maximum m and sum l of the softmax; when m grows, l and the accumulator shrink by
// exp(m_old - m_new), so one pass suffices.
// Backward, with p = exp(s - lse) recomputed and delta_i = sum_d dout_id out_id:
//   dv = p^T dout,  ds = scale p (dout v^T - delta),  dq = ds k,  dk = ds^T q
// One kernel owns query tiles (dq) and one owns key tiles (dk, dv; it walks the queries of all
// the heads that share the key head), so every gradient has one writer and no atomics.
//
// Tiles lie in shared memory as f32 with rows of D + 4 floats: the 16 threads that read 16
// neighbouring rows with 16-byte loads then touch all banks evenly. Rows past a sequence's
// length are stored as zeros, so what the tensors hold there never enters a product. Each of
// the 16 x 16 threads computes an R x R piece of the BT x BT scores (R = BT / 16). Bound: the
// f32 FMA lanes (4 D FLOPs a pair forward, 14 D backward with the scores made twice) and the
// shared-memory reads that feed them: an 8-byte operand for 4 FMAs. 4 x 1024 tokens of 8 heads of
// 256, f32: forward 3.80 ms (9 TFLOP/s of 80), backward 10.9 ms (8 counted, 11 as run). Head
// lengths over 128 are not among the measured workloads; tiles split between the warps as in
// k_attn_mma.cu would be the next step.
#include "attn_geom.cuh"

namespace fconv {
namespace ops {
namespace {

// acc[r][c] = sum_d a[ty R + r][d] * b[tx + 16 c][d]
template <int R>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, int Dp, int ty, int tx,
                                         float (&acc)[R][R]) {
  const int pitch = Dp + 4;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < R; ++c) acc[r][c] = 0.0f;
#pragma unroll 2
  for (int d = 0; d < Dp; d += 4) {
    float4 x[R], y[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      x[r] = *reinterpret_cast<const float4*>(a + (ty * R + r) * pitch + d);
#pragma unroll
    for (int c = 0; c < R; ++c)
      y[c] = *reinterpret_cast<const float4*>(b + (tx + 16 * c) * pitch + d);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < R; ++c) {
        float s = acc[r][c];
        s = fmaf(x[r].x, y[c].x, s);
        s = fmaf(x[r].y, y[c].y, s);
        s = fmaf(x[r].z, y[c].z, s);
        acc[r][c] = fmaf(x[r].w, y[c].w, s);
      }
  }
}

// acc[r][e] += sum_j p[ty R + r][j] * t[j][2 tx + 32 e ..]; TR: p is read transposed
template <int BT, int NE, bool TR>
__device__ __forceinline__ void mix_tile(const float* p, const float* t, int Dp, int ty, int tx,
                                         float2 (&acc)[BT / 16][NE]) {
  constexpr int R = BT / 16;
  const int pitch = Dp + 4;
  for (int j0 = 0; j0 < BT; j0 += 4) {
    float w[4][R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!TR) {
        const float4 v = *reinterpret_cast<const float4*>(p + (ty * R + r) * (BT + 4) + j0);
        w[0][r] = v.x;
        w[1][r] = v.y;
        w[2][r] = v.z;
        w[3][r] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i][r] = p[(j0 + i) * (BT + 4) + ty * R + r];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const int d = tx * 2 + 32 * e;
        if (d >= Dp) break;
        const float2 y = *reinterpret_cast<const float2*>(t + (j0 + i) * pitch + d);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r][e].x = fmaf(w[i][r], y.x, acc[r][e].x);
          acc[r][e].y = fmaf(w[i][r], y.y, acc[r][e].y);
        }
      }
  }
}

template <typename T, int BT, int NE>
__device__ __forceinline__ void store_rows(T* dst, int64_t row_stride, int64_t row0, int64_t rows,
                                           const float2 (&acc)[BT / 16][NE], const float* mul,
                                           int D, int ty, int tx) {
  constexpr int R = BT / 16;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = row0 + ty * R + r;
    if (row >= rows) continue;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int d = tx * 2 + 32 * e;
      if (d < D) dst[row * row_stride + d] = from_f<T>(acc[r][e].x * mul[r]);
      if (d + 1 < D) dst[row * row_stride + d + 1] = from_f<T>(acc[r][e].y * mul[r]);
    }
  }
}

template <int R, int NE>
__device__ __forceinline__ void clear(float2 (&acc)[R][NE]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < NE; ++e) acc[r][e] = make_float2(0.0f, 0.0f);
}

template <typename T, int BT, int NE>
__global__ void __launch_bounds__(256, 1)
    attn_fma_forward(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                     T* __restrict__ o, float* __restrict__ lse, const Geom g) {
  constexpr int R = BT / 16;
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);
  const int pitch = g.Dp + 4;
  float* ks = qs + BT * pitch;
  float* vs = ks + BT * pitch;
  float* ps = vs + BT * pitch;
  const int64_t tiles = (g.Lq + BT - 1) / BT;
  int64_t u = blockIdx.x;
  const int64_t i0 = u % tiles * BT;
  u /= tiles;
  const int h = (int)(u % g.Hq);
  const int64_t b = u / g.Hq;
  const Lens L = lens_of(g, b);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;

  int64_t nk = i0 < L.q ? L.k : 0;
  if (g.causal && nk > 0) {
    const int64_t last = (i0 + BT < L.q ? i0 + BT : L.q) - 1 + L.shift;  // last key seen
    nk = last + 1 < nk ? last + 1 : nk;
  }
  float2 acc[R][NE];
  clear(acc);
  float m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
  }
  const T* qp = q + b * g.q[0] + h * g.q[2];
  const T* kp = k + b * g.k[0] + (h / g.G) * g.k[2];
  const T* vp = v + b * g.v[0] + (h / g.G) * g.v[2];
  load_tile<T, BT, 8, false>(qs, qp, g.q[1], i0, 0, L.q, g);
  const float c = g.scale * kLog2e;
  // the next keys are fetched when this tile's scores are made, the next values when its
  // probabilities are used up
  load_tile<T, BT, 8, false>(ks, kp, g.k[1], 0, 0, L.k, g);
  load_tile<T, BT, 8, false>(vs, vp, g.v[1], 0, 0, L.k, g);
  for (int64_t j0 = 0; j0 < nk; j0 += BT) {
    __syncthreads();
    float s[R][R];
    dot_tile<R>(qs, ks, g.Dp, ty, tx, s);
    __syncthreads();
    load_tile<T, BT, 8, false>(ks, kp, g.k[1], j0 + BT, 0, L.k, g);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t i = i0 + ty * R + r;
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < R; ++e) {
        const int64_t j = j0 + tx + 16 * e;
        const bool ok = i < L.q && j < L.k && (!g.causal || j <= i + L.shift);
        s[r][e] = ok ? s[r][e] * c : -INFINITY;
        top = fmaxf(top, s[r][e]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float mn = fmaxf(m[r], top);
      const float ref = mn == -INFINITY ? 0.0f : mn;  // a row without keys so far
      const float shrink = exp2f(m[r] - ref);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < R; ++e) {
        const float p = exp2f(s[r][e] - ref);
        sum += p;
        ps[(ty * R + r) * (BT + 4) + tx + 16 * e] = p;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[r] = l[r] * shrink + sum;
      m[r] = mn;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        acc[r][e].x *= shrink;
        acc[r][e].y *= shrink;
      }
    }
    __syncthreads();
    mix_tile<BT, NE, false>(ps, vs, g.Dp, ty, tx, acc);
    __syncthreads();
    load_tile<T, BT, 8, false>(vs, vp, g.v[1], j0 + BT, 0, L.k, g);
  }
  float mul[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mul[r] = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
    const int64_t i = i0 + ty * R + r;
    if (lse && tx == 0 && i < g.Lq)
      lse[(b * g.Hq + h) * g.Lq + i] = l[r] == 0.0f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
  }
  store_rows<T, BT, NE>(o + b * g.o[0] + h * g.o[2], g.o[1], i0, g.Lq, acc, mul, g.D, ty, tx);
}

// p and ds of one tile pair (query rows ty R + r, keys tx + 16 e): s holds the scores and dp
// the products dout v^T; both are replaced.
template <int R>
__device__ __forceinline__ void grad_tile(float (&s)[R][R], float (&dp)[R][R], int64_t i0,
                                          int64_t j0, const Lens& L, const Geom& g,
                                          const float* lse_row, const float* delta_row, int ty,
                                          int tx) {
  const float c = g.scale * kLog2e;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = i0 + ty * R + r;
    const float lse = i < L.q ? lse_row[i] * kLog2e : 0.0f, delta = i < L.q ? delta_row[i] : 0.0f;
#pragma unroll
    for (int e = 0; e < R; ++e) {
      const int64_t j = j0 + tx + 16 * e;
      const bool ok = i < L.q && j < L.k && (!g.causal || j <= i + L.shift);
      const float p = ok ? exp2f(s[r][e] * c - lse) : 0.0f;
      s[r][e] = p;
      dp[r][e] = ok ? p * (dp[r][e] - delta) : 0.0f;
    }
  }
}

template <typename T, int BT, int NE>
__global__ void __launch_bounds__(256, 1)
    attn_fma_dq(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                const T* __restrict__ dout, const float* __restrict__ lse,
                const float* __restrict__ delta, T* __restrict__ dq, const Geom g) {
  constexpr int R = BT / 16;
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);
  const int pitch = g.Dp + 4;
  float* gs = qs + BT * pitch;
  float* ks = gs + BT * pitch;
  float* vs = ks + BT * pitch;
  float* ps = vs + BT * pitch;
  const int64_t tiles = (g.Lq + BT - 1) / BT;
  int64_t u = blockIdx.x;
  const int64_t i0 = u % tiles * BT;
  u /= tiles;
  const int h = (int)(u % g.Hq);
  const int64_t b = u / g.Hq;
  const Lens L = lens_of(g, b);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  int64_t nk = i0 < L.q ? L.k : 0;
  if (g.causal && nk > 0) {
    const int64_t last = (i0 + BT < L.q ? i0 + BT : L.q) - 1 + L.shift;
    nk = last + 1 < nk ? last + 1 : nk;
  }
  float2 acc[R][NE];
  clear(acc);
  load_tile<T, BT, 8, false>(qs, q + b * g.q[0] + h * g.q[2], g.q[1], i0, 0, L.q, g);
  load_tile<T, BT, 8, false>(gs, dout + b * g.g[0] + h * g.g[2], g.g[1], i0, 0, L.q, g);
  const T* kp = k + b * g.k[0] + (h / g.G) * g.k[2];
  const T* vp = v + b * g.v[0] + (h / g.G) * g.v[2];
  const float* lse_row = lse + (b * g.Hq + h) * g.Lq;
  const float* delta_row = delta + (b * g.Hq + h) * g.Lq;
  load_tile<T, BT, 8, false>(vs, vp, g.v[1], 0, 0, L.k, g);
  load_tile<T, BT, 8, false>(ks, kp, g.k[1], 0, 0, L.k, g);
  for (int64_t j0 = 0; j0 < nk; j0 += BT) {
    __syncthreads();
    float s[R][R], dp[R][R];
    dot_tile<R>(qs, ks, g.Dp, ty, tx, s);
    dot_tile<R>(gs, vs, g.Dp, ty, tx, dp);
    __syncthreads();
    load_tile<T, BT, 8, false>(vs, vp, g.v[1], j0 + BT, 0, L.k, g);
    grad_tile<R>(s, dp, i0, j0, L, g, lse_row, delta_row, ty, tx);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < R; ++e) ps[(ty * R + r) * (BT + 4) + tx + 16 * e] = dp[r][e];
    __syncwarp();  // a warp reads back only the rows that it wrote
    mix_tile<BT, NE, false>(ps, ks, g.Dp, ty, tx, acc);
    __syncthreads();
    load_tile<T, BT, 8, false>(ks, kp, g.k[1], j0 + BT, 0, L.k, g);
  }
  float mul[R];
#pragma unroll
  for (int r = 0; r < R; ++r) mul[r] = g.scale;
  store_rows<T, BT, NE>(dq + b * g.dq[0] + h * g.dq[2], g.dq[1], i0, g.Lq, acc, mul, g.D, ty, tx);
}

template <typename T, int BT, int NE>
__global__ void __launch_bounds__(256, 1)
    attn_fma_dkv(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                 const T* __restrict__ dout, const float* __restrict__ lse,
                 const float* __restrict__ delta, T* __restrict__ dk, T* __restrict__ dv,
                 const Geom g) {
  constexpr int R = BT / 16;
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);
  const int pitch = g.Dp + 4;
  float* gs = qs + BT * pitch;
  float* ks = gs + BT * pitch;
  float* vs = ks + BT * pitch;
  float* ps = vs + BT * pitch;
  float* ds = ps + BT * (BT + 4);
  const int64_t tiles = (g.Lk + BT - 1) / BT;
  int64_t u = blockIdx.x;
  const int64_t j0 = u % tiles * BT;
  u /= tiles;
  const int hk = (int)(u % g.Hk);
  const int64_t b = u / g.Hk;
  const Lens L = lens_of(g, b);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float2 ak[R][NE], av[R][NE];
  clear(ak);
  clear(av);
  load_tile<T, BT, 8, false>(ks, k + b * g.k[0] + hk * g.k[2], g.k[1], j0, 0, L.k, g);
  load_tile<T, BT, 8, false>(vs, v + b * g.v[0] + hk * g.v[2], g.v[1], j0, 0, L.k, g);
  int64_t first = 0;                                 // first query that sees key j0
  if (g.causal) first = j0 - L.shift;
  if (first < 0) first = 0;
  // queries that see no key at all take no part either (their scores are all hidden)
  const int64_t lead = g.causal && L.shift < 0 ? -L.shift : 0;
  const int64_t end = j0 < L.k ? L.q : 0;
  const int64_t start = first / BT * BT, steps = end > start ? (end - start + BT - 1) / BT : 0;
  const int64_t all = steps * g.G;
  auto head_of = [&](int64_t n) { return hk * g.G + (int)(n / steps); };
  auto row_of = [&](int64_t n) { return start + n % steps * BT; };
  auto load_q = [&](int64_t n) {
    if (n < all)
      load_tile<T, BT, 8, false>(qs, q + b * g.q[0] + head_of(n) * g.q[2], g.q[1], row_of(n),
                                 lead, L.q, g);
  };
  auto load_g = [&](int64_t n) {
    if (n < all)
      load_tile<T, BT, 8, false>(gs, dout + b * g.g[0] + head_of(n) * g.g[2], g.g[1], row_of(n),
                                 lead, L.q, g);
  };
  load_q(0);
  load_g(0);
  for (int64_t n = 0; n < all; ++n) {
    const int64_t i0 = row_of(n), row = (b * g.Hq + head_of(n)) * g.Lq;
    __syncthreads();
    float s[R][R], dp[R][R];
    dot_tile<R>(qs, ks, g.Dp, ty, tx, s);
    dot_tile<R>(gs, vs, g.Dp, ty, tx, dp);
    grad_tile<R>(s, dp, i0, j0, L, g, lse + row, delta + row, ty, tx);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < R; ++e) {
        ps[(ty * R + r) * (BT + 4) + tx + 16 * e] = s[r][e];
        ds[(ty * R + r) * (BT + 4) + tx + 16 * e] = dp[r][e];
      }
    __syncthreads();
    mix_tile<BT, NE, true>(ps, gs, g.Dp, ty, tx, av);
    __syncthreads();
    load_g(n + 1);
    mix_tile<BT, NE, true>(ds, qs, g.Dp, ty, tx, ak);
    __syncthreads();
    load_q(n + 1);
  }
  float one[R], mul[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    one[r] = 1.0f;
    mul[r] = g.scale;
  }
  store_rows<T, BT, NE>(dk + b * g.dk[0] + hk * g.dk[2], g.dk[1], j0, g.Lk, ak, mul, g.D, ty, tx);
  store_rows<T, BT, NE>(dv + b * g.dv[0] + hk * g.dv[2], g.dv[1], j0, g.Lk, av, one, g.D, ty, tx);
}

size_t tile_bytes(const Geom& g, int BT, int tiles, int squares) {
  return sizeof(float) * ((size_t)tiles * BT * (g.Dp + 4) + (size_t)squares * BT * (BT + 4));
}

template <typename T, int BT, int NE>
int forward_t(const Geom& g, const AttnArgs& a, cudaStream_t s) {
  const long long blocks = g.B * g.Hq * ((g.Lq + BT - 1) / BT);
  if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
  const size_t smem = tile_bytes(g, BT, 3, 1);
  auto kern = attn_fma_forward<T, BT, NE>;
  const int e = allow_smem((const void*)kern, smem);
  if (e) return e;
  kern<<<(unsigned)blocks, 256, smem, s>>>((const T*)a.q, (const T*)a.k, (const T*)a.v, (T*)a.o,
                                           a.lse, g);
  return (int)cudaGetLastError();
}

template <typename T, int BT, int NE>
int backward_t(const Geom& g, const AttnArgs& a, cudaStream_t s) {
  const long long rows = g.B * g.Hq * g.Lq;
  const long long bq = g.B * g.Hq * ((g.Lq + BT - 1) / BT);
  const long long bk = g.B * g.Hk * ((g.Lk + BT - 1) / BT);
  float* delta = (float*)a.ws;
  if (rows > 0) {
    const size_t smem = tile_bytes(g, BT, 4, 1);
    auto kern = attn_fma_dq<T, BT, NE>;
    const int e = allow_smem((const void*)kern, smem);
    if (e) return e;
    if (!grid_ok((rows + 7) / 8) || !grid_ok(bq)) return (int)cudaErrorInvalidValue;
    attn_delta<T><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>((const T*)a.out, (const T*)a.dout,
                                                             delta, g);
    kern<<<(unsigned)bq, 256, smem, s>>>((const T*)a.q, (const T*)a.k, (const T*)a.v,
                                         (const T*)a.dout, a.lse, delta, (T*)a.dq, g);
  }
  if (bk > 0) {
    const size_t smem = tile_bytes(g, BT, 4, 2);
    auto kern = attn_fma_dkv<T, BT, NE>;
    const int e = allow_smem((const void*)kern, smem);
    if (e) return e;
    if (!grid_ok(bk)) return (int)cudaErrorInvalidValue;
    kern<<<(unsigned)bk, 256, smem, s>>>((const T*)a.q, (const T*)a.k, (const T*)a.v,
                                         (const T*)a.dout, a.lse, delta, (T*)a.dk, (T*)a.dv, g);
  }
  return (int)cudaGetLastError();
}

}  // namespace

int launch_attn_fma_forward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s) {
  const Geom g = geom_of(d, a);
#define FCONV_M(T) return forward_t<T, 32, 8>(g, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

int launch_attn_fma_backward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s) {
  const Geom g = geom_of(d, a);
#define FCONV_M(T) return backward_t<T, 32, 8>(g, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
