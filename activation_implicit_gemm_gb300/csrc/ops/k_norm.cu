// Layer norm forward and backward (include/fconv_ops.h). x is (outer, channels, inner).
//
//   mean = sum(x) / C,  rstd = (sum((x - mean)^2) / C + eps)^-1/2,  y = (x - mean) rstd w + b
//   g = dy w,  h = (x - mean) rstd,  dx = rstd (g - mean(g) - h mean(g h))
//   dw = sum(dy h),  db = sum(dy)   over all positions
// The variance comes from the centred values: a one-pass sum of squares would cancel when the
// mean is far from zero. All sums are f32, each output is rounded once.
//
// Bound: HBM (x in, y out; dy and x in, dx out). Every kernel reads its data once from HBM:
//  * rows (inner = 1, C <= 8192): a row stays in the registers of 32, 256 or 512 threads, E
//    elements each. Blocks are persistent, so w (and b) are read once a block and the partial
//    sums of dw and db stay in registers until the end; the next three or four rows are on
//    their way to shared memory as bulk copies (with one row ahead in registers instead, 24 KB
//    in flight an SM, 32768 rows of 4096 ran at half the copy rate).
//  * long rows (C > 8192): a block a row, read again from L2 in each pass.
//  * planes (inner > 1): lanes along the positions, 4 bytes each, channels split over the
//    warps; up to 256 channels the next tiles come through a ring in shared memory, beyond that
//    (or with odd 16-bit planes) a tile is read again from L2 in each pass.
// dw and db: every block writes one partial sum, norm_dparam_join adds them in order.
//
// Measured: 32768 rows of 4096 in bf16, forward 85 us (6.3 TB/s) and backward 132 us with the join
// (6.1 TB/s), 0.93 and 0.90 of the copy rate. 5001 rows of 1001 in f32 (no 16-byte units:
// a row ahead in registers), 12 us, 16 and 5: the 2.7 MB of partial sums and the launches are as
// long as the data. 32 x 128 channels x 56 x 56 in f16, forward 17 us, backward 27 and 3.7: the
// data (51 and 77 MB) is largely in L2, and the conversions, sums and products of two positions a
// lane bound it (issue slots 64 % and 57 % busy).
#include "ops_common.cuh"
#include "ops_internal.h"

#include "../fconv_internal.h"
#include "../ptx.cuh"
#include "row_feed.cuh"
#include "waits.cuh"

namespace fconv {
namespace ops {
namespace {

__device__ __forceinline__ float param_at(const void* p, int f32, int64_t i, int dtype) {
  if (f32) return ((const float*)p)[i];
  return dtype == FCONV_F16 ? to_f(((const __half*)p)[i]) : to_f(((const __nv_bfloat16*)p)[i]);
}

struct NormGeom {
  const void* x;
  const void* dy;
  const void* w;
  const void* b;
  void* y;  // y, or dx
  float* mean;
  float* rstd;
  float* part;  // [block][dw, db][C], null when not wanted
  int64_t outer, C, inner;
  int dtype, param_f32;
  float eps;
};

// ------------------------------------------------------------------------------ rows

template <int TPR>
__host__ __device__ constexpr int row_threads() { return TPR == 32 ? 128 : TPR; }

// Sum of N values over the TPR threads of a row. `red` has 2 * N * 16 floats and alternates
// between its halves: a half is written again only after the barrier of the next use, by when
// every thread has read it. ASK: whether `ok` holds in all those threads, the same answer in each.
template <int TPR, bool ASK, int N>
__device__ __forceinline__ bool row_sum(float (&v)[N], float* red, int& turn, bool ok) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = warp_sum(v[n]);
  if (TPR == 32) return !ASK || __all_sync(0xffffffffu, ok);
  float* r = red + turn * (N * 16);
  turn ^= 1;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) r[n * 16 + warp] = v[n];
  }
  if (ASK) ok = __syncthreads_and(ok);
  else __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v[n] += r[n * 16 + i];
  }
  return !ASK || ok;
}

// Thread t of a row owns chunks t, t + TPR, ... of VEC elements, E elements in all.
template <typename T, int VEC, int E, int TPR>
struct Row {
  static constexpr int NV = E / VEC;
  __device__ __forceinline__ static void get(float (&f)[E], const T* p, int t, int C) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      Vec<T, VEC> raw;
      if (c < C) raw = *reinterpret_cast<const Vec<T, VEC>*>(p + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[i * VEC + e] = c < C ? to_f(raw.v[e]) : 0.0f;
    }
  }
  __device__ __forceinline__ static void put(T* p, const float (&f)[E], int t, int C) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (c >= C) continue;
      Vec<T, VEC> o;
#pragma unroll
      for (int e = 0; e < VEC; ++e) o.v[e] = from_f<T>(f[i * VEC + e]);
      *reinterpret_cast<Vec<T, VEC>*>(p + c) = o;
    }
  }
  __device__ __forceinline__ static void params(float (&f)[E], const void* p, float none,
                                                const NormGeom& g, int t, int C) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (i * TPR + t) * VEC + e;
        f[i * VEC + e] = c >= C ? 0.0f : p ? param_at(p, g.param_f32, c, g.dtype) : none;
      }
  }
};

constexpr int kFwdStages = 4, kBwdStages = 3;

// Blocks an SM holds: as many as leave a thread the registers for E values of x and of the
// parameters (forward), and of dy and the two partial sums as well (backward).
__host__ __device__ constexpr int row_blocks(int E, int TPR, bool bwd) {
  const int threads = bwd ? (E <= 8 ? 768 : E <= 16 ? 512 : 384)
                          : (E <= 8 ? 1024 : E <= 16 ? 768 : 512);
  const int nt = TPR == 32 ? 128 : TPR;
  return threads / nt > 0 ? threads / nt : 1;
}

template <typename T, int VEC, int E, int TPR>
__global__ void __launch_bounds__(row_threads<TPR>(), row_blocks(E, TPR, false))
    norm_rows_forward(const NormGeom g) {
  constexpr int NT = row_threads<TPR>(), RPB = NT / TPR;
  extern __shared__ __align__(16) uint8_t dsmem[];
  __shared__ float red[2 * 16];
  __shared__ int abort_flag;
  using R = Row<T, VEC, E, TPR>;
  const int t = threadIdx.x % TPR, C = (int)g.C;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  Feed<T, 1, kFwdStages, TPR, (VEC > 1)> feed;
  feed.init(dsmem, threadIdx.x / TPR, RPB, t, row, g.outer, step, C);
  feed.src[0] = (const T*)g.x + row * C;
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_trigger();
  feed.start();
  float w[E], b[E];
  R::params(w, g.w, 1.0f, g, t, C);
  R::params(b, g.b, 0.0f, g, t, C);
  const float inv = 1.0f / (float)C;
  int turn = 0;
  float ahead[VEC > 1 ? 1 : E];  // without a ring the next row waits in registers
  if constexpr (VEC == 1)
    if (row < g.outer) R::get(ahead, (const T*)g.x + row * C, t, C);
  for (; row < g.outer; row += step) {
    float f[E];
    bool ok = true;
    if constexpr (VEC > 1) {
      ok = feed.wait(&abort_flag);
      R::get(f, feed.row(dsmem, 0), t, C);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = ahead[e];
      if (row + step < g.outer) R::get(ahead, (const T*)g.x + (row + step) * C, t, C);
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int e = 0; e < E; ++e) s[0] += f[e];
    ok = row_sum<TPR, (VEC > 1)>(s, red, turn, ok);
    feed.next(ok);
    const float m = s[0] * inv;
    s[0] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      f[e] = (e / VEC * TPR + t) * VEC < C ? f[e] - m : 0.0f;
      s[0] = fmaf(f[e], f[e], s[0]);
    }
    row_sum<TPR, false>(s, red, turn, true);
    const float r = rsqrtf(s[0] * inv + g.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = fmaf(f[e] * r, w[e], b[e]);
    if (!ok) break;  // here: before the row's arithmetic the branch cost up to a quarter
    if (t == 0) {
      if (g.mean) g.mean[row] = m;
      if (g.rstd) g.rstd[row] = r;
    }
    R::put((T*)g.y + row * C, f, t, C);
  }
  if (abort_flag) feed.drain();
}

template <typename T, int VEC, int E, int TPR>
__global__ void __launch_bounds__(row_threads<TPR>(), row_blocks(E, TPR, true))
    norm_rows_backward(const NormGeom g) {
  constexpr int NT = row_threads<TPR>(), RPB = NT / TPR;
  extern __shared__ __align__(16) uint8_t dsmem[];
  __shared__ float red[TPR == 32 ? 2 * E * 32 : 2 * 2 * 16];
  __shared__ int abort_flag;
  using R = Row<T, VEC, E, TPR>;
  const int t = threadIdx.x % TPR, lane = threadIdx.x & 31, C = (int)g.C;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  Feed<T, 2, kBwdStages, TPR, (VEC > 1)> feed;
  feed.init(dsmem, threadIdx.x / TPR, RPB, t, row, g.outer, step, C);
  feed.src[0] = (const T*)g.x + row * C;
  feed.src[1] = (const T*)g.dy + row * C;
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_trigger();
  feed.start();
  float w[E], aw[E], ab[E];
  R::params(w, g.w, 1.0f, g, t, C);
#pragma unroll
  for (int e = 0; e < E; ++e) aw[e] = ab[e] = 0.0f;
  const float inv = 1.0f / (float)C;
  int turn = 0;
  float ahead[2][VEC > 1 ? 1 : E];  // without a ring the next row waits in registers
  if constexpr (VEC == 1)
    if (row < g.outer) {
      R::get(ahead[0], (const T*)g.x + row * C, t, C);
      R::get(ahead[1], (const T*)g.dy + row * C, t, C);
    }
  float lm = 0.0f, lr = 0.0f;  // lane i: the statistics of the row i steps past a group of 32
  for (uint32_t k = 0; row < g.outer; row += step, ++k) {
    if ((k & 31) == 0) {
      const int64_t at = row + lane * step;
      lm = at < g.outer ? g.mean[at] : 0.0f;
      lr = at < g.outer ? g.rstd[at] : 0.0f;
    }
    const float m = __shfl_sync(0xffffffffu, lm, k & 31), r = __shfl_sync(0xffffffffu, lr, k & 31);
    float h[E], d[E];
    bool ok = true;
    if constexpr (VEC > 1) {
      ok = feed.wait(&abort_flag);
      R::get(h, feed.row(dsmem, 0), t, C);
      R::get(d, feed.row(dsmem, 1), t, C);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        h[e] = ahead[0][e];
        d[e] = ahead[1][e];
      }
      if (row + step < g.outer) {
        R::get(ahead[0], (const T*)g.x + (row + step) * C, t, C);
        R::get(ahead[1], (const T*)g.dy + (row + step) * C, t, C);
      }
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      h[e] = (h[e] - m) * r;
      aw[e] = fmaf(d[e], h[e], aw[e]);
      ab[e] += d[e];
      d[e] *= w[e];  // 0 past the row's end, where h is not
      s[0] += d[e];
      s[1] = fmaf(d[e], h[e], s[1]);
    }
    ok = row_sum<TPR, (VEC > 1)>(s, red, turn, ok);
    feed.next(ok);
    const float a = s[0] * inv, c = s[1] * inv;
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] = r * (d[e] - a - h[e] * c);
    if (!ok) break;
    R::put((T*)g.y + row * C, d, t, C);
  }
  if (abort_flag) feed.drain();
  if (!g.part) return;
  float* part = g.part + (int64_t)blockIdx.x * 2 * C;
  if (TPR == 32) {  // the block's warps add up in order
    for (int k = 0; k < RPB; ++k) {
      __syncthreads();
      if (threadIdx.x / TPR == k)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float* p = red + e * 32 + t;
          p[0] = k ? p[0] + aw[e] : aw[e];
          p[E * 32] = k ? p[E * 32] + ab[e] : ab[e];
        }
    }
    if (threadIdx.x / TPR != RPB - 1) return;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      aw[e] = red[e * 32 + t];
      ab[e] = red[(E + e) * 32 + t];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (e / VEC * TPR + t) * VEC + e % VEC;
    if (c < C) {
      part[c] = aw[e];
      part[C + c] = ab[e];
    }
  }
}

// ------------------------------------------------------------------------------ long rows

constexpr int kLong = 512;

template <typename T>
__global__ void __launch_bounds__(kLong) norm_long_forward(const NormGeom g) {
  __shared__ float red[kLong / 32];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int64_t row = blockIdx.x, C = g.C;
  const T* x = (const T*)g.x + row * C;
  T* y = (T*)g.y + row * C;
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < C; c += kLong) s += to_f(x[c]);
  const float m = block_sum<kLong>(s, red) / (float)C;
  s = 0.0f;
  for (int64_t c = threadIdx.x; c < C; c += kLong) {
    const float d = to_f(x[c]) - m;
    s = fmaf(d, d, s);
  }
  const float r = rsqrtf(block_sum<kLong>(s, red) / (float)C + g.eps);
  if (threadIdx.x == 0) {
    if (g.mean) g.mean[row] = m;
    if (g.rstd) g.rstd[row] = r;
  }
  for (int64_t c = threadIdx.x; c < C; c += kLong) {
    const float w = g.w ? param_at(g.w, g.param_f32, c, g.dtype) : 1.0f;
    const float b = g.b ? param_at(g.b, g.param_f32, c, g.dtype) : 0.0f;
    y[c] = from_f<T>(fmaf((to_f(x[c]) - m) * r, w, b));
  }
}

// A block adds its rows' dy h and dy to its partial sums in the workspace, which only it uses.
template <typename T>
__global__ void __launch_bounds__(kLong) norm_long_backward(const NormGeom g) {
  __shared__ float red[kLong / 32];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int64_t C = g.C;
  float* part = g.part ? g.part + (int64_t)blockIdx.x * 2 * C : nullptr;
  for (int64_t row = blockIdx.x; row < g.outer; row += gridDim.x) {
    const T* x = (const T*)g.x + row * C;
    const T* dy = (const T*)g.dy + row * C;
    T* dx = (T*)g.y + row * C;
    const float m = g.mean[row], r = g.rstd[row];
    float s = 0.0f, u = 0.0f;
    for (int64_t c = threadIdx.x; c < C; c += kLong) {
      const float d = to_f(dy[c]), h = (to_f(x[c]) - m) * r;
      const float k = d * (g.w ? param_at(g.w, g.param_f32, c, g.dtype) : 1.0f);
      s += k;
      u = fmaf(k, h, u);
      if (part) {
        const bool first = row == blockIdx.x;
        part[c] = first ? d * h : fmaf(d, h, part[c]);
        part[C + c] = first ? d : part[C + c] + d;
      }
    }
    s = block_sum<kLong>(s, red) / (float)C;
    u = block_sum<kLong>(u, red) / (float)C;
    for (int64_t c = threadIdx.x; c < C; c += kLong) {
      const float k = to_f(dy[c]) * (g.w ? param_at(g.w, g.param_f32, c, g.dtype) : 1.0f);
      const float h = (to_f(x[c]) - m) * r;
      dx[c] = from_f<T>(r * (k - s - h * u));
    }
  }
}

// ------------------------------------------------------------------------------ planes

// A lane has VP positions (a 4-byte access where the type and the plane allow it). Sums over
// the warps that share them.
template <int VP>
__device__ __forceinline__ void plane_sum(float (&v)[VP], float* red, int warps) {
#pragma unroll
  for (int i = 0; i < VP; ++i) red[(threadIdx.y * VP + i) * 32 + threadIdx.x] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < VP; ++i) v[i] = 0.0f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < VP; ++i) v[i] += red[(w * VP + i) * 32 + threadIdx.x];
  __syncthreads();
}

// Sums N values (a power of two) over the 32 lanes; lane l ends with the sum of value l % N.
// Each step folds the half of the values that the other lane keeps: N - 1 shuffles and a tail
// of log2(32 / N) instead of 5 N.
template <int N>
__device__ __forceinline__ float fold(float (&v)[N]) {
  const int lane = threadIdx.x;
#pragma unroll
  for (int n = N / 2; n >= 1; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n];
      const float keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, n);
    }
  }
  float s = v[0];
#pragma unroll
  for (int o = N; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

struct Tile {
  int64_t base, pos;  // element of channel 0 and position index of the lane's first value
  int live;           // positions of the lane that exist
};
template <int VP>
__device__ __forceinline__ Tile tile_of(const NormGeom& g, int64_t u) {
  const int64_t tiles = (g.inner + 32 * VP - 1) / (32 * VP);
  const int64_t n = u / tiles, i = (u - n * tiles) * (32 * VP) + threadIdx.x * VP;
  Tile t;
  t.live = (int)max((int64_t)0, min((int64_t)VP, g.inner - i));
  t.base = n * g.C * g.inner + i;
  t.pos = n * g.inner + i;
  return t;
}
template <typename T, int VP>
__device__ __forceinline__ Vec<T, VP> plane_load(const T* p, bool live) {
  Vec<T, VP> v;
#pragma unroll
  for (int i = 0; i < VP; ++i) v.v[i] = from_f<T>(0.0f);
  if (live) v = *reinterpret_cast<const Vec<T, VP>*>(p);
  return v;
}

constexpr int kPlaneWarps = 16;
constexpr int kCpw = 16;  // channels a warp holds
constexpr int kStaged = kPlaneWarps * kCpw;

// Tiles of up to kStaged channels x 32 lanes of 4 bytes, on their way to shared memory while
// earlier ones are worked on: each thread copies, waits for and reads only its own words, so
// the ring needs no barriers. N tensors, S stages.
template <int N, int S>
struct TileRing {
  uint32_t at;      // this thread's first word
  uint32_t pitch;   // bytes between a thread's words
  __device__ __forceinline__ void init(const void* dsmem) {
    const uint32_t threads = blockDim.x * blockDim.y;
    at = ptx::smem_addr(dsmem) + (threadIdx.y * 32 + threadIdx.x) * 4;
    pitch = threads * 4;
  }
  __device__ __forceinline__ uint32_t word(uint32_t stage, int n, int c) const {
    return at + ((stage * N + n) * kCpw + c) * pitch;
  }
  template <typename T>
  __device__ __forceinline__ void ask(uint32_t stage, int n, const T* p, int64_t step, int C,
                                      bool live) const {
    const int warps = blockDim.y;
#pragma unroll
    for (int c = 0; c < kCpw; ++c) {
      const int ch = c * warps + threadIdx.y;
      const bool ok = live && ch < C;
      ptx::cp_async4(word(stage, n, c), ok ? p + ch * step : p, ok ? 4 : 0);
    }
  }
};

// The positions of a lane: one f32, or two that the packed f32 instructions work on at once.
template <int VP>
struct Lane;
template <>
struct Lane<1> {
  using V = float;
  static __device__ __forceinline__ V all(float x) { return x; }
  static __device__ __forceinline__ V add(V a, V b) { return a + b; }
  static __device__ __forceinline__ V mul(V a, V b) { return a * b; }
  static __device__ __forceinline__ V fma(V a, V b, V c) { return fmaf(a, b, c); }
  static __device__ __forceinline__ float sum(V a) { return a; }
  static __device__ __forceinline__ float at(V a, int) { return a; }
  static __device__ __forceinline__ V from(const float (&f)[1]) { return f[0]; }
};
template <>
struct Lane<2> {
  using V = uint64_t;
  static __device__ __forceinline__ V all(float x) { return pair(x, x); }
  static __device__ __forceinline__ V add(V a, V b) { return add2(a, b); }
  static __device__ __forceinline__ V mul(V a, V b) { return mul2(a, b); }
  static __device__ __forceinline__ V fma(V a, V b, V c) { return fma2(a, b, c); }
  static __device__ __forceinline__ float sum(V a) { return low(a) + high(a); }
  static __device__ __forceinline__ float at(V a, int i) { return i ? high(a) : low(a); }
  static __device__ __forceinline__ V from(const float (&f)[2]) { return pair(f[0], f[1]); }
};
// A 4-byte word of T as the lane's values, and back.
template <typename T, int VP>
__device__ __forceinline__ typename Lane<VP>::V lane_get(uint32_t word) {
  const Vec<T, VP> v = *reinterpret_cast<const Vec<T, VP>*>(&word);
  float f[VP];
#pragma unroll
  for (int i = 0; i < VP; ++i) f[i] = to_f(v.v[i]);
  return Lane<VP>::from(f);
}
template <typename T, int VP>
__device__ __forceinline__ void lane_put(T* p, typename Lane<VP>::V a) {
  Vec<T, VP> v;
#pragma unroll
  for (int i = 0; i < VP; ++i) v.v[i] = from_f<T>(Lane<VP>::at(a, i));
  *reinterpret_cast<Vec<T, VP>*>(p) = v;
}
constexpr int kTileFwdStages = 3, kTileBwdStages = 2;

// The parameters of the block's channels in shared memory, as f32.
template <int STRIDE>
__device__ __forceinline__ void stage_params(float* dst, const void* p, float none,
                                             const NormGeom& g) {
  for (int c = threadIdx.y * 32 + threadIdx.x; c < kStaged; c += blockDim.y * 32)
    dst[c * STRIDE] = p && c < g.C ? param_at(p, g.param_f32, c, g.dtype) : none;
}

template <typename T, int VP>
__global__ void __launch_bounds__(kPlaneWarps * 32, 2)
    norm_tiles_forward(const NormGeom g, int64_t tiles) {
  extern __shared__ __align__(16) uint8_t dsmem[];
  __shared__ float red[kPlaneWarps * VP * 32];
  __shared__ float2 wb[kStaged];
  using L = Lane<VP>;
  constexpr int S = kTileFwdStages;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int warps = blockDim.y, C = (int)g.C;
  const int64_t step = g.inner;
  const float inv = 1.0f / (float)C;
  // channels of this warp that exist: the first `mine` of its kCpw
  const int mine = (C - (int)threadIdx.y + warps - 1) / warps;
  TileRing<1, S> ring;
  ring.init(dsmem);
  auto ask = [&](int64_t u, uint32_t stage) {
    if (u < tiles) {
      const Tile k = tile_of<VP>(g, u);
      ring.ask(stage, 0, (const T*)g.x + (k.live ? k.base : 0), step, C, k.live);
    }
    ptx::cp_async_commit();
  };
  for (int i = 0; i < S - 1; ++i) ask(blockIdx.x + (int64_t)i * gridDim.x, i);
  stage_params<2>(&wb[0].x, g.w, 1.0f, g);
  stage_params<2>(&wb[0].y, g.b, 0.0f, g);
  uint32_t stage = 0;
  for (int64_t u = blockIdx.x; u < tiles; u += gridDim.x) {
    ask(u + (int64_t)(S - 1) * gridDim.x, (stage + S - 1) % S);
    ptx::cp_async_wait<S - 1>();
    const Tile k = tile_of<VP>(g, u);
    typename L::V f[kCpw], acc = L::all(0.0f);
    const uint32_t word = ring.word(stage, 0, 0);
#pragma unroll
    for (int c = 0; c < kCpw; ++c) {  // channels that do not exist arrived as zeros
      f[c] = lane_get<T, VP>(ptx::ld_shared_u32(word + c * ring.pitch));
      acc = L::add(acc, f[c]);
    }
    float m[VP], r[VP];
#pragma unroll
    for (int i = 0; i < VP; ++i) m[i] = L::at(acc, i);
    plane_sum<VP>(m, red, warps);
#pragma unroll
    for (int i = 0; i < VP; ++i) m[i] = -m[i] * inv;
    const typename L::V nm = L::from(m);
    acc = L::all(0.0f);
    if (mine == kCpw) {
#pragma unroll
      for (int c = 0; c < kCpw; ++c) {
        f[c] = L::add(f[c], nm);
        acc = L::fma(f[c], f[c], acc);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kCpw; ++c)
        if (c < mine) {
          f[c] = L::add(f[c], nm);
          acc = L::fma(f[c], f[c], acc);
        }
    }
#pragma unroll
    for (int i = 0; i < VP; ++i) r[i] = L::at(acc, i);
    plane_sum<VP>(r, red, warps);
#pragma unroll
    for (int i = 0; i < VP; ++i) r[i] = rsqrtf(r[i] * inv + g.eps);
    if (k.live) {
      if (threadIdx.y == 0) {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          if (g.mean) g.mean[k.pos + i] = -m[i];
          if (g.rstd) g.rstd[k.pos + i] = r[i];
        }
      }
      const typename L::V rr = L::from(r);
      T* y = (T*)g.y + k.base + threadIdx.y * step;
#pragma unroll
      for (int c = 0; c < kCpw; ++c, y += warps * step) {
        if (c >= mine) break;
        const float2 p = wb[c * warps + threadIdx.y];
        lane_put<T, VP>(y, L::fma(L::mul(f[c], rr), L::all(p.x), L::all(p.y)));
      }
    }
    stage = (stage + 1) % S;
  }
}

// A warp folds the sums of its kCpw channels over its lanes; lane l keeps those of channel l
// in registers to the end.
template <typename T, int VP>
__global__ void __launch_bounds__(kPlaneWarps * 32, 1)
    norm_tiles_backward(const NormGeom g, int64_t tiles) {
  extern __shared__ __align__(16) uint8_t dsmem[];
  __shared__ float red[kPlaneWarps * 2 * VP * 32], w[kStaged];
  constexpr int S = kTileBwdStages;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int warps = blockDim.y, lane = threadIdx.x, C = (int)g.C;
  const int64_t step = g.inner;
  const float inv = 1.0f / (float)C;
  const int mine = (C - (int)threadIdx.y + warps - 1) / warps;
  using L = Lane<VP>;
  TileRing<2, S> ring;
  ring.init(dsmem);
  auto ask = [&](int64_t u, uint32_t stage) {
    if (u < tiles) {
      const Tile k = tile_of<VP>(g, u);
      ring.ask(stage, 0, (const T*)g.x + (k.live ? k.base : 0), step, C, k.live);
      ring.ask(stage, 1, (const T*)g.dy + (k.live ? k.base : 0), step, C, k.live);
    }
    ptx::cp_async_commit();
  };
  ask(blockIdx.x, 0);
  stage_params<1>(w, g.w, 1.0f, g);
  __syncthreads();
  float aw = 0.0f, ab = 0.0f;
  uint32_t stage = 0;
  for (int64_t u = blockIdx.x; u < tiles; u += gridDim.x) {
    const Tile k = tile_of<VP>(g, u);
    float m[VP], r[VP], s[2 * VP];
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      m[i] = k.live ? -g.mean[k.pos + i] : 0.0f;
      r[i] = k.live ? g.rstd[k.pos + i] : 0.0f;
    }
    ask(u + gridDim.x, stage ^ 1);
    const typename L::V nm = L::from(m), rr = L::from(r);
    ptx::cp_async_wait<S - 1>();
    const uint32_t wx = ring.word(stage, 0, 0), wd = ring.word(stage, 1, 0);
    typename L::V s1 = L::all(0.0f), s2 = L::all(0.0f);
    float p[kCpw], q[kCpw];
#pragma unroll
    for (int c = 0; c < kCpw; ++c) {  // channels that do not exist arrived with dy = 0
      const typename L::V x = lane_get<T, VP>(ptx::ld_shared_u32(wx + c * ring.pitch));
      const typename L::V d = lane_get<T, VP>(ptx::ld_shared_u32(wd + c * ring.pitch));
      const typename L::V wc = L::all(w[c * warps + threadIdx.y]);
      const typename L::V h = L::mul(L::add(x, nm), rr), k2 = L::mul(d, wc);
      p[c] = L::sum(L::mul(d, h));
      q[c] = L::sum(d);
      s1 = L::add(s1, k2);
      s2 = L::fma(k2, h, s2);
    }
    if (g.part) {
      aw += fold<kCpw>(p);
      ab += fold<kCpw>(q);
    }
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      s[i] = L::at(s1, i);
      s[VP + i] = L::at(s2, i);
    }
    plane_sum<2 * VP>(s, red, warps);
    if (k.live) {
      float a1[VP], a2[VP];
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        a1[i] = -s[i] * inv;
        a2[i] = -s[VP + i] * inv;
      }
      const typename L::V n1 = L::from(a1), n2 = L::from(a2);
      T* dx = (T*)g.y + k.base + threadIdx.y * step;
#pragma unroll
      for (int c = 0; c < kCpw; ++c, dx += warps * step) {
        if (c >= mine) break;
        const typename L::V x = lane_get<T, VP>(ptx::ld_shared_u32(wx + c * ring.pitch));
        const typename L::V d = lane_get<T, VP>(ptx::ld_shared_u32(wd + c * ring.pitch));
        const typename L::V h = L::mul(L::add(x, nm), rr);
        const typename L::V t = L::fma(d, L::all(w[c * warps + threadIdx.y]), n1);
        lane_put<T, VP>(dx, L::mul(L::fma(h, n2, t), rr));
      }
    }
    stage ^= 1;
  }
  const int ch = lane * warps + threadIdx.y;
  if (g.part && lane < kCpw && ch < C) {
    float* part = g.part + (int64_t)blockIdx.x * 2 * C;
    part[ch] = aw;
    part[C + ch] = ab;
  }
}

// Planes that no 4-byte lanes fit or with more than kStaged channels: the channels are walked
// kCpw a warp at a time in each pass, from L2 after the first.
template <typename T, int VP>
__global__ void __launch_bounds__(kPlaneWarps * 32, 1) norm_planes_forward(const NormGeom g) {
  __shared__ float red[kPlaneWarps * VP * 32];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int C = (int)g.C;
  const Tile k = tile_of<VP>(g, blockIdx.x);
  const T* x = (const T*)g.x + k.base;
  T* y = (T*)g.y + k.base;
  const int64_t step = g.inner;
  const float inv = 1.0f / (float)C;
  Vec<T, VP> v[kCpw];
  auto at = [&](int c0, int c) { return c0 + c * kPlaneWarps + (int)threadIdx.y; };
  auto fetch = [&](int c0) {
#pragma unroll
    for (int c = 0; c < kCpw; ++c)
      v[c] = plane_load<T, VP>(x + at(c0, c) * step, k.live && at(c0, c) < C);
  };
  float m[VP], r[VP];
#pragma unroll
  for (int i = 0; i < VP; ++i) m[i] = r[i] = 0.0f;
  for (int c0 = 0; c0 < C; c0 += kStaged) {
    fetch(c0);
#pragma unroll
    for (int c = 0; c < kCpw; ++c)
#pragma unroll
      for (int i = 0; i < VP; ++i) m[i] += to_f(v[c].v[i]);
  }
  plane_sum<VP>(m, red, kPlaneWarps);
#pragma unroll
  for (int i = 0; i < VP; ++i) m[i] *= inv;
  for (int c0 = 0; c0 < C; c0 += kStaged) {
    fetch(c0);
#pragma unroll
    for (int c = 0; c < kCpw; ++c)
      if (at(c0, c) < C)
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          const float d = to_f(v[c].v[i]) - m[i];
          r[i] = fmaf(d, d, r[i]);
        }
  }
  plane_sum<VP>(r, red, kPlaneWarps);
#pragma unroll
  for (int i = 0; i < VP; ++i) r[i] = rsqrtf(r[i] * inv + g.eps);
  if (!k.live) return;
  if (threadIdx.y == 0) {
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      if (g.mean) g.mean[k.pos + i] = m[i];
      if (g.rstd) g.rstd[k.pos + i] = r[i];
    }
  }
  for (int c0 = 0; c0 < C; c0 += kStaged) {
    fetch(c0);
#pragma unroll
    for (int c = 0; c < kCpw; ++c) {
      const int ch = at(c0, c);
      if (ch >= C) break;
      const float w = g.w ? param_at(g.w, g.param_f32, ch, g.dtype) : 1.0f;
      const float b = g.b ? param_at(g.b, g.param_f32, ch, g.dtype) : 0.0f;
      float o[VP];
#pragma unroll
      for (int i = 0; i < VP; ++i) o[i] = fmaf((to_f(v[c].v[i]) - m[i]) * r[i], w, b);
      store_f<T, VP>(y + ch * step, o);
    }
  }
}

// The folded channel sums go to the block's own partial sums in the workspace.
template <typename T, int VP>
__global__ void __launch_bounds__(kPlaneWarps * 32, 1)
    norm_planes_backward(const NormGeom g, int64_t tiles) {
  __shared__ float red[kPlaneWarps * 2 * VP * 32];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int lane = threadIdx.x, C = (int)g.C;
  const int64_t step = g.inner;
  const float inv = 1.0f / (float)C;
  auto at = [&](int c0, int c) { return c0 + c * kPlaneWarps + (int)threadIdx.y; };
  float* part = g.part ? g.part + (int64_t)blockIdx.x * 2 * C : nullptr;
  for (int64_t u = blockIdx.x; u < tiles; u += gridDim.x) {
    const Tile k = tile_of<VP>(g, u);
    const T* x = (const T*)g.x + k.base;
    const T* dy = (const T*)g.dy + k.base;
    T* dx = (T*)g.y + k.base;
    Vec<T, VP> vx[kCpw], vd[kCpw];
    auto fetch = [&](int c0) {
#pragma unroll
      for (int c = 0; c < kCpw; ++c) {
        const bool ok = k.live && at(c0, c) < C;
        vx[c] = plane_load<T, VP>(x + at(c0, c) * step, ok);
        vd[c] = plane_load<T, VP>(dy + at(c0, c) * step, ok);
      }
    };
    float m[VP], r[VP], s[2 * VP];
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      m[i] = k.live ? g.mean[k.pos + i] : 0.0f;
      r[i] = k.live ? g.rstd[k.pos + i] : 0.0f;
      s[i] = s[VP + i] = 0.0f;
    }
    for (int c0 = 0; c0 < C; c0 += kStaged) {
      fetch(c0);
      float p[kCpw];
#pragma unroll
      for (int c = 0; c < kCpw; ++c) {
        const int ch = at(c0, c);
        const float w = g.w && ch < C ? param_at(g.w, g.param_f32, ch, g.dtype) : 1.0f;
        p[c] = 0.0f;
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          const float d = to_f(vd[c].v[i]), h = (to_f(vx[c].v[i]) - m[i]) * r[i];
          p[c] = fmaf(d, h, p[c]);
          s[i] = fmaf(d, w, s[i]);
          s[VP + i] = fmaf(d * w, h, s[VP + i]);
        }
      }
      if (part) {
        const float a = fold<kCpw>(p);
#pragma unroll
        for (int c = 0; c < kCpw; ++c) {
          p[c] = 0.0f;
#pragma unroll
          for (int i = 0; i < VP; ++i) p[c] += to_f(vd[c].v[i]);
        }
        const float b = fold<kCpw>(p);
        if (lane < kCpw && at(c0, lane) < C) {
          float* q = part + at(c0, lane);
          const bool first = u == blockIdx.x;
          q[0] = first ? a : q[0] + a;
          q[C] = first ? b : q[C] + b;
        }
      }
    }
    plane_sum<2 * VP>(s, red, kPlaneWarps);
#pragma unroll
    for (int i = 0; i < 2 * VP; ++i) s[i] *= inv;
    for (int c0 = 0; c0 < C; c0 += kStaged) {
      fetch(c0);
      if (!k.live) continue;
#pragma unroll
      for (int c = 0; c < kCpw; ++c) {
        const int ch = at(c0, c);
        if (ch >= C) break;
        const float w = g.w ? param_at(g.w, g.param_f32, ch, g.dtype) : 1.0f;
        float o[VP];
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          const float h = (to_f(vx[c].v[i]) - m[i]) * r[i];
          o[i] = r[i] * (to_f(vd[c].v[i]) * w - s[i] - h * s[VP + i]);
        }
        store_f<T, VP>(dx + ch * step, o);
      }
    }
  }
}

// ------------------------------------------------------------------------------ join

// dw (blockIdx.y 0) and db (1) from the blocks' partial sums: 32 interleaved sequences a
// channel, then those in order.
__global__ void __launch_bounds__(1024)
    norm_dparam_join(const float* __restrict__ part, void* dw, void* db, int dtype, int f32,
                     int64_t C, int blocks) {
  __shared__ float red[32][32];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  void* out = blockIdx.y ? db : dw;
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < C && out) {
#pragma unroll 8
    for (int i = threadIdx.y; i < blocks; i += 32) s += part[(2 * (int64_t)i + blockIdx.y) * C + c];
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y || c >= C || !out) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
  if (f32) ((float*)out)[c] = s;
  else if (dtype == FCONV_F16) ((__half*)out)[c] = from_f<__half>(s);
  else ((__nv_bfloat16*)out)[c] = from_f<__nv_bfloat16>(s);
}

// ------------------------------------------------------------------------------ host side

enum Kind { kRows, kLongRows, kTiles, kPlanes };
constexpr int kMaxRow = 8192;

// Positions a lane: 4 bytes where the plane length and the addresses allow it.
int plane_vp(const fconv_norm_desc& d, const NormArgs& a) {
  if (d.dtype == FCONV_F32 || d.inner % 2) return 1;
  const uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.dy;
  return bits & 3 ? 1 : 2;
}
Kind kind_of(const fconv_norm_desc& d, int vp) {
  if (d.inner == 1) return d.channels <= kMaxRow ? kRows : kLongRows;
  return d.channels <= kStaged && (d.dtype == FCONV_F32 || vp == 2) ? kTiles : kPlanes;
}

// E elements a thread and threads a row. 16-bit rows of up to 1024 channels fit a warp (no
// barriers). A thread that also keeps two rows in flight and two partial sums has registers for
// 16 values of 32 bits, and for 8 when every element is a load of its own (vec 1).
void row_shape(int64_t C, int vec, int* e, int* tpr) {
  const int64_t warp = vec == 8 ? 1024 : vec == 4 ? 512 : 256;
  if (C <= warp) {
    *tpr = 32;
    *e = C <= 256 ? 8 : C <= 512 ? 16 : C <= 768 ? 24 : 32;
  } else {
    *tpr = C <= 4096 ? 256 : 512;
    *e = C <= 2048 ? 8 : 16;
  }
}
int row_vec(const fconv_norm_desc& d, const NormArgs& a) {
  const int v = d.dtype == FCONV_F32 ? 4 : 8;
  const uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.dy;
  return d.channels % v == 0 && (bits & 15) == 0 ? v : 1;
}

int64_t plane_tiles(const fconv_norm_desc& d, int vp) {
  return d.outer * ((d.inner + 32 * vp - 1) / (32 * vp));
}
// Tiles: warps of a block, its shared memory and how many an SM holds (of 228 KB, 8 KB of
// which are the blocks' own and static).
int tile_warps(const fconv_norm_desc& d) { return (int)((d.channels + kCpw - 1) / kCpw); }
size_t tile_smem(const fconv_norm_desc& d, bool bwd) {
  return (size_t)(bwd ? 2 * kTileBwdStages : kTileFwdStages) * kCpw * tile_warps(d) * 128;
}
int64_t tile_blocks(const fconv_norm_desc& d, bool bwd) {
  const int64_t threads = (bwd ? 768 : 1024) / (32 * tile_warps(d));
  const int64_t room = 180 * 1024 / (int64_t)tile_smem(d, bwd);
  const int64_t n = threads < room ? threads : room;
  return n < 1 ? 1 : n > 16 ? 16 : n;
}

// Blocks of the backward pass over rows of `vec` elements a load, or over planes of `vp`
// positions a lane (each block writes one partial sum).
int64_t backward_blocks(const fconv_norm_desc& d, int sms, int vec, int vp) {
  int64_t work, per_sm;
  switch (kind_of(d, vp)) {
    case kRows: {
      int e, tpr;
      row_shape(d.channels, vec, &e, &tpr);
      const int nt = tpr == 32 ? 128 : tpr;
      work = (d.outer * tpr + nt - 1) / nt;
      per_sm = row_blocks(e, tpr, true);
      break;
    }
    case kLongRows:
      work = d.outer;
      per_sm = 4;
      break;
    case kTiles:
      work = plane_tiles(d, vp);
      per_sm = tile_blocks(d, true);
      break;
    default:
      work = plane_tiles(d, vp);
      per_sm = 1;
      break;
  }
  if (per_sm < 1) per_sm = 1;
  int64_t n = work < per_sm * sms ? work : per_sm * sms;
  return n < 1 ? 1 : n;
}

template <typename T, int VEC, bool BWD, int E, int TPR>
int rows_launch(const NormGeom& g, int64_t blocks, cudaStream_t s) {
  constexpr int NT = row_threads<TPR>();
  auto kern = BWD ? norm_rows_backward<T, VEC, E, TPR> : norm_rows_forward<T, VEC, E, TPR>;
  size_t smem = 0;
  if (VEC > 1)
    smem = BWD ? feed_bytes<2, kBwdStages>(NT / TPR, g.C * sizeof(T))
               : feed_bytes<1, kFwdStages>(NT / TPR, g.C * sizeof(T));
  const int e = allow_smem((const void*)kern, smem);
  if (e) return e;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(NT), smem, s, g);
}

template <typename T, int VEC, bool BWD>
int rows_t(const NormGeom& g, int64_t blocks, int sms, cudaStream_t s) {
  int e, tpr;
  row_shape(g.C, VEC, &e, &tpr);
  const int nt = tpr == 32 ? 128 : tpr;
  if (!BWD) {
    const int64_t work = (g.outer * tpr + nt - 1) / nt;
    const int64_t cap = (int64_t)row_blocks(e, tpr, false) * sms;
    blocks = work < cap ? work : cap;
  }
#define FCONV_ROW(E_, TPR_) \
  if (e == E_ && tpr == TPR_) return rows_launch<T, VEC, BWD, E_, TPR_>(g, blocks, s)
  FCONV_ROW(8, 32);
  if constexpr (VEC > 1) FCONV_ROW(16, 32);
  if constexpr (VEC == 8) {
    FCONV_ROW(24, 32);
    FCONV_ROW(32, 32);
  }
  FCONV_ROW(8, 256);
  FCONV_ROW(16, 256);
  FCONV_ROW(16, 512);
#undef FCONV_ROW
  return (int)cudaErrorInvalidValue;
}

template <typename T, bool BWD>
int norm_t(const fconv_norm_desc& d, int sms, const NormArgs& a, cudaStream_t s) {
  NormGeom g{};
  g.x = a.x;
  g.dy = a.dy;
  g.w = a.w;
  g.b = a.b;
  g.y = a.y;
  g.mean = a.mean;
  g.rstd = a.rstd;
  g.part = a.dw || a.db ? a.ws : nullptr;
  g.outer = d.outer;
  g.C = d.channels;
  g.inner = d.inner;
  g.dtype = d.dtype;
  g.param_f32 = d.param_dtype == FCONV_F32;
  g.eps = d.eps;
  const int vp = plane_vp(d, a);
  const Kind kind = kind_of(d, vp);
  const int64_t most = backward_blocks(d, sms, row_vec(d, a), vp);
  if (kind == kRows) {
    if (row_vec(d, a) > 1) return rows_t<T, 16 / sizeof(T), BWD>(g, most, sms, s);
    return rows_t<T, 1, BWD>(g, most, sms, s);
  }
  if (kind == kLongRows) {
    if (BWD) return launch_pdl(norm_long_backward<T>, dim3((unsigned)most), dim3(kLong), 0, s, g);
    return launch_pdl(norm_long_forward<T>, dim3((unsigned)d.outer), dim3(kLong), 0, s, g);
  }
  const int64_t tiles = plane_tiles(d, vp);
  if (!grid_ok(tiles)) return (int)cudaErrorInvalidValue;
  if (kind == kTiles) {
    constexpr int VP = 4 / sizeof(T);
    auto kern = BWD ? norm_tiles_backward<T, VP> : norm_tiles_forward<T, VP>;
    const size_t smem = tile_smem(d, BWD);
    const int e = allow_smem((const void*)kern, smem);
    if (e) return e;
    const int64_t cap = tile_blocks(d, BWD) * sms;
    return launch_pdl(kern, dim3((unsigned)(tiles < cap ? tiles : cap)),
                      dim3(32, tile_warps(d)), smem, s, g, tiles);
  }
#define FCONV_PLANE(VP_)                                                                       \
  if (vp == VP_) {                                                                             \
    if (BWD)                                                                                   \
      return launch_pdl(norm_planes_backward<T, VP_>, dim3((unsigned)most),                    \
                        dim3(32, kPlaneWarps), 0, s, g, tiles);                                \
    return launch_pdl(norm_planes_forward<T, VP_>, dim3((unsigned)tiles),                      \
                      dim3(32, kPlaneWarps), 0, s, g);                                         \
  }
  if constexpr (sizeof(T) == 2) {
    FCONV_PLANE(2)
  }
  FCONV_PLANE(1)
#undef FCONV_PLANE
  return (int)cudaErrorInvalidValue;
}

}  // namespace

int read_and_clear_norm_error(cudaStream_t s, unsigned* v) { return read_and_clear_error(s, v); }

size_t norm_workspace(const fconv_norm_desc& d, int sms) {
  // unaligned calls may take more blocks than aligned ones, or fewer
  int64_t n = 0;
  for (int vec : {1, d.dtype == FCONV_F32 ? 4 : 8})
    for (int vp : {1, 2}) {
      const int64_t b = backward_blocks(d, sms, vec, vp);
      n = b > n ? b : n;
    }
  return (size_t)n * 2 * (size_t)d.channels * sizeof(float);
}

int launch_norm_forward(const fconv_norm_desc& d, int sms, const NormArgs& a, cudaStream_t s) {
#define FCONV_M(T) return norm_t<T, false>(d, sms, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

int launch_norm_backward(const fconv_norm_desc& d, int sms, const NormArgs& a, cudaStream_t s) {
  int e = 0;
  if (d.outer > 0) {
#define FCONV_M(T) e = norm_t<T, true>(d, sms, a, s)
    FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
  }
  if (e || (!a.dw && !a.db)) return e;
  // without rows there are no partial sums and both gradients are zero
  const int blocks =
      d.outer > 0 ? (int)backward_blocks(d, sms, row_vec(d, a), plane_vp(d, a)) : 0;
  return launch_pdl(norm_dparam_join, dim3((unsigned)((d.channels + 31) / 32), 2), dim3(32, 32), 0,
                    s, (const float*)a.ws, a.dw, a.db, d.dtype, (int)(d.param_dtype == FCONV_F32),
                    d.channels, blocks);
}

}  // namespace ops
}  // namespace fconv
