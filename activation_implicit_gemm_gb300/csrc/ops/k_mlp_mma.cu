// The gated feed-forward block without tcgen05 (include/fconv_ops.h), every type, size, stride and
// address: all calls of a plan made for it. Others come here only with an f16 or bf16 operand in rows
// that TMA takes at an address off 16 bytes, which it does not (operands in other rows, and f32, are
// copied first), and without tokens, for gradients of zero. 16384 x 4096 x 10240 in bf16, forward:
// 122 ms, against 2.4 ms on tcgen05.
//
// Every product is one kernel, D = A B^T with any strides of both, on m16n8k8 TF32 instructions.
// An f32 value is hi (rounded to TF32) + lo; a product is lo hi + hi lo + hi hi, which drops about
// 2^-23 of it, and 16-bit values are TF32 values as they are. The instructions' sums round towards
// zero, so they run over 16 products only and are then added in plain f32.
//
// A block owns 128 x 64 of D, a warp 32 x 32 in registers. Tiles are split on their way into
// shared memory, once for all warps that read them, as pairs (hi, lo) in rows of 20: both the
// pairs of f32 and the single values of 16-bit types are then read without bank conflicts. The
// next tile's loads are on their way while the current one's products run. In the gated product
// the 64 columns are groups of 8 of the gate and 8 of the up projection in turn, so that a thread
// has both values of its outputs.
#include "mlp_math.cuh"
#include "split_tf32.cuh"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kM = 128, kN = 64, kK = 16, kPitch = kK + 4, kThreads = 256;

enum { kPlain, kGated, kGrad };

struct Operand {
  const void* p;
  int64_t row, k;  // strides in elements
};
struct Product {
  Operand a[2], b[2];  // the terms of a sum; with kGated b holds the gate and the up weights
  int terms;
  int64_t M, N, K;
  const void* bias[2];
  void* out[3];  // rows of out_row elements; kGrad: dg, du and h
  int64_t out_row;
  float* saved;
  int64_t quads;
  int act;
  float alpha;
};

template <bool SPLIT>
struct Cell;
template <>
struct Cell<true> {
  using Type = float2;
  static __device__ __forceinline__ float2 of(float v) {
    uint32_t hi, lo;
    split_tf32(v, hi, lo);
    return make_float2(__uint_as_float(hi), __uint_as_float(lo));
  }
};
template <>
struct Cell<false> {
  using Type = float;
  static __device__ __forceinline__ float of(float v) { return v; }
};
__device__ __forceinline__ uint32_t hi_of(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t hi_of(float2 v) { return __float_as_uint(v.x); }
__device__ __forceinline__ uint32_t lo_of(float) { return 0; }
__device__ __forceinline__ uint32_t lo_of(float2 v) { return __float_as_uint(v.y); }

// A thread's part of a tile of ROWS x kK on its way from global memory.
template <typename T, int ROWS>
struct Part {
  float v[ROWS * kK / kThreads];
  // threads run along the axis that is contiguous
  static __device__ __forceinline__ int row_of(int i, bool along_k) {
    return along_k ? (int)threadIdx.x / kK + i * (kThreads / kK) : (int)threadIdx.x % ROWS;
  }
  static __device__ __forceinline__ int k_of(int i, bool along_k) {
    return along_k ? (int)threadIdx.x % kK
                   : (int)threadIdx.x / ROWS + i * (kThreads / ROWS);
  }
  template <typename Row>
  __device__ __forceinline__ void load(int64_t k0, int64_t K, bool along_k, Row row) {
#pragma unroll
    for (int i = 0; i < ROWS * kK / kThreads; ++i) {
      const int64_t k = k0 + k_of(i, along_k);
      const T* p = row(row_of(i, along_k), k);
      v[i] = p && k < K ? to_f(*p) : 0.0f;
    }
  }
  template <bool SPLIT>
  __device__ __forceinline__ void store(typename Cell<SPLIT>::Type* tile, bool along_k) const {
#pragma unroll
    for (int i = 0; i < ROWS * kK / kThreads; ++i)
      tile[row_of(i, along_k) * kPitch + k_of(i, along_k)] = Cell<SPLIT>::of(v[i]);
  }
};

template <typename T, int EPI>
__global__ void __launch_bounds__(kThreads, 2) mlp_mma(const __grid_constant__ Product q) {
  constexpr bool SPLIT = sizeof(T) == 4;
  using C = typename Cell<SPLIT>::Type;
  extern __shared__ float4 smem4[];
  C* as = reinterpret_cast<C*>(smem4);  // two stages of A, then of B
  C* bs = as + 2 * kM * kPitch;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  constexpr int kCols = EPI == kGated ? kN / 2 : kN;  // columns of D
  const int64_t ntiles = (q.N + kCols - 1) / kCols;
  const int64_t m0 = blockIdx.x / ntiles * kM, n0 = blockIdx.x % ntiles * kCols;
  const int64_t ksteps = (q.K + kK - 1) / kK;
  const int64_t steps = ksteps * (EPI == kPlain ? q.terms : 1);

  Part<T, kM> pa;
  Part<T, kN> pb;
  auto load = [&](int64_t step) {
    const int term = EPI == kPlain && step >= ksteps ? 1 : 0;
    const int64_t k0 = (step - term * ksteps) * kK;
    const Operand& a = q.a[term];
    pa.load(k0, q.K, a.k == 1, [&](int r, int64_t k) -> const T* {
      const int64_t m = m0 + r;
      return m < q.M ? (const T*)a.p + m * a.row + k * a.k : nullptr;
    });
    const bool along = q.b[term].k == 1;
    pb.load(k0, q.K, along, [&](int r, int64_t k) -> const T* {
      const int64_t n = EPI == kGated ? n0 + (r >> 4) * 8 + (r & 7) : n0 + r;
      const Operand& b = q.b[EPI == kGated ? (r >> 3) & 1 : term];
      return n < q.N ? (const T*)b.p + n * b.row + k * b.k : nullptr;
    });
  };
  auto store = [&](int64_t step) {
    const int term = EPI == kPlain && step >= ksteps ? 1 : 0, stage = (int)(step & 1);
    pa.template store<SPLIT>(as + stage * kM * kPitch, q.a[term].k == 1);
    pb.template store<SPLIT>(bs + stage * kN * kPitch, q.b[term].k == 1);
  };

  const int warp = threadIdx.x >> 5, gr = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const int wm = (warp >> 1) * 32, wn = (warp & 1) * 32;
  float acc[2][4][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.0f;
  if (steps > 0) {
    load(0);
    store(0);
  }
  __syncthreads();
  for (int64_t step = 0; step < steps; ++step) {
    if (step + 1 < steps) load(step + 1);
    const C* a = as + (step & 1) * kM * kPitch + (wm + gr) * kPitch + t;
    const C* b = bs + (step & 1) * kN * kPitch + (wn + gr) * kPitch + t;
    uint32_t bh[2][4][2], bl[2][4][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const C v = b[n * 8 * kPitch + k * 8 + e * 4];
          bh[k][n][e] = hi_of(v);
          bl[k][n][e] = lo_of(v);
        }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float z[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[n][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const C v = a[(i * 16 + (e & 1) * 8) * kPitch + k * 8 + (e >> 1) * 4];
          ah[e] = hi_of(v);
          al[e] = lo_of(v);
        }
        if (SPLIT) {
#pragma unroll
          for (int n = 0; n < 4; ++n) mma_tf32(z[n], al, bh[k][n]);
#pragma unroll
          for (int n = 0; n < 4; ++n) mma_tf32(z[n], ah, bl[k][n]);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) mma_tf32(z[n], ah, bh[k][n]);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][n][e] += z[n][e];
    }
    if (step + 1 < steps) store(step + 1);
    __syncthreads();
  }

#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t row = m0 + wm + i * 16 + half * 8 + gr;
      if (row >= q.M) continue;
#pragma unroll
      for (int n = 0; n < 4; n += EPI == kGated ? 2 : 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = (int)n0 + (EPI == kGated ? (wn + n * 8) / 2 : wn + n * 8) + 2 * t + e;
          if (col >= q.N) continue;
          const int64_t at = row * q.out_row + col;
          const float v = acc[i][n][half * 2 + e];
          if (EPI == kPlain) {
            const float bias = q.bias[0] ? to_f(((const T*)q.bias[0])[col]) : 0.0f;
            ((T*)q.out[0])[at] = from_f<T>(v + bias);
          } else if (EPI == kGated) {
            float g = v, u = acc[i][(n + 1) & 3][half * 2 + e], unused;
            if (q.bias[0]) g += to_f(((const T*)q.bias[0])[col]);
            if (q.bias[1]) u += to_f(((const T*)q.bias[1])[col]);
            if (q.saved) {
              q.saved[saved_index(row, col, q.quads, 0)] = g;
              q.saved[saved_index(row, col, q.quads, 1)] = u;
            }
            if (q.out[0])
              ((T*)q.out[0])[at] = from_f<T>(act_of<false>(q.act, q.alpha, g, unused) * u);
          } else {
            const float g = q.saved[saved_index(row, col, q.quads, 0)];
            const float u = q.saved[saved_index(row, col, q.quads, 1)];
            float slope;
            const float a = act_of<true>(q.act, q.alpha, g, slope);
            ((T*)q.out[0])[at] = from_f<T>(v * u * slope);
            ((T*)q.out[1])[at] = from_f<T>(v * a);
            ((T*)q.out[2])[at] = from_f<T>(a * u);
          }
        }
    }
}

template <typename T, int EPI>
int run(const Product& q, cudaStream_t s) {
  constexpr int kCols = EPI == kGated ? kN / 2 : kN;
  const long long blocks = ((q.M + kM - 1) / kM) * ((q.N + kCols - 1) / kCols);
  if (blocks == 0) return 0;
  if (!grid_ok(blocks)) return (int)cudaErrorInvalidValue;
  const size_t smem = 2 * (kM + kN) * kPitch * (sizeof(T) == 4 ? 8 : 4);
  const void* kernel = (const void*)mlp_mma<T, EPI>;
  if (const int e = allow_smem(kernel, smem)) return e;
  return launch_pdl(mlp_mma<T, EPI>, dim3((unsigned)blocks), dim3(kThreads), smem, s, q);
}

// The workspace: h, and in the backward pass dg and du, rows of `hidden` values; then the sums.
size_t matrix_bytes(const fconv_mlp_desc& d) {
  const size_t n = (size_t)d.tokens * (size_t)d.hidden * (d.dtype == FCONV_F32 ? 4 : 2);
  return (n + 255) / 256 * 256;
}
void* matrix(const fconv_mlp_desc& d, const MlpArgs& a, int i) {
  return (char*)a.ws + i * matrix_bytes(d);
}

// The gated product: h (may be null) and, where `saved` is given, the projections.
template <typename T>
int gated(const fconv_mlp_desc& d, const MlpArgs& a, float* saved, void* h, cudaStream_t s) {
  Product q{};
  q.a[0] = {a.x, d.x_stride, 1};
  q.b[0] = {a.w_gate, d.gate_stride, 1};
  q.b[1] = {a.w_up, d.up_stride, 1};
  q.terms = 1;
  q.M = d.tokens;
  q.N = d.hidden;
  q.K = d.features;
  q.bias[0] = a.b_gate;
  q.bias[1] = a.b_up;
  q.out[0] = h;
  q.out_row = d.hidden;
  q.saved = saved;
  q.quads = (d.hidden + 3) / 4;
  q.act = d.activation;
  q.alpha = d.alpha;
  return run<T, kGated>(q, s);
}

template <typename T>
int forward(const fconv_mlp_desc& d, const MlpArgs& a, cudaStream_t s) {
  void* h = matrix(d, a, 0);
  if (const int e = gated<T>(d, a, a.saved, h, s)) return e;
  Product q{};
  q.a[0] = {h, d.hidden, 1};
  q.b[0] = {a.w_down, d.down_stride, 1};
  q.terms = 1;
  q.M = d.tokens;
  q.N = d.out_features;
  q.K = d.hidden;
  q.bias[0] = a.b_down;
  q.out[0] = a.y;
  q.out_row = d.y_stride;
  return run<T, kPlain>(q, s);
}

template <typename T>
int backward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  void *h = matrix(d, a, 0), *dg = matrix(d, a, 1), *du = matrix(d, a, 2);
  int e = 0;
  if (a.remake) e = gated<T>(d, a, a.saved, nullptr, s);
  Product q{};
  if (!e) {
    q.a[0] = {a.dy, d.dy_stride, 1};
    q.b[0] = {a.w_down, 1, d.down_stride};
    q.terms = 1;
    q.M = d.tokens;
    q.N = d.hidden;
    q.K = d.out_features;
    q.out[0] = dg;
    q.out[1] = du;
    q.out[2] = h;
    q.out_row = d.hidden;
    q.saved = a.saved;
    q.quads = (d.hidden + 3) / 4;
    q.act = d.activation;
    q.alpha = d.alpha;
    e = run<T, kGrad>(q, s);
  }
  if (!e && a.dx) {
    q = Product{};
    q.a[0] = {dg, d.hidden, 1};
    q.a[1] = {du, d.hidden, 1};
    q.b[0] = {a.w_gate, 1, d.gate_stride};
    q.b[1] = {a.w_up, 1, d.up_stride};
    q.terms = 2;
    q.M = d.tokens;
    q.N = d.features;
    q.K = d.hidden;
    q.out[0] = a.dx;
    q.out_row = d.dx_stride;
    e = run<T, kPlain>(q, s);
  }
  // the weights' gradients: sums over tokens
  auto weight = [&](const void* g, int64_t g_row, int64_t m, const void* in, int64_t in_row,
                    int64_t n, void* out) {
    if (e || !out) return;
    q = Product{};
    q.a[0] = {g, 1, g_row};
    q.b[0] = {in, 1, in_row};
    q.terms = 1;
    q.M = m;
    q.N = n;
    q.K = d.tokens;
    q.out[0] = out;
    q.out_row = n;
    e = run<T, kPlain>(q, s);
  };
  weight(dg, d.hidden, d.hidden, a.x, d.x_stride, d.features, a.dw_gate);
  weight(du, d.hidden, d.hidden, a.x, d.x_stride, d.features, a.dw_up);
  weight(a.dy, d.dy_stride, d.out_features, h, d.hidden, d.hidden, a.dw_down);
  if (e) return e;
  const SumsArgs m[3] = {{dg, d.hidden, d.hidden, 0, a.db_gate},
                         {du, d.hidden, d.hidden, 0, a.db_up},
                         {a.dy, d.dy_stride, d.out_features, 0, a.db_down}};
  return launch_column_sums(d.dtype, false, false, m, d.tokens, (float*)matrix(d, a, 3), sms, s);
}

}  // namespace

size_t mlp_saved_bytes(const fconv_mlp_desc& d) {
  return (size_t)saved_floats(d.tokens, d.hidden) * sizeof(float);
}

size_t mlp_simple_workspace(const fconv_mlp_desc& d, bool backward, int sms) {
  if (!backward) return matrix_bytes(d);
  const int64_t cols[3] = {d.hidden, d.hidden, d.out_features};
  return 3 * matrix_bytes(d) + column_sums_workspace(cols, sms);
}

int launch_mlp_simple_forward(const fconv_mlp_desc& d, const MlpArgs& a, cudaStream_t s) {
#define FCONV_M(T) return forward<T>(d, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

int launch_mlp_simple_backward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
#define FCONV_M(T) return backward<T>(d, sms, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
