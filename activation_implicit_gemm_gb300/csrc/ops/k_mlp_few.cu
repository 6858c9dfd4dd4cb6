// The gated feed-forward block for few tokens (include/fconv_ops.h): up to 32, f16 and bf16 with
// sizes and strides of whole 16-byte units.
//
//   h = act(x Wg^T + bg) * (x Wu^T + bu),  y = h Wd^T + bd
// Bound: HBM, every weight is read once for all tokens. Weights go from global memory straight
// into the A operand of m16n8k16 instructions, tokens are the 8 columns of B. Lane (g, t) of a warp
// takes 16 bytes of rows g and g + 8 and of token g, elements 8 t to 8 t + 7 of a step of 32; their
// words 0 and 1 feed one instruction and 2 and 3 another, with the same order of K in both
// operands, so neither has to be moved between lanes. In the gated product rows 0 to 7 are the
// gate's and 8 to 15 the up projection's of the same 8 hidden values.
//
// The eight warps of a block share the same rows and split K; their f32 sums are joined through
// shared memory in a fixed order, then come biases, gate and the one rounding. With more than 8
// tokens a warp takes two row groups, so that tokens are read half as often.
#include "mlp_math.cuh"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

struct Few {
  const void* x;  // tokens x K
  const void* w[2];
  const void* bias[2];
  void* out;      // tokens x N
  float* saved;
  int64_t x_row, w_row[2], out_row, quads;
  int tokens, K, N;
  int act;
  float alpha;
};

__device__ __forceinline__ uint4 load_weight(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
template <typename T>
constexpr bool kIsBf16 = false;
template <>
constexpr bool kIsBf16<__nv_bfloat16> = true;
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kIsBf16<T>) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// NT: groups of 8 tokens. MT: row groups of a warp. U: steps of K whose loads go out together.
template <typename T, bool GATED, int NT, int MT, int U>
__global__ void __launch_bounds__(kThreads, 2) mlp_few(const __grid_constant__ Few q) {
  __shared__ float sums[kWarps][MT * 16][NT * 8 + 1];
  constexpr int kRows = GATED ? 8 : 16;  // outputs of a row group
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows * MT;
  // this lane's rows of weights; rows past the end read the last one, for outputs no one writes
  const T* wp[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int which = GATED ? i : 0;
      const int row = min(n0 + m * kRows + (GATED ? 0 : i * 8) + gr, q.N - 1);
      wp[m][i] = (const T*)q.w[which] + row * q.w_row[which] + t * 8;
    }
  const T* xp[NT];
  bool there[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    there[n] = n * 8 + gr < q.tokens;
    xp[n] = (const T*)q.x + (there[n] ? n * 8 + gr : 0) * q.x_row + t * 8;
  }
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.0f;
  ptx::pdl_wait();
  ptx::pdl_trigger();

  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = warp * 32 * U; k0 < q.K; k0 += kWarps * 32 * U) {
    uint4 w[U][MT][2], x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32;
      const bool in = k + t * 8 < q.K;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) w[u][m][i] = in ? load_weight(wp[m][i] + k) : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        x[u][n] = in && there[n] ? *reinterpret_cast<const uint4*>(xp[n] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 a = w[u][m][0], b = w[u][m][1], c = x[u][n];
          mma<T>(acc[m][n], a.x, b.x, a.y, b.y, c.x, c.y);
          mma<T>(acc[m][n], a.z, b.z, a.w, b.w, c.z, c.w);
        }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sums[warp][m * 16 + gr + (e >> 1) * 8][n * 8 + 2 * t + (e & 1)] = acc[m][n][e];
  __syncthreads();

  // outputs: neighbouring threads have neighbouring rows of one token
  for (int i = threadIdx.x; i < kRows * MT * NT * 8; i += kThreads) {
    const int r = i % (kRows * MT), token = i / (kRows * MT), col = n0 + r;
    if (token >= q.tokens || col >= q.N) continue;
    const int at = GATED ? r / 8 * 16 + r % 8 : r;
    float v = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      v += sums[w][at][token];
      if (GATED) u += sums[w][at + 8][token];
    }
    if (q.bias[0]) v += to_f(((const T*)q.bias[0])[col]);
    if (GATED) {
      if (q.bias[1]) u += to_f(((const T*)q.bias[1])[col]);
      if (q.saved) {
        q.saved[saved_index(token, col, q.quads, 0)] = v;
        q.saved[saved_index(token, col, q.quads, 1)] = u;
      }
      float unused;
      v = act_of<false>(q.act, q.alpha, v, unused) * u;
    }
    ((T*)q.out)[token * q.out_row + col] = from_f<T>(v);
  }
}

template <typename T, bool GATED>
int run(const Few& q, cudaStream_t s) {
  const int rows = GATED ? 8 : 16;
  auto grid = [&](int mt) { return dim3((unsigned)((q.N + rows * mt - 1) / (rows * mt))); };
  if (q.tokens <= 8) return launch_pdl(mlp_few<T, GATED, 1, 1, 4>, grid(1), dim3(kThreads), 0, s, q);
  if (q.tokens <= 16)
    return launch_pdl(mlp_few<T, GATED, 2, 2, 2>, grid(2), dim3(kThreads), 0, s, q);
  return launch_pdl(mlp_few<T, GATED, 4, 2, 2>, grid(2), dim3(kThreads), 0, s, q);
}

template <typename T>
int gated(const fconv_mlp_desc& d, const MlpArgs& a, cudaStream_t s) {
  Few q{};
  q.x = a.x;
  q.w[0] = a.w_gate;
  q.w[1] = a.w_up;
  q.bias[0] = a.b_gate;
  q.bias[1] = a.b_up;
  q.out = a.h;
  q.saved = a.saved;
  q.x_row = d.x_stride;
  q.w_row[0] = d.gate_stride;
  q.w_row[1] = d.up_stride;
  q.out_row = d.hidden;
  q.quads = (d.hidden + 3) / 4;
  q.tokens = (int)d.tokens;
  q.K = (int)d.features;
  q.N = (int)d.hidden;
  q.act = d.activation;
  q.alpha = d.alpha;
  return run<T, true>(q, s);
}

template <typename T>
int down(const fconv_mlp_desc& d, const MlpArgs& a, cudaStream_t s) {
  Few q{};
  q.x = a.h;
  q.w[0] = a.w_down;
  q.bias[0] = a.b_down;
  q.out = a.y;
  q.x_row = d.hidden;
  q.w_row[0] = d.down_stride;
  q.out_row = d.y_stride;
  q.tokens = (int)d.tokens;
  q.K = (int)d.hidden;
  q.N = (int)d.out_features;
  return run<T, false>(q, s);
}

}  // namespace

int launch_mlp_few_gated(const fconv_mlp_desc& d, const MlpArgs& a, cudaStream_t s) {
  return d.dtype == FCONV_BF16 ? gated<__nv_bfloat16>(d, a, s) : gated<__half>(d, a, s);
}

int launch_mlp_few_down(const fconv_mlp_desc& d, const MlpArgs& a, cudaStream_t s) {
  return d.dtype == FCONV_BF16 ? down<__nv_bfloat16>(d, a, s) : down<__half>(d, a, s);
}

}  // namespace ops
}  // namespace fconv
