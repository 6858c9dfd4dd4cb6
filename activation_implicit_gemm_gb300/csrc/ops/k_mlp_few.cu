// The gated feed-forward block for up to 32 tokens (include/fconv_ops.h), every type, size and
// stride.
//
//   h = act(x Wg^T + bg) * (x Wu^T + bu),  y = h Wd^T + bd
// Bound: HBM, every weight is read once for all tokens. Weights go from global memory straight
// into the A operand of warp-level tensor instructions, tokens are the 8 columns of B. Lane (g, t)
// of a warp takes 16 bytes of rows g and g + 8 and of token g, of the 64 bytes of a step those from
// 16 t on; words 0 and 1 feed one instruction and 2 and 3 another, with the same order of K in both
// operands, so neither has to be moved between lanes. In the gated product rows 0 to 7 are the
// gate's and 8 to 15 the up projection's of the same 8 hidden values. One token through 4096 x
// 10240 in bf16: 41 us with the launches, 6.1 TB/s.
//
// f16 and bf16 are m16n8k16 operands as they are; f32 is split for m16n8k8 TF32 (hi + lo, three
// products, sums of 16 products at a time as the instructions round towards zero). Where rows do
// not start on 16 bytes the same bytes come an element at a time.
//
// h of the 16-bit types goes from one product to the other in two 16-bit parts, and the second one
// adds up both, so that nothing but y is rounded to 16 bits. With one part, outputs were off by 1.4
// times their own rounding on average and 1.8 at the most; the second one costs nothing for up to 8
// tokens (4096 x 10240 in bf16 in a captured graph: 40.6 us for one and 42 for 8, before and after),
// at 16 tokens 55 us instead of 50 and at 32 tokens 85 instead of 74.
//
// The eight warps of a block share the same rows and split K; their f32 sums are joined through
// shared memory in a fixed order, then come biases, gate and the one rounding. Tokens are read from
// L1 for every row group; with two row groups a warp, which reads them half as often, 16 tokens took
// 67 us instead of 58 (fewer blocks than the SMs hold), 32 tokens 83 instead of 81.
#include "mlp_math.cuh"
#include "split_tf32.cuh"

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
  int64_t plane;  // from h to its second part, 16-bit types
  int tokens, K, N;
  int act;
  float alpha;
};

__device__ __forceinline__ float load_l2(const float* p) { return __ldcg(p); }
__device__ __forceinline__ __half load_l2(const __half* p) { return __ldcg(p); }
__device__ __forceinline__ __nv_bfloat16 load_l2(const __nv_bfloat16* p) { return __ldcg(p); }

// How a row is read: weights once (a plain load that leaves L1 alone takes 51 us for one token
// through 4096 x 10240, one through L2 only 60, with L2 full of other data); EARLY ones through L2
// only, as nothing orders this SM's L1 before the wait; tokens through L1.
enum { kTokens, kWeights, kEarly };

// 16 bytes of a row from element k on where `in` (WIDE: a row has no rest), zeros past K.
template <typename T, bool WIDE, int HOW>
__device__ __forceinline__ uint4 load_row(const T* p, int k, int K, bool in) {
  if constexpr (WIDE) {
    if (!in) return make_uint4(0, 0, 0, 0);
    if (HOW == kTokens) return *reinterpret_cast<const uint4*>(p + k);
    if (HOW == kEarly) return __ldcg(reinterpret_cast<const uint4*>(p + k));
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p + k));
    return v;
  } else {
    constexpr int E = 16 / sizeof(T);
    Vec<T, E> e;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      e.v[i] = from_f<T>(0.0f);
      if (in && k + i < K) e.v[i] = HOW == kEarly ? load_l2(p + k + i) : p[k + i];
    }
    return *reinterpret_cast<const uint4*>(&e);
  }
}

// The same of a row of h in a 16-bit type, which starts on 16 bytes and is followed by whatever lies up
// to the next unit's end: a wide access whatever the weights allow (16 tokens of 767 x 2047: 25.4 us an
// element at a time, 15.3 so; f32, with four elements to mask for four loaded, 17.4 and 20.4).
template <typename T, bool WIDE>
__device__ __forceinline__ uint4 load_hidden(const T* p, int k, int K, bool in) {
  constexpr int E = 16 / sizeof(T);
  if (!in) return make_uint4(0, 0, 0, 0);
  const uint4 v = *reinterpret_cast<const uint4*>(p + k);
  if (WIDE || k + E <= K) return v;
  Vec<T, E> e = *reinterpret_cast<const Vec<T, E>*>(&v);
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (k + i >= K) e.v[i] = from_f<T>(0.0f);
  return *reinterpret_cast<const uint4*>(&e);
}

template <typename T>
constexpr bool kIsBf16 = false;
template <>
constexpr bool kIsBf16<__nv_bfloat16> = true;

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
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

// h of the 16-bit types in two parts, v to within 2^-16 (bf16) or 2^-22 (f16) of itself. The second
// one of f16 is scaled so that it keeps its bits under 6e-5, where f16 has fewer, and is added up by
// itself. Values past the type's largest keep that as their first part.
template <typename T>
constexpr float kLowScale = kIsBf16<T> ? 1.0f : 2048.0f;
template <typename T>
constexpr float kLargest = kIsBf16<T> ? 3.3895313892515355e38f : 65504.0f;  // (2 - 2^-7) 2^127
template <typename T>
__device__ __forceinline__ void split_16(float v, T& hi, T& lo) {
  hi = from_f<T>(within(v, kLargest<T>));
  lo = from_f<T>((v - to_f(hi)) * kLowScale<T>);
}

// acc += a step's products: rows a (g) and b (g + 8), tokens c.
template <typename T>
__device__ __forceinline__ void step(float (&acc)[4], const uint4& a, const uint4& b,
                                     const uint4& c) {
  if constexpr (sizeof(T) == 2) {
    mma16<T>(acc, a.x, b.x, a.y, b.y, c.x, c.y);
    mma16<T>(acc, a.z, b.z, a.w, b.w, c.z, c.w);
  } else {
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
    const uint32_t cv[4] = {c.x, c.y, c.z, c.w};
    float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      uint32_t ah[4], al[4], ch[2], cl[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        split_tf32(__uint_as_float(av[i + e]), ah[2 * e], al[2 * e]);
        split_tf32(__uint_as_float(bv[i + e]), ah[2 * e + 1], al[2 * e + 1]);
        split_tf32(__uint_as_float(cv[i + e]), ch[e], cl[e]);
      }
      mma_tf32(z, al, ch);
      mma_tf32(z, ah, cl);
      mma_tf32(z, ah, ch);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += z[e];
  }
}

// NT: groups of 8 tokens. U: steps of K whose loads go out together.
template <typename T, bool WIDE, bool GATED, int NT, int U>
__global__ void __launch_bounds__(kThreads, 2) mlp_few(const __grid_constant__ Few q) {
  constexpr int kElems = 16 / sizeof(T), kStep = 4 * kElems;  // of a lane, of a step
  __shared__ float sums[kWarps][16][NT * 8 + 1];
  constexpr int kRows = GATED ? 8 : 16;  // outputs of a block
  constexpr int kParts = !GATED && sizeof(T) == 2 ? 2 : 1;  // of a token's values
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows;
  // this lane's rows of weights; rows past the end read the last one, for outputs no one writes
  const T* wp[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int which = GATED ? i : 0;
    const int row = min(n0 + (GATED ? 0 : i * 8) + gr, q.N - 1);
    wp[i] = (const T*)q.w[which] + row * q.w_row[which];
  }
  const T* xp[NT];
  bool there[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    there[n] = n * 8 + gr < q.tokens;
    xp[n] = (const T*)q.x + (there[n] ? n * 8 + gr : 0) * q.x_row;
  }
  float acc[kParts][NT][4];
#pragma unroll
  for (int p = 0; p < kParts; ++p)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[p][n][e] = 0.0f;
  uint4 w[U][2];
  auto load_weights = [&](int k0, bool early) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kStep + t * kElems;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[u][i] = early ? load_row<T, WIDE, kEarly>(wp[i], k, q.K, k < q.K)
                        : load_row<T, WIDE, kWeights>(wp[i], k, q.K, k < q.K);
    }
  };
  const int first = warp * kStep * U;
  // The second product's first weights do not wait for the first product: that has waited for all
  // that came before it when this kernel may start.
  if (!GATED) load_weights(first, true);
  ptx::pdl_wait();
  ptx::pdl_trigger();

  for (int k0 = first; k0 < q.K; k0 += kWarps * kStep * U) {
    uint4 x[kParts][U][NT];
    if (GATED || k0 != first) load_weights(k0, false);
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * kStep + t * kElems;
        const bool in = k < q.K;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          x[p][u][n] = kParts == 2
                           ? load_hidden<T, WIDE>(xp[n] + p * q.plane, k, q.K, in && there[n])
                           : load_row<T, WIDE, kTokens>(xp[n], k, q.K, in && there[n]);
      }
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) step<T>(acc[p][n], w[u][0], w[u][1], x[p][u][n]);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = acc[0][n][e];
      if (kParts == 2) v += acc[kParts - 1][n][e] * (1.0f / kLowScale<T>);
      sums[warp][gr + (e >> 1) * 8][n * 8 + 2 * t + (e & 1)] = v;
    }
  __syncthreads();

  // outputs: neighbouring threads have neighbouring rows of one token
  for (int i = threadIdx.x; i < kRows * NT * 8; i += kThreads) {
    const int r = i % kRows, token = i / kRows, col = n0 + r;
    if (token >= q.tokens || col >= q.N) continue;
    float v = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      v += sums[w][r][token];
      if (GATED) u += sums[w][r + 8][token];
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
    if (!q.out) continue;
    T* to = (T*)q.out + token * q.out_row + col;
    if constexpr (GATED && sizeof(T) == 2) split_16(v, to[0], to[q.plane]);
    else *to = from_f<T>(v);
  }
}

template <typename T, bool WIDE, bool GATED>
int run_as(const Few& q, cudaStream_t s) {
  const int rows = GATED ? 8 : 16;
  const dim3 grid((unsigned)((q.N + rows - 1) / rows)), block(kThreads);
  if (q.tokens <= 8) return launch_pdl(mlp_few<T, WIDE, GATED, 1, 4>, grid, block, 0, s, q);
  if (q.tokens <= 16) return launch_pdl(mlp_few<T, WIDE, GATED, 2, 4>, grid, block, 0, s, q);
  return launch_pdl(mlp_few<T, WIDE, GATED, 4, 2>, grid, block, 0, s, q);
}

// 16-byte accesses where every row of weights and tokens starts on one and has no rest.
template <typename T, bool GATED>
int run(const Few& q, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  bool wide = q.K % E == 0 && (uintptr_t)q.x % 16 == 0 && (q.tokens == 1 || q.x_row % E == 0);
  for (int i = 0; i < (GATED ? 2 : 1); ++i)
    wide = wide && (uintptr_t)q.w[i] % 16 == 0 && (q.N == 1 || q.w_row[i] % E == 0);
  return wide ? run_as<T, true, GATED>(q, s) : run_as<T, false, GATED>(q, s);
}

template <typename T>
int gated(const fconv_mlp_desc& d, const MlpArgs& a, void* h, int64_t h_row, int64_t h_plane,
          cudaStream_t s) {
  Few q{};
  q.plane = h_plane;
  q.x = a.x;
  q.w[0] = a.w_gate;
  q.w[1] = a.w_up;
  q.bias[0] = a.b_gate;
  q.bias[1] = a.b_up;
  q.out = h;
  q.saved = a.saved;
  q.x_row = d.x_stride;
  q.w_row[0] = d.gate_stride;
  q.w_row[1] = d.up_stride;
  q.out_row = h_row;
  q.quads = (d.hidden + 3) / 4;
  q.tokens = (int)d.tokens;
  q.K = (int)d.features;
  q.N = (int)d.hidden;
  q.act = d.activation;
  q.alpha = d.alpha;
  return run<T, true>(q, s);
}

template <typename T>
int down(const fconv_mlp_desc& d, const MlpArgs& a, const void* h, int64_t h_row, int64_t h_plane,
         cudaStream_t s) {
  Few q{};
  q.plane = h_plane;
  q.x = h;
  q.w[0] = a.w_down;
  q.bias[0] = a.b_down;
  q.out = a.y;
  q.x_row = h_row;
  q.w_row[0] = d.down_stride;
  q.out_row = d.y_stride;
  q.tokens = (int)d.tokens;
  q.K = (int)d.hidden;
  q.N = (int)d.out_features;
  return run<T, false>(q, s);
}

}  // namespace

int launch_mlp_few_gated(const fconv_mlp_desc& d, const MlpArgs& a, void* h, int64_t h_row,
                         int64_t h_plane, cudaStream_t s) {
#define FCONV_M(T) return gated<T>(d, a, h, h_row, h_plane, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

int launch_mlp_few_down(const fconv_mlp_desc& d, const MlpArgs& a, const void* h, int64_t h_row,
                        int64_t h_plane, cudaStream_t s) {
#define FCONV_M(T) return down<T>(d, a, h, h_row, h_plane, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
