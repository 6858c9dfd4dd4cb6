// Sums over the rows of up to three matrices at once: the bias gradients of the gated
// feed-forward block. Bound: HBM, each matrix read once. A warp adds 32 accesses' columns of its share
// of the rows, four rows on their way; the shares' f32 sums are joined in order by a second launch.
//
// The first launch uses no shared memory, so that with `early` its blocks fit beside those of the
// products launched before it (226 KB each), from which it needs nothing: the training pass of an
// image batch (6304 rows of 2048 + 2048 + 768, f16) takes 186.4 us with that and 190.6 without, one
// of 999 rows of 777 + 777 + 333 in f32 122.8 and 131.0. (Started beside the input's gradient in the
// same way, the weights' gradients gained nothing: 187.5 and 122.6.)
#include "ops_common.cuh"
#include "ops_internal.h"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPad = 256;  // columns of a matrix's sums are a multiple of

struct Sums {
  SumsArgs m[3];
  float* part;       // shares x first[3] * kPad
  int64_t rows;
  int first[4];      // first group of kPad columns of each matrix
  int shares, early;
};
__device__ __forceinline__ int matrix_of(const Sums& q, int group) {
  return group >= q.first[2] ? 2 : group >= q.first[1] ? 1 : 0;
}

// VEC elements in one access through L2: an early launch reads before anything orders its SM's L1.
template <typename T, int VEC>
__device__ __forceinline__ void load_l2(const T* p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_f(__ldcg(p));
  } else {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p));
    const Vec<T, VEC> x = *reinterpret_cast<const Vec<T, VEC>*>(&v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f(x.v[i]);
  }
}

// blockIdx.x: 32 VEC columns; blockIdx.y: the shares of its warps.
template <typename T, int VEC, int PLANES>
__global__ void __launch_bounds__(kThreads) column_sums(const __grid_constant__ Sums q) {
  constexpr int kCols = 32 * VEC, kAhead = 4;
  if (!q.early) ptx::pdl_wait();
  ptx::pdl_trigger();
  const int group = (int)(blockIdx.x * kCols / kPad), which = matrix_of(q, group);
  const SumsArgs& m = q.m[which];
  const int lane = threadIdx.x & 31, share = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const int64_t at = (int64_t)blockIdx.x * kCols + lane * VEC;       // among all columns
  const int64_t c = at - (int64_t)q.first[which] * kPad;             // of this matrix
  const int64_t each = (q.rows + q.shares - 1) / q.shares;
  const int64_t r1 = min((share + 1) * each, q.rows);
  if (share < q.shares && c < m.cols) {  // a row is whole accesses; what lies past it is no one's
    float sum[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] = 0.0f;
#pragma unroll 1
    for (int k = 0; k < PLANES; ++k) {
      const T* p = (const T*)m.p + k * m.plane + c;
      int64_t r = share * each;
      for (; r + kAhead <= r1; r += kAhead) {
        float x[kAhead][VEC];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_l2<T, VEC>(p + (r + i) * m.row, x[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) sum[e] += x[i][e];
      }
      for (; r < r1; ++r) {
        float x[VEC];
        load_l2<T, VEC>(p + r * m.row, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[e] += x[e];
      }
    }
    float* to = q.part + (int64_t)share * q.first[3] * kPad + at;
#pragma unroll
    for (int e = 0; e < VEC; ++e) to[e] = sum[e];
  }
  if (q.early) ptx::pdl_wait();  // it ends after the launch before it, too
}

// 32 columns a block, 32 shares at a time.
template <typename T>
__global__ void __launch_bounds__(1024) column_join(const __grid_constant__ Sums q) {
  __shared__ float sums[32][33];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int which = matrix_of(q, (int)(blockIdx.x / (kPad / 32)));
  const SumsArgs& m = q.m[which];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int64_t at = (int64_t)blockIdx.x * 32 + lane, c = at - (int64_t)q.first[which] * kPad;
  float v = 0.0f;
  if (c < m.cols)
    for (int i = row; i < q.shares; i += 32)
      v += __ldcg(q.part + (int64_t)i * q.first[3] * kPad + at);
  sums[row][lane] = v;
  __syncthreads();
  if (row > 0 || c >= m.cols) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += sums[i][lane];
  ((T*)m.out)[c] = from_f<T>(v);
}

int64_t groups_of(int64_t cols) { return (cols + kPad - 1) / kPad; }

// Shares of the rows: about 24 warps an SM over all groups of columns, of 16 rows at least.
int64_t shares_of(int64_t groups, int64_t rows, int sms) {
  int64_t n = (24 * (int64_t)sms + groups - 1) / (groups > 0 ? groups : 1);
  const int64_t most = (rows + 15) / 16;
  if (n > most) n = most;
  if (n > 4096) n = 4096;
  return n < 1 ? 1 : n;
}

}  // namespace

// For any subset of matrices of these widths: fewer matrices make more shares, but not more sums
// than 24 warps an SM and one group of columns for each share.
size_t column_sums_workspace(const int64_t cols[3], int sms) {
  int64_t groups = 0;
  for (int i = 0; i < 3; ++i) groups += groups_of(cols[i]);
  return (size_t)(24 * (int64_t)sms + 2 * groups) * kPad * sizeof(float);
}

int launch_column_sums(int dtype, bool planes, bool early, const SumsArgs m[3], int64_t rows,
                       float* part, int sms, cudaStream_t s) {
  Sums q{};
  q.part = part;
  q.rows = rows;
  q.early = early;
  for (int i = 0; i < 3; ++i) {
    q.m[i] = m[i];
    q.first[i + 1] = q.first[i] + (int)(m[i].out ? groups_of(m[i].cols) : 0);
  }
  if (q.first[3] == 0) return 0;
  q.shares = (int)shares_of(q.first[3], rows, sms);
  const dim3 block(kThreads);
  auto grid = [&](int vec) {
    return dim3((unsigned)(q.first[3] * (kPad / (32 * vec))),
                (unsigned)((q.shares + kWarps - 1) / kWarps));
  };
  int e = 0;
  if (planes) {  // rows of whole 16-byte units
    e = launch_pdl(column_sums<__nv_bfloat16, 8, 3>, grid(8), block, 0, s, q);
  } else {
    // 16-byte accesses where every row of every matrix starts on one and has no rest
    const int full = dtype == FCONV_F32 ? 4 : 8;
    bool wide = true;
    for (int i = 0; i < 3; ++i)
      if (m[i].out)
        wide = wide && m[i].cols % full == 0 && m[i].row % full == 0 && (uintptr_t)m[i].p % 16 == 0;
#define FCONV_M(T)                                                                              \
  e = wide ? launch_pdl(column_sums<T, 16 / (int)sizeof(T), 1>, grid(full), block, 0, s, q)     \
           : launch_pdl(column_sums<T, 1, 1>, grid(1), block, 0, s, q)
    FCONV_OPS_TYPE(dtype, FCONV_M)
#undef FCONV_M
  }
  if (e) return e;
  const dim3 join((unsigned)q.first[3] * (kPad / 32));
#define FCONV_M(T) e = launch_pdl(column_join<T>, join, dim3(1024), 0, s, q)
  FCONV_OPS_TYPE(dtype, FCONV_M)
#undef FCONV_M
  return e;
}

}  // namespace ops
}  // namespace fconv
