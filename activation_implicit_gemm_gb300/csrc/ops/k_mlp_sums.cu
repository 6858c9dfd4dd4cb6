// Sums over the rows of up to three matrices at once: the bias gradients of the gated
// feed-forward block. Bound: HBM, each matrix read once. A block adds 64 columns of its share of
// the rows; the shares' f32 sums are joined in order by a second launch.
#include "ops_common.cuh"
#include "ops_internal.h"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kCols = 64, kRowsAtOnce = 16;  // 32 lanes of two columns each, 16 warps

struct Sums {
  SumsArgs m[3];
  float* part;
  int64_t rows;
  int first[4];  // first block of 64 columns of each matrix
  int shares;
};
__device__ __forceinline__ int matrix_of(const Sums& q, int block) {
  return block >= q.first[2] ? 2 : block >= q.first[1] ? 1 : 0;
}

template <typename T>
__global__ void __launch_bounds__(32 * kRowsAtOnce)
    column_sums(const __grid_constant__ Sums q) {
  __shared__ float sums[kRowsAtOnce][kCols + 1];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int which = matrix_of(q, blockIdx.x);
  const SumsArgs& m = q.m[which];
  const int64_t c0 = (int64_t)(blockIdx.x - q.first[which]) * kCols;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = c0 + 2 * lane;
  const int64_t each = (q.rows + q.shares - 1) / q.shares;
  const int64_t r1 = min(((int64_t)blockIdx.y + 1) * each, q.rows);
  float a = 0.0f, b = 0.0f;
  const T* p = (const T*)m.p + c;
  for (int64_t r = blockIdx.y * each + warp; r < r1; r += kRowsAtOnce) {
    if (c < m.cols) a += to_f(p[r * m.row]);
    if (c + 1 < m.cols) b += to_f(p[r * m.row + 1]);
  }
  sums[warp][2 * lane] = a;
  sums[warp][2 * lane + 1] = b;
  __syncthreads();
  if (threadIdx.x >= kCols) return;
  float v = 0.0f;
  for (int i = 0; i < kRowsAtOnce; ++i) v += sums[i][threadIdx.x];
  q.part[((int64_t)blockIdx.y * q.first[3] + blockIdx.x) * kCols + threadIdx.x] = v;
}

template <typename T>
__global__ void __launch_bounds__(kCols) column_join(const __grid_constant__ Sums q) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int which = matrix_of(q, blockIdx.x);
  const SumsArgs& m = q.m[which];
  const int64_t c = (int64_t)(blockIdx.x - q.first[which]) * kCols + threadIdx.x;
  if (c >= m.cols) return;
  float v = 0.0f;
  for (int i = 0; i < q.shares; ++i)
    v += __ldcg(q.part + ((int64_t)i * q.first[3] + blockIdx.x) * kCols + threadIdx.x);
  ((T*)m.out)[c] = from_f<T>(v);
}

int64_t blocks_of(int64_t cols) { return (cols + kCols - 1) / kCols; }

// Shares of the rows: about two blocks an SM, of 64 rows at least.
int shares_of(int64_t blocks, int64_t rows, int sms) {
  int64_t n = (2 * sms + blocks - 1) / (blocks > 0 ? blocks : 1);
  const int64_t most = (rows + 63) / 64;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

}  // namespace

// For any subset of matrices of these widths: fewer matrices make more shares.
size_t column_sums_workspace(const int64_t cols[3], int sms) {
  int64_t blocks = 0;
  for (int i = 0; i < 3; ++i) blocks += blocks_of(cols[i]);
  return (size_t)(2 * (int64_t)sms + 2 * blocks) * kCols * sizeof(float);
}

int launch_column_sums(int dtype, const SumsArgs m[3], int64_t rows, float* part, int sms,
                       cudaStream_t s) {
  Sums q{};
  q.part = part;
  q.rows = rows;
  for (int i = 0; i < 3; ++i) {
    q.m[i] = m[i];
    q.first[i + 1] = q.first[i] + (int)(m[i].out ? blocks_of(m[i].cols) : 0);
  }
  if (q.first[3] == 0) return 0;
  q.shares = shares_of(q.first[3], rows, sms);
  int e = 0;
#define FCONV_M(T)                                                                            \
  e = launch_pdl(column_sums<T>, dim3((unsigned)q.first[3], (unsigned)q.shares),              \
                 dim3(32 * kRowsAtOnce), 0, s, q);                                            \
  if (!e) e = launch_pdl(column_join<T>, dim3((unsigned)q.first[3]), dim3(kCols), 0, s, q)
  FCONV_OPS_TYPE(dtype, FCONV_M)
#undef FCONV_M
  return e;
}

}  // namespace ops
}  // namespace fconv
