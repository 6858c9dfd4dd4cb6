// Sums over the rows of up to three matrices at once: the bias gradients of the gated
// feed-forward block. Bound: HBM, each matrix read once. A block adds 128 columns of its share of
// the rows (256 bytes of a 16-bit row at a time); the shares' f32 sums are joined in order by a
// second launch.
#include "ops_common.cuh"
#include "ops_internal.h"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kThreads = 256, kCols = 128;

struct Sums {
  SumsArgs m[3];
  float* part;
  int64_t rows;
  int first[4];  // first block of kCols columns of each matrix
  int shares;
};
__device__ __forceinline__ int matrix_of(const Sums& q, int block) {
  return block >= q.first[2] ? 2 : block >= q.first[1] ? 1 : 0;
}

// VEC columns a thread in one access, kCols / VEC threads a row, four rows on their way at a time.
template <typename T, int VEC>
__device__ __forceinline__ void sum_rows(const T* p, int64_t row, int64_t cols, int64_t c,
                                         int64_t r, int64_t r1, float (&sum)[VEC]) {
  constexpr int kRows = kThreads / (kCols / VEC), kAhead = 4;
  if (c >= cols) return;  // a row is whole accesses, the last columns may be no one's
  p += c;
  for (; r + (kAhead - 1) * kRows < r1; r += kAhead * kRows) {
    float x[kAhead][VEC];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_f<T, VEC>(p + (r + i * kRows) * row, x[i]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[e] += x[i][e];
  }
  for (; r < r1; r += kRows) {
    float x[VEC];
    load_f<T, VEC>(p + r * row, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] += x[e];
  }
}

template <typename T, int VEC, int PLANES>
__global__ void __launch_bounds__(kThreads) column_sums(const __grid_constant__ Sums q) {
  constexpr int kAcross = kCols / VEC, kRows = kThreads / kAcross;
  __shared__ float sums[kRows][kCols + 1];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int which = matrix_of(q, blockIdx.x);
  const SumsArgs& m = q.m[which];
  const int64_t c0 = (int64_t)(blockIdx.x - q.first[which]) * kCols;
  const int across = threadIdx.x % kAcross, down = threadIdx.x / kAcross;
  const int64_t each = (q.rows + q.shares - 1) / q.shares;
  const int64_t r1 = min(((int64_t)blockIdx.y + 1) * each, q.rows);
  float sum[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) sum[e] = 0.0f;
#pragma unroll
  for (int i = 0; i < PLANES; ++i)
    sum_rows<T, VEC>((const T*)m.p + i * m.plane, m.row, m.cols, c0 + across * VEC,
                     blockIdx.y * each + down, r1, sum);
#pragma unroll
  for (int e = 0; e < VEC; ++e) sums[down][across * VEC + e] = sum[e];
  __syncthreads();
  if (threadIdx.x >= kCols) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) v += sums[i][threadIdx.x];
  q.part[((int64_t)blockIdx.y * q.first[3] + blockIdx.x) * kCols + threadIdx.x] = v;
}

// 32 columns a block, 32 shares at a time.
template <typename T>
__global__ void __launch_bounds__(1024) column_join(const __grid_constant__ Sums q) {
  __shared__ float sums[32][33];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int block = blockIdx.x / (kCols / 32), which = matrix_of(q, block);
  const SumsArgs& m = q.m[which];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int in_block = blockIdx.x % (kCols / 32) * 32 + lane;
  const int64_t c = (int64_t)(block - q.first[which]) * kCols + in_block;
  float v = 0.0f;
  for (int i = row; i < q.shares; i += 32)
    v += __ldcg(q.part + ((int64_t)i * q.first[3] + block) * kCols + in_block);
  sums[row][lane] = v;
  __syncthreads();
  if (row > 0 || c >= m.cols) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += sums[i][lane];
  ((T*)m.out)[c] = from_f<T>(v);
}

int64_t blocks_of(int64_t cols) { return (cols + kCols - 1) / kCols; }

// Shares of the rows: about eight blocks an SM, of 32 rows at least.
int shares_of(int64_t blocks, int64_t rows, int sms) {
  int64_t n = (8 * sms + blocks - 1) / (blocks > 0 ? blocks : 1);
  const int64_t most = (rows + 31) / 32;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

}  // namespace

// For any subset of matrices of these widths: fewer matrices make more shares.
size_t column_sums_workspace(const int64_t cols[3], int sms) {
  int64_t blocks = 0;
  for (int i = 0; i < 3; ++i) blocks += blocks_of(cols[i]);
  return (size_t)(8 * (int64_t)sms + 2 * blocks) * kCols * sizeof(float);
}

int launch_column_sums(int dtype, bool planes, const SumsArgs m[3], int64_t rows, float* part,
                       int sms, cudaStream_t s) {
  Sums q{};
  q.part = part;
  q.rows = rows;
  for (int i = 0; i < 3; ++i) {
    q.m[i] = m[i];
    q.first[i + 1] = q.first[i] + (int)(m[i].out ? blocks_of(m[i].cols) : 0);
  }
  if (q.first[3] == 0) return 0;
  q.shares = shares_of(q.first[3], rows, sms);
  const dim3 grid((unsigned)q.first[3], (unsigned)q.shares), block(kThreads);
  int e = 0;
  if (planes) {  // rows of whole 16-byte units
    e = launch_pdl(column_sums<__nv_bfloat16, 8, 3>, grid, block, 0, s, q);
  } else {
    // 16-byte accesses where every row of every matrix starts on one and has no rest
    const int full = dtype == FCONV_F32 ? 4 : 8;
    bool wide = true;
    for (int i = 0; i < 3; ++i)
      if (m[i].out)
        wide = wide && m[i].cols % full == 0 && m[i].row % full == 0 && (uintptr_t)m[i].p % 16 == 0;
#define FCONV_M(T)                                                                   \
  e = wide ? launch_pdl(column_sums<T, 16 / (int)sizeof(T), 1>, grid, block, 0, s, q) \
           : launch_pdl(column_sums<T, 1, 1>, grid, block, 0, s, q)
    FCONV_OPS_TYPE(dtype, FCONV_M)
#undef FCONV_M
  }
  if (e) return e;
#define FCONV_M(T) e = launch_pdl(column_join<T>, dim3((unsigned)q.first[3] * (kCols / 32)), dim3(1024), 0, s, q)
  FCONV_OPS_TYPE(dtype, FCONV_M)
#undef FCONV_M
  return e;
}

}  // namespace ops
}  // namespace fconv
