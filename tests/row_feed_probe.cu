// The norm kernels' row feed with two groups of 32 threads: group 0's rows are asked for, group
// 1's are not, so that its wait runs out (after its limit of seconds) and the block ends by itself.
#include "../activation_implicit_gemm_gb300/csrc/ops/row_feed.cuh"

using namespace fconv::ops;

__global__ void probe(const float* x, float* y, int* ok, int rows, int asked) {
  constexpr int kColumns = 64, kStages = 4;
  extern __shared__ __align__(16) uint8_t dsmem[];
  __shared__ int abort_flag;
  const int group = threadIdx.x / 32, t = threadIdx.x % 32;
  Feed<float, 1, kStages, 32, true> feed;
  feed.init(dsmem, group, 2, t, group, rows, 2, kColumns);
  feed.src[0] = x + group * kColumns;
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  if (group < asked) feed.start();
  bool good = true;
  for (int row = group; row < rows; row += 2) {
    good = __all_sync(0xffffffffu, feed.wait(&abort_flag));
    if (!good) {
      feed.drain();
      break;
    }
    const float* r = feed.row(dsmem, 0);
    y[row * kColumns + t] = r[t];
    y[row * kColumns + 32 + t] = r[32 + t];
    __syncwarp();
    feed.next();
  }
  if (t == 0) ok[group] = good;
}

extern "C" int run_probe(const float* x, float* y, int* ok, int rows, int asked) {
  probe<<<1, 64, feed_bytes<1, 4>(2, 64 * sizeof(float))>>>(x, y, ok, rows, asked);
  return (int)cudaGetLastError();
}
extern "C" int read_probe(unsigned* word) { return read_and_clear_error(nullptr, word); }
