// The ring that feeds rows to the norm kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../ptx.cuh"
#include "waits.cuh"

namespace fconv {
namespace ops {
namespace {

// A call of its own: with its loop inline in the kernels the backward ones spilled up to 552 bytes.
__device__ __noinline__ bool wait_row(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return wait_bar(bar, parity, abort_flag);
}

// Rows on their way to a group of TPR threads: a ring of S stages in shared memory filled by
// bulk copies (N tensors a stage), so that the loads in flight do not depend on registers or
// on the group's barriers. Rows that are not whole 16-byte units do not use it (RING false).
// A wait that runs out sets the block's abort flag: every thread then leaves its rows, and the
// group waits for its copies in flight (drain).
template <typename T, int N, int S, int TPR, bool RING>
struct Feed {
  const T* src[N];
  int64_t step, C, left;  // left: rows not yet asked for
  uint32_t ring, bars, bytes, k;
  int t;
  __device__ __forceinline__ void ask(uint32_t stage) {
    const uint32_t bar = bars + stage * 8;
    ptx::mbar_arrive_expect_tx(bar, N * bytes);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      bulk_load(ring + (stage * N + n) * bytes, src[n], bytes, bar);
      src[n] += step * C;
    }
    --left;
  }
  // dsmem: the block's dynamic shared memory; group: this group's index of `groups`.
  __device__ __forceinline__ void init(uint8_t* dsmem, int group, int groups, int t_, int64_t row,
                                       int64_t rows, int64_t step_, int64_t C_) {
    t = t_;
    step = step_;
    C = C_;
    k = 0;
    bytes = (uint32_t)(C * sizeof(T));
    left = row < rows ? (rows - row + step - 1) / step : 0;
    bars = ptx::smem_addr(dsmem) + group * S * 8;
    ring = ptx::smem_addr(dsmem) + ((groups * S * 8 + 15) & ~15) + group * S * N * bytes;
    if (RING && t == 0) {
      for (int i = 0; i < S; ++i) ptx::mbar_init(bars + i * 8, 1);
      ptx::fence_mbar_init();
    }
  }
  __device__ __forceinline__ void start() {
    if (RING && t == 0)
      for (int i = 0; i < S && left > 0; ++i) ask(i);
  }
  // All threads of the group wait for the current row; false when the wait was given up.
  __device__ __forceinline__ bool wait(volatile int* abort_flag) {
    const uint32_t bar = bars + k % S * 8, parity = (k / S) & 1;
    return !RING || ptx::mbar_try_wait(bar, parity) || wait_row(bar, parity, abort_flag);
  }
  // On the way out after that, before next() or after it: the copies in flight land before the
  // block's shared memory is given back (a stage that was not asked for again runs into the drain's
  // short limit).
  __device__ __forceinline__ void drain() {
    if (RING && t == 0)
      for (uint32_t i = k > 0 ? k - 1 : 0; i < k + S; ++i) drain_bar(bars + i % S * 8, (i / S) & 1);
  }
  // The current row of tensor n.
  __device__ __forceinline__ const T* row(const uint8_t* dsmem, int n) const {
    return reinterpret_cast<const T*>(dsmem + (ring - ptx::smem_addr(dsmem)) +
                                      (k % S * N + n) * bytes);
  }
  // After a barrier of the group past the last read of the current row; ok: its wait was not given
  // up (else its stage is left alone).
  __device__ __forceinline__ void next(bool ok = true) {
    if (RING && t == 0 && ok && left > 0) ask(k % S);
    ++k;
  }
};
template <int N, int S>
size_t feed_bytes(int groups, int64_t row_bytes) {
  return ((size_t)groups * S * 8 + 15) / 16 * 16 + (size_t)groups * S * N * row_bytes;
}

}  // namespace
}  // namespace ops
}  // namespace fconv
