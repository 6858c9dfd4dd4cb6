// Bounded mbarrier waits with an error word for the translation unit that includes this.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 200000000ull;

// Set by a wait that ran out; read and cleared by read_and_clear_error.
__device__ unsigned g_wait_error = 0;

// Wait for a phase of an mbarrier, for at most kWaitLimitNs; gives up early when another warp
// of the block has. A wait that runs out sets the flag and the error word.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort_flag) return false;
      if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(&g_wait_error, 1u);
        return false;
      }
    }
  }
}

// On the way out: wait for operations this block has already issued (they always complete). Goes
// on after its limit, with the error word set.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity) {
  if (ptx::mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return;
    if ((i & 63u) == 0 && ptx::globaltimer_ns() - t0 > kDrainLimitNs) {
      atomicOr(&g_wait_error, 1u);
      return;
    }
  }
}

// Contiguous copy of `bytes` (a multiple of 16, both addresses 16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

inline int read_and_clear_error(cudaStream_t s, unsigned* value) {
  unsigned v = 0, zero = 0;
  cudaError_t e =
      cudaMemcpyFromSymbolAsync(&v, g_wait_error, sizeof(v), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && v)
    e = cudaMemcpyToSymbolAsync(g_wait_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *value = v;
  return (int)e;
}

}  // namespace
}  // namespace ops
}  // namespace fconv
