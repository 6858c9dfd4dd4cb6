// Instruction wrappers beyond ../ptx.cuh that the tensor-core kernels of the token-side operators
// share: descriptors, MMAs, TMEM loads and stores, bulk stores, register shares.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

// Shared-memory descriptors in the 128-byte swizzle, 8-row atoms of 1024 bytes. The upper word
// is the same for all (stride offset 1024 >> 4, version 1, layout 2), so only the lower one is
// kept and advanced: the issuing thread has few registers, and 64-bit descriptors kept for
// every step of an unrolled product made it spill. K-major (64 elements of a row along K): the
// leading offset is unused. MN-major (rows run along K, 64 elements along M or N contiguous):
// it leads to the next 64 elements along M or N, one box further.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (1u << 16);
}
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t box_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | ((box_bytes >> 4) << 16);
}

// Instruction descriptor of kind::f16: f32 accumulator, A and B both f16 (0) or both bf16 (1),
// B K-major or (bmn) MN-major.
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, int M, int N, bool bmn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (bmn ? 1u << 16 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The issuing warp runs its loop with all lanes and values that the compiler can see are the
// same in all of them (uni), and only the instruction itself is one lane's: the operands then
// live in uniform registers. With a loop of one lane every product of 8 instructions took 800
// cycles to issue, operand by operand, against the 512 that it takes to run.
__device__ __forceinline__ int uni(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint32_t uni(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ bool all_lanes(bool v) { return __all_sync(0xffffffffu, v); }
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= A[smem] * B[smem]^T, lower descriptor words; issued by one thread.
__device__ __forceinline__ void mma_ss(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: A's rows are TMEM lanes, two 16-bit elements a column.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// 4-D tiled TMA load (c0 innermost).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int c0, int c1, int c2,
                                            int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"((uint64_t)tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// 4-D tiled TMA store of a box from shared memory (elements outside the tensor are left out),
// its group, and the wait until the group's boxes have been read / written.
__device__ __forceinline__ void tma_store_4d(const void* tmap, uint32_t src, int c0, int c1, int c2,
                                             int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
          (uint64_t)tmap),
      "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// One thread's 16-bit row of 32 columns (64 bytes) of a swizzled box of 128-byte rows.
__device__ __forceinline__ void stage_row(uint32_t box, int row, int c0, const uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ptx::st_shared_v4(box + row * 128 + (((c0 / 8 + i) ^ (row & 7)) << 4), w[4 * i], w[4 * i + 1],
                      w[4 * i + 2], w[4 * i + 3]);
}

#define FCONV_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), \
                       "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define FCONV_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), \
                       "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
#define FCONV_P8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), \
                       "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])

// Whole warp: starts the load of 32 lanes x 32 columns (thread t gets lane base + t). The
// registers hold the values only after tmem_arrived() on them.
__device__ __forceinline__ void tmem_fetch32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : FCONV_R8(r, 0), FCONV_R8(r, 8), FCONV_R8(r, 16), FCONV_R8(r, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_fetch8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : FCONV_R8(r, 0)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[8]) {
  asm volatile("" : FCONV_P8(r, 0)::"memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::FCONV_I8(
          r, 0),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Ties the registers to the wait that precedes: no use of them moves above it.
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[32]) {
  asm volatile("" : FCONV_P8(r, 0), FCONV_P8(r, 8), FCONV_P8(r, 16), FCONV_P8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::FCONV_I8(r, 0),
      FCONV_I8(r, 8), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Registers a thread of the calling warpgroup may use from here on (all its warps call it).
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 2^x by the special-function unit (within 2 ulp; results below 2^-126 become 0).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values rounded to 16 bits, the first in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

}  // namespace
}  // namespace ops
}  // namespace fconv
