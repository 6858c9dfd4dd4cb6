// The gated feed-forward block on tcgen05 tensor cores (include/fconv_ops.h).
//
//   forward   h = act(x Wg^T + bg) * (x Wu^T + bu)      both products in one accumulator
//             y = h Wd^T + bd
//   backward  dh = dy Wd;  dg = dh u act'(g), du = dh act(g), h = act(g) u   in its epilogue
//             dx = dg Wg + du Wu                         one sum over both
//             dWg = dg^T x, dWu = du^T x, dWd = dy^T h   one launch, with dx where that is quicker
// All of them are one kernel, D = A B^T with operands that run along K or along M and N in memory
// (the descriptors transpose, nothing is copied), f32 sums in TMEM and an epilogue that adds
// biases, gates, and rounds once.
//
// Two SMs work on a tile of 256 x 256 (CG 2): each loads 128 rows of A and 128 of B and one of
// them issues the products of both, which halves what has to come out of L2 for each product
// (32 KB a 64-deep step and SM against 48 for 128 x 256 tiles of one). Tiles of 128 x 128 on one
// SM (CG 1) are for calls with too few of the others. Per block: a load warp keeps a ring of
// 32 KB stages full, an MMA warp issues, eight warps empty one accumulator while the next tile's
// products fill the other. Blocks are persistent and take tiles in groups of 8 rows of tiles, so
// that blocks at work at one time share operands in L2. Where one-SM tiles are few, a cluster of
// blocks shares a tile (SPLIT): each takes a part of K, leaves its sums in shared memory and finishes
// some of the columns, adding the blocks' parts in their order.
//
// Bound: the tensor pipe, busy throughout at 16384 x 4096 x 10240 in bf16 (1375 to 1390 and 718 to 728 us
// alone, 1.9 to 2.0 PFLOP/s; 2.31 to 2.41 ms in passes under the power cap). Short sums (768 of K) leave the
// epilogues and their traffic to bound it: 48 us for the gated product of 6304 x 768 x 2048 with g
// and u going out in f32, 27 without.
//
// f32 (F32) comes as three bf16 planes that add up to it (k_mlp_prep.cu; h, dg and du are split in
// the epilogues). Six products of planes, the smallest first, leave out less than 2^-23 of a
// product. The tensor core's f32 sums cut off instead of rounding (measured: 1.7e-8 of the result
// for each instruction of 16 products, always towards zero), so after 128 of K they are added to
// registers in plain f32 (after 512 the errors were twice as large, at the same speed).
//
// What is cut adds up where terms have one sign: 1.0e-7 of the result for each instruction (measured,
// positive values), 1.7e-3 for a weight's gradient over 2^18 tokens, 3.5 times f16's rounding. So in
// 16-bit types, too, a sum of more than kLong steps comes in passes of at most 16384 products (1.0e-4).
// A thread's part of a tile does not fit its registers there: the sums so far lie in the workspace,
// each thread reads and writes its own, and all blocks' 20 MB stay in L2. Passes of at most 4096, 8192
// and 16384: 2122, 2105 and 2067 us for 16384 x 4096 x 10240 forward (its down projection sums 10240
// values), 950, 915 and 866 us for 2048 x 16384 x 8192; 2070 and 870 without passes. Calls whose sums
// take one pass have kernels without that code (LONG), which costs them 1 %: 2380 and 2402 us for the
// first shape in passes under the power cap, 184 and 185.6 for both passes of 6304 x 768 x 2048.
#include "mlp_math.cuh"
#include "split_bf16.cuh"
#include "tc_instr.cuh"
#include "waits.cuh"

#include "../fconv_internal.h"
#include "../ptx.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kStep = 64;                  // K of a stage
constexpr uint32_t kSide = 128 * kStep * 2;  // bytes of 128 rows (or columns) of one operand
constexpr uint32_t kBox = kSide / 2;       // 64 of them where they run along M or N
constexpr uint32_t kSlot = 32 * 64;        // staged output of a warp: 32 rows of 32 values
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8, kFirstEpiWarp = 4;

enum { kPlain, kGated, kGrad };

constexpr int kPlanes = 3, kTerms = 6;  // of f32
constexpr int kChunk = 2;               // steps of K whose sums stay in TMEM, f32
constexpr int kLong = 256;              // and in 16-bit types

template <int EPI, bool F32>  // of an epilogue warp
constexpr int kSlots = EPI == kPlain ? 2 : EPI == kGated ? (F32 ? kPlanes : 2) : F32 ? 2 * kPlanes : 3;
template <int EPI, bool F32>
constexpr int kStages = kSlots<EPI, F32> > 3 ? 4 : kSlots<EPI, F32> == 3 ? 5 : 6;

struct Problem {
  CUtensorMap a[2], b[2], c[3];  // products of a sum (kGated: gate and up), outputs as boxes
  int mt, nt, steps;             // tiles, steps of a product
  int products;
  int a_mn, b_mn;                // whether operands run along M or N in memory, not along K
  int64_t M;
  int N;
  const void* bias[2];
  void* out;                     // where boxes do not go: rows of any stride
  int64_t out_row;
};
struct Job {
  Problem p[4];
  int problems, tiles;
  int splits;  // blocks of a tile, SPLIT
  float* saved;
  float* sums;  // of passes, 128 rows of each block's columns
  int64_t quads;
  float alpha;
  int act, bf16;
};

template <int S>
struct Control {
  uint64_t full[S], empty[S], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort_flag;
};

// ------------------------------------------------------------- pairs of blocks (CG 2)

__device__ __forceinline__ uint32_t block_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address, for the whole cluster, of what lies at `addr` in the first block.
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ uint32_t in_block(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_take(uint32_t dst, uint32_t cols) {
  if (CG == 1) {
    ptx::tmem_alloc(dst, cols);
    ptx::tmem_relinquish();
  } else {
    asm volatile(
        "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
        "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(dst),
        "r"(cols)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_give(uint32_t addr, uint32_t cols) {
  if (CG == 1)
    ptx::tmem_dealloc(addr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  if (CG == 1) {
    mma_ss(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
  }
}
// Arrives on `bar` (of both blocks) when the products issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if (CG == 1) {
    ptx::mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  }
}
// A box into this block's shared memory, its bytes counted on a barrier of the first block.
template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                         int plane, uint32_t bar) {
  if (CG == 1) {
    ptx::tma_load_3d(dst, map, c0, c1, plane, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(plane), "r"(bar)
        : "memory");
  }
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int c0, int c1,
                                          int plane) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          (uint64_t)map),
      "r"(src), "r"(c0), "r"(c1), "r"(plane)
      : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read_but() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// A wait for arrivals from the other block too.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag) {
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000)
        : "memory");
    if (ok) return true;
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

// ------------------------------------------------------------------------- the tiles

struct Tile {
  int which, m, n;
};
// Tile `id` of a job: problem by problem, in groups of 8 rows of tiles.
__device__ __forceinline__ Tile tile_of(const Job& j, int id) {
  Tile t;
  t.which = 0;
  while (t.which + 1 < j.problems && id >= j.p[t.which].mt * j.p[t.which].nt) {
    id -= j.p[t.which].mt * j.p[t.which].nt;
    ++t.which;
  }
  constexpr int kGroup = 8;
  const int mt = j.p[t.which].mt, nt = j.p[t.which].nt;
  const int group = id / (kGroup * nt), first = group * kGroup, rows = min(kGroup, mt - first);
  const int at = id - group * kGroup * nt;
  t.m = first + at % rows;
  t.n = at / rows;
  return t;
}

// The steps [lo, hi) of a tile's products that a block takes, product by product.
struct Range {
  int lo, hi;
};
__device__ __forceinline__ Range range_of(const Problem& p, int products, int rank, int splits) {
  const int all = products * p.steps;
  Range r;
  r.lo = (int)((int64_t)all * rank / splits);
  r.hi = (int)((int64_t)all * (rank + 1) / splits);
  return r;
}
// They come in passes, each into an accumulator of its own: for 16-bit types as few and as even ones
// as kLong allows, for f32 one for every kChunk steps (of one product), six terms each.
template <bool F32>
__device__ __forceinline__ int pass_steps(const Problem& p, const Range& r, int at) {
  if (!F32) {
    const int all = r.hi - r.lo;
    if (all <= kLong) return all;
    const int passes = (all + kLong - 1) / kLong;
    return min((all + passes - 1) / passes, r.hi - at);
  }
  return min(min(kChunk, r.hi - at), p.steps - at % p.steps);
}
struct Step {
  int product, k, a_plane, b_plane;
};
// Load i of the pass of `len` steps from step `at` on.
template <bool F32>
__device__ __forceinline__ Step step_of(const Problem& p, int at, int len, int i) {
  const int term = F32 ? i / len : 0, g = at + i - term * len;
  Step s;
  s.product = g >= p.steps;
  s.k = g - s.product * p.steps;
  s.a_plane = F32 ? (0x001102 >> (4 * term)) & 3 : 0;  // 2 0 1 1 0 0
  s.b_plane = F32 ? (0x010120 >> (4 * term)) & 3 : 0;  // 0 2 1 0 1 0
  return s;
}

__device__ __forceinline__ uint32_t pack16(bool bf16, float a, float b) {
  return bf16 ? pack2<true>(a, b) : pack2<false>(a, b);
}
// N words of a row (64 bytes, 32 values) of a staged box in the 64-byte swizzle, from word w0 on.
template <int N>
__device__ __forceinline__ void stage(uint32_t slot, int row, int w0, const uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    ptx::st_shared_v4(slot + row * 64 + ((((w0 + i) >> 2) ^ ((row >> 1) & 3)) << 4), w[i], w[i + 1],
                      w[i + 2], w[i + 3]);
}
// 8 f32 values from column c0 on as their three bf16 planes, in three slots.
__device__ __forceinline__ void stage_planes(uint32_t slots, int row, int c0, const float* x) {
  uint32_t w[kPlanes][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a[kPlanes], b[kPlanes];
    split_bf16(x[2 * i], a);
    split_bf16(x[2 * i + 1], b);
#pragma unroll
    for (int q = 0; q < kPlanes; ++q) w[q][i] = pack2<true>(a[q], b[q]);
  }
#pragma unroll
  for (int q = 0; q < kPlanes; ++q) stage(slots + q * kSlot, row, c0 / 2, w[q]);
}
// The staged rows of a warp to global memory, a row of 32 columns at a time, at any alignment.
template <bool F32>
__device__ __forceinline__ void store_rows(uint32_t slot, void* out, int64_t out_row, int64_t grow0,
                                           int64_t M, int col, int N, int lane) {
  __syncwarp();
  const bool in = col + lane < N;
#pragma unroll 4
  for (int i = 0; i < 32; ++i) {
    if (grow0 + i >= M) break;
    const int64_t at = (grow0 + i) * out_row + col + lane;
    if (F32) {
      const uint32_t v =
          ptx::ld_shared_u32(slot + i * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4);
      if (in) ((uint32_t*)out)[at] = v;
    } else {
      const uint32_t v = ptx::ld_shared_u16(slot + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) +
                                            (lane & 7) * 2);
      if (in) ((uint16_t*)out)[at] = (uint16_t)v;
    }
  }
  __syncwarp();
}

// x[i] += bias[col + i] for 32 columns, those past N left alone. A lane reads one.
template <bool F32>
__device__ __forceinline__ void add_bias(float (&x)[32], const void* bias, int col, int N, bool bf16,
                                         int lane) {
  if (!bias) return;
  float v = 0.0f;
  if (col + lane < N) {
    if (F32) v = ((const float*)bias)[col + lane];
    else if (bf16) v = to_f(((const __nv_bfloat16*)bias)[col + lane]);
    else v = to_f(((const __half*)bias)[col + lane]);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] += __shfl_sync(0xffffffffu, v, i);
}

__device__ __forceinline__ void as_floats(float (&x)[32], const uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
}

// 32 values of h from g and u, two a word.
template <int ACT>
__device__ __forceinline__ void gate(uint32_t (&w)[16], const float (&g)[32], const float (&u)[32],
                                     float alpha, bool bf16) {
  float unused;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    w[i] = pack16(bf16, act_fast<ACT, false>(alpha, g[2 * i], unused) * u[2 * i],
                  act_fast<ACT, false>(alpha, g[2 * i + 1], unused) * u[2 * i + 1]);
}
// 8 values of dg, du and h from those of dh, g and u.
template <int ACT>
__device__ __forceinline__ void gate_grad(uint32_t (&wg)[4], uint32_t (&wu)[4], uint32_t (&wh)[4],
                                          const float* dh, const float4 (&g)[2],
                                          const float4 (&u)[2], float alpha, bool bf16) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float gs[4] = {g[k].x, g[k].y, g[k].z, g[k].w}, us[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
    float dg[4], du[4], h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float slope;
      const float a = act_fast<ACT, true>(alpha, gs[e], slope), d = dh[k * 4 + e];
      dg[e] = d * us[e] * slope;
      du[e] = d * a;
      h[e] = a * us[e];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      wg[2 * k + e] = pack16(bf16, dg[2 * e], dg[2 * e + 1]);
      wu[2 * k + e] = pack16(bf16, du[2 * e], du[2 * e + 1]);
      wh[2 * k + e] = pack16(bf16, h[2 * e], h[2 * e + 1]);
    }
  }
}

// The same for f32, staged as planes: 32 values of h; 8 of dg, or of du and h.
template <int ACT>
__device__ __forceinline__ void gate_planes(uint32_t slots, int row, const float (&g)[32],
                                            const float (&u)[32], float alpha) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    float h[8], unused;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = act_exact<ACT, false>(alpha, g[i + e], unused) * u[i + e];
    stage_planes(slots, row, i, h);
  }
}
template <int ACT, bool GATE>
__device__ __forceinline__ void gate_grad_planes(uint32_t slots, int row, int c0, const float* dh,
                                                 const float (&g)[8], const float (&u)[8],
                                                 float alpha) {
  float v[8], h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float slope = 0.0f;
    const float a = act_exact<ACT, GATE>(alpha, g[e], slope);
    v[e] = GATE ? dh[e] * u[e] * slope : dh[e] * a;
    h[e] = a * u[e];
  }
  stage_planes(slots, row, c0, v);
  if (!GATE) stage_planes(slots + kPlanes * kSlot, row, c0, h);
}

// LONG: a 16-bit tile's sums may come in several passes (without SPLIT).
template <int CG, int EPI, bool F32, bool SPLIT, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) mlp_tc(const __grid_constant__ Job j) {
  constexpr int S = kStages<EPI, F32>, BN = 128 * CG;
  constexpr int kCols = EPI == kGated ? BN / 2 : BN;  // of a tile of D
  constexpr uint32_t kStageBytes = 2 * kSide;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Control<S> ctl;
  const uint32_t ring = ptx::smem_addr(smem);
  if (ring & 1023u) {  // the swizzle's atoms: the same for all threads
    if (threadIdx.x == 0) atomicOr(&g_wait_error, 2u);
    return;
  }
  const int warp = uni((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : block_rank();
  const int splits = SPLIT ? j.splits : 1, part = SPLIT ? (int)block_rank() : 0;
  volatile int* abort_flag = &ctl.abort_flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.acc_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.acc_empty[i]), CG * kEpiWarps);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl.done), 1);
    ctl.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    const Problem& p = j.p[0];
    ptx::prefetch_tmap(&p.a[0]);
    ptx::prefetch_tmap(&p.b[0]);
    if (EPI == kGated) ptx::prefetch_tmap(&p.b[1]);
  }
  if (warp == 2) tmem_take<CG>(ptx::smem_addr(&ctl.tmem), 2 * BN);
  ptx::tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int first = (int)blockIdx.x / (CG * splits), stride = (int)gridDim.x / (CG * splits);

  if (warp == 0) {  // loads
    int it = 0;
    bool ok = true;
    for (int id = first; ok && id < j.tiles; id += stride) {
      const Tile t = tile_of(j, id);
      const Problem& p = j.p[t.which];
      const int m0 = (t.m * CG + (int)rank) * 128;
      const int n0 = EPI == kGated ? t.n * kCols : t.n * BN + (int)rank * 128;
      const Range r = range_of(p, EPI == kGated ? 1 : p.products, part, splits);
      for (int at = r.lo, len; ok && at < r.hi; at += len) {
        len = pass_steps<F32>(p, r, at);
        const int steps = len * (F32 ? kTerms : 1);
        for (int i = 0; i < steps; ++i, ++it) {
          const Step st = step_of<F32>(p, at, len, i);
          const int s = it % S;
          ok = all_lanes(wait_bar(ptx::smem_addr(&ctl.empty[s]), ((it / S) & 1) ^ 1, abort_flag));
          if (!ok) break;
          const uint32_t own = ptx::smem_addr(&ctl.full[s]);
          const uint32_t bar = CG == 1 ? own : in_first(own);
          const uint32_t sa = ring + s * kStageBytes, sb = sa + kSide;
          const CUtensorMap *ma = &p.a[st.product], *mb = &p.b[st.product];
          const int k = st.k * kStep, pa = st.a_plane, pb = st.b_plane;
          if (elect_lane()) {
            if (rank == 0) ptx::mbar_arrive_expect_tx(own, CG * kStageBytes);
            if (EPI == kPlain && p.a_mn) {
              load_box<CG>(sa, ma, m0, k, pa, bar);
              load_box<CG>(sa + kBox, ma, m0 + 64, k, pa, bar);
            } else {
              load_box<CG>(sa, ma, k, m0, pa, bar);
            }
            if (EPI != kGated && p.b_mn) {
              load_box<CG>(sb, mb, n0, k, pb, bar);
              load_box<CG>(sb + kBox, mb, n0 + 64, k, pb, bar);
            } else if (EPI == kGated && CG == 1) {
              load_box<CG>(sb, &p.b[0], k, n0, pb, bar);
              load_box<CG>(sb + kBox, &p.b[1], k, n0, pb, bar);
            } else if (EPI == kGated) {
              load_box<CG>(sb, &p.b[rank], k, n0, pb, bar);
            } else {
              load_box<CG>(sb, mb, k, n0, pb, bar);
            }
          }
          __syncwarp();
        }
      }
    }
    // the last arrivals on this block's barriers, and on the way out of a wait given up its copies
    if (*abort_flag) {
      if (rank == 0)
        for (int s = 0; s < S && s < it; ++s)
          drain_bar(ptx::smem_addr(&ctl.full[s]), ((it - 1 - s) / S) & 1);
    } else {
      for (int s = 0; s < S && s < it; ++s)
        wait_bar(ptx::smem_addr(&ctl.empty[s]), ((it - 1 - s) / S) & 1, abort_flag);
    }
  } else if (warp == 1) {  // products
    if (rank == 0) {
      int it = 0, n = 0;
      bool ok = true;
      for (int id = first; ok && id < j.tiles; id += stride) {
        const Tile t = tile_of(j, id);
        const Problem& p = j.p[t.which];
        const bool amn = EPI == kPlain && p.a_mn, bmn = EPI != kGated && p.b_mn;
        const uint32_t idesc =
            uni(idesc_16(F32 || j.bf16, 128 * CG, BN, bmn) | (amn ? 1u << 15 : 0u));
        // a step of 16 of K: 32 bytes of a row, or 16 rows
        const uint32_t a_next = uni(amn ? 128u : 2u), b_next = uni(bmn ? 128u : 2u);
        const Range r = range_of(p, EPI == kGated ? 1 : p.products, part, splits);
        for (int at = r.lo, len; ok && at < r.hi; at += len, ++n) {
          len = pass_steps<F32>(p, r, at);
          const int steps = len * (F32 ? kTerms : 1);
          const uint32_t d = tmem + (n & 1) * BN;
          ok = all_lanes(wait_cluster(ptx::smem_addr(&ctl.acc_empty[n & 1]), ((n >> 1) & 1) ^ 1,
                                      abort_flag));
          ptx::tc_fence_after();
          for (int k = 0; ok && k < steps; ++k, ++it) {
            const int s = it % S;
            ok = all_lanes(wait_bar(ptx::smem_addr(&ctl.full[s]), (it / S) & 1, abort_flag));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t sa = ring + s * kStageBytes, sb = sa + kSide;
            const uint32_t a = uni(amn ? desc_mn(sa, kBox) : desc_k(sa));
            const uint32_t b = uni(bmn ? desc_mn(sb, kBox) : desc_k(sb));
            if (elect_lane()) {
#pragma unroll
              for (int i = 0; i < kStep / 16; ++i)
                mma<CG>(d, a + i * a_next, b + i * b_next, idesc, k > 0 || i > 0);
              commit<CG>(ptx::smem_addr(&ctl.empty[s]));
              if (k + 1 == steps) commit<CG>(ptx::smem_addr(&ctl.acc_full[n & 1]));
            }
            __syncwarp();
          }
        }
      }
      if (!ok) {  // the products issued so far read both blocks' shared memory
        if (elect_lane()) commit<CG>(ptx::smem_addr(&ctl.done));
        __syncwarp();
        drain_bar(ptx::smem_addr(&ctl.done), 0);
      }
    }
  } else if (warp >= kFirstEpiWarp) {
    // Each warp for itself: a quarter of the rows (its TMEM lanes) of half of the columns, its own
    // slots and its own stores.
    const int half = (warp - kFirstEpiWarp) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t slots =
        ring + S * kStageBytes + (uint32_t)((warp - kFirstEpiWarp) * kSlots<EPI, F32>) * kSlot;
    const bool bf16 = j.bf16;
    const int act = j.act;
    const float alpha = j.alpha;
    constexpr int kParts = kCols / 64;  // 32-column parts of a warp's half of the tile
    constexpr int kUps = EPI == kGated ? kParts : 1;
    int n = 0, slot = 0;
    bool ok = true;
    for (int id = first; ok && id < j.tiles; id += stride) {
      const Tile t = tile_of(j, id);
      const Problem& p = j.p[t.which];
      const int m0 = (t.m * CG + (int)rank) * 128 + quarter * 32;  // this warp's first row
      const int64_t grow = (int64_t)m0 + lane;
      const int first_part = SPLIT ? half * splits + part : half * kParts;
      // saved values of this warp's rows: block of 32 rows, a row a lane
      float* saved = nullptr;
      if (EPI != kPlain && j.saved)
        saved = j.saved + (grow >> 5) * j.quads * 256 + lane * 4;
      // kGrad: those of 32 columns, in 16-bit types on their way since the part before (f32 has no
      // registers for that)
      constexpr bool kEarly = EPI == kGrad && !F32;
      float4 gs[kEarly ? 8 : 1], us[kEarly ? 8 : 1];
      auto load_saved = [&](int c, int i, float4& g, float4& v) {
        g = v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int col = t.n * kCols + c * 32 + 4 * i;
        if (grow < p.M && col < p.N) {
          const float* from = saved + (int64_t)(col >> 2) * 256;
          g = __ldcg(reinterpret_cast<const float4*>(from));
          v = __ldcg(reinterpret_cast<const float4*>(from + 128));
        }
      };
      if (kEarly) {
#pragma unroll
        for (int i = 0; i < 8; ++i) load_saved(first_part, i, gs[i], us[i]);
      }

      auto arrive = [&]() {
        ok = all_lanes(
            wait_bar(ptx::smem_addr(&ctl.acc_full[n & 1]), (n >> 1) & 1, abort_flag));
        ptx::tc_fence_after();
        return ok;
      };
      auto release = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = ptx::smem_addr(&ctl.acc_empty[n & 1]);
          if (CG == 1) ptx::mbar_arrive(bar);
          else arrive_cluster(in_first(bar));
        }
      };
      auto fetch = [&](int c, uint32_t (&r0)[32], uint32_t (&r1)[32]) {
        const uint32_t acc = tmem + (n & 1) * BN + ((uint32_t)(quarter * 32) << 16);
        const int tcol = half * (kCols / 2) + c * 32;
        tmem_fetch32(acc + tcol, r0);
        if (EPI == kGated) tmem_fetch32(acc + BN / 2 + tcol, r1);
        tmem_wait_ld();
        tmem_arrived(r0);
        if (EPI == kGated) tmem_arrived(r1);
      };
      // Slots that may be written again.
      auto reuse = [&]() {
        if (lane == 0) bulk_wait_read_but<kSlots<EPI, F32> == 2 ? 1 : 0>();
        __syncwarp();
      };
      auto store = [&](const CUtensorMap* map, int col, int boxes, uint32_t from, bool planes) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && m0 < p.M) {
          for (int i = 0; i < boxes; ++i)
            store_box(planes ? map : map + i, from + i * kSlot, col, m0, planes ? i : 0);
          bulk_commit();
        }
      };
      // 32 columns of the tile, of which this warp takes `next` after them; x (and with kGated u)
      // are sums of products.
      auto finish = [&](int c, int next, float (&x)[32], float (&u)[32]) {
        const int col = t.n * kCols + c * 32;
        if (col >= p.N) return;
        if (EPI == kPlain) {
          add_bias<F32>(x, p.bias[0], col, p.N, bf16, lane);
          uint32_t w[16];
          if (F32) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              ptx::st_shared_v4(slots + lane * 128 + (((i >> 2) ^ (lane & 7)) << 4),
                                __float_as_uint(x[i]), __float_as_uint(x[i + 1]),
                                __float_as_uint(x[i + 2]), __float_as_uint(x[i + 3]));
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack16(bf16, x[2 * i], x[2 * i + 1]);
          }
          if (F32 || p.out) {
            if (!F32) {  // boxes of another problem's tile may be on their way
              if (lane == 0) bulk_wait_read_but<0>();
              __syncwarp();
              stage(slots, lane, 0, w);
            }
            store_rows<F32>(slots, p.out, p.out_row, m0, p.M, col, p.N, lane);
          } else {
            reuse();
            stage(slots + slot * kSlot, lane, 0, w);
            store(&p.c[0], col, 1, slots + slot * kSlot, false);
            slot ^= 1;
          }
        } else if (EPI == kGated) {
          add_bias<F32>(x, p.bias[0], col, p.N, bf16, lane);
          add_bias<F32>(u, p.bias[1], col, p.N, bf16, lane);
          reuse();
          if (F32) {
#define FCONV_M(ACT) gate_planes<ACT>(slots, lane, x, u, alpha)
            FCONV_GATE_SWITCH(act, FCONV_M)
#undef FCONV_M
            store(&p.c[0], col, kPlanes, slots, true);
          } else {
            uint32_t w[16];
#define FCONV_M(ACT) gate<ACT>(w, x, u, alpha, bf16)
            FCONV_GATE_SWITCH(act, FCONV_M)
#undef FCONV_M
            stage(slots + slot * kSlot, lane, 0, w);
            store(&p.c[0], col, 1, slots + slot * kSlot, false);
            slot ^= 1;
          }
          if (saved && grow < p.M) {  // after the fence, which would wait for them
            float* to = saved + (int64_t)(col >> 2) * 256;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              if (col + i >= p.N) break;
              *reinterpret_cast<float4*>(to + i * 64) =
                  make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
              *reinterpret_cast<float4*>(to + i * 64 + 128) =
                  make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]);
            }
          }
        } else if (F32) {
          auto values = [&](int i, float (&g)[8], float (&v)[8]) {
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
              float4 g4, v4;
              load_saved(c, (i + k) / 4, g4, v4);
              g[k] = g4.x, g[k + 1] = g4.y, g[k + 2] = g4.z, g[k + 3] = g4.w;
              v[k] = v4.x, v[k + 1] = v4.y, v[k + 2] = v4.z, v[k + 3] = v4.w;
            }
          };
          // dg, then du and h: there is no room for nine planes at once
#define FCONV_M(ACT)                                                     \
  reuse();                                                               \
  _Pragma("unroll") for (int i = 0; i < 32; i += 8) {                    \
    float g[8], v[8];                                                    \
    values(i, g, v);                                                     \
    gate_grad_planes<ACT, true>(slots, lane, i, x + i, g, v, alpha);     \
  }                                                                      \
  store(&p.c[0], col, kPlanes, slots, true);                             \
  reuse();                                                               \
  _Pragma("unroll") for (int i = 0; i < 32; i += 8) {                    \
    float g[8], v[8];                                                    \
    values(i, g, v);                                                     \
    gate_grad_planes<ACT, false>(slots, lane, i, x + i, g, v, alpha);    \
  }                                                                      \
  store(&p.c[1], col, kPlanes, slots, true);                             \
  store(&p.c[2], col, kPlanes, slots + kPlanes * kSlot, true)
          FCONV_GATE_SWITCH(act, FCONV_M)
#undef FCONV_M
        } else {
          reuse();
#define FCONV_M(ACT)                                                                             \
  _Pragma("unroll") for (int i = 0; i < 32; i += 8) {                                            \
    uint32_t wg[4], wu[4], wh[4];                                                                \
    const float4 g[2] = {gs[i / 4], gs[i / 4 + 1]}, v[2] = {us[i / 4], us[i / 4 + 1]};           \
    if (next >= 0) {                                                                             \
      load_saved(next, i / 4, gs[i / 4], us[i / 4]);                                             \
      load_saved(next, i / 4 + 1, gs[i / 4 + 1], us[i / 4 + 1]);                                 \
    }                                                                                            \
    gate_grad<ACT>(wg, wu, wh, x + i, g, v, alpha, bf16);                                        \
    stage(slots, lane, i / 2, wg);                                                               \
    stage(slots + kSlot, lane, i / 2, wu);                                                       \
    stage(slots + 2 * kSlot, lane, i / 2, wh);                                                   \
  }
          FCONV_GATE_SWITCH(act, FCONV_M)
#undef FCONV_M
          store(&p.c[0], col, 3, slots, false);
        }
      };

      // The sums of the passes so far, each thread's own, 16 bytes a lane (16-bit types: the columns
      // of a row that a thread has do not fit its registers).
      auto sums_of = [&](int c) {
        constexpr int kEach = EPI == kGated ? 16 : 8;  // accesses of a part
        const int64_t first_access =
            ((int64_t)blockIdx.x * kEpiWarps + (warp - kFirstEpiWarp)) * kParts + c;
        return reinterpret_cast<float4*>(j.sums) + first_access * kEach * 32 + lane;
      };
      auto add_sums = [&](int c, float (&x)[32], float (&u)[32]) {
        const float4* from = sums_of(c);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 v = __ldcg(from + i / 4 * 32);
          x[i] += v.x, x[i + 1] += v.y, x[i + 2] += v.z, x[i + 3] += v.w;
          if (EPI == kGated) {
            const float4 w = __ldcg(from + (8 + i / 4) * 32);
            u[i] += w.x, u[i + 1] += w.y, u[i + 2] += w.z, u[i + 3] += w.w;
          }
        }
      };
      auto put_sums = [&](int c, const float (&x)[32], const float (&u)[32]) {
        float4* to = sums_of(c);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          __stcg(to + i / 4 * 32, make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
          if (EPI == kGated)
            __stcg(to + (8 + i / 4) * 32, make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]));
        }
      };

      // All sums of this warp's part of the tile.
      auto collect = [&](float (&x)[kParts][32], float (&u)[kUps][32]) {
        const Range r = range_of(p, EPI == kGated ? 1 : p.products, part, splits);
        for (int at = r.lo; at < r.hi; at += pass_steps<F32>(p, r, at), ++n) {
          if (!arrive()) return;
#pragma unroll
          for (int c = 0; c < kParts; ++c) {
            uint32_t r0[32], r1[32];
            fetch(c, r0, r1);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              x[c][i] = (at > r.lo ? x[c][i] : 0.0f) + __uint_as_float(r0[i]);
              if (EPI == kGated) u[c][i] = (at > r.lo ? u[c][i] : 0.0f) + __uint_as_float(r1[i]);
            }
          }
          release();
        }
      };

      if constexpr (SPLIT) {
        // columns c of 32 of the tile: rows of 16 bytes, a row a lane, 128 rows after each other
        auto sums_at = [&](int c, int which) {
          return (uint32_t)((c * (EPI == kGated ? 2 : 1) + which) * 128 * 32 * 4 + row * 16);
        };
        {
          float x[kParts][32], u[kUps][32];
          collect(x, u);
          if (ok) {  // the ring is free: nothing more is loaded, and what was has been read
#pragma unroll
            for (int c = 0; c < kParts; ++c)
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const uint32_t to = ring + sums_at(half * kParts + c, 0) + i * 512;
                ptx::st_shared_v4(to, __float_as_uint(x[c][i]), __float_as_uint(x[c][i + 1]),
                                  __float_as_uint(x[c][i + 2]), __float_as_uint(x[c][i + 3]));
                if (EPI == kGated) {
                  const uint32_t at = ring + sums_at(half * kParts + c, 1) + i * 512;
                  ptx::st_shared_v4(at, __float_as_uint(u[c][i]), __float_as_uint(u[c][i + 1]),
                                    __float_as_uint(u[c][i + 2]), __float_as_uint(u[c][i + 3]));
                }
              }
          }
        }
        __syncwarp();
        cluster_sync();  // with the other warps, below
        // columns c go to block c % splits, there to half c / splits of the warps
        const int c = first_part;
        if (ok && c < 2 * kParts) {
          float x[32], u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = u[i] = 0.0f;
          for (int b = 0; b < splits; ++b) {
            const uint32_t from = in_block(ring, b);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 v = load_cluster(from + sums_at(c, 0) + i * 512);
              x[i] += v.x, x[i + 1] += v.y, x[i + 2] += v.z, x[i + 3] += v.w;
              if (EPI == kGated) {
                const float4 w = load_cluster(from + sums_at(c, 1) + i * 512);
                u[i] += w.x, u[i + 1] += w.y, u[i + 2] += w.z, u[i + 3] += w.w;
              }
            }
          }
          finish(c, -1, x, u);
        }
        break;  // one tile
      } else if constexpr (F32) {
        float x[kParts][32], u[kUps][32];
        collect(x, u);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < kParts; ++c)
          finish(first_part + c, c + 1 < kParts ? first_part + c + 1 : -1, x[c],
                 u[EPI == kGated ? c : 0]);
      } else {
        const Range r = range_of(p, EPI == kGated ? 1 : p.products, part, splits);
        for (int at = r.lo, len; at < r.hi; at += len, ++n) {
          len = LONG ? pass_steps<F32>(p, r, at) : r.hi - at;
          if (!arrive()) break;
#pragma unroll 1
          for (int c = 0; c < kParts; ++c) {
            uint32_t r0[32], r1[32];
            float x[32], u[32];
            fetch(c, r0, r1);
            if (c + 1 == kParts) release();
            as_floats(x, r0);
            if (EPI == kGated) as_floats(u, r1);
            if (LONG && at > r.lo) add_sums(c, x, u);
            if (LONG && at + len < r.hi)
              put_sums(c, x, u);
            else
              finish(first_part + c, c + 1 < kParts ? first_part + c + 1 : -1, x, u);
          }
        }
        if (!ok) break;
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  if (SPLIT && warp < kFirstEpiWarp) {  // the sums of all blocks are in shared memory
    __syncwarp();
    cluster_sync();
  }
  __syncthreads();
  ptx::tc_fence_before();
  // nothing of the other blocks is on its way here any more, and they have read what they need
  if (CG == 2 || SPLIT) cluster_sync();
  ptx::tc_fence_after();
  if (warp == 2) tmem_give<CG>(tmem, 2 * BN);
}

// -------------------------------------------------------------------------- host side

// A matrix of 16-bit elements in `planes` planes: rows of `cols` elements `stride` apart.
struct Matrix {
  const void* p;
  int64_t rows, cols, stride, plane;
};
bool map_of(EncodeTiledFn enc, CUtensorMap* m, const Matrix& x, bool bf16, int planes,
            int box_inner, int box_rows) {
  auto bytes = [](int64_t stride, int64_t extent) {
    return (cuuint64_t)(extent > 1 ? stride * 2 : 16);
  };
  const cuuint64_t dims[3] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {bytes(x.stride, x.rows), bytes(x.plane, planes)};
  const cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(x.p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_inner == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of a call: pairs of SMs (CG 2), single ones, or clusters of `splits` for each tile.
struct Shape {
  int cg, splits;
  double cost;
};

template <int CG, int EPI, bool F32>
struct Builder {
  EncodeTiledFn enc = tensor_map_encoder();
  Job j{};
  bool ok = enc != nullptr, bf16;
  static constexpr int kCols = EPI == kGated ? 64 * CG : 128 * CG;

  Builder(const fconv_mlp_desc& d, float* saved, float* pass_sums) {
    j.saved = saved;
    j.sums = pass_sums;
    j.quads = (d.hidden + 3) / 4;
    j.act = d.activation;
    j.alpha = d.alpha;
    j.bf16 = d.dtype == FCONV_BF16;
    bf16 = F32 || j.bf16;
  }
  // A new problem, D of M x N as sums over K, and how its operands lie.
  Problem& add(int64_t M, int64_t N, int64_t K, bool a_mn, bool b_mn) {
    Problem& p = j.p[j.problems++];
    p.a_mn = a_mn;
    p.b_mn = b_mn;
    p.mt = (int)((M + 128 * CG - 1) / (128 * CG));
    p.nt = (int)((N + kCols - 1) / kCols);
    p.steps = (int)((K + kStep - 1) / kStep);
    p.M = M;
    p.N = (int)N;
    j.tiles += p.mt * p.nt;
    return p;
  }
  void operand(CUtensorMap* m, const Matrix& x, bool mn, int rows) {
    ok = ok && map_of(enc, m, x, bf16, F32 ? kPlanes : 1, 64, mn ? 64 : rows);
  }
  void product(Problem& p, const Matrix& a, const Matrix& b) {
    operand(&p.a[p.products], a, p.a_mn, 128);
    operand(&p.b[p.products], b, p.b_mn, EPI == kGated && CG == 1 ? 64 : 128);
    ++p.products;
  }
  // An operand of a later product.
  void inner(Problem& p, int i, const Matrix& c) {
    ok = ok && map_of(enc, &p.c[i], c, bf16, F32 ? kPlanes : 1, 32, 32);
  }
  // A result of the call: by boxes where its rows are whole 16-byte units (a box writes the unit that
  // a row ends in as a whole) and start on one.
  void result(Problem& p, void* out, int64_t rows, int64_t cols, int64_t stride) {
    if (!F32 && cols % 8 == 0 && (uintptr_t)out % 16 == 0 && (rows <= 1 || stride % 8 == 0)) {
      inner(p, 0, {out, rows, cols, stride, 0});
    } else {
      p.out = out;
      p.out_row = stride;
    }
  }
  int launch(int sms, int splits, cudaStream_t s) {
    if (!ok) return (int)cudaErrorInvalidValue;
    if (j.tiles == 0) return 0;
    j.splits = splits;
    if constexpr (CG == 1) {
      if (splits > 1) return start<true, false>(j.tiles * splits, splits, s);
    }
    const int most = sms / CG, blocks = (j.tiles < most ? j.tiles : most) * CG;
    if constexpr (!F32) {
      bool passes = false;
      for (int i = 0; i < j.problems; ++i)
        passes = passes || j.p[i].products * j.p[i].steps > kLong;
      if (passes && !j.sums) return (int)cudaErrorInvalidValue;  // the layout has no room for them
      if (passes) return start<false, true>(blocks, CG, s);
    }
    return start<false, false>(blocks, CG, s);
  }
  template <bool SPLIT, bool LONG>
  int start(int blocks, int cluster, cudaStream_t s) {
    const size_t smem = kStages<EPI, F32> * 2 * kSide + kEpiWarps * kSlots<EPI, F32> * kSlot;
    auto kernel = mlp_tc<CG, EPI, F32, SPLIT, LONG>;
    if (const int e = allow_smem((const void*)kernel, smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, j);
  }
};

// What the products read: the call's tensors, or their copies in the workspace.
struct Inputs {
  Matrix x, gate, up, down, dy;
  Matrix h, dg, du;
  float* pass_sums;  // of 16-bit types where a sum is long, else null
};

// h, and where `saved` is given the projections.
template <int CG, bool F32>
int gated(const fconv_mlp_desc& d, int sms, int splits, const MlpArgs& a, const Inputs& in,
          cudaStream_t s) {
  Builder<CG, kGated, F32> b(d, a.saved, in.pass_sums);
  Problem& p = b.add(d.tokens, d.hidden, d.features, false, false);
  b.product(p, in.x, in.gate);
  b.operand(&p.b[1], in.up, false, CG == 1 ? 64 : 128);
  p.bias[0] = a.b_gate;
  p.bias[1] = a.b_up;
  b.inner(p, 0, in.h);
  return b.launch(sms, splits, s);
}

template <int CG, bool F32>
int down(const fconv_mlp_desc& d, int sms, int splits, const MlpArgs& a, const Inputs& in,
         cudaStream_t s) {
  Builder<CG, kPlain, F32> b(d, nullptr, in.pass_sums);
  Problem& p = b.add(d.tokens, d.out_features, d.hidden, false, false);
  b.product(p, in.h, in.down);
  p.bias[0] = a.b_down;
  b.result(p, a.y, d.tokens, d.out_features, d.y_stride);
  return b.launch(sms, splits, s);
}

template <int CG, bool F32>
int grads_of_projections(const fconv_mlp_desc& d, int sms, int splits, const MlpArgs& a,
                         const Inputs& in, cudaStream_t s) {
  Builder<CG, kGrad, F32> b(d, a.saved, in.pass_sums);
  Problem& p = b.add(d.tokens, d.hidden, d.out_features, false, true);
  b.product(p, in.dy, in.down);
  b.inner(p, 0, in.dg);
  b.inner(p, 1, in.du);
  b.inner(p, 2, in.h);
  return b.launch(sms, splits, s);
}

// dx and the weights' gradients, of which `a` may leave some out.
template <int CG, bool F32>
int gradients(const fconv_mlp_desc& d, int sms, int splits, const MlpArgs& a, const Inputs& in,
              cudaStream_t s) {
  Builder<CG, kPlain, F32> b(d, nullptr, in.pass_sums);
  if (a.dx) {
    Problem& p = b.add(d.tokens, d.features, d.hidden, false, true);
    b.product(p, in.dg, in.gate);
    b.product(p, in.du, in.up);
    b.result(p, a.dx, d.tokens, d.features, d.dx_stride);
  }
  auto weight = [&](const Matrix& g, const Matrix& x, void* out) {
    if (!out) return;
    Problem& p = b.add(g.cols, x.cols, d.tokens, true, true);
    b.product(p, g, x);
    b.result(p, out, g.cols, x.cols, x.cols);
  };
  weight(in.dg, in.x, a.dw_gate);
  weight(in.du, in.x, a.dw_up);
  weight(in.dy, in.h, a.dw_down);
  return b.launch(sms, splits, s);
}

// Tiles of one length: those of a product of M x N (in columns of accumulators: gated ones have two
// for each of D), of one SM and of a pair, and their steps of K.
struct Group {
  int64_t tiles1, tiles2, steps;
};
Group group_of(int64_t M, int64_t N, int64_t K, int products) {
  auto tiles = [&](int side) { return ((M + side - 1) / side) * ((N + side - 1) / side); };
  return Group{tiles(128), tiles(256), products * ((K + kStep - 1) / kStep)};
}

// The blocks of a launch: what takes the least time, counted in steps of a single SM's tile (0.19 us
// where operands come from HBM). A step of a pair of SMs takes 1.2 of them, a round of tiles 4 to 6
// more, a cluster's start and its exchange of sums 12 to 24 (196 tokens, each product launched by itself:
// 2048 to 768 takes 13.7 us with 12 blocks, 12.2, 10.9 and 12.0 with 2, 4 and 8 times as many, 768 to 2048
// in 64 tiles 9.9 and 11.4; in a captured graph, where one starts as the other ends, both take 15).
// Clusters of 4 and 8 leave SMs of a GPC unused.
Shape shape_of(const fconv_mlp_desc& d, const Group* g, int n, int sms) {
  constexpr double kRound = 4.0, kSplitRound = 6.0, kPair = 1.2, kGain = 0.93;
  const double terms = d.dtype == FCONV_F32 ? kTerms : 1;
  // rounds of `slots` tiles, each as long as the longest of them
  auto cost = [&](bool pairs, int64_t slots, double round, double step, int splits) {
    double sum = 0.0;
    int64_t over = 0;  // slots of the last round that the next group can use
    for (int i = 0; i < n; ++i) {
      int64_t tiles = pairs ? g[i].tiles2 : g[i].tiles1;
      const int64_t used = tiles < over ? tiles : over;
      over -= used;
      tiles -= used;
      const int64_t rounds = (tiles + slots - 1) / slots;
      sum += (double)rounds * (round + step * (double)((g[i].steps + splits - 1) / splits));
      if (rounds > 0) over = rounds * slots - tiles;
    }
    return sum;
  };
  int64_t least_steps = g[0].steps, tiles = 0;
  for (int i = 0; i < n; ++i) {
    if (g[i].steps < least_steps) least_steps = g[i].steps;
    tiles += g[i].tiles1;
  }
  Shape best{1, 1, cost(false, sms, kRound, terms, 1)};
  for (int splits = 2; splits <= 8; splits *= 2) {
    const int64_t slots = sms / splits - (splits == 8 ? 3 : splits == 4 ? 2 : 0);
    if (slots < 1 || least_steps < 2 * splits || tiles * splits > (1 << 30)) break;
    const double c = 8 + 2 * splits + cost(false, slots, kSplitRound, terms, splits);
    if (c < kGain * best.cost) best = Shape{1, splits, c};
  }
  if (d.dtype != FCONV_F32 && sms > 1) {
    const double c = cost(true, sms / 2, kRound, kPair, 1);
    if (c <= best.cost) best = Shape{2, 1, c};
  }
  return best;
}
Shape shape_of(const fconv_mlp_desc& d, int64_t M, int64_t N, int64_t K, int sms) {
  const Group g = group_of(M, N, K, 1);
  return shape_of(d, &g, 1, sms);
}
#define FCONV_BY_SHAPE(v, call)                                          \
  (d.dtype == FCONV_F32 ? call<1, true>(d, sms, (v).splits, a, l.in, s)  \
   : (v).cg == 2        ? call<2, false>(d, sms, 1, a, l.in, s)          \
                        : call<1, false>(d, sms, (v).splits, a, l.in, s))

// Rows in the workspace start on 128 bytes: a box's row then is one line of L2, not parts of two.
int64_t whole_row(int64_t cols) { return (cols + 63) / 64 * 64; }
size_t whole256(size_t n) { return (n + 255) / 256 * 256; }

// A tensor of the call that TMA does not take as it is: f32, rows that do not start on 16 bytes or
// that overlap.
bool needs_copy(const fconv_mlp_desc& d, int64_t rows, int64_t cols, int64_t stride) {
  if (d.dtype == FCONV_F32) return true;
  return rows > 1 && (stride % 8 != 0 || stride < cols || stride >= (1LL << 39));
}

// The workspace, and the operands in it or where the call has them. Copies come in `prep`.
struct Layout {
  size_t bytes = 0;
  Inputs in{};
  PrepArgs prep{};
  float* sums = nullptr;
};
Layout layout(const fconv_mlp_desc& d, const MlpArgs& a, bool backward, int sms) {
  Layout l;
  const bool few = d.tokens <= kMlpFewTokens;
  // of what the workspace holds: f32 operands in three parts, 16-bit h of few tokens in two
  const int planes = d.dtype == FCONV_F32 ? kPlanes : few && !backward ? 2 : 1;
  char* base = (char*)a.ws;
  auto take = [&](size_t bytes) {
    char* p = base + l.bytes;
    l.bytes += whole256(bytes);
    return p;
  };
  auto fresh = [&](int64_t rows, int64_t cols) {
    Matrix m{nullptr, rows, cols, whole_row(cols), 0};
    m.plane = rows * m.stride;
    m.p = take((size_t)m.plane * planes * 2);
    return m;
  };
  auto input = [&](const void* p, int64_t rows, int64_t cols, int64_t stride) {
    if (!needs_copy(d, rows, cols, stride)) return Matrix{p, rows, cols, stride, 0};
    const Matrix m = fresh(rows, cols);
    l.prep.m[l.prep.count++] = {p, const_cast<void*>(m.p), rows, cols, stride, m.stride, m.plane};
    return m;
  };
  l.in.h = fresh(d.tokens, d.hidden);
  // each block's share of the largest tile: 128 rows of 256 columns (few tokens: of the backward pass)
  int64_t longest = d.features > d.hidden ? d.features : d.hidden;
  if (backward) {  // over tokens and outputs too, and over both projections of hidden values
    for (int64_t k : {2 * d.hidden, d.tokens, d.out_features}) longest = k > longest ? k : longest;
  }
  if (planes == 1 && longest > kLong * kStep)
    l.in.pass_sums = (float*)take((size_t)sms * 128 * 256 * sizeof(float));
  if (backward) {
    l.in.dg = fresh(d.tokens, d.hidden);
    l.in.du = fresh(d.tokens, d.hidden);
    const int64_t cols[3] = {d.hidden, d.hidden, d.out_features};
    l.sums = (float*)take(column_sums_workspace(cols, sms));
    l.in.dy = input(a.dy, d.tokens, d.out_features, d.dy_stride);
  } else if (few) {
    return l;  // the weight-streaming kernels read everything where it is
  }
  l.in.x = input(a.x, d.tokens, d.features, d.x_stride);
  l.in.gate = input(a.w_gate, d.hidden, d.features, d.gate_stride);
  l.in.up = input(a.w_up, d.hidden, d.features, d.up_stride);
  l.in.down = input(a.w_down, d.out_features, d.hidden, d.down_stride);
  return l;
}

int gradients_by_shape(const fconv_mlp_desc& d, int sms, const Shape& v, const MlpArgs& a,
                       const Layout& l, cudaStream_t s) {
  return FCONV_BY_SHAPE(v, gradients);
}
// A call that wants dx alone, or the weights' gradients alone.
MlpArgs only(const MlpArgs& a, bool dx) {
  MlpArgs v = a;
  if (dx)
    v.dw_gate = v.dw_up = v.dw_down = nullptr;
  else
    v.dx = nullptr;
  return v;
}

// g, u and h (few tokens: if wanted).
int projections(const fconv_mlp_desc& d, int sms, const MlpArgs& a, const Layout& l, bool want_h,
                cudaStream_t s) {
  if (d.tokens <= kMlpFewTokens)
    return launch_mlp_few_gated(d, a, want_h ? const_cast<void*>(l.in.h.p) : nullptr,
                                l.in.h.stride, l.in.h.plane, s);
  return FCONV_BY_SHAPE(shape_of(d, d.tokens, 2 * d.hidden, d.features, sms), gated);
}

}  // namespace

bool mlp_tc_supported(const fconv_mlp_desc& d, const MlpArgs& a, bool backward) {
  if (d.tokens == 0) return false;
  auto there = [&](const void* p, int64_t rows, int64_t cols, int64_t stride) {
    return (uintptr_t)p % 16 == 0 || needs_copy(d, rows, cols, stride);
  };
  if (!backward && d.tokens <= kMlpFewTokens) return true;
  return there(a.x, d.tokens, d.features, d.x_stride) &&
         there(a.w_gate, d.hidden, d.features, d.gate_stride) &&
         there(a.w_up, d.hidden, d.features, d.up_stride) &&
         there(a.w_down, d.out_features, d.hidden, d.down_stride) &&
         (!backward || there(a.dy, d.tokens, d.out_features, d.dy_stride));
}

size_t mlp_tc_workspace(const fconv_mlp_desc& d, bool backward, int sms) {
  return layout(d, MlpArgs{}, backward, sms).bytes;
}

int launch_mlp_tc_forward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  const Layout l = layout(d, a, false, sms);
  int e = launch_mlp_prep(d.dtype, l.prep, s);
  if (!e) e = projections(d, sms, a, l, true, s);
  if (e) return e;
  if (d.tokens <= kMlpFewTokens) return launch_mlp_few_down(d, a, l.in.h.p, l.in.h.stride, l.in.h.plane, s);
  return FCONV_BY_SHAPE(shape_of(d, d.tokens, d.out_features, d.hidden, sms), down);
}

int launch_mlp_tc_backward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  const int64_t T = d.tokens, D = d.features, F = d.hidden, O = d.out_features;
  const Layout l = layout(d, a, true, sms);
  int e = launch_mlp_prep(d.dtype, l.prep, s);
  // made again, the projections are the forward pass's bit by bit
  if (!e && a.remake) e = projections(d, sms, a, l, false, s);
  if (!e) e = FCONV_BY_SHAPE(shape_of(d, T, F, O, sms), grads_of_projections);
  // Nothing of dx goes into the weights' gradients or back, so tiles of all may share the GPU in one
  // launch of persistent blocks, unless their lengths want shapes of their own (few tokens: long sums
  // for dx, short ones for the weights). Both passes of 6304 x 768 x 2048 in f16: 186 us with two
  // launches, 182 with one; the gradients of 100 x 3000 x 4000 in f32: 259 and 406 us; clusters that
  // took both gained nothing (999 x 333 x 777, f32, both passes: 123 and 130).
  Group g[4];
  int n = 0;  // in the order of the launch's problems
  if (a.dx) g[n++] = group_of(T, D, F, 2);
  const int after_dx = n;
  if (a.dw_gate) g[n++] = group_of(F, D, T, 1);
  if (a.dw_up) g[n++] = group_of(F, D, T, 1);
  if (a.dw_down) g[n++] = group_of(O, F, T, 1);
  if (!e && n > 0) {
    constexpr double kLaunch = 10.0;  // steps that a launch of its own costs
    const Shape all = shape_of(d, g, n, sms);
    const Shape first = after_dx > 0 ? shape_of(d, g, after_dx, sms) : all;
    const Shape rest = n > after_dx ? shape_of(d, g + after_dx, n - after_dx, sms) : all;
    if (after_dx > 0 && n > after_dx &&
        (all.splits > 1 || first.cost + rest.cost + kLaunch < all.cost)) {
      e = gradients_by_shape(d, sms, first, only(a, true), l, s);
      if (!e) e = gradients_by_shape(d, sms, rest, only(a, false), l, s);
    } else {
      e = gradients_by_shape(d, sms, all, a, l, s);
    }
  }
  if (e) return e;
  const Matrix* from[3] = {&l.in.dg, &l.in.du, &l.in.dy};
  void* to[3] = {a.db_gate, a.db_up, a.db_down};
  SumsArgs m[3];
  for (int i = 0; i < 3; ++i) m[i] = {from[i]->p, from[i]->stride, from[i]->cols, from[i]->plane, to[i]};
  const bool early = n > 0;  // the launch before has waited for dg, du and dy
  return launch_column_sums(d.dtype, d.dtype == FCONV_F32, early, m, T, l.sums, sms, s);
}

int read_and_clear_mlp_error(cudaStream_t s, unsigned* value) {
  return read_and_clear_error(s, value);
}

}  // namespace ops
}  // namespace fconv
