// The gated feed-forward block on tcgen05 tensor cores (include/fconv_ops.h): f16 and bf16 with
// sizes and strides of whole 16-byte units.
//
//   forward   h = act(x Wg^T + bg) * (x Wu^T + bu)      both products in one accumulator
//             y = h Wd^T + bd
//   backward  dh = dy Wd;  dg = dh u act'(g), du = dh act(g), h = act(g) u   in its epilogue
//             dx = dg Wg + du Wu                         one sum over both
//             dWg = dg^T x, dWu = du^T x, dWd = dy^T h   one launch
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
// that blocks at work at one time share operands in L2.
#include "mlp_math.cuh"
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
constexpr uint32_t kSlot = 128 * 64;       // staged output: 128 rows of 32 values
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8, kFirstEpiWarp = 4;

enum { kPlain, kGated, kGrad };

template <int EPI>
constexpr int kStages = EPI == kGrad ? 5 : 6;
template <int EPI>
constexpr int kSlots = EPI == kGrad ? 3 : 2;  // of each epilogue warpgroup

struct Problem {
  CUtensorMap a[2], b[2], c[3];  // terms of a sum (kGated: gate and up), outputs
  int mt, nt, steps;             // tiles, steps of a term
  int terms;
  int64_t M;
  int N;
  const void* bias[2];
};
struct Job {
  Problem p[3];
  int problems, tiles;
  float* saved;
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
                                         uint32_t bar) {
  if (CG == 1) {
    ptx::tma_load_2d(dst, map, c0, c1, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  }
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::
                   "l"((uint64_t)map),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read_but() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// The same answer for `count` threads (whole warps): whether all of them have `ok`.
__device__ __forceinline__ bool bar_and(uint32_t id, uint32_t count, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(count), "r"((uint32_t)ok)
      : "memory");
  return all != 0;
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

__device__ __forceinline__ uint32_t pack16(bool bf16, float a, float b) {
  return bf16 ? pack2<true>(a, b) : pack2<false>(a, b);
}
__device__ __forceinline__ float2 unpack16(bool bf16, uint32_t v) {
  if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// A row's 8 N / 4... values: N words of a 32-column row (64 bytes) of a staged box in the 64-byte
// swizzle, from word w0 on.
template <int N>
__device__ __forceinline__ void stage(uint32_t slot, int row, int w0, const uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    ptx::st_shared_v4(slot + row * 64 + ((((w0 + i) >> 2) ^ ((row >> 1) & 3)) << 4), w[i], w[i + 1],
                      w[i + 2], w[i + 3]);
}

// x[i] += bias[col + i] for 32 columns, those past N left alone (N is a multiple of 8).
__device__ __forceinline__ void add_bias(float (&x)[32], const void* bias, int col, int N,
                                         bool bf16) {
  if (!bias) return;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    if (col + i >= N) break;
    const uint4 v = ptx::ldg_nc_v4((const uint16_t*)bias + col + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack16(bf16, w[k]);
      x[i + 2 * k] += f.x;
      x[i + 2 * k + 1] += f.y;
    }
  }
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

template <int CG, bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(kThreads, 1) mlp_tc(const __grid_constant__ Job j) {
  constexpr int S = kStages<EPI>, BN = 128 * CG;
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
  if (warp == 2) tmem_take<CG>(ptx::smem_addr(&ctl.tmem), 2 * BN);
  ptx::tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int first = (int)blockIdx.x / CG, stride = (int)gridDim.x / CG;

  if (warp == 0) {  // loads
    int it = 0;
    bool ok = true;
    for (int id = first; ok && id < j.tiles; id += stride) {
      const Tile t = tile_of(j, id);
      const Problem& p = j.p[t.which];
      const int m0 = (t.m * CG + (int)rank) * 128;
      const int n0 = EPI == kGated ? t.n * kCols : t.n * BN + (int)rank * 128;
      const int terms = EPI == kGated ? 1 : p.terms;
      for (int term = 0; ok && term < terms; ++term) {
        for (int k = 0; k < p.steps; ++k, ++it) {
          const int s = it % S;
          ok = all_lanes(wait_bar(ptx::smem_addr(&ctl.empty[s]), ((it / S) & 1) ^ 1, abort_flag));
          if (!ok) break;
          const uint32_t own = ptx::smem_addr(&ctl.full[s]);
          const uint32_t bar = CG == 1 ? own : in_first(own);
          const uint32_t sa = ring + s * kStageBytes, sb = sa + kSide;
          if (elect_lane()) {
            if (rank == 0) ptx::mbar_arrive_expect_tx(own, CG * kStageBytes);
            if (AMN) {
              load_box<CG>(sa, &p.a[term], m0, k * kStep, bar);
              load_box<CG>(sa + kBox, &p.a[term], m0 + 64, k * kStep, bar);
            } else {
              load_box<CG>(sa, &p.a[term], k * kStep, m0, bar);
            }
            if (BMN) {
              load_box<CG>(sb, &p.b[term], n0, k * kStep, bar);
              load_box<CG>(sb + kBox, &p.b[term], n0 + 64, k * kStep, bar);
            } else if (EPI == kGated && CG == 1) {
              load_box<CG>(sb, &p.b[0], k * kStep, n0, bar);
              load_box<CG>(sb + kBox, &p.b[1], k * kStep, n0, bar);
            } else if (EPI == kGated) {
              load_box<CG>(sb, &p.b[rank], k * kStep, n0, bar);
            } else {
              load_box<CG>(sb, &p.b[term], k * kStep, n0, bar);
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
      const uint32_t idesc = idesc_16(j.bf16, 128 * CG, BN, BMN) | (AMN ? 1u << 15 : 0u);
      int it = 0, n = 0;
      bool ok = true;
      for (int id = first; ok && id < j.tiles; id += stride, ++n) {
        const Tile t = tile_of(j, id);
        const Problem& p = j.p[t.which];
        const int steps = p.steps * (EPI == kGated ? 1 : p.terms);
        const uint32_t d = tmem + (n & 1) * BN;
        ok = all_lanes(
            wait_cluster(ptx::smem_addr(&ctl.acc_empty[n & 1]), ((n >> 1) & 1) ^ 1, abort_flag));
        ptx::tc_fence_after();
        for (int k = 0; ok && k < steps; ++k, ++it) {
          const int s = it % S;
          ok = all_lanes(wait_bar(ptx::smem_addr(&ctl.full[s]), (it / S) & 1, abort_flag));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t sa = ring + s * kStageBytes, sb = sa + kSide;
          const uint32_t a = uni(AMN ? desc_mn(sa, kBox) : desc_k(sa));
          const uint32_t b = uni(BMN ? desc_mn(sb, kBox) : desc_k(sb));
          if (elect_lane()) {
#pragma unroll
            for (int i = 0; i < kStep / 16; ++i)  // 16 elements of a row, or 16 rows
              mma<CG>(d, a + i * (AMN ? 128 : 2), b + i * (BMN ? 128 : 2), idesc, k > 0 || i > 0);
            commit<CG>(ptx::smem_addr(&ctl.empty[s]));
            if (k + 1 == steps) commit<CG>(ptx::smem_addr(&ctl.acc_full[n & 1]));
          }
          __syncwarp();
        }
      }
      if (!ok) {  // the products issued so far read both blocks' shared memory
        if (elect_lane()) commit<CG>(ptx::smem_addr(&ctl.done));
        __syncwarp();
        drain_bar(ptx::smem_addr(&ctl.done), 0);
      }
    }
  } else if (warp >= kFirstEpiWarp) {
    const int half = (warp - kFirstEpiWarp) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t slots = ring + S * kStageBytes + half * kSlots<EPI> * kSlot;
    const bool bf16 = j.bf16;
    const bool issues = threadIdx.x == (kFirstEpiWarp + 4 * half) * 32;
    const int act = j.act;
    const float alpha = j.alpha;
    int n = 0, slot = 0;
    for (int id = first; id < j.tiles; id += stride, ++n) {
      const Tile t = tile_of(j, id);
      const Problem& p = j.p[t.which];
      const int m0 = (t.m * CG + (int)rank) * 128;
      const int64_t grow = (int64_t)m0 + row;
      // saved values of this warp's rows: block of 32 rows, a row a lane
      float* saved = nullptr;
      if (EPI != kPlain && j.saved)
        saved = j.saved + (grow >> 5) * j.quads * 256 + lane * 4;
      // the warps of a group, which meet at barriers below, go on or give up together
      if (!bar_and(1 + half, 128,
                   wait_bar(ptx::smem_addr(&ctl.acc_full[n & 1]), (n >> 1) & 1, abort_flag)))
        break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + (n & 1) * BN + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < kCols / 64; ++c) {
        const int tcol = half * (kCols / 2) + c * 32, col = t.n * kCols + tcol;
        uint32_t r0[32], r1[32];
        tmem_fetch32(acc + tcol, r0);
        if (EPI == kGated) tmem_fetch32(acc + BN / 2 + tcol, r1);
        tmem_wait_ld();
        tmem_arrived(r0);
        if (EPI == kGated) tmem_arrived(r1);
        if (c + 1 == kCols / 64) {  // the accumulator is free
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            const uint32_t bar = ptx::smem_addr(&ctl.acc_empty[n & 1]);
            if (CG == 1) ptx::mbar_arrive(bar);
            else arrive_cluster(in_first(bar));
          }
        }
        if (col >= p.N) continue;  // the same for the whole warpgroup
        if (issues) bulk_wait_read_but<EPI == kGrad ? 0 : kSlots<EPI> - 1>();
        ptx::bar_sync(1 + half, 128);
        if (EPI == kPlain) {
          float x[32];
          as_floats(x, r0);
          add_bias(x, p.bias[0], col, p.N, bf16);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack16(bf16, x[2 * i], x[2 * i + 1]);
          stage(slots + slot * kSlot, row, 0, w);
        } else if (EPI == kGated) {
          float g[32], u[32];
          as_floats(g, r0);
          as_floats(u, r1);
          add_bias(g, p.bias[0], col, p.N, bf16);
          add_bias(u, p.bias[1], col, p.N, bf16);
          if (saved && grow < p.M) {
            float* to = saved + (int64_t)(col >> 2) * 256;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              if (col + i >= p.N) break;
              *reinterpret_cast<float4*>(to + i * 64) =
                  make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]);
              *reinterpret_cast<float4*>(to + i * 64 + 128) =
                  make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]);
            }
          }
          uint32_t w[16];
#define FCONV_M(ACT) gate<ACT>(w, g, u, alpha, bf16)
          FCONV_GATE_SWITCH(act, FCONV_M)
#undef FCONV_M
          stage(slots + slot * kSlot, row, 0, w);
        } else {
          const float* from = saved + (int64_t)(col >> 2) * 256;
          float dh[32];
          as_floats(dh, r0);
#define FCONV_M(ACT)                                                                        \
  _Pragma("unroll") for (int i = 0; i < 32; i += 8) {                                       \
    uint32_t wg[4], wu[4], wh[4];                                                           \
    float4 g[2] = {}, u[2] = {};                                                            \
    if (grow < p.M && col + i < p.N) {                                                      \
      _Pragma("unroll") for (int k = 0; k < 2; ++k) {                                       \
        g[k] = __ldcg(reinterpret_cast<const float4*>(from + (i + 4 * k) * 64));            \
        u[k] = __ldcg(reinterpret_cast<const float4*>(from + (i + 4 * k) * 64 + 128));      \
      }                                                                                     \
    }                                                                                       \
    gate_grad<ACT>(wg, wu, wh, dh + i, g, u, alpha, bf16);                                  \
    stage(slots, row, i / 2, wg);                                                           \
    stage(slots + kSlot, row, i / 2, wu);                                                   \
    stage(slots + 2 * kSlot, row, i / 2, wh);                                               \
  }
          FCONV_GATE_SWITCH(act, FCONV_M)
#undef FCONV_M
        }
        ptx::fence_proxy_async_smem();
        ptx::bar_sync(1 + half, 128);
        if (issues && m0 < p.M) {
          if (EPI == kGrad) {
#pragma unroll
            for (int i = 0; i < 3; ++i) store_box(&p.c[i], slots + i * kSlot, col, m0);
          } else {
            store_box(&p.c[0], slots + slot * kSlot, col, m0);
          }
          bulk_commit();
        }
        if (EPI != kGrad) slot ^= 1;
      }
    }
    if (issues) bulk_wait_all();
  }
  __syncthreads();
  ptx::tc_fence_before();
  if (CG == 2) cluster_sync();  // nothing of the other block is on its way here any more
  ptx::tc_fence_after();
  if (warp == 2) tmem_give<CG>(tmem, 2 * BN);
}

// -------------------------------------------------------------------------- host side

// A matrix of `rows` rows of `inner` elements `stride` apart, in boxes of box_inner x box_rows.
bool map_of(EncodeTiledFn enc, CUtensorMap* m, const void* p, bool bf16, int64_t inner,
            int64_t rows, int64_t stride, int box_inner, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? stride : inner) * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows};
  const cuuint32_t one[2] = {1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
             const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_inner == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Matrix {
  const void* p;
  int64_t rows, cols, stride;
};

template <int CG, bool AMN, bool BMN, int EPI>
struct Builder {
  EncodeTiledFn enc = tensor_map_encoder();
  Job j{};
  bool ok = enc != nullptr;
  static constexpr int kCols = EPI == kGated ? 64 * CG : 128 * CG;

  Builder(const fconv_mlp_desc& d, float* saved) {
    j.saved = saved;
    j.quads = (d.hidden + 3) / 4;
    j.act = d.activation;
    j.alpha = d.alpha;
    j.bf16 = d.dtype == FCONV_BF16;
  }
  // A new problem, D of M x N as sums over K.
  Problem& add(int64_t M, int64_t N, int64_t K) {
    Problem& p = j.p[j.problems++];
    p.mt = (int)((M + 128 * CG - 1) / (128 * CG));
    p.nt = (int)((N + kCols - 1) / kCols);
    p.steps = (int)((K + kStep - 1) / kStep);
    p.terms = 0;
    p.M = M;
    p.N = (int)N;
    j.tiles += p.mt * p.nt;
    return p;
  }
  void operand(CUtensorMap* m, const Matrix& x, bool mn, int rows) {
    ok = ok && map_of(enc, m, x.p, j.bf16, x.cols, x.rows, x.stride, 64, mn ? 64 : rows);
  }
  void term(Problem& p, const Matrix& a, const Matrix& b) {
    operand(&p.a[p.terms], a, AMN, 128);
    operand(&p.b[p.terms], b, BMN, EPI == kGated && CG == 1 ? 64 : 128);
    ++p.terms;
  }
  void output(Problem& p, int i, const Matrix& c) {
    ok = ok && map_of(enc, &p.c[i], c.p, j.bf16, c.cols, c.rows, c.stride, 32, 128);
  }
  int launch(int sms, cudaStream_t s) {
    if (!ok) return (int)cudaErrorInvalidValue;
    if (j.tiles == 0) return 0;
    const size_t smem = kStages<EPI> * 2 * kSide + 2 * kSlots<EPI> * kSlot;
    auto kernel = mlp_tc<CG, AMN, BMN, EPI>;
    if (const int e = allow_smem((const void*)kernel, smem)) return e;
    const int most = sms / CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((j.tiles < most ? j.tiles : most) * CG));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, j);
  }
};

// h, and where `saved` is given the projections.
template <int CG>
int gated(const fconv_mlp_desc& d, int sms, const MlpArgs& a, void* h, cudaStream_t s) {
  Builder<CG, false, false, kGated> b(d, a.saved);
  Problem& p = b.add(d.tokens, d.hidden, d.features);
  b.term(p, {a.x, d.tokens, d.features, d.x_stride}, {a.w_gate, d.hidden, d.features, d.gate_stride});
  b.operand(&p.b[1], {a.w_up, d.hidden, d.features, d.up_stride}, false, CG == 1 ? 64 : 128);
  p.bias[0] = a.b_gate;
  p.bias[1] = a.b_up;
  b.output(p, 0, {h, d.tokens, d.hidden, d.hidden});
  return b.launch(sms, s);
}

template <int CG>
int down(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  Builder<CG, false, false, kPlain> b(d, nullptr);
  Problem& p = b.add(d.tokens, d.out_features, d.hidden);
  b.term(p, {a.h, d.tokens, d.hidden, d.hidden}, {a.w_down, d.out_features, d.hidden, d.down_stride});
  p.bias[0] = a.b_down;
  b.output(p, 0, {a.y, d.tokens, d.out_features, d.y_stride});
  return b.launch(sms, s);
}

template <int CG>
int grads_of_projections(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  Builder<CG, false, true, kGrad> b(d, a.saved);
  Problem& p = b.add(d.tokens, d.hidden, d.out_features);
  b.term(p, {a.dy, d.tokens, d.out_features, d.dy_stride},
         {a.w_down, d.out_features, d.hidden, d.down_stride});
  const void* out[3] = {a.dg, a.du, a.h};
  for (int i = 0; i < 3; ++i) b.output(p, i, {out[i], d.tokens, d.hidden, d.hidden});
  return b.launch(sms, s);
}

template <int CG>
int grad_of_input(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  Builder<CG, false, true, kPlain> b(d, nullptr);
  Problem& p = b.add(d.tokens, d.features, d.hidden);
  b.term(p, {a.dg, d.tokens, d.hidden, d.hidden}, {a.w_gate, d.hidden, d.features, d.gate_stride});
  b.term(p, {a.du, d.tokens, d.hidden, d.hidden}, {a.w_up, d.hidden, d.features, d.up_stride});
  b.output(p, 0, {a.dx, d.tokens, d.features, d.dx_stride});
  return b.launch(sms, s);
}

template <int CG>
int grads_of_weights(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  Builder<CG, true, true, kPlain> b(d, nullptr);
  auto one = [&](const Matrix& g, const Matrix& in, void* out) {
    if (!out) return;
    Problem& p = b.add(g.cols, in.cols, d.tokens);
    b.term(p, g, in);
    b.output(p, 0, {out, g.cols, in.cols, in.cols});
  };
  const Matrix x = {a.x, d.tokens, d.features, d.x_stride};
  one({a.dg, d.tokens, d.hidden, d.hidden}, x, a.dw_gate);
  one({a.du, d.tokens, d.hidden, d.hidden}, x, a.dw_up);
  one({a.dy, d.tokens, d.out_features, d.dy_stride}, {a.h, d.tokens, d.hidden, d.hidden}, a.dw_down);
  return b.launch(sms, s);
}

// Pairs of SMs where their tiles of 256 x (256, gated: 128) fill half of the GPU at least.
bool pairs_fill(int64_t M, int64_t N, int sms) {
  return ((M + 255) / 256) * ((N + 255) / 256) * 4 >= sms;
}

// g, u and h.
int projections(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  if (d.tokens <= kMlpFewTokens) return launch_mlp_few_gated(d, a, s);
  return pairs_fill(d.tokens, 2 * d.hidden, sms) ? gated<2>(d, sms, a, a.h, s)
                                                 : gated<1>(d, sms, a, a.h, s);
}

}  // namespace

bool mlp_tc_supported(const fconv_mlp_desc& d) {
  if (d.dtype == FCONV_F32) return false;
  auto whole = [](int64_t rows, int64_t cols, int64_t stride) {
    if (cols % 8 != 0) return false;
    return rows <= 1 || (stride % 8 == 0 && stride >= cols && stride < (1LL << 39));
  };
  if (!whole(d.tokens, d.features, d.x_stride) || !whole(d.tokens, d.out_features, d.y_stride) ||
      !whole(d.hidden, d.features, d.gate_stride) || !whole(d.hidden, d.features, d.up_stride) ||
      !whole(d.out_features, d.hidden, d.down_stride) || d.hidden % 8 != 0)
    return false;
  return !d.training || (whole(d.tokens, d.out_features, d.dy_stride) &&
                         whole(d.tokens, d.features, d.dx_stride));
}

int launch_mlp_tc_forward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  if (const int e = projections(d, sms, a, s)) return e;
  if (d.tokens <= kMlpFewTokens) return launch_mlp_few_down(d, a, s);
  return pairs_fill(d.tokens, d.out_features, sms) ? down<2>(d, sms, a, s) : down<1>(d, sms, a, s);
}

int launch_mlp_tc_backward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s) {
  const int64_t T = d.tokens;
  // made again, the projections are the forward pass's bit by bit (h, too, is written again)
  int e = a.remake ? projections(d, sms, a, s) : 0;
  if (!e)
    e = pairs_fill(T, d.hidden, sms) ? grads_of_projections<2>(d, sms, a, s)
                                     : grads_of_projections<1>(d, sms, a, s);
  if (!e && a.dx)
    e = pairs_fill(T, d.features, sms) ? grad_of_input<2>(d, sms, a, s)
                                       : grad_of_input<1>(d, sms, a, s);
  if (!e && (a.dw_gate || a.dw_up || a.dw_down))
    e = pairs_fill(2 * d.hidden + d.out_features, d.features, sms)
            ? grads_of_weights<2>(d, sms, a, s)
            : grads_of_weights<1>(d, sms, a, s);
  return e;
}

int read_and_clear_mlp_error(cudaStream_t s, unsigned* value) {
  return read_and_clear_error(s, value);
}

}  // namespace ops
}  // namespace fconv
