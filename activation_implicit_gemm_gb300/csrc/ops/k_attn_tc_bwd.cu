// Attention backward on the tcgen05 tensor cores (f16 and bf16, head_dim a multiple of 8 up to
// 128), the probabilities made again from lse:
//   p = exp(scale q k^T - lse),  dp = dout v^T,  ds = p (dp - delta),  delta_i = dout_i . out_i
//   dv = p^T dout,  dk = scale ds^T q,  dq = scale ds k
//
// attn_tc_delta writes -lse (in log2) and -delta per packed query row.
// attn_tc_dkv owns 128 keys of a (batch, key head) and walks the query tiles of all the heads
// that share them; attn_tc_dq owns 128 packed query rows and walks the key tiles. dq needs
// nothing of dkv's: its blocks start as dkv's end, and it waits for dkv only before it ends (f16
// images of 197 tokens: 86 -> 82 us a training pass; the causal size below: 699 -> 690). Every
// gradient element has one writer that adds in a fixed order: no atomics, the same bits every
// time. The price is that q k^T and dout v^T are made twice: 7 products of 128 x 128 x D a tile
// pair instead of 5, while one kernel for all five would add dq in f32 atomics (32 bits a value
// of extra traffic, an order that changes from run to run, and a conversion pass).
//
// Both kernels turn the score tile so that its rows are what they own. p and ds are rounded to
// 16 bits into TMEM over the scores they come from and are the A operand of the products that
// follow, whose B operand is the tile already in shared memory read MN-major: no transposes and
// no shared-memory round trip.
//   dkv: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q     (512 TMEM columns in all)
//   dq:  S = Q K^T (two buffers), dP = dO V^T, dQ += dS K
// The MMA warp orders them so that elementwise work always overlaps two products:
//   dkv: dV(i) S(i+1) | dK(i) dP(i+1)      dq: S(j+1) | dP(j+1) dQ(j)
// Eight elementwise warps split a tile: warp w has TMEM lanes 32 (w % 4).., columns
// 64 (w / 4)... Roles: warps 0-7 elementwise, 8 MMA, 9 TMA.
//
// f16 range: p is scaled by 2^12 and ds by the power of two that puts the largest possible
// |dp - delta| (from the largest norms of dout and v rows of the head) at 2^15, undone exactly
// in the epilogue: small gradients do not fall into f16's subnormals and none overflows. bf16
// needs neither.
//
// Bound: tensor (14 D FLOPs a pair as run, 10 D counted). 2 x 4096 tokens in causal order, 32
// heads of 128 on 8, bf16 (4096 and 2631 valid): delta 22 us, dkv 280, dq 241. In dkv the tensor
// pipe waits for p and ds between its products (4096 tokens of 19 heads: 219 us, the products
// alone 180); dq waits for its K and V tiles, each from L2 for one query tile (there 214 us, 193
// without elementwise work, 128 without the loads as well). 32 x 197 tokens, 12 heads of 64, f16:
// delta 10 us, dkv 33, dq 24: 768 items of two tiles, a chain of latencies each, on 152 SMs.
#include "attn_tc.cuh"

#include <climits>
#include <cmath>
#include <cstring>

namespace fconv {
namespace ops {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kLaunchRegs = 168, kWorkRegs = 216, kOtherRegs = 72;
static_assert(2 * kWorkRegs + kOtherRegs <= 3 * kLaunchRegs, "within the launch's registers");
constexpr int kPShift = 12;               // log2 of p's scale in f16
constexpr uint32_t kStatBytes = 2 * kTile * 4;

struct BwdArgs {
  TcGeom g;
  int splits, per;   // splits of the walked axis, tiles of a split
  int items;
  int* counter;      // of the items handed out, or null
  const float* stat;   // [b][hk][query tile]: 128 of -lse (log2, with p's scale), 128 of -delta
  const float* gmax;   // f16: [b][hk][query tile] largest |dout row|^2
  const float* vmax;   // f16: [b][hk][key tile] largest |v row|^2
  int64_t o1[3], o2[3];
  void* out1;          // dq, or dk
  void* out2;          // dv
  float* part1;        // splits > 1: [split][b][head][token][D]
  float* part2;
};

// ------------------------------------------------------------------------------ delta

struct DeltaArgs {
  TcGeom g;
  int64_t o[3], d[3], v[3];
  const uint16_t* out;
  const uint16_t* dout;
  const uint16_t* val;
  const float* lse;
  float* stat;
  float* gmax;
  float* vmax;
  int* counters;  // two, set to zero for the kernels that follow
};

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// A block per query tile of a (batch, key head); in f16 also one per key tile for the largest
// value norm. LPR lanes share a row, eight elements each, so RP rows go at a time.
template <bool BF16, int LPR>
__global__ void __launch_bounds__(256, 4) attn_tc_delta(const DeltaArgs a) {
  constexpr int RP = 256 / LPR, N = kTile / RP;
  __shared__ float top[RP];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x < 2) a.counters[threadIdx.x] = 0;
  const TcGeom& g = a.g;
  const int per = g.qtiles + (BF16 ? 0 : g.ktiles);
  const int bh = blockIdx.x / per, tile = blockIdx.x - bh * per;
  const int b = bh / g.Hk, hk = bh - b * g.Hk;
  const TcLens l = tc_lens(g, b);
  const int sub = threadIdx.x / LPR, at = threadIdx.x % LPR, d = at * 8;
  float most = 0.0f;
  if (tile < g.qtiles) {
    float* stat = a.stat + ((int64_t)bh * g.qtiles + tile) * (2 * kTile);
    // four rows of a lane in flight, and the lse of all that it shares
    float lse = -INFINITY;
    {
      const int n = at, r = sub + n * RP, tok = r / g.G, i = tile * g.toks + tok;
      if (n < N && r < g.rows && i >= l.lead && i < l.q)
        lse = a.lse[((int64_t)b * g.Hq + (int64_t)hk * g.G + (r - tok * g.G)) * g.Lq + i];
    }
    const uint16_t* out = a.out + b * a.o[0] + (int64_t)hk * g.G * a.o[2] + d;
    const uint16_t* dout = a.dout + b * a.d[0] + (int64_t)hk * g.G * a.d[2] + d;
    float delta = 0.0f;
#pragma unroll 1
    for (int n0 = 0; n0 < N; n0 += 4) {
      uint4 x[4], y[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int r = sub + (n0 + n) * RP, tok = r / g.G, i = tile * g.toks + tok;
        const int64_t h = r - tok * g.G;
        x[n] = y[n] = make_uint4(0, 0, 0, 0);
        if (r < g.rows && i >= l.lead && i < l.q && d < g.D) {
          x[n] = ptx::ldg_nc_v4(out + i * a.o[1] + h * a.o[2]);
          y[n] = ptx::ldg_nc_v4(dout + i * a.d[1] + h * a.d[2]);
        }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t xs[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
        const uint32_t ys[4] = {y[n].x, y[n].y, y[n].z, y[n].w};
        float s = 0.0f, z = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u = unpack2<BF16>(xs[e]), v = unpack2<BF16>(ys[e]);
          s = fmaf(u.x, v.x, fmaf(u.y, v.y, s));
          z = fmaf(v.x, v.x, fmaf(v.y, v.y, z));
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
          s += __shfl_xor_sync(0xffffffffu, s, o);
          if (!BF16) z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        most = fmaxf(most, z);
        if (at == n0 + n) delta = s;
      }
    }
    const int n = at;
    if (n < N) {
      // -lse is added to the scores; a row that sees nothing (or only scores of -inf) gets
      // -inf: its p is 0
      stat[sub + n * RP] =
          lse == -INFINITY ? -INFINITY : (BF16 ? 0.0f : (float)kPShift) - lse * kLog2e;
      stat[kTile + sub + n * RP] = -delta;  // 0 where the row takes no part
    }
  } else {
    const int j0 = (tile - g.qtiles) * kTile;
    uint4 y[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int j = j0 + sub + n * RP;
      y[n] = make_uint4(0, 0, 0, 0);
      if (j < l.k && d < g.D)
        y[n] = ptx::ldg_nc_v4(a.val + b * a.v[0] + (int64_t)j * a.v[1] + hk * a.v[2] + d);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t ys[4] = {y[n].x, y[n].y, y[n].z, y[n].w};
      float z = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = unpack2<BF16>(ys[e]);
        z = fmaf(v.x, v.x, fmaf(v.y, v.y, z));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      most = fmaxf(most, z);
    }
  }
  if (BF16) return;
  if (at == 0) top[sub] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 0; i < RP; ++i) most = fmaxf(most, top[i]);
    if (tile < g.qtiles) a.gmax[(int64_t)bh * g.qtiles + tile] = most;
    else a.vmax[(int64_t)bh * g.ktiles + tile - g.qtiles] = most;
  }
}

// k such that 2^k (dp - delta) stays below 2^15: |dp - delta| <= 2 |dout| |v|.
__device__ __forceinline__ int grad_shift(const BwdArgs& a, int bh, int lane) {
  float x = 0.0f, y = 0.0f;
  for (int i = lane; i < a.g.qtiles; i += 32)
    x = fmaxf(x, __ldcg(a.gmax + (int64_t)bh * a.g.qtiles + i));
  for (int i = lane; i < a.g.ktiles; i += 32)
    y = fmaxf(y, __ldcg(a.vmax + (int64_t)bh * a.g.ktiles + i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
  }
  const float top = 2.0f * sqrtf(x) * sqrtf(y);
  if (!(top > 0.0f) || top == INFINITY) return 0;
  const int e = (int)(__float_as_uint(top) >> 23) - 127;  // top < 2^(e + 1)
  return min(max(14 - e, -100), 100);
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// ------------------------------------------------------------------------------ shared parts

// D[128 x 128] = A B^T over head_dim, both K-major tiles in shared memory.
template <int H>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b, int dk,
                                           uint32_t idesc) {
  const uint32_t x = desc_k(a), y = desc_k(b);
#pragma unroll
  for (int s = 0; s < 4 * H; ++s)
    if (s < dk) mma_ss(d, x + k_step(s), y + k_step(s), idesc, s > 0);
}

// D[128 x head_dim] (+)= A B over the 128 columns of a score tile: A in TMEM, its two column
// halves 64 columns apart, B a tile read MN-major. PART 0 and 1: the first and the last 32 of
// each half's columns.
template <int PART>
__device__ __forceinline__ void mma_grads(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                          bool first) {
  const uint32_t y = desc_mn(b);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int h = n >> 1, s = PART * 2 + (n & 1);  // half, K step of the half
    mma_ts(d, a + h * 64 + s * 8, y + (h * 4 + s) * (2048 >> 4), idesc, !first || PART || n);
  }
}

// One thread's row of an accumulator, columns [c0, c0 + 32 H), times mul: to a 16-bit row or
// to an f32 partial row. `ok`: the row exists; `keep`: it has a gradient (else zeros).
template <bool BF16, int H>
__device__ __forceinline__ void store_grad(uint32_t at, int c0, int D, float mul, bool ok,
                                           bool keep, bool fetch, uint16_t* out, float* part) {
#pragma unroll
  for (int q = 0; q < H; ++q) {
    const int d0 = c0 + q * 32;
    if (d0 >= D) return;
    uint32_t o[32];
    if (fetch) {
      tmem_fetch32(at + d0, o);
      tmem_wait_ld();
      tmem_arrived(o);
    }
    if (!ok) continue;
    float f[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) f[e] = keep ? __uint_as_float(o[e]) * mul : 0.0f;
    if (part) {
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        if (d0 + e < D)
          *reinterpret_cast<float4*>(part + d0 + e) =
              make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < 32; e += 8)
        if (d0 + e < D)
          ptx::st_global_v4(out + d0 + e,
                            make_uint4(pack2<BF16>(f[e], f[e + 1]), pack2<BF16>(f[e + 2], f[e + 3]),
                                       pack2<BF16>(f[e + 4], f[e + 5]),
                                       pack2<BF16>(f[e + 6], f[e + 7])));
    }
  }
}

// One thread's half row of an accumulator, columns [32 H half, 32 H (half + 1)), times mul, into
// a staged tile of H boxes of 64 columns.
template <bool BF16, int H>
__device__ __forceinline__ void stage_grad(uint32_t at, int half, int row, float mul, bool keep,
                                           uint32_t tile) {
#pragma unroll
  for (int q = 0; q < H; ++q) {
    const int d0 = half * 32 * H + q * 32;
    uint32_t o[32], w[16];
    tmem_fetch32(at + d0, o);
    tmem_wait_ld();
    tmem_arrived(o);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      w[e] = keep ? pack2<BF16>(__uint_as_float(o[2 * e]) * mul, __uint_as_float(o[2 * e + 1]) * mul)
                  : 0u;
    stage_row(tile + (d0 >> 6) * kHalfBytes, row, d0 & 63, w);
  }
}

// All eight warps have written what they store (or read what they free): true in warp 0 when
// they have, in the others at once.
__device__ __forceinline__ bool store_ready(uint64_t& bar, uint32_t n, int warp, int lane,
                                            volatile int* abort_flag) {
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&bar));
  return warp != 0 || wait_bar(ptx::smem_addr(&bar), n & 1, abort_flag);
}

// ------------------------------------------------------------------------------ dq

struct DqItem {
  int valid, b, hk, split, t0, tile, jb, n, shift;  // shift: log2 of ds's scale (f16)
  TcLens l;
};

__device__ __forceinline__ void dq_item(const BwdArgs& a, int u, DqItem& it) {
  it.valid = u < a.items;
  if (!it.valid) return;
  it.split = u % a.splits;
  u /= a.splits;
  const int bh = (int)a.g.B * a.g.Hk;
  if (a.g.causal) {  // the query tiles with most keys first
    it.tile = a.g.qtiles - 1 - u / bh;
    u %= bh;
  } else {
    it.tile = u % a.g.qtiles;
    u /= a.g.qtiles;
  }
  it.hk = u % a.g.Hk;
  it.b = u / a.g.Hk;
  it.l = tc_lens(a.g, it.b);
  it.t0 = it.tile * a.g.toks;
  it.jb = it.split * a.per;
  it.n = max(min(key_tiles(a.g, it.l, it.t0) - it.jb, a.per), 0);
}

template <int H>
struct DqPlan {
  static constexpr uint32_t tile = H * kHalfBytes;
  static constexpr int own = H == 1 ? 2 : 1;    // buffers of (Q, dO)
  static constexpr int slots = H == 1 ? 8 : 5;  // ring of K and V tiles
};
template <int H>
struct DqCtl {
  uint64_t full[DqPlan<H>::slots], empty[DqPlan<H>::slots];
  uint64_t own_full[2], own_empty[2];
  uint64_t tail, drain, s_full[2], dp_full, dp_free, done;
  uint64_t ds_ready[2][2];  // [step's parity][column part]: a warp may be a step ahead of another
  uint64_t out_ready;
  Sched<DqItem> sched;
  uint32_t tmem;
  int abort_flag;
};
template <int H>
constexpr uint32_t dq_smem() {
  return (2 * DqPlan<H>::own + DqPlan<H>::slots) * DqPlan<H>::tile + sizeof(DqCtl<H>);
}
static_assert(dq_smem<2>() <= 232448 && dq_smem<1>() <= 232448, "one block's shared memory");

template <bool BF16, int H>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_dq(const BwdArgs a, const __grid_constant__ CUtensorMap tm_q,
               const __grid_constant__ CUtensorMap tm_g, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ CUtensorMap tm_o1) {
  using Plan = DqPlan<H>;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  if (!smem_ok(dsmem)) return;
  DqCtl<H>& ctl = *reinterpret_cast<DqCtl<H>*>(dsmem + (2 * Plan::own + Plan::slots) * Plan::tile);
  const TcGeom& g = a.g;
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;
  const uint32_t own = ptx::smem_addr(dsmem), ring = own + 2 * Plan::own * Plan::tile;
  volatile int* abort_flag = &ctl.abort_flag;

  if (tid == 0) {
    for (int i = 0; i < Plan::slots; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.own_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.own_empty[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.s_full[i]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl.tail), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.drain), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.dp_full), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.dp_free), 8);
    for (int i = 0; i < 4; ++i) ptx::mbar_init(ptx::smem_addr(&ctl.ds_ready[i >> 1][i & 1]), 8);
    ptx::mbar_init(ptx::smem_addr(&ctl.done), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.out_ready), 8);
    sched_init(ctl.sched);
    ctl.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_addr(&ctl.tmem), 512);
    ptx::tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_g);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = uni(ctl.tmem);
  // No wait for the launch before: that is attn_tc_dkv, which let this one start after its own
  // wait for the delta pass, so all that is read here is complete (read from L2, since nothing
  // orders this SM's L1 after the delta pass).

  if (warp >= 8) {
    regs_fewer<kOtherRegs>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- TMA producer
      uint32_t c = 0, items = 0, tails = 0;
      DqItem it;
      bool stop = false;
      auto make = [&](int u, DqItem& x) {
        dq_item(a, u, x);
        x.shift = !BF16 && x.valid ? grad_shift(a, x.b * g.Hk + x.hk, lane) : 0;
      };
      for (int k = 0; !stop && sched_make(ctl.sched, k, it, a.counter, lane, abort_flag, make);
           ++k) {
        if (it.n == 0) continue;
        const uint32_t ob = items % Plan::own;
        if (!wait_bar(ptx::smem_addr(&ctl.own_empty[ob]), ((items / Plan::own) & 1) ^ 1,
                      abort_flag))
          break;
        ++items;
        if (lane == 0) {
          const uint32_t bar = ptx::smem_addr(&ctl.own_full[ob]);
          ptx::mbar_arrive_expect_tx(bar, 2 * H * (uint32_t)g.rows * 128);
          for (int h = 0; h < H; ++h) {
            const uint32_t dst = own + ob * 2 * Plan::tile + h * kHalfBytes;
            tma_load_4d(dst, &tm_q, h * 64, it.hk * g.G, it.t0, it.b * g.qb, bar);
            tma_load_4d(dst + Plan::tile, &tm_g, h * 64, it.hk * g.G, it.t0, it.b * g.gb, bar);
          }
        }
        for (int j = 0; j < 2 * it.n; ++j, ++c) {
          const uint32_t s = c % Plan::slots;
          if (!wait_bar(ptx::smem_addr(&ctl.empty[s]), ((c / Plan::slots) & 1) ^ 1, abort_flag)) {
            stop = true;
            break;
          }
          const int key0 = (it.jb + (j >> 1)) * kTile;
          const uint32_t dst = ring + s * Plan::tile;
          const bool is_v = j & 1;
          // rows of K past the sequence meet ds = 0 in dq += ds k: a NaN there must not count
          const bool ragged = !is_v && key0 + kTile > it.l.k && it.l.k < g.Lk;
          const uint32_t full = ptx::smem_addr(&ctl.full[s]);
          const uint32_t bar = ragged ? ptx::smem_addr(&ctl.tail) : full;
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(bar, Plan::tile);
            for (int h = 0; h < H; ++h)
              tma_load_4d(dst + h * kHalfBytes, is_v ? &tm_v : &tm_k, h * 64,
                          it.hk * (is_v ? g.vh : g.kh), key0, it.b * (is_v ? g.vb : g.kb), bar);
          }
          if (ragged) {
            if (!wait_bar(bar, tails & 1, abort_flag)) {
              drain_bar(bar, tails & 1);
              stop = true;
              break;
            }
            ++tails;
            zero_rows(dst, H, it.l.k - key0, kTile, lane);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full);
          }
        }
      }
      if (*abort_flag) {
        for (uint32_t i = c > Plan::slots ? c - Plan::slots : 0; i < c; ++i)
          drain_bar(ptx::smem_addr(&ctl.full[i % Plan::slots]), (i / Plan::slots) & 1);
        for (uint32_t i = items > Plan::own ? items - Plan::own : 0; i < items; ++i)
          drain_bar(ptx::smem_addr(&ctl.own_full[i % Plan::own]), (i / Plan::own) & 1);
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issue
      const bool leader = elect_lane();
      const int dk = (g.D + 15) / 16;
      const uint32_t id_s = idesc_16(BF16, kTile, kTile, false);
      const uint32_t id_g = idesc_16(BF16, kTile, dk * 16, true);
      const uint32_t dp = tmem + 256, dq = tmem + 384;
      uint32_t c = 0, items = 0, steps = 0;
      DqItem it;
      bool stop = false;
      auto wait = [&](uint64_t& bar, uint32_t parity) {
        return all_lanes(wait_bar(ptx::smem_addr(&bar), parity, abort_flag));
      };
      auto commit = [&](uint64_t& bar) {
        if (leader) ptx::mma_commit(ptx::smem_addr(&bar));
      };
      auto wait_slot = [&](uint32_t i) {
        return wait(ctl.full[i % Plan::slots], (i / Plan::slots) & 1);
      };
      auto slot = [&](uint32_t i) { return ring + i % Plan::slots * Plan::tile; };
      auto free_slot = [&](uint32_t i) { commit(ctl.empty[i % Plan::slots]); };
      for (int k = 0; !stop && sched_take(ctl.sched, k, it, lane, abort_flag); ++k) {
        const int n = uni(it.n);
        if (n == 0) continue;
        const uint32_t ob = items % Plan::own;
        if (!wait(ctl.own_full[ob], (items / Plan::own) & 1) || !wait_slot(c) || !wait_slot(c + 1))
          break;
        ++items;
        const uint32_t q = own + ob * 2 * Plan::tile, go = q + Plan::tile;
        ptx::tc_fence_after();
        if (leader) mma_scores<H>(tmem + (steps & 1) * 128, q, slot(c), dk, id_s);
        commit(ctl.s_full[steps & 1]);
        if (leader) mma_scores<H>(dp, go, slot(c + 1), dk, id_s);
        commit(ctl.dp_full);
        free_slot(c + 1);
        for (int j = 0; j < n; ++j, c += 2, ++steps) {
          const bool more = j + 1 < n;
          if (more) {
            if (!wait_slot(c + 2)) {
              stop = true;
              break;
            }
            ptx::tc_fence_after();
            if (leader) mma_scores<H>(tmem + ((steps + 1) & 1) * 128, q, slot(c + 2), dk, id_s);
            commit(ctl.s_full[(steps + 1) & 1]);
            if (!wait(ctl.dp_free, steps & 1) || !wait_slot(c + 3)) {
              stop = true;
              break;
            }
            ptx::tc_fence_after();
            if (leader) mma_scores<H>(dp, go, slot(c + 3), dk, id_s);
            commit(ctl.dp_full);
            free_slot(c + 3);
          }
          const uint32_t ds = tmem + (steps & 1) * 128;
          if (!wait(ctl.ds_ready[steps & 1][0], (steps >> 1) & 1)) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          if (leader) mma_grads<0>(dq, ds, slot(c), id_g, j == 0);
          if (!wait(ctl.ds_ready[steps & 1][1], (steps >> 1) & 1)) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          if (leader) mma_grads<1>(dq, ds, slot(c), id_g, j == 0);
          free_slot(c);
          if (!more) commit(ctl.done);
        }
      }
      commit(ctl.drain);
      drain_bar(ptx::smem_addr(&ctl.drain), 0);
    }
  } else {
    // ------------------------------------------------------------------ elementwise, epilogue
    regs_more<kWorkRegs>();
    const int half = warp >> 2, row = tid & 127, tok = row / g.G, head = row - tok * g.G;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint64_t c2 = pair(g.scale * kLog2e, g.scale * kLog2e);
    uint32_t steps = 0, items = 0;
    DqItem it;
    for (int k = 0; sched_take(ctl.sched, k, it, lane, abort_flag); ++k) {
      const int i = it.t0 + tok, bh = it.b * g.Hk + it.hk;
      const int limit = row < g.rows ? key_limit(g, it.l, i) : 0;
      const float* stat = a.stat + ((int64_t)bh * g.qtiles + it.tile) * (2 * kTile);
      const float nl = __ldcg(stat + row);
      const uint64_t nlse = pair(nl, nl);
      const int shift = it.shift;
      const float gs = BF16 ? 1.0f : pow2i(shift - kPShift), nd = __ldcg(stat + kTile + row) * gs;
      const uint64_t gs2 = pair(gs, gs), nd2 = pair(nd, nd);
      bool stop = false;
      for (int j = 0; j < it.n; ++j, ++steps) {
        const uint32_t s_at = tmem + (steps & 1) * 128 + half * 64 + lanes;
        const uint32_t dp_at = tmem + 256 + half * 64 + lanes;
        if (!wait_bar(ptx::smem_addr(&ctl.s_full[steps & 1]), (steps >> 1) & 1, abort_flag)) {
          stop = true;
          break;
        }
        ptx::tc_fence_after();
        uint32_t s[2][32], dp[2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_fetch32(s_at + q * 32, s[q]);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tmem_arrived(s[q]);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x = fma2(pair(s[q][e], s[q][e + 1]), c2, nlse);
            s[q][e] = __float_as_uint(exp2_fast(low(x)));
            s[q][e + 1] = __float_as_uint(exp2_fast(high(x)));
          }
        }
        if (!wait_bar(ptx::smem_addr(&ctl.dp_full), steps & 1, abort_flag)) {
          stop = true;
          break;
        }
        ptx::tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_fetch32(dp_at + q * 32, dp[q]);
        tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.dp_free));
        const int seen = limit - (it.jb + j) * kTile - half * 64;
        const bool masked = __any_sync(0xffffffffu, seen < 64);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tmem_arrived(dp[q]);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            uint64_t x = pair(dp[q][e], dp[q][e + 1]);
            x = BF16 ? add2(x, nd2) : fma2(x, gs2, nd2);
            x = mul2(x, pair(s[q][e], s[q][e + 1]));
            dp[q][e] = (uint32_t)x;
            dp[q][e + 1] = (uint32_t)(x >> 32);
          }
          if (masked) {  // hidden columns, whatever their scores and products are
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e >= seen) dp[q][e] = 0;
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack2<BF16>(__uint_as_float(dp[q][2 * e]), __uint_as_float(dp[q][2 * e + 1]));
          tmem_store16(s_at + q * 16, w);
          tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.ds_ready[steps & 1][q]));
        }
      }
      if (stop) break;
      if (it.n > 0) {
        if (!wait_bar(ptx::smem_addr(&ctl.done), items & 1, abort_flag)) break;
        ++items;
        ptx::tc_fence_after();
      }
      const bool keep = limit > 0;
      const float mul = g.scale * (BF16 ? 1.0f : pow2i(-shift));
      if (a.splits == 1 && it.n > 0) {
        // over Q, which has been read last, and out as one box
        const uint32_t ob = (items - 1) % Plan::own, box = own + ob * 2 * Plan::tile;
        stage_grad<BF16, H>(tmem + 384 + lanes, half, row, mul, keep, box);
        if (!store_ready(ctl.out_ready, items - 1, warp, lane, abort_flag)) break;
        if (tid == 0) {
          for (int x = 0; x < H; ++x)
            tma_store_4d(&tm_o1, box + x * kHalfBytes, x * 64, it.hk * g.G, it.t0, it.b);
          bulk_commit();
          bulk_wait_read();
          ptx::mbar_arrive(ptx::smem_addr(&ctl.own_empty[ob]));
        }
        continue;
      }
      const bool ok = row < g.rows && i < g.Lq;
      const int64_t h = (int64_t)it.hk * g.G + head;
      uint16_t* out = (uint16_t*)a.out1 + it.b * a.o1[0] + i * a.o1[1] + h * a.o1[2];
      float* part = nullptr;
      if (a.splits > 1)
        part = a.part1 + ((((int64_t)it.split * g.B + it.b) * g.Hq + h) * g.Lq + i) * g.D;
      store_grad<BF16, H>(tmem + 384 + lanes, half * 32 * H, g.D, mul, ok, it.n > 0 && keep,
                          it.n > 0, out, part);
      if (it.n > 0) {  // Q and dO are free once every warp is here
        if (!store_ready(ctl.out_ready, items - 1, warp, lane, abort_flag)) break;
        if (tid == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.own_empty[(items - 1) % Plan::own]));
      }
    }
    if (tid == 0) bulk_wait_all();
  }

  ptx::pdl_wait();  // attn_tc_dkv: what follows this kernel follows both
  ptx::pdl_trigger();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------ dk, dv

struct DkvItem {
  int valid, b, hk, split, tile, ib, n, shift;  // query tiles [ib, ib + n)
  TcLens l;
};

__device__ __forceinline__ void dkv_item(const BwdArgs& a, int u, DkvItem& it) {
  it.valid = u < a.items;
  if (!it.valid) return;
  it.split = u % a.splits;
  u /= a.splits;
  const int bh = (int)a.g.B * a.g.Hk;
  if (a.g.causal) {  // the first keys are seen by most queries
    it.tile = u / bh;
    u %= bh;
  } else {
    it.tile = u % a.g.ktiles;
    u /= a.g.ktiles;
  }
  it.hk = u % a.g.Hk;
  it.b = u / a.g.Hk;
  it.l = tc_lens(a.g, it.b);
  const int j0 = it.tile * kTile;
  // queries [first, q) see a key of the tile
  const int first = max(it.l.lead, a.g.causal ? j0 - it.l.shift : 0);
  int lo = first / a.g.toks, hi = (it.l.q + a.g.toks - 1) / a.g.toks;
  if (j0 >= it.l.k || first >= it.l.q) hi = lo = 0;
  it.ib = max(lo, it.split * a.per);
  it.n = max(min(hi, (it.split + 1) * a.per) - it.ib, 0);
}

template <int H>
struct DkvPlan {
  static constexpr uint32_t tile = H * kHalfBytes;
  static constexpr int own = H == 1 ? 2 : 1;   // buffers of (K, V)
  static constexpr int qs = H == 1 ? 4 : 3, gs = H == 1 ? 4 : 2;  // Q and dO tiles in flight
  static constexpr int stats = 2;
  static constexpr uint32_t stat_at = (2 * own + qs + gs) * tile;
  static constexpr uint32_t ctl_at = stat_at + stats * kStatBytes;
};
template <int H>
struct DkvCtl {
  uint64_t q_full[DkvPlan<H>::qs], q_empty[DkvPlan<H>::qs];
  uint64_t g_full[DkvPlan<H>::gs], g_empty[DkvPlan<H>::gs];
  uint64_t st_full[2], st_empty[2];
  uint64_t own_full[2], own_empty[2];
  uint64_t tail, drain, s_full, dp_full, p_ready[2], ds_ready[2], done;
  uint64_t out_ready;
  Sched<DkvItem> sched;
  uint32_t tmem;
  int abort_flag;
};
template <int H>
constexpr uint32_t dkv_smem() {
  return DkvPlan<H>::ctl_at + sizeof(DkvCtl<H>);
}
static_assert(dkv_smem<2>() <= 232448 && dkv_smem<1>() <= 232448, "one block's shared memory");

template <bool BF16, int H>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_dkv(const BwdArgs a, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ CUtensorMap tm_g, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_o1,
                const __grid_constant__ CUtensorMap tm_o2) {
  using Plan = DkvPlan<H>;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  if (!smem_ok(dsmem)) return;
  DkvCtl<H>& ctl = *reinterpret_cast<DkvCtl<H>*>(dsmem + Plan::ctl_at);
  const TcGeom& g = a.g;
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;
  const uint32_t own = ptx::smem_addr(dsmem);
  const uint32_t qring = own + 2 * Plan::own * Plan::tile, gring = qring + Plan::qs * Plan::tile;
  const uint32_t stats = own + Plan::stat_at;
  volatile int* abort_flag = &ctl.abort_flag;

  if (tid == 0) {
    for (int i = 0; i < Plan::qs; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.q_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.q_empty[i]), 1);
    }
    for (int i = 0; i < Plan::gs; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.g_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.g_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.st_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.st_empty[i]), 8);
      ptx::mbar_init(ptx::smem_addr(&ctl.own_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.own_empty[i]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl.tail), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.drain), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.s_full), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.dp_full), 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.p_ready[i]), 8);
      ptx::mbar_init(ptx::smem_addr(&ctl.ds_ready[i]), 8);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl.done), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.out_ready), 8);
    sched_init(ctl.sched);
    ctl.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  // rows that no box ever fills (G not a power of two) meet p = 0 in the products over the
  // query rows: they hold zeros from here on
  if (g.rows < kTile && warp < 8) {
    for (int i = warp; i < Plan::qs + Plan::gs; i += 8)
      zero_rows(qring + i * Plan::tile, H, g.rows, kTile, lane);
    ptx::fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_addr(&ctl.tmem), 512);
    ptx::tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_g);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = uni(ctl.tmem);
  ptx::pdl_wait();
  ptx::pdl_trigger();  // attn_tc_dq's blocks take the SMs as this kernel's leave them

  if (warp >= 8) {
    regs_fewer<kOtherRegs>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- TMA producer
      uint32_t c = 0, items = 0, tails = 0;  // c: query tiles loaded so far
      DkvItem it;
      bool stop = false;
      auto make = [&](int u, DkvItem& x) {
        dkv_item(a, u, x);
        x.shift = !BF16 && x.valid ? grad_shift(a, x.b * g.Hk + x.hk, lane) : 0;
      };
      for (int k = 0; !stop && sched_make(ctl.sched, k, it, a.counter, lane, abort_flag, make);
           ++k) {
        if (it.n == 0) continue;
        const uint32_t ob = items % Plan::own;
        if (!wait_bar(ptx::smem_addr(&ctl.own_empty[ob]), ((items / Plan::own) & 1) ^ 1,
                      abort_flag))
          break;
        ++items;
        if (lane == 0) {
          const uint32_t bar = ptx::smem_addr(&ctl.own_full[ob]);
          ptx::mbar_arrive_expect_tx(bar, 2 * Plan::tile);
          for (int h = 0; h < H; ++h) {
            const uint32_t dst = own + ob * 2 * Plan::tile + h * kHalfBytes;
            tma_load_4d(dst, &tm_k, h * 64, it.hk * g.kh, it.tile * kTile, it.b * g.kb, bar);
            tma_load_4d(dst + Plan::tile, &tm_v, h * 64, it.hk * g.vh, it.tile * kTile,
                        it.b * g.vb, bar);
          }
        }
        const int bh = it.b * g.Hk + it.hk;
        for (int i = 0; i < it.n && !stop; ++i, ++c) {
          const int tile = it.ib + i, t0 = tile * g.toks;
          // rows of queries that take no part meet p = ds = 0: a NaN there must not count
          const int lo = min(max(it.l.lead - t0, 0), g.toks) * g.G;
          const int hi = it.l.q < g.Lq ? min(it.l.q - t0, g.toks) * g.G : g.rows;
          const bool ragged = lo > 0 || hi < g.rows;
          const uint32_t ss = c & 1;
          for (int x = 0; x < 2; ++x) {  // Q with the row statistics, then dO
            const uint32_t n = x ? Plan::gs : Plan::qs, s = c % n, ph = (c / n) & 1;
            const uint32_t full = ptx::smem_addr(x ? &ctl.g_full[s] : &ctl.q_full[s]);
            const uint32_t empty = ptx::smem_addr(x ? &ctl.g_empty[s] : &ctl.q_empty[s]);
            const uint32_t dst = (x ? gring : qring) + s * Plan::tile;
            if (!wait_bar(empty, ph ^ 1, abort_flag) ||
                (x == 0 && !wait_bar(ptx::smem_addr(&ctl.st_empty[ss]), ((c >> 1) & 1) ^ 1,
                                     abort_flag))) {
              stop = true;
              break;
            }
            const uint32_t bar = ragged ? ptx::smem_addr(&ctl.tail) : full;
            if (lane == 0) {
              if (x == 0) {
                const uint32_t sb = ptx::smem_addr(&ctl.st_full[ss]);
                ptx::mbar_arrive_expect_tx(sb, kStatBytes);
                bulk_load(stats + ss * kStatBytes,
                          a.stat + ((int64_t)bh * g.qtiles + tile) * (2 * kTile), kStatBytes, sb);
              }
              ptx::mbar_arrive_expect_tx(bar, H * (uint32_t)g.rows * 128);
              for (int h = 0; h < H; ++h)
                tma_load_4d(dst + h * kHalfBytes, x ? &tm_g : &tm_q, h * 64, it.hk * g.G, t0,
                            it.b * (x ? g.gb : g.qb), bar);
            }
            if (ragged) {
              if (!wait_bar(bar, tails & 1, abort_flag)) {
                drain_bar(bar, tails & 1);
                stop = true;
                break;
              }
              ++tails;
              zero_rows(dst, H, 0, lo, lane);
              zero_rows(dst, H, hi, g.rows, lane);
              ptx::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(full);
            }
          }
        }
      }
      if (*abort_flag) {
        // loads in flight land before the block's shared memory is given back; a slot that
        // was never armed runs into the drain's short limit
        for (uint32_t i = c > Plan::qs ? c - Plan::qs : 0; i < c; ++i)
          drain_bar(ptx::smem_addr(&ctl.q_full[i % Plan::qs]), (i / Plan::qs) & 1);
        for (uint32_t i = c > Plan::gs ? c - Plan::gs : 0; i < c; ++i)
          drain_bar(ptx::smem_addr(&ctl.g_full[i % Plan::gs]), (i / Plan::gs) & 1);
        for (uint32_t i = c > 2 ? c - 2 : 0; i < c; ++i)
          drain_bar(ptx::smem_addr(&ctl.st_full[i & 1]), (i >> 1) & 1);
        for (uint32_t i = items > Plan::own ? items - Plan::own : 0; i < items; ++i)
          drain_bar(ptx::smem_addr(&ctl.own_full[i % Plan::own]), (i / Plan::own) & 1);
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issue
      const bool leader = elect_lane();
      const int dk = (g.D + 15) / 16;
      const uint32_t id_s = idesc_16(BF16, kTile, kTile, false);
      const uint32_t id_g = idesc_16(BF16, kTile, dk * 16, true);
      const uint32_t st = tmem, dp = tmem + 128, dv = tmem + 256, dkk = tmem + 384;
      uint32_t c = 0, items = 0;
      DkvItem it;
      bool stop = false;
      auto wait = [&](uint64_t& bar, uint32_t parity) {
        return all_lanes(wait_bar(ptx::smem_addr(&bar), parity, abort_flag));
      };
      auto commit = [&](uint64_t& bar) {
        if (leader) ptx::mma_commit(ptx::smem_addr(&bar));
      };
      auto wait_q = [&](uint32_t i) { return wait(ctl.q_full[i % Plan::qs], (i / Plan::qs) & 1); };
      auto wait_g = [&](uint32_t i) { return wait(ctl.g_full[i % Plan::gs], (i / Plan::gs) & 1); };
      auto q_tile = [&](uint32_t i) { return qring + i % Plan::qs * Plan::tile; };
      auto g_tile = [&](uint32_t i) { return gring + i % Plan::gs * Plan::tile; };
      for (int k = 0; !stop && sched_take(ctl.sched, k, it, lane, abort_flag); ++k) {
        const int n = uni(it.n);
        if (n == 0) continue;
        const uint32_t ob = items % Plan::own;
        if (!wait(ctl.own_full[ob], (items / Plan::own) & 1) || !wait_q(c)) break;
        ++items;
        const uint32_t kt = own + ob * 2 * Plan::tile, vt = kt + Plan::tile;
        ptx::tc_fence_after();
        if (leader) mma_scores<H>(st, kt, q_tile(c), dk, id_s);
        commit(ctl.s_full);
        if (!wait_g(c)) break;
        ptx::tc_fence_after();
        if (leader) mma_scores<H>(dp, vt, g_tile(c), dk, id_s);
        commit(ctl.dp_full);
        for (int i = 0; i < n; ++i, ++c) {
          const bool more = i + 1 < n;
          if (!wait(ctl.p_ready[0], c & 1)) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          if (leader) mma_grads<0>(dv, st, g_tile(c), id_g, i == 0);
          if (!wait(ctl.p_ready[1], c & 1)) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          if (leader) mma_grads<1>(dv, st, g_tile(c), id_g, i == 0);
          commit(ctl.g_empty[c % Plan::gs]);
          if (more) {
            if (!wait_q(c + 1)) {
              stop = true;
              break;
            }
            ptx::tc_fence_after();
            if (leader) mma_scores<H>(st, kt, q_tile(c + 1), dk, id_s);
            commit(ctl.s_full);
          }
          if (!wait(ctl.ds_ready[0], c & 1)) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          if (leader) mma_grads<0>(dkk, dp, q_tile(c), id_g, i == 0);
          if (!wait(ctl.ds_ready[1], c & 1)) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          if (leader) mma_grads<1>(dkk, dp, q_tile(c), id_g, i == 0);
          commit(ctl.q_empty[c % Plan::qs]);
          if (more) {
            if (!wait_g(c + 1)) {
              stop = true;
              break;
            }
            ptx::tc_fence_after();
            if (leader) mma_scores<H>(dp, vt, g_tile(c + 1), dk, id_s);
            commit(ctl.dp_full);
          } else {
            commit(ctl.done);
          }
        }
      }
      commit(ctl.drain);
      drain_bar(ptx::smem_addr(&ctl.drain), 0);
    }
  } else {
    // ------------------------------------------------------------------ elementwise, epilogue
    regs_more<kWorkRegs>();
    const int half = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = tmem + half * 64 + lanes, dp_at = s_at + 128;
    const uint64_t c2 = pair(g.scale * kLog2e, g.scale * kLog2e);
    uint32_t steps = 0, items = 0;
    DkvItem it;
    for (int k = 0; sched_take(ctl.sched, k, it, lane, abort_flag); ++k) {
      const int j = it.tile * kTile + row, bh = it.b * g.Hk + it.hk;
      const int shift = it.shift;
      const float gs = BF16 ? 1.0f : pow2i(shift - kPShift);
      const uint64_t gs2 = pair(gs, gs);
      bool stop = false;
      for (int i = 0; i < it.n; ++i, ++steps) {
        const uint32_t ss = steps & 1;
        const ulonglong2* nlse = reinterpret_cast<const ulonglong2*>(dsmem + Plan::stat_at +
                                                                     ss * kStatBytes) + half * 16;
        const ulonglong2* ndelta = nlse + kTile / 4;
        if (!wait_bar(ptx::smem_addr(&ctl.st_full[ss]), (steps >> 1) & 1, abort_flag)) {
          stop = true;
          break;
        }
        // the columns' statistics are in registers before the scores are there
        ulonglong2 n[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) n[e] = nlse[e];
        if (!wait_bar(ptx::smem_addr(&ctl.s_full), steps & 1, abort_flag)) {
          stop = true;
          break;
        }
        ptx::tc_fence_after();
        uint32_t s[2][32];
        tmem_fetch32(s_at, s[0]);
        // columns [0, hide) are queries before the first that sees key j
        int hide = 0;
        if (g.causal)
          hide = min(max(j - it.l.shift - (it.ib + i) * g.toks, 0), g.toks) * g.G - half * 64;
        const bool masked = __any_sync(0xffffffffu, hide > 0);
        tmem_wait_ld();
        tmem_arrived(s[0]);
        tmem_fetch32(s_at + 32, s[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1) {
            tmem_wait_ld();
            tmem_arrived(s[1]);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const uint64_t x = fma2(pair(s[q][e], s[q][e + 1]), c2, n[q * 8 + e / 4].x);
            const uint64_t y = fma2(pair(s[q][e + 2], s[q][e + 3]), c2, n[q * 8 + e / 4].y);
            s[q][e] = __float_as_uint(exp2_fast(low(x)));
            s[q][e + 1] = __float_as_uint(exp2_fast(high(x)));
            s[q][e + 2] = __float_as_uint(exp2_fast(low(y)));
            s[q][e + 3] = __float_as_uint(exp2_fast(high(y)));
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e < hide) s[q][e] = 0;
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack2<BF16>(__uint_as_float(s[q][2 * e]), __uint_as_float(s[q][2 * e + 1]));
          tmem_store16(s_at + q * 16, w);
          tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.p_ready[q]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = ndelta[e];
        if (!wait_bar(ptx::smem_addr(&ctl.dp_full), steps & 1, abort_flag)) {
          stop = true;
          break;
        }
        ptx::tc_fence_after();
        uint32_t dp[2][32];
        tmem_fetch32(dp_at, dp[0]);
        tmem_wait_ld();
        tmem_arrived(dp[0]);
        tmem_fetch32(dp_at + 32, dp[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] = ndelta[8 + e];
            tmem_wait_ld();
            tmem_arrived(dp[1]);
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            uint64_t x = add2(pair(dp[q][e], dp[q][e + 1]), n[e / 4].x);
            uint64_t y = add2(pair(dp[q][e + 2], dp[q][e + 3]), n[e / 4].y);
            x = mul2(x, pair(s[q][e], s[q][e + 1]));
            y = mul2(y, pair(s[q][e + 2], s[q][e + 3]));
            if (!BF16) {
              x = mul2(x, gs2);
              y = mul2(y, gs2);
            }
            w[e / 2] = pack2<BF16>(low(x), high(x));
            w[e / 2 + 1] = pack2<BF16>(low(y), high(y));
          }
          tmem_store16(dp_at + q * 16, w);
          tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.ds_ready[q]));
        }
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.st_empty[ss]));
      }
      if (stop) break;
      if (it.n > 0) {
        if (!wait_bar(ptx::smem_addr(&ctl.done), items & 1, abort_flag)) break;
        ++items;
        ptx::tc_fence_after();
      }
      const bool keep = it.n > 0 && j < it.l.k;
      const float mul_v = BF16 ? 1.0f : pow2i(-kPShift);
      const float mul_k = g.scale * (BF16 ? 1.0f : pow2i(-shift));
      if (a.splits == 1 && it.n > 0) {
        // dk over K and dv over V, which have been read last, and out as boxes
        const uint32_t ob = (items - 1) % Plan::own, box = own + ob * 2 * Plan::tile;
        stage_grad<BF16, H>(tmem + 384 + lanes, half, row, mul_k, keep, box);
        stage_grad<BF16, H>(tmem + 256 + lanes, half, row, mul_v, keep, box + Plan::tile);
        if (!store_ready(ctl.out_ready, items - 1, warp, lane, abort_flag)) break;
        if (tid == 0) {
          for (int x = 0; x < H; ++x) {
            tma_store_4d(&tm_o1, box + x * kHalfBytes, x * 64, it.hk, it.tile * kTile, it.b);
            tma_store_4d(&tm_o2, box + Plan::tile + x * kHalfBytes, x * 64, it.hk,
                         it.tile * kTile, it.b);
          }
          bulk_commit();
          bulk_wait_read();
          ptx::mbar_arrive(ptx::smem_addr(&ctl.own_empty[ob]));
        }
        continue;
      }
      const bool ok = j < g.Lk;
      uint16_t* o1 = (uint16_t*)a.out1 + it.b * a.o1[0] + j * a.o1[1] + it.hk * a.o1[2];
      uint16_t* o2 = (uint16_t*)a.out2 + it.b * a.o2[0] + j * a.o2[1] + it.hk * a.o2[2];
      float *p1 = nullptr, *p2 = nullptr;
      if (a.splits > 1) {
        const int64_t at = ((((int64_t)it.split * g.B + it.b) * g.Hk + it.hk) * g.Lk + j) * g.D;
        p1 = a.part1 + at;
        p2 = a.part2 + at;
      }
      store_grad<BF16, H>(tmem + 256 + lanes, half * 32 * H, g.D, mul_v, ok, keep, it.n > 0, o2,
                          p2);
      store_grad<BF16, H>(tmem + 384 + lanes, half * 32 * H, g.D, mul_k, ok, keep, it.n > 0, o1,
                          p1);
      if (it.n > 0) {  // K and V are free once every warp is here
        if (!store_ready(ctl.out_ready, items - 1, warp, lane, abort_flag)) break;
        if (tid == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.own_empty[(items - 1) % Plan::own]));
      }
    }
    if (tid == 0) bulk_wait_all();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------ join

struct JoinArgs {
  const float* part[2];
  uint16_t* out[2];
  int64_t st[2][3];
  int64_t rows, len;  // rows = batch * heads * len
  int heads, D, splits, count;
};

// Adds the partial gradients of each row in split order; four elements a thread.
template <bool BF16>
__global__ void __launch_bounds__(256) attn_tc_sum(const JoinArgs a) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int quads = a.D / 4;
  const int64_t total = a.rows * quads;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total * a.count;
       u += (int64_t)gridDim.x * 256) {
    const int w = u >= total;
    const int64_t v = w ? u - total : u, at = v / quads;
    const int d = (int)(v - at * quads) * 4;
    const float* p = (w ? a.part[1] : a.part[0]) + at * a.D + d;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < a.splits; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(p + (int64_t)i * a.rows * a.D);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    const int64_t t = at % a.len, bh = at / a.len, h = bh % a.heads, b = bh / a.heads;
    const int64_t* st = w ? a.st[1] : a.st[0];
    uint16_t* o = (w ? a.out[1] : a.out[0]) + b * st[0] + t * st[1] + h * st[2] + d;
    *reinterpret_cast<uint2*>(o) = make_uint2(pack2<BF16>(s.x, s.y), pack2<BF16>(s.z, s.w));
  }
}

// ------------------------------------------------------------------------------ host side

// Splits of the walked axis: the count with the shortest schedule, in steps of about a
// microsecond (a tile pair). An item costs its tiles and 2 more for its loads and epilogue; the
// last round is whole with a fixed order, and costs about a quarter of an item with a running
// counter (longest items first, `fill` of the tiles needed on average); partial sums of
// `floats` values a split are written and read once.
int split_count(long long base, int tiles, double floats, bool dynamic, double fill, int sms) {
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= tiles && s <= 64; ++s) {
    const int per = (tiles + s - 1) / s;
    if ((tiles + per - 1) / per != s) continue;
    double cost;
    if (dynamic && base * s > sms)
      cost = (double)base * (tiles * fill + 2.0 * s) / sms + per * 0.25;
    else
      cost = (double)((base * s + sms - 1) / sms) * (per + 2.0);
    if (s > 1) cost += 4.0 + s * floats * 8.0 / 6.7e6;
    if (cost < least - 1e-9) {
      least = cost;
      best = s;
    }
  }
  return best;
}

struct BwdPlan {
  TcGeom g;
  int dq_splits, dkv_splits;
  size_t counters, stat, gmax, vmax, part_q, part_k, part_v, total;  // offsets in floats
};

BwdPlan bwd_plan(const fconv_attn_desc& d, int sms, const AttnArgs& a) {
  BwdPlan p{};
  p.g = tc_geom(d, a);
  const long long bh = (long long)p.g.B * p.g.Hk;
  const size_t D = (size_t)p.g.D;
  const bool dynamic = d.causal || d.has_q_lens || d.has_kv_lens;
  const double fill = d.causal ? 0.5 : 0.75;
  p.dq_splits = split_count(bh * p.g.qtiles, p.g.ktiles, (double)p.g.B * p.g.Hq * p.g.Lq * D,
                            dynamic, fill, sms);
  p.dkv_splits = split_count(bh * p.g.ktiles, p.g.qtiles, 2.0 * bh * p.g.Lk * D, dynamic, fill,
                             sms);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 3) / 4 * 4;
    return o;
  };
  p.counters = take(4);
  p.stat = take((size_t)bh * p.g.qtiles * 2 * kTile);
  p.gmax = take((size_t)bh * p.g.qtiles);
  p.vmax = take((size_t)bh * p.g.ktiles);
  const size_t k = p.dkv_splits > 1 ? (size_t)p.dkv_splits * bh * p.g.Lk * D : 0;
  p.part_k = take(k);
  p.part_v = take(k);
  p.part_q = take(p.dq_splits > 1 ? (size_t)p.dq_splits * p.g.B * p.g.Hq * p.g.Lq * D : 0);
  p.total = at;
  return p;
}

template <int OUTS, typename K>
int start(K kern, uint32_t smem, int items, int sms, const BwdArgs& b, const CUtensorMap* m,
          cudaStream_t s) {
  const int e = allow_smem((const void*)kern, smem);
  if (e) return e;
  const dim3 grid(items < sms ? items : sms);
  if constexpr (OUTS == 1)
    return launch_pdl(kern, grid, dim3(kThreads), smem, s, b, m[0], m[1], m[2], m[3], m[4]);
  else
    return launch_pdl(kern, grid, dim3(kThreads), smem, s, b, m[0], m[1], m[2], m[3], m[5], m[6]);
}

int join(bool bf, const JoinArgs& j, int sms, cudaStream_t s) {
  long long blocks = (j.rows * (j.D / 4) * j.count + 255) / 256;
  if (blocks > 8LL * sms) blocks = 8LL * sms;
  return launch_pdl(bf ? attn_tc_sum<true> : attn_tc_sum<false>, dim3((unsigned)blocks), dim3(256),
                    0, s, j);
}

}  // namespace

bool attn_tc_backward_supported(const fconv_attn_desc& d) {
  if (!attn_tc_supported(d)) return false;
  auto ok = [&](const int64_t st[3], int64_t len, int64_t heads, bool zero) {
    const int64_t ext[3] = {d.batch, len, heads};
    for (int i = 0; i < 3; ++i)
      if (ext[i] > 1 && (st[i] % 8 != 0 || st[i] >= (int64_t)1 << 38 ||
                         (st[i] == 0 && !(zero && i == 0))))
        return false;
    return true;
  };
  if (!ok(d.dout_stride, d.len_q, d.heads_q, true) || !ok(d.dq_stride, d.len_q, d.heads_q, false) ||
      !ok(d.dk_stride, d.len_k, d.heads_kv, false) || !ok(d.dv_stride, d.len_k, d.heads_kv, false))
    return false;
  const int64_t toks = kTile / (d.heads_q / d.heads_kv);
  const int64_t tiles = (d.len_q + toks - 1) / toks + (d.len_k + kTile - 1) / kTile;
  return d.batch * d.heads_kv * tiles <= INT_MAX / 128;
}

size_t attn_tc_backward_workspace(const fconv_attn_desc& d, int sms) {
  return bwd_plan(d, sms, AttnArgs{}).total * sizeof(float);
}

int launch_attn_tc_backward(const fconv_attn_desc& d, int sms, const AttnArgs& a, cudaStream_t s) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return (int)cudaErrorNotSupported;
  BwdPlan p = bwd_plan(d, sms, a);
  TcGeom& g = p.g;
  float* ws = (float*)a.ws;
  const bool bf = d.dtype == FCONV_BF16;
  CUtensorMap m[7];  // q, dout, k, v, dq, dk, dv
  int whole;
  std::memset(m, 0, sizeof(m));
  if (!make_map(enc, &m[0], a.q, d.dtype, g.D, g.Hq, g.Lq, g.B, d.q_stride, g.G, g.toks, nullptr,
                &g.qb) ||
      !make_map(enc, &m[1], a.dout, d.dtype, g.D, g.Hq, g.Lq, g.B, d.dout_stride, g.G, g.toks,
                nullptr, &g.gb) ||
      !make_map(enc, &m[2], a.k, d.dtype, g.D, g.Hk, g.Lk, g.B, d.k_stride, 1, kTile, &g.kh,
                &g.kb) ||
      !make_map(enc, &m[3], a.v, d.dtype, g.D, g.Hk, g.Lk, g.B, d.v_stride, 1, kTile, &g.vh,
                &g.vb) ||
      !make_map(enc, &m[4], a.dq, d.dtype, g.D, g.Hq, g.Lq, g.B, d.dq_stride, g.G, g.toks, nullptr,
                &whole) ||
      !make_map(enc, &m[5], a.dk, d.dtype, g.D, g.Hk, g.Lk, g.B, d.dk_stride, 1, kTile, nullptr,
                &whole) ||
      !make_map(enc, &m[6], a.dv, d.dtype, g.D, g.Hk, g.Lk, g.B, d.dv_stride, 1, kTile, nullptr,
                &whole))
    return (int)cudaErrorInvalidValue;

  DeltaArgs da{};
  da.g = g;
  for (int i = 0; i < 3; ++i) {
    da.o[i] = d.out_stride[i];
    da.d[i] = d.dout_stride[i];
    da.v[i] = d.v_stride[i];
  }
  da.out = (const uint16_t*)a.out;
  da.dout = (const uint16_t*)a.dout;
  da.val = (const uint16_t*)a.v;
  da.lse = a.lse;
  da.stat = ws + p.stat;
  da.gmax = ws + p.gmax;
  da.vmax = ws + p.vmax;
  da.counters = (int*)(ws + p.counters);
  const long long bh = (long long)g.B * g.Hk;
  auto pre = d.head_dim <= 64 ? (bf ? attn_tc_delta<true, 8> : attn_tc_delta<false, 8>)
                              : (bf ? attn_tc_delta<true, 16> : attn_tc_delta<false, 16>);
  int e = launch_pdl(pre, dim3((unsigned)(bh * (g.qtiles + (bf ? 0 : g.ktiles)))), dim3(256), 0, s,
                     da);
  if (e) return e;

  BwdArgs b{};
  b.g = g;
  b.stat = da.stat;
  b.gmax = da.gmax;
  b.vmax = da.vmax;
  b.splits = p.dkv_splits;
  b.per = (g.qtiles + b.splits - 1) / b.splits;
  b.items = (int)(bh * g.ktiles * b.splits);
  b.counter = sched_dynamic(d, b.items, sms) ? da.counters : nullptr;
  for (int i = 0; i < 3; ++i) {
    b.o1[i] = d.dk_stride[i];
    b.o2[i] = d.dv_stride[i];
  }
  b.out1 = a.dk;
  b.out2 = a.dv;
  b.part1 = ws + p.part_k;
  b.part2 = ws + p.part_v;
  if (d.head_dim <= 64)
    e = bf ? start<2>(attn_tc_dkv<true, 1>, dkv_smem<1>(), b.items, sms, b, m, s)
           : start<2>(attn_tc_dkv<false, 1>, dkv_smem<1>(), b.items, sms, b, m, s);
  else
    e = bf ? start<2>(attn_tc_dkv<true, 2>, dkv_smem<2>(), b.items, sms, b, m, s)
           : start<2>(attn_tc_dkv<false, 2>, dkv_smem<2>(), b.items, sms, b, m, s);
  if (e) return e;
  b.splits = p.dq_splits;
  b.per = (g.ktiles + b.splits - 1) / b.splits;
  b.items = (int)(bh * g.qtiles * b.splits);
  b.counter = sched_dynamic(d, b.items, sms) ? da.counters + 1 : nullptr;
  for (int i = 0; i < 3; ++i) b.o1[i] = d.dq_stride[i];
  b.out1 = a.dq;
  b.part1 = ws + p.part_q;
  if (d.head_dim <= 64)
    e = bf ? start<1>(attn_tc_dq<true, 1>, dq_smem<1>(), b.items, sms, b, m, s)
           : start<1>(attn_tc_dq<false, 1>, dq_smem<1>(), b.items, sms, b, m, s);
  else
    e = bf ? start<1>(attn_tc_dq<true, 2>, dq_smem<2>(), b.items, sms, b, m, s)
           : start<1>(attn_tc_dq<false, 2>, dq_smem<2>(), b.items, sms, b, m, s);
  if (e) return e;

  JoinArgs j{};
  j.D = g.D;
  if (p.dkv_splits > 1) {
    j.part[0] = ws + p.part_k;
    j.part[1] = ws + p.part_v;
    j.out[0] = (uint16_t*)a.dk;
    j.out[1] = (uint16_t*)a.dv;
    for (int i = 0; i < 3; ++i) {
      j.st[0][i] = d.dk_stride[i];
      j.st[1][i] = d.dv_stride[i];
    }
    j.rows = bh * g.Lk;
    j.len = g.Lk;
    j.heads = g.Hk;
    j.splits = p.dkv_splits;
    j.count = 2;
    e = join(bf, j, sms, s);
    if (e) return e;
  }
  if (p.dq_splits == 1) return 0;
  j.part[0] = j.part[1] = ws + p.part_q;
  j.out[0] = j.out[1] = (uint16_t*)a.dq;
  for (int i = 0; i < 3; ++i) j.st[0][i] = j.st[1][i] = d.dq_stride[i];
  j.rows = (int64_t)g.B * g.Hq * g.Lq;
  j.len = g.Lq;
  j.heads = g.Hq;
  j.splits = p.dq_splits;
  j.count = 1;
  return join(bf, j, sms, s);
}

int read_and_clear_attn_backward_error(cudaStream_t s, unsigned* v) {
  return read_and_clear_error(s, v);
}

}  // namespace ops
}  // namespace fconv
