// Attention forward on the tcgen05 tensor cores (f16 and bf16, head_dim a multiple of 8 up to
// 128).
//
// A persistent block (one per SM) owns a pair of 128-row query tiles of one (batch, key head)
// and walks the keys in tiles of 128:
//   S_t = Q_t K^T (both operands in shared memory), 128 x 128 f32 in TMEM
//   P_t = exp2(scale log2e S_t - m)  rounded to 16 bits, written over S_t in TMEM
//   O_t += P_t V (P from TMEM, V from shared memory as the MN-major operand)
// The two tiles share every K and V tile and take turns: while the 128 softmax threads of one
// tile work (a thread owns a row: no shuffles), the tensor core runs P V and the next Q K^T of
// the other. m is the running row maximum, less kLift; O and the row sum are rescaled only when
// it grew by more than 8 in log2 (the sums stay below 2^15 times their final size, far inside f32,
// and P below 2^(8 + kLift), inside its type), which is exact in the same way as rescaling always:
// m cancels in O / l. P's rounding is the only one before the output's; the row sum adds the
// unrounded values. In f16 kLift is 7: a probability keeps all its bits down to 2^-21 of the row's
// largest and some down to 2^-32, so that the keys under a dominant one that carries no value
// still count (2^-14 and 2^-25 without it). bf16 has f32's range.
//
// Roles: warps 0-3 and 4-7 softmax and epilogue of tile 0 and 1, warp 8 MMA, warp 9 TMA (10 and
// 11 only complete the warpgroup).
// TMEM: S0 S1 O0 O1, 128 columns each. Shared memory: the Q tiles (of the next item too for
// head_dim up to 64), a ring of K and V tiles, a box of output a tile.
// When there are fewer blocks than SMs the keys are split; partial O (normalised, f32) and the
// log2 of their sums go to the workspace and attn_tc_join adds them in order. With few queries
// (one tile a key head) a split's even key tiles go through S0, P0, O0 and its odd ones through
// S1, P1, O1 with the same Q (FOLD), two chains of products and exponentials instead of one, each
// with a partial sum of its own.
//
// Bound: tensor (4 D FLOPs a pair) for long queries, HBM (K and V) for few, latency for short
// sequences. 16384 tokens, 16 heads of 128, bf16: 1.35 to 1.40 ms from GPU to GPU, 1570 to 1630
// TFLOP/s, 0.92 to 0.96 of what a long run of library products keeps up; head length 64 has the same exponentials for half the products
// (4 x 4096 tokens, 16 heads: 280 us, 980 TFLOP/s). One query and up to 8192 keys of 16
// sequences, 8 key heads of 128 for 32: 64 us and 6 for the join, 5.4 TB/s. 196 tokens of 12
// heads of 64: 8.9 us, one tile's chain of two key tiles.
// Signalling each half of a tile's probabilities as it is ready (so that P V starts earlier) ran
// 3 % slower at a head length of 128 and 1.5 % faster at 64: not done. With 168 registers at launch
// ptxas spills 36 bytes in every instance.
#include "attn_tc.cuh"

#include <climits>
#include <cmath>
#include <cstring>

namespace fconv {
namespace ops {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
// A softmax thread holds a row of 128 scores; three warps a scheduler leave 168 registers a
// thread, so the third warpgroup hands some over: 2 * 216 + 72 = 3 * 168.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "within the launch's registers");

struct FwdArgs {
  TcGeom g;
  int pairs, splits, per;  // query tile pairs (FOLD: tiles); key splits, key tiles of a split
  int fold, parts;         // parts: partial sums of a row
  int items;
  int* counter;
  int64_t o[3];
  void* out;
  float* lse;
  float* part;      // splits > 1: [split][B][Hq][Lq][D]
  float* part_lse;  // [split][B][Hq][Lq], log2
  size_t counter_floats, part_floats;  // of the workspace
};

struct FwdItem {
  int valid, b, hk, split, t0[2], n[2], jb;
  TcLens l;
};

// In causal order the long query tiles come first; otherwise neighbouring blocks share a
// head's keys in L2.
__device__ __forceinline__ void fwd_item(const FwdArgs& a, int u, FwdItem& it) {
  it.valid = u < a.items;
  if (!it.valid) return;
  it.split = u % a.splits;
  u /= a.splits;
  const int bh = (int)a.g.B * a.g.Hk;
  int pair;
  if (a.g.causal) {
    pair = a.pairs - 1 - u / bh;
    u %= bh;
  } else {
    pair = u % a.pairs;
    u /= a.pairs;
  }
  it.hk = u % a.g.Hk;
  it.b = u / a.g.Hk;
  it.l = tc_lens(a.g, it.b);
  it.jb = it.split * a.per;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.t0[t] = (a.fold ? pair : 2 * pair + t) * a.g.toks;
    it.n[t] = max(min(key_tiles(a.g, it.l, it.t0[t]) - it.jb, a.per), 0);
    if (a.fold) it.n[t] = (it.n[t] + 1 - t) / 2;  // tiles jb + t, jb + t + 2, ...
  }
}

template <int H>
struct FwdPlan {
  static constexpr uint32_t tile_bytes = H * kHalfBytes;
  static constexpr int own = H == 1 ? 2 : 1;    // buffers of the two Q tiles
  static constexpr int slots = H == 1 ? 6 : 4;  // ring of K and V tiles
  static constexpr uint32_t ring_at = 2 * own * tile_bytes;
  static constexpr uint32_t out_at = ring_at + slots * tile_bytes;  // a box of 64 columns a tile
  static constexpr uint32_t ctl_at = out_at + 2 * kHalfBytes;
  // FOLD: one Q tile, and the rest of the space a ring
  static constexpr int fold_slots = (ctl_at - tile_bytes) / tile_bytes;
};

template <int H>
struct FwdCtl {
  uint64_t full[FwdPlan<H>::fold_slots], empty[FwdPlan<H>::fold_slots];
  uint64_t q_full[2], q_empty[2], tail, drain;
  uint64_t s_full[2], p_ready[2], o_done[2], out_ready[2], out_free[2];
  Sched<FwdItem> sched;
  uint32_t tmem;
  int abort_flag;
};
template <int H>
constexpr uint32_t fwd_smem() {
  return FwdPlan<H>::ctl_at + sizeof(FwdCtl<H>);
}
static_assert(fwd_smem<2>() <= 232448 && fwd_smem<1>() <= 232448, "one block's shared memory");

template <bool BF16, int H, bool FOLD>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_forward(const FwdArgs a, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_o) {
  using Plan = FwdPlan<H>;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  if (!smem_ok(dsmem)) return;
  FwdCtl<H>& ctl = *reinterpret_cast<FwdCtl<H>*>(dsmem + Plan::ctl_at);
  const TcGeom& g = a.g;
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;
  const uint32_t own = ptx::smem_addr(dsmem);
  constexpr int kOwn = FOLD ? 1 : Plan::own, kSlots = FOLD ? Plan::fold_slots : Plan::slots;
  constexpr float kLift = BF16 ? 0.0f : 7.0f;
  const uint32_t ring = own + (FOLD ? Plan::tile_bytes : Plan::ring_at);
  volatile int* abort_flag = &ctl.abort_flag;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl.full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.empty[i]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl.tail), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl.drain), 1);
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(ptx::smem_addr(&ctl.q_full[t]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.q_empty[t]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.s_full[t]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.p_ready[t]), 4);
      ptx::mbar_init(ptx::smem_addr(&ctl.o_done[t]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl.out_ready[t]), 4);
      ptx::mbar_init(ptx::smem_addr(&ctl.out_free[t]), 1);
    }
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
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    ptx::prefetch_tmap(&tm_o);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = uni(ctl.tmem);
  ptx::pdl_wait();

  if (warp >= 8) {
    regs_fewer<kOtherRegs>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- TMA producer
      uint32_t c = 0, q_items = 0, tails = 0;
      FwdItem it;
      bool stop = false;
      auto make = [&](int u, FwdItem& x) { fwd_item(a, u, x); };
      for (int k = 0; !stop && sched_make(ctl.sched, k, it, a.counter, lane, abort_flag, make);
           ++k) {
        const int n = max(it.n[0], it.n[1]);
        if (n == 0) continue;
        const uint32_t ob = q_items % kOwn;
        if (!wait_bar(ptx::smem_addr(&ctl.q_empty[ob]), ((q_items / kOwn) & 1) ^ 1,
                      abort_flag))
          break;
        ++q_items;
        if (lane == 0) {
          const uint32_t bar = ptx::smem_addr(&ctl.q_full[ob]);
          const uint32_t box = (uint32_t)g.rows * 128;
          const int tiles = FOLD ? 1 : (it.n[0] > 0) + (it.n[1] > 0);
          ptx::mbar_arrive_expect_tx(bar, tiles * H * box);
#pragma unroll
          for (int t = 0; t < (FOLD ? 1 : 2); ++t)
            if (it.n[t] > 0)
              for (int h = 0; h < H; ++h)
                tma_load_4d(own + (ob * 2 + t) * Plan::tile_bytes + h * kHalfBytes, &tm_q, h * 64,
                            it.hk * g.G, it.t0[t], it.b * g.qb, bar);
        }
        // K, V of each step; FOLD: K, K, V, V of its two tiles (the last step may have one)
        const int loads = FOLD ? 2 * (it.n[0] + it.n[1]) : 2 * n;
        for (int j = 0; j < loads; ++j, ++c) {
          const uint32_t s = c % kSlots, ph = (c / kSlots) & 1;
          if (!wait_bar(ptx::smem_addr(&ctl.empty[s]), ph ^ 1, abort_flag)) {
            stop = true;
            break;
          }
          int tile = j >> 1;
          bool is_v = j & 1;
          if (FOLD) {
            const bool two = (j >> 2) < it.n[1];
            is_v = two ? j & 2 : j & 1;
            tile = 2 * (j >> 2) + (two ? j & 1 : 0);
          }
          const int key0 = (it.jb + tile) * kTile;
          const uint32_t dst = ring + s * Plan::tile_bytes;
          // rows of V past the sequence would meet P = 0: a NaN there must not reach the product
          const bool ragged = is_v && key0 + kTile > it.l.k && it.l.k < g.Lk;
          const uint32_t full = ptx::smem_addr(&ctl.full[s]);
          const uint32_t bar = ragged ? ptx::smem_addr(&ctl.tail) : full;
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(bar, Plan::tile_bytes);
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
        // loads in flight land before the block's shared memory is given back
        for (uint32_t i = c > kSlots ? c - kSlots : 0; i < c; ++i)
          drain_bar(ptx::smem_addr(&ctl.full[i % kSlots]), (i / kSlots) & 1);
        for (uint32_t i = q_items > kOwn ? q_items - kOwn : 0; i < q_items; ++i)
          drain_bar(ptx::smem_addr(&ctl.q_full[i % kOwn]), (i / kOwn) & 1);
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issue
      const bool leader = elect_lane();
      const uint32_t id_s = idesc_16(BF16, kTile, kTile, false);
      const int dk = (g.D + 15) / 16;  // K steps of Q K^T, N / 16 of P V
      const uint32_t id_o = idesc_16(BF16, kTile, dk * 16, true);
      uint32_t c = 0, q_items = 0, pv0 = 0, pv1 = 0;
      FwdItem it;
      bool stop = false;
      auto wait = [&](uint64_t& bar, uint32_t parity) {
        return all_lanes(wait_bar(ptx::smem_addr(&bar), parity, abort_flag));
      };
      auto commit = [&](uint64_t& bar) {
        if (leader) ptx::mma_commit(ptx::smem_addr(&bar));
      };
      for (int k = 0; !stop && sched_take(ctl.sched, k, it, lane, abort_flag); ++k) {
        const int n0 = uni(it.n[0]), n1 = uni(it.n[1]), n = max(n0, n1);
        if (n == 0) continue;
        const uint32_t ob = q_items % kOwn;
        const uint32_t q0 = own + ob * 2 * Plan::tile_bytes;
        auto scores = [&](int t, uint32_t ktile) {
          const uint32_t q = desc_k(q0 + (FOLD ? 0 : t) * Plan::tile_bytes), kt = desc_k(ktile);
          if (leader) {
#pragma unroll
            for (int d = 0; d < 4 * H; ++d)
              if (d < dk) mma_ss(tmem + t * 128, q + k_step(d), kt + k_step(d), id_s, d > 0);
          }
          commit(ctl.s_full[t]);
        };
        if (!wait(ctl.q_full[ob], (q_items / kOwn) & 1)) break;
        ++q_items;
        if (FOLD) {
          auto wait_slot = [&](uint32_t i) { return wait(ctl.full[i % kSlots], (i / kSlots) & 1); };
          auto slot = [&](uint32_t i) { return ring + i % kSlots * Plan::tile_bytes; };
          // scores of step j, whose loads start at `at`, for chain t
          auto fold_scores = [&](int t, uint32_t at, bool last) {
            if (!wait_slot(at + t)) return false;
            ptx::tc_fence_after();
            scores(t, slot(at + t));
            commit(ctl.empty[(at + t) % kSlots]);
            if (last) commit(ctl.q_empty[ob]);
            return true;
          };
          const int all = n0 + n1;
          if (!fold_scores(0, c, all == 1) || (n1 > 0 && !fold_scores(1, c, all == 2))) break;
          for (int j = 0; j < n0; ++j) {
            const int two = j < n1 ? 2 : 1;
            const uint32_t next = c + 2 * two;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (t >= two) continue;
              if (!wait_slot(c + two + t) || !wait(ctl.p_ready[t], (t ? pv1 : pv0) & 1)) {
                stop = true;
                break;
              }
              ++(t ? pv1 : pv0);
              ptx::tc_fence_after();
              const uint32_t v = desc_mn(slot(c + two + t));
              if (leader) {
#pragma unroll
                for (int s = 0; s < kTile / 16; ++s)
                  mma_ts(tmem + 256 + t * 128, tmem + t * 128 + s * 8, v + s * (2048 >> 4), id_o,
                         j > 0 || s > 0);
              }
              commit(ctl.empty[(c + two + t) % kSlots]);
              if (j + 1 == (t ? n1 : n0)) {
                commit(ctl.o_done[t]);
              } else if (!fold_scores(t, next, 2 * (j + 1) + t + 1 == all)) {
                stop = true;
                break;
              }
            }
            if (stop) break;
            c = next;
          }
          continue;
        }
        if (!wait(ctl.full[c % kSlots], (c / kSlots) & 1)) break;
        ptx::tc_fence_after();
        if (n0 > 0) scores(0, ring + c % kSlots * Plan::tile_bytes);
        if (n1 > 0) scores(1, ring + c % kSlots * Plan::tile_bytes);
        commit(ctl.empty[c % kSlots]);
        if (n == 1) commit(ctl.q_empty[ob]);
        for (int j = 0; j < n; ++j, c += 2) {
          const uint32_t vs = (c + 1) % kSlots, ks = (c + 2) % kSlots;
          if (!wait(ctl.full[vs], ((c + 1) / kSlots) & 1) ||
              (j + 1 < n && !wait(ctl.full[ks], ((c + 2) / kSlots) & 1))) {
            stop = true;
            break;
          }
          const uint32_t v = desc_mn(ring + vs * Plan::tile_bytes);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? n1 : n0;
            if (j >= nt) continue;
            if (!wait(ctl.p_ready[t], (t ? pv1 : pv0) & 1)) {
              stop = true;
              break;
            }
            ++(t ? pv1 : pv0);
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
              for (int s = 0; s < kTile / 16; ++s)
                mma_ts(tmem + 256 + t * 128, tmem + t * 128 + s * 8, v + s * (2048 >> 4), id_o,
                       j > 0 || s > 0);
            }
            if (j == nt - 1) commit(ctl.o_done[t]);
            if (j + 1 < nt) scores(t, ring + ks * Plan::tile_bytes);
          }
          if (stop) break;
          commit(ctl.empty[vs]);
          if (j + 1 < n) commit(ctl.empty[ks]);
          if (j + 2 == n) commit(ctl.q_empty[ob]);
        }
      }
      commit(ctl.drain);
      drain_bar(ptx::smem_addr(&ctl.drain), 0);
    }
  } else {
    // ------------------------------------------------------------------ softmax, epilogue
    regs_more<kSoftmaxRegs>();
    const int t = warp >> 2;
    const int row = tid & 127, tok = row / g.G, head = row - tok * g.G;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    const uint32_t s_at = tmem + t * 128 + lanes, o_at = tmem + 256 + t * 128 + lanes;
    const uint32_t box = own + Plan::out_at + t * kHalfBytes;
    const float c = g.scale * kLog2e;
    uint32_t steps = 0, done = 0, boxes = 0;
    FwdItem it;
    for (int k = 0; sched_take(ctl.sched, k, it, lane, abort_flag); ++k) {
      const int n = t ? it.n[1] : it.n[0], t0 = t ? it.t0[1] : it.t0[0], i = t0 + tok;
      const int limit = row < g.rows ? key_limit(g, it.l, i) : 0;
      // a few query tokens leave most warps without a row
      const bool warp_live = __any_sync(0xffffffffu, limit > 0);
      float m = -INFINITY, l = 0.0f;
      bool stop = false;
      for (int j = 0; j < n; ++j) {
        if (!wait_bar(ptx::smem_addr(&ctl.s_full[t]), steps & 1, abort_flag)) {
          stop = true;
          break;
        }
        ++steps;
        ptx::tc_fence_after();
        if (!warp_live) {  // rows that no one reads: their P is whatever lies there
          ptx::tc_fence_before();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.p_ready[t]));
          continue;
        }
        uint32_t s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_fetch32(s_at + q * 32, s[q]);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_arrived(s[q]);
        const int tile = it.jb + (FOLD ? 2 * j + t : j);
        const int seen = limit - tile * kTile;  // columns of this tile that the row sees
        if (__any_sync(0xffffffffu, seen < kTile)) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e >= seen) s[q][e] = 0xff800000u;  // -inf
        }
        float top[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          top[q] = __uint_as_float(s[q][0]);
#pragma unroll
          for (int e = 1; e < 32; ++e) top[q] = fmaxf(top[q], __uint_as_float(s[q][e]));
        }
        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const float mn = fmaxf(m, fmaf(most, c, -kLift));
        if (__any_sync(0xffffffffu, mn > m + 8.0f)) {
          // the scores of this tile are complete, so every earlier P V is too
          const float f = mn == -INFINITY ? 1.0f : exp2_fast(m - mn);
          l *= f;
          m = mn;
          if (j > 0)
#pragma unroll 1
            for (int q = 0; q < (g.D + 7) / 8; ++q) {
              uint32_t o[8];
              tmem_fetch8(o_at + q * 8, o);
              tmem_wait_ld();
              tmem_arrived(o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_store8(o_at + q * 8, o);
            }
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        const uint64_t c2 = pair(c, c), r2 = pair(-ref, -ref);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint64_t x = fma2(pair(s[q][2 * e], s[q][2 * e + 1]), c2, r2);
            const float u = exp2_fast(low(x)), v = exp2_fast(high(x));
            sum[e & 1] = add2(sum[e & 1], pair(u, v));
            p[e] = pack2<BF16>(u, v);
          }
          tmem_store16(s_at + q * 16, p);
        }
        sum[0] = add2(sum[0], sum[1]);
        l += low(sum[0]) + high(sum[0]);
        tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.p_ready[t]));
      }
      if (stop) break;
      if (n > 0) {
        if (!wait_bar(ptx::smem_addr(&ctl.o_done[t]), done & 1, abort_flag)) break;
        ++done;
        ptx::tc_fence_after();
      }
      const bool live = row < g.rows && i < g.Lq;
      const int64_t h = (int64_t)it.hk * g.G + head;
      const int64_t at = ((int64_t)it.b * g.Hq + h) * g.Lq + i;
      const bool any = n > 0 && limit > 0 && l != 0.0f;  // l: NaN counts as present
      const float inv = any ? 1.0f / l : 0.0f;
      const float lse2 = any ? m + log2f(l) : -INFINITY;
      const int64_t rows = g.B * g.Hq * g.Lq;
      const int64_t part_at = (int64_t)(FOLD ? 2 * it.split + t : it.split) * rows + at;
      if (live) {
        if (a.parts > 1) a.part_lse[part_at] = lse2;
        else if (a.lse) a.lse[at] = lse2 * kLn2;
      }
      if (a.parts > 1) {
        float* part = a.part + part_at * g.D;
        for (int q = 0; q < (g.D + 31) / 32; ++q) {
          uint32_t o[32];
          if (n > 0) {
            tmem_fetch32(o_at + q * 32, o);
            tmem_wait_ld();
            tmem_arrived(o);
          }
          if (!live) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = any ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            if (q * 32 + e < g.D)
              ptx::st_global_v4(part + q * 32 + e, make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
        }
        continue;
      }
      // 64 columns at a time through shared memory to a TMA store; a thread's own 16-byte
      // stores, one row a lane, kept the store unit busy for 4000 cycles a tile
      for (int x = 0; x < H; ++x, ++boxes) {
        if (t0 >= g.Lq) break;  // the pair's second tile may not exist
        if (!wait_bar(ptx::smem_addr(&ctl.out_free[t]), (boxes & 1) ^ 1, abort_flag)) {
          stop = true;
          break;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t o[32], w[16];
          if (n > 0) {
            tmem_fetch32(o_at + x * 64 + q * 32, o);
            tmem_wait_ld();
            tmem_arrived(o);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = any ? pack2<BF16>(__uint_as_float(o[2 * e]) * inv,
                                     __uint_as_float(o[2 * e + 1]) * inv)
                       : 0u;
          stage_row(box, row, q * 32, w);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl.out_ready[t]));
        if ((warp & 3) == 0) {
          if (!wait_bar(ptx::smem_addr(&ctl.out_ready[t]), boxes & 1, abort_flag)) {
            stop = true;
            break;
          }
          if (lane == 0) {
            tma_store_4d(&tm_o, box, x * 64, it.hk * g.G, t0, it.b);
            bulk_commit();
            bulk_wait_read();
            ptx::mbar_arrive(ptx::smem_addr(&ctl.out_free[t]));
          }
        }
      }
      if (stop) break;
    }
    if ((warp & 3) == 0 && lane == 0) bulk_wait_all();
  }

  ptx::pdl_trigger();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Joins the key splits of a row: out = sum_s w_s part_s / sum_s w_s, w_s = 2^(lse_s - max).
// One warp per row, splits in order, eight at a time on their way (8.3 -> 6.1 us for 512 rows).
template <bool BF16>
__global__ void __launch_bounds__(256) attn_tc_join(const FwdArgs a) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const TcGeom& g = a.g;
  const int64_t rows = g.B * g.Hq * g.Lq;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (at >= rows) return;
  float top = -INFINITY;
  for (int s = lane; s < a.parts; s += 32) top = fmaxf(top, a.part_lse[(int64_t)s * rows + at]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -INFINITY ? 0.0f : top;
  float total = 0.0f;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int d = lane * 4;
  for (int s0 = 0; s0 < a.parts; s0 += 32) {
    const int n = min(32, a.parts - s0);
    const float mine =
        lane < n ? exp2f(a.part_lse[(int64_t)(s0 + lane) * rows + at] - ref) : 0.0f;
    for (int s = 0; s < n; s += 8) {  // eight loads in flight
      float w[8];
      float4 p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = __shfl_sync(0xffffffffu, mine, s + i);
        p[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (w[i] != 0.0f && d < g.D)  // a split without keys has written nothing
          p[i] = *reinterpret_cast<const float4*>(a.part + ((int64_t)(s0 + s + i) * rows + at) *
                                                               g.D + d);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        total += w[i];
        acc[0] = fmaf(w[i], p[i].x, acc[0]);
        acc[1] = fmaf(w[i], p[i].y, acc[1]);
        acc[2] = fmaf(w[i], p[i].z, acc[2]);
        acc[3] = fmaf(w[i], p[i].w, acc[3]);
      }
    }
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t i = at % g.Lq, bh = at / g.Lq, h = bh % g.Hq, b = bh / g.Hq;
  if (d < g.D) {
    uint16_t* out = (uint16_t*)a.out + b * a.o[0] + i * a.o[1] + h * a.o[2] + d;
    const uint2 v = make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv),
                               pack2<BF16>(acc[2] * inv, acc[3] * inv));
    *reinterpret_cast<uint2*>(out) = v;
  }
  if (a.lse && lane == 0)
    a.lse[at] = total == 0.0f ? -INFINITY : (ref + log2f(total)) * kLn2;
}

// Key splits: the count with the shortest schedule, in steps of about a microsecond (a key
// tile). An item costs its tiles and 1.5 more for its loads and epilogue; the last round is
// whole with a fixed order, and costs about half an item with a running counter; partial sums
// are written and read once, and joined in about 4.
int split_count(const TcGeom& g, bool dynamic, int sms, int pairs) {
  const double tile = g.qtiles == 1 ? 0.7 : 1.0;  // two chains
  const long long base = (long long)g.B * g.Hk * pairs;
  const double floats = (double)g.B * g.Hq * g.Lq * g.D, fill = g.causal ? 0.5 : 0.75;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= g.ktiles && s <= 64; ++s) {
    const int per = (g.ktiles + s - 1) / s;
    if ((g.ktiles + per - 1) / per != s) continue;
    double cost;
    if (dynamic && base * s > sms)
      cost = (double)base * (g.ktiles * fill * tile + 1.5 * s) / sms + per * tile * 0.5;
    else
      cost = (double)((base * s + sms - 1) / sms) * (per * tile + 1.5);
    if (s > 1) cost += 4.0 + s * floats * 8.0 / 6.7e6;
    if (cost < least - 1e-9) {
      least = cost;
      best = s;
    }
  }
  return best;
}

FwdArgs fwd_args(const fconv_attn_desc& d, int sms, const AttnArgs& a) {
  FwdArgs f{};
  f.g = tc_geom(d, a);
  f.pairs = (f.g.qtiles + 1) / 2;
  f.splits = split_count(f.g, d.causal || d.has_q_lens || d.has_kv_lens, sms, f.pairs);
  f.per = (f.g.ktiles + f.splits - 1) / f.splits;
  f.fold = f.g.qtiles == 1 && f.splits > 1 && f.per > 1;
  f.parts = f.splits * (f.fold ? 2 : 1);
  f.items = (int)((long long)f.g.B * f.g.Hk * f.pairs * f.splits);
  for (int i = 0; i < 3; ++i) f.o[i] = d.out_stride[i];
  f.out = a.o;
  f.lse = a.lse;
  const size_t rows = (size_t)f.g.B * f.g.Hq * f.g.Lq;
  float* ws = (float*)a.ws;
  if (sched_dynamic(d, f.items, sms)) {
    f.counter = (int*)ws;
    f.counter_floats = 4;
    if (ws) ws += 4;
  }
  if (f.parts > 1) {
    f.part_lse = ws;
    f.part_floats = ((size_t)f.parts * rows + 3) / 4 * 4;
    if (ws) f.part = ws + f.part_floats;
    f.part_floats += (size_t)f.parts * rows * f.g.D;
  }
  return f;
}

template <bool BF16, int H>
int launch_t(const FwdArgs& f, int sms, const CUtensorMap* m, cudaStream_t s) {
  auto kern = f.fold ? attn_tc_forward<BF16, H, true> : attn_tc_forward<BF16, H, false>;
  const int e = allow_smem((const void*)kern, fwd_smem<H>());
  if (e) return e;
  const int grid = f.items < sms ? f.items : sms;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), fwd_smem<H>(), s, f, m[0], m[1], m[2], m[3]);
}

}  // namespace

// Strides of axes that are walked must be whole 16-byte units; 0 only on an axis of K or V
// that a block does not walk (batch, head).
bool attn_tc_supported(const fconv_attn_desc& d) {
  if (d.dtype == FCONV_F32 || d.head_dim % 8 != 0 || d.head_dim > 128) return false;
  if (d.heads_q / d.heads_kv > kTile || d.len_q == 0 || d.len_k == 0 || d.batch == 0) return false;
  auto unit = [](int64_t stride, int64_t extent, bool zero) {
    return extent == 1 || (stride % 8 == 0 && stride < (int64_t)1 << 38 && (stride > 0 || zero));
  };
  auto ok = [&](const int64_t st[3], int64_t len, int64_t heads, bool zero_head) {
    return unit(st[0], d.batch, true) && unit(st[1], len, false) && unit(st[2], heads, zero_head);
  };
  const int64_t h = d.heads_q, kh = d.heads_kv;
  if (!ok(d.q_stride, d.len_q, h, false) || !ok(d.k_stride, d.len_k, kh, true) ||
      !ok(d.v_stride, d.len_k, kh, true) || !ok(d.out_stride, d.len_q, h, false))
    return false;
  // blocks' items, up to 64 key splits each, count in 32 bits
  const int64_t toks = kTile / (h / kh);
  return d.batch * kh * ((d.len_q + toks - 1) / toks / 2 + 1) <= INT_MAX / 128;
}

size_t attn_tc_forward_workspace(const fconv_attn_desc& d, int sms) {
  const FwdArgs f = fwd_args(d, sms, AttnArgs{});
  return (f.counter_floats + f.part_floats) * sizeof(float);
}

int launch_attn_tc_forward(const fconv_attn_desc& d, int sms, const AttnArgs& a, cudaStream_t s) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return (int)cudaErrorNotSupported;
  FwdArgs f = fwd_args(d, sms, a);
  int e, whole;
  CUtensorMap m[4];  // q, k, v, out
  std::memset(m, 0, sizeof(m));
  if (!make_map(enc, &m[0], a.q, d.dtype, d.head_dim, d.heads_q, d.len_q, d.batch, d.q_stride,
                f.g.G, f.g.toks, nullptr, &f.g.qb) ||
      !make_map(enc, &m[1], a.k, d.dtype, d.head_dim, d.heads_kv, d.len_k, d.batch, d.k_stride, 1,
                kTile, &f.g.kh, &f.g.kb) ||
      !make_map(enc, &m[2], a.v, d.dtype, d.head_dim, d.heads_kv, d.len_k, d.batch, d.v_stride, 1,
                kTile, &f.g.vh, &f.g.vb) ||
      !make_map(enc, &m[3], a.o, d.dtype, d.head_dim, d.heads_q, d.len_q, d.batch, d.out_stride,
                f.g.G, f.g.toks, nullptr, &whole))
    return (int)cudaErrorInvalidValue;
  if (f.counter) {
    e = (int)cudaMemsetAsync(f.counter, 0, sizeof(int), s);
    if (e) return e;
  }
  const bool bf = d.dtype == FCONV_BF16;
  if (d.head_dim <= 64)
    e = bf ? launch_t<true, 1>(f, sms, m, s) : launch_t<false, 1>(f, sms, m, s);
  else
    e = bf ? launch_t<true, 2>(f, sms, m, s) : launch_t<false, 2>(f, sms, m, s);
  if (e || f.parts == 1) return e;
  const long long rows = (long long)f.g.B * f.g.Hq * f.g.Lq;
  return launch_pdl(bf ? attn_tc_join<true> : attn_tc_join<false>, dim3((unsigned)((rows + 7) / 8)),
                    dim3(256), 0, s, f);
}

int read_and_clear_attn_forward_error(cudaStream_t s, unsigned* v) {
  return read_and_clear_error(s, v);
}

}  // namespace ops
}  // namespace fconv
