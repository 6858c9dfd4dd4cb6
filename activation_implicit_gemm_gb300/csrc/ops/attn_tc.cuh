// Pieces shared by the tensor-core attention kernels: the packing of query rows, work items,
// tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../fconv_internal.h"
#include "../ptx.cuh"
#include "ops_common.cuh"
#include "ops_internal.h"
#include "tc_instr.cuh"
#include "waits.cuh"

namespace fconv {
namespace ops {
namespace {

constexpr int kTile = 128;                 // rows of a query tile, keys of a key tile
constexpr uint32_t kHalfBytes = kTile * 128;  // 128 rows of 64 elements: one 128-byte-row box
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------------- instructions

__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr) { return desc_mn(saddr, kHalfBytes); }

// Byte offset of K step s (16 elements) in a K-major tile of 64-element boxes, in descriptor
// units of 16 bytes.
__host__ __device__ constexpr uint32_t k_step(int s) {
  return (uint32_t)(s >> 2) * (kHalfBytes >> 4) + (uint32_t)(s & 3) * 2;
}

// ------------------------------------------------------------------------------ geometry

// Query rows are packed: a tile of key head hk takes `toks` tokens of all G heads that read it,
// row r = token * G + head in group, so shared heads fill a tile together and read each key
// tile once. toks = 128 / G; rows toks * G .. 127 (G not a power of two) stay empty.
struct TcGeom {
  int64_t B, Lq, Lk;
  int Hq, Hk, G, D;
  int toks, rows;              // tokens and rows of a query tile
  int qtiles;                  // query tiles of a (batch, key head)
  int ktiles;                  // key tiles of the longest sequence
  float scale;
  int causal;
  const int32_t* q_lens;
  const int32_t* kv_lens;
  int kb, kh, vb, vh, qb, gb;  // coordinate multipliers: 0 where a tensor broadcasts the axis
};

struct TcLens {
  int q, k, shift;  // causal: query i sees keys j <= i + shift
  int lead;         // queries before it see no key (causal order with more queries than keys)
};
__device__ __forceinline__ TcLens tc_lens(const TcGeom& g, int b) {
  TcLens l;
  l.q = (int)g.Lq;
  l.k = (int)g.Lk;
  if (g.q_lens) l.q = min(max(__ldcg(g.q_lens + b), 0), (int)g.Lq);
  if (g.kv_lens) l.k = min(max(__ldcg(g.kv_lens + b), 0), (int)g.Lk);
  l.shift = l.k - l.q;
  l.lead = g.causal && l.shift < 0 ? -l.shift : 0;
  if (l.k == 0) l.lead = l.q;
  return l;
}
// Keys that query i sees: [0, limit). Queries outside [lead, q) see none.
__device__ __forceinline__ int key_limit(const TcGeom& g, const TcLens& l, int i) {
  if (i < l.lead || i >= l.q) return 0;
  return g.causal ? min(l.k, i + l.shift + 1) : l.k;
}
// Key tiles that the query tile starting at token t0 needs.
__device__ __forceinline__ int key_tiles(const TcGeom& g, const TcLens& l, int t0) {
  if (t0 >= l.q) return 0;
  const int last = min(t0 + g.toks, l.q) - 1;
  return (key_limit(g, l, last) + kTile - 1) / kTile;
}

// A block's dynamic shared memory must start on the swizzle atom's 1024 bytes.
__device__ __forceinline__ bool smem_ok(const uint8_t* p) {
  if ((ptx::smem_addr(p) & 1023u) == 0) return true;
  if (threadIdx.x == 0) atomicOr(&g_wait_error, 2u);
  return false;
}

// Work items on their way from the load warp, which makes them (a running counter in global
// memory where items differ in length, else a fixed order; lengths and index divisions), to
// the MMA warp and the eight others, two ahead.
template <typename Item>
struct Sched {
  uint64_t full[2], empty[2];
  Item slot[2];
};
constexpr int kSchedReaders = 9;  // warps
template <typename Item>
__device__ __forceinline__ void sched_init(Sched<Item>& s) {
  for (int i = 0; i < 2; ++i) {
    ptx::mbar_init(ptx::smem_addr(&s.full[i]), 1);
    ptx::mbar_init(ptx::smem_addr(&s.empty[i]), kSchedReaders);
  }
}
// Whole load warp (make runs in all lanes): makes and hands on item k; false at the end (handed
// on as well).
template <typename Item, typename Make>
__device__ __forceinline__ bool sched_make(Sched<Item>& s, int k, Item& it, int* counter, int lane,
                                           volatile int* abort_flag, Make make) {
  const int i = k & 1;
  if (!all_lanes(wait_bar(ptx::smem_addr(&s.empty[i]), ((k >> 1) & 1) ^ 1, abort_flag)))
    return false;
  // rounds run forwards and backwards in turn: the blocks' sums come out even
  int at = k * (int)gridDim.x + ((k & 1) ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x);
  if (counter) {
    if (lane == 0) at = atomicAdd(counter, 1);
    at = uni(at);
  }
  make(at, it);
  if (lane == 0) s.slot[i] = it;
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&s.full[i]));
  return it.valid;
}
template <typename Item>
__device__ __forceinline__ bool sched_take(Sched<Item>& s, int k, Item& it, int lane,
                                           volatile int* abort_flag) {
  const int i = k & 1;
  if (!all_lanes(wait_bar(ptx::smem_addr(&s.full[i]), (k >> 1) & 1, abort_flag))) return false;
  it = s.slot[i];
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&s.empty[i]));
  return it.valid;
}
// Whether items differ enough in length for a running counter.
inline bool sched_dynamic(const fconv_attn_desc& d, long long items, int sms) {
  return items > sms && (d.causal || d.has_q_lens || d.has_kv_lens);
}

// Zeroes rows [lo, hi) of a tile made of `halves` boxes of 128-byte rows (the swizzle moves
// 16-byte units within a row only). Whole warp.
__device__ __forceinline__ void zero_rows(uint32_t tile, int halves, int lo, int hi, int lane) {
  for (int h = 0; h < halves; ++h)
    for (int e = lo * 8 + lane; e < hi * 8; e += 32)
      ptx::st_shared_v4(tile + h * kHalfBytes + (uint32_t)e * 16, 0, 0, 0, 0);
}

// ------------------------------------------------------------------------------ host side

// Tensor map of a (batch, token, head, D) tensor seen as (D, head, token, batch), with boxes
// of 64 elements x `heads` x `toks`. An axis with stride 0 gets extent 1 and multiplier 0.
inline bool make_map(EncodeTiledFn enc, CUtensorMap* m, const void* base, int dtype, int64_t D,
                     int64_t heads, int64_t len, int64_t batch, const int64_t st[3], int box_heads,
                     int box_toks, int* mul_head, int* mul_batch) {
  if (mul_head) {
    *mul_head = st[2] == 0 ? 0 : 1;
    if (!*mul_head) heads = 1;
  }
  *mul_batch = st[0] == 0 ? 0 : 1;
  if (!*mul_batch) batch = 1;
  auto bytes = [&](int64_t stride, int64_t extent) {
    return (cuuint64_t)(extent > 1 ? stride * 2 : 16);
  };
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)len,
                              (cuuint64_t)batch};
  const cuuint64_t strides[3] = {bytes(st[2], heads), bytes(st[1], len), bytes(st[0], batch)};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_toks, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m,
             dtype == FCONV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             4, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline TcGeom tc_geom(const fconv_attn_desc& d, const AttnArgs& a) {
  TcGeom g{};
  g.B = d.batch;
  g.Lq = d.len_q;
  g.Lk = d.len_k;
  g.Hq = (int)d.heads_q;
  g.Hk = (int)d.heads_kv;
  g.G = g.Hq / g.Hk;
  g.D = (int)d.head_dim;
  g.toks = kTile / g.G;
  g.rows = g.toks * g.G;
  g.qtiles = (int)((g.Lq + g.toks - 1) / g.toks);
  g.ktiles = (int)((g.Lk + kTile - 1) / kTile);
  g.scale = d.scale;
  g.causal = d.causal;
  g.q_lens = a.q_lens;
  g.kv_lens = a.kv_lens;
  return g;
}

}  // namespace
}  // namespace ops
}  // namespace fconv
