// C ABI and planner of the token-side operators (include/fconv_ops.h). Nothing is allocated on
// the device; every rule is checked here, before anything is launched.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <mutex>

#include "api_common.h"

using namespace fconv::ops;

struct fconv_norm_plan {
  fconv_norm_desc d;
  int sms;
  size_t workspace;
};
struct fconv_rope_plan {
  fconv_rope_desc d;
  int sms;
};
struct fconv_attn_plan {
  fconv_attn_desc d;
  int sms;
  int want;            // the route asked for
  bool fwd_tc, bwd_tc;  // tensor cores for calls with aligned addresses
  size_t fwd_ws, bwd_ws;
};

namespace {

fconv_status check_norm(const fconv_norm_desc& d) {
  if (!known_type(d.dtype) || !known_type(d.param_dtype) ||
      (d.param_dtype != d.dtype && d.param_dtype != FCONV_F32))
    return FCONV_E_UNSUPPORTED;
  if (d.outer < 0 || !small(d.channels, 1) || !small(d.inner, 1)) return FCONV_E_EXTENT;
  if (!(d.eps > 0.0f) || !std::isfinite(d.eps)) return FCONV_E_ATTR_VALUE;
  if (d.outer > INT_MAX || d.outer * ((d.inner + 31) / 32) > INT_MAX) return FCONV_E_UNSUPPORTED;
  return FCONV_OK;
}

fconv_status check_rope(const fconv_rope_desc& d) {
  if (!known_type(d.dtype)) return FCONV_E_UNSUPPORTED;
  if (!small(d.batch, 0) || !small(d.len, 0) || !small(d.heads_q, 1) || !small(d.heads_k, 0) ||
      !small(d.head_dim, 1) || (d.pos_batch != 1 && d.pos_batch != d.batch))
    return FCONV_E_EXTENT;
  if (d.axes < 1 || d.axes > 3 || d.pairing < FCONV_ROPE_INTERLEAVED ||
      d.pairing > FCONV_ROPE_HALF_PER_AXIS || d.pos_type < FCONV_POS_I32 ||
      d.pos_type > FCONV_POS_F32)
    return FCONV_E_ATTR_VALUE;
  int64_t pairs = 0;
  for (int i = 0; i < d.axes; ++i) {
    if (!small(d.section[i], 0)) return FCONV_E_ATTR_VALUE;
    pairs += d.section[i];
  }
  if (pairs > d.head_dim / 2) return FCONV_E_EXTENT;
  const int64_t eq[3] = {d.batch, d.len, d.heads_q}, ek[3] = {d.batch, d.len, d.heads_k};
  if (!strides_ok(d.q_stride, eq, d.head_dim, false) ||
      !strides_ok(d.q_out_stride, eq, d.head_dim, true) ||
      (d.heads_k && (!strides_ok(d.k_stride, ek, d.head_dim, false) ||
                     !strides_ok(d.k_out_stride, ek, d.head_dim, true))))
    return FCONV_E_STRIDE;
  if (d.batch * d.len > INT_MAX || d.batch * d.len * d.head_dim / 256 >= INT_MAX)
    return FCONV_E_UNSUPPORTED;
  return FCONV_OK;
}

fconv_status check_attn(const fconv_attn_desc& d) {
  if (!known_type(d.dtype)) return FCONV_E_UNSUPPORTED;
  if (!small(d.batch, 0) || !small(d.len_q, 0) || !small(d.len_k, 0) || !small(d.heads_q, 1) ||
      !small(d.heads_kv, 1) || d.heads_q % d.heads_kv != 0 || !small(d.head_dim, 1))
    return FCONV_E_EXTENT;
  if (d.head_dim > 256) return FCONV_E_UNSUPPORTED;
  if (!(d.scale > 0.0f) || !std::isfinite(d.scale)) return FCONV_E_ATTR_VALUE;
  const int64_t eq[3] = {d.batch, d.len_q, d.heads_q}, ek[3] = {d.batch, d.len_k, d.heads_kv};
  if (!strides_ok(d.q_stride, eq, d.head_dim, false) ||
      !strides_ok(d.k_stride, ek, d.head_dim, false) ||
      !strides_ok(d.v_stride, ek, d.head_dim, false) ||
      !strides_ok(d.out_stride, eq, d.head_dim, true))
    return FCONV_E_STRIDE;
  if (d.training && (!strides_ok(d.dout_stride, eq, d.head_dim, false) ||
                     !strides_ok(d.dq_stride, eq, d.head_dim, true) ||
                     !strides_ok(d.dk_stride, ek, d.head_dim, true) ||
                     !strides_ok(d.dv_stride, ek, d.head_dim, true)))
    return FCONV_E_STRIDE;
  // one block at most per 32 rows of a head, delta rows in blocks of 8
  const double rows = (double)d.batch * (double)d.heads_q;
  if (rows * ((double)d.len_q / 8 + 2) > INT_MAX || rows * ((double)d.len_k / 32 + 2) > INT_MAX)
    return FCONV_E_UNSUPPORTED;
  return FCONV_OK;
}

// The checks that the forward and the backward pass of attention share.
fconv_status attn_inputs(const fconv_attn_desc& d, const void* q, const void* k, const void* v,
                         const int32_t* q_lens, const int32_t* kv_lens) {
  const bool nq = d.batch * d.len_q > 0, nk = d.batch * d.len_k > 0;
  if ((nq && !q) || (nk && (!k || !v))) return FCONV_E_NULL;
  if (d.batch > 0 && ((d.has_q_lens != 0) != (q_lens != nullptr) ||
                      (d.has_kv_lens != 0) != (kv_lens != nullptr)))
    return FCONV_E_MASK;
  const size_t e = type_size(d.dtype);
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(q_lens, 4) ||
      misaligned(kv_lens, 4))
    return FCONV_E_ALIGNMENT;
  return FCONV_OK;
}

}  // namespace

namespace fconv {
namespace ops {

int allow_smem(const void* kernel, size_t bytes) {
  if (bytes <= 24 * 1024) return 0;  // with static shared memory within the default 48 KB
  struct Seen {
    const void* kernel;
    int device;
    size_t bytes;
  };
  static std::mutex mu;
  static Seen seen[256];
  static int count = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return (int)e;
  std::lock_guard<std::mutex> lock(mu);
  Seen* at = nullptr;
  for (int i = 0; i < count && !at; ++i)
    if (seen[i].kernel == kernel && seen[i].device == device) at = &seen[i];
  if (at && at->bytes >= bytes) return 0;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return (int)e;
  if (!at && count < 256) {
    at = &seen[count++];
    at->kernel = kernel;
    at->device = device;
  }
  if (at) at->bytes = bytes;
  return 0;
}

}  // namespace ops
}  // namespace fconv

extern "C" {

const char* fconv_ops_status_string(int s) {
  switch (s) {
    case FCONV_E_EXTENT: return "an extent is below its minimum, or sizes do not fit together";
    case FCONV_E_STRIDE: return "a stride is negative or makes elements of an output overlap";
    case FCONV_E_MASK: return "lengths were given that the plan does not have, or the reverse";
    case FCONV_E_ATTR_VALUE: return "an attribute has a value outside its range";
    case FCONV_E_BIAS_SHAPE:
      return "a weight, a bias or a gradient of one was given that the plan does not have";
    case FCONV_E_ALIGNMENT: return "a device pointer is not aligned as its type or route needs";
    case FCONV_E_ALIAS: return "an output must not be an input or another output";
    default: return fconv_status_string((fconv_status)s);
  }
}

fconv_status fconv_ops_check_device(void* stream) {
  unsigned n = 0, f = 0, b = 0, m = 0;
  if (read_and_clear_norm_error((cudaStream_t)stream, &n) != 0 ||
      read_and_clear_attn_forward_error((cudaStream_t)stream, &f) != 0 ||
      read_and_clear_attn_backward_error((cudaStream_t)stream, &b) != 0 ||
      read_and_clear_mlp_error((cudaStream_t)stream, &m) != 0)
    return FCONV_E_CUDA;
  return n || f || b || m ? FCONV_E_DEVICE_TIMEOUT : FCONV_OK;
}

// ---------------------------------------------------------------------------- layer norm

fconv_status fconv_norm_plan_create(const fconv_norm_desc* desc, int device,
                                    fconv_norm_plan** out) {
  const fconv_status st = new_plan(desc, device, check_norm, out);
  if (st == FCONV_OK) (*out)->workspace = norm_workspace((*out)->d, (*out)->sms);
  return st;
}

fconv_status fconv_norm_workspace_size(const fconv_norm_plan* p, size_t* bytes) {
  if (!p || !bytes) return FCONV_E_NULL;
  *bytes = p->workspace;
  return FCONV_OK;
}

fconv_status fconv_norm_forward(const fconv_norm_plan* p, const void* x, const void* w,
                                const void* b, void* y, float* mean, float* rstd, void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_norm_desc& d = p->d;
  if ((d.outer && (!x || !y)) || (d.has_weight && !w) || (d.has_bias && !b)) return FCONV_E_NULL;
  if ((!d.has_weight && w) || (!d.has_bias && b)) return FCONV_E_BIAS_SHAPE;
  const size_t e = type_size(d.dtype), pe = type_size(d.param_dtype);
  if (misaligned(x, e) || misaligned(y, e) || misaligned(w, pe) || misaligned(b, pe) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return FCONV_E_ALIGNMENT;
  if (y && (y == w || y == b || y == mean || y == rstd || (mean && mean == rstd)))
    return FCONV_E_ALIAS;
  if (d.outer == 0) return FCONV_OK;
  NormArgs a{};
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return done(launch_norm_forward(d, p->sms, a, (cudaStream_t)stream));
}

fconv_status fconv_norm_backward(const fconv_norm_plan* p, const void* dy, const void* x,
                                 const void* w, const float* mean, const float* rstd, void* dx,
                                 void* dw, void* db, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_norm_desc& d = p->d;
  if ((d.outer && (!x || !dy || !mean || !rstd || !dx)) || (d.has_weight && !w))
    return FCONV_E_NULL;
  if ((!d.has_weight && (w || dw)) || (!d.has_bias && db)) return FCONV_E_BIAS_SHAPE;
  const size_t e = type_size(d.dtype), pe = type_size(d.param_dtype);
  if (misaligned(x, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(w, pe) ||
      misaligned(dw, pe) || misaligned(db, pe) || misaligned(mean, 4) || misaligned(rstd, 4) ||
      misaligned(workspace, 16))
    return FCONV_E_ALIGNMENT;
  if ((dx && (dx == x || dx == w || dx == mean || dx == rstd || dx == dw || dx == db)) ||
      (dw && (dw == w || dw == db)))
    return FCONV_E_ALIAS;
  if ((dw || db) && (!workspace || workspace_bytes < p->workspace)) return FCONV_E_WORKSPACE;
  NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.w = w;
  a.y = dx;
  a.dw = dw;
  a.db = db;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.ws = (float*)workspace;
  return done(launch_norm_backward(d, p->sms, a, (cudaStream_t)stream));
}

void fconv_norm_destroy(fconv_norm_plan* p) { delete p; }

// ------------------------------------------------------------------------------ positions

fconv_status fconv_rope_plan_create(const fconv_rope_desc* desc, int device,
                                    fconv_rope_plan** out) {
  return new_plan(desc, device, check_rope, out);
}

fconv_status fconv_rope_run(const fconv_rope_plan* p, const void* q, const void* k,
                            const void* positions, const float* inv_freq, void* q_out,
                            void* k_out, void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_rope_desc& d = p->d;
  if (d.batch * d.len == 0) return FCONV_OK;
  if (!q || !q_out || !positions || !inv_freq || (d.heads_k && (!k || !k_out)))
    return FCONV_E_NULL;
  if (!d.heads_k && (k || k_out)) return FCONV_E_EXTENT;
  const size_t e = type_size(d.dtype), pe = d.pos_type == FCONV_POS_I64 ? 8 : 4;
  if (misaligned(q, e) || misaligned(k, e) || misaligned(q_out, e) || misaligned(k_out, e) ||
      misaligned(positions, pe) || misaligned(inv_freq, 4))
    return FCONV_E_ALIGNMENT;
  if ((q_out == q && !same_strides(d.q_stride, d.q_out_stride)) ||
      (k && k_out == k && !same_strides(d.k_stride, d.k_out_stride)) || (k && q_out == k) ||
      (k && k_out == q) || (k && k_out == q_out) || q_out == positions || k_out == positions ||
      q_out == inv_freq || k_out == inv_freq)
    return FCONV_E_ALIAS;
  RopeArgs a{q, k, positions, inv_freq, q_out, k_out};
  return done(launch_rope(d, p->sms, a, (cudaStream_t)stream));
}

void fconv_rope_destroy(fconv_rope_plan* p) { delete p; }

// ------------------------------------------------------------------------------ attention

fconv_status fconv_attn_plan_create(const fconv_attn_desc* desc, int device, int route,
                                    fconv_attn_plan** out) {
  const fconv_status st = new_plan(desc, device, check_attn, out);
  if (st != FCONV_OK) return st;
  fconv_attn_plan* p = *out;
  const bool fwd = attn_tc_supported(p->d);
  const bool bwd = p->d.training && attn_tc_backward_supported(p->d);
  if (route < FCONV_ATTN_AUTO || route > FCONV_ATTN_TC ||
      (route == FCONV_ATTN_TC && (!fwd || (p->d.training && !bwd)))) {
    delete p;
    *out = nullptr;
    return FCONV_E_UNSUPPORTED;
  }
  p->want = route;
  p->fwd_tc = fwd && route != FCONV_ATTN_SIMPLE;
  p->bwd_tc = bwd && route != FCONV_ATTN_SIMPLE;
  p->fwd_ws = p->fwd_tc ? attn_tc_forward_workspace(p->d, p->sms) : 0;
  if (p->d.training) {
    p->bwd_ws = attn_simple_backward_workspace(p->d);
    if (p->bwd_tc) {  // a call with unaligned addresses takes the simple route
      const size_t n = attn_tc_backward_workspace(p->d, p->sms);
      if (n > p->bwd_ws) p->bwd_ws = n;
    }
  }
  return FCONV_OK;
}

fconv_status fconv_attn_plan_route(const fconv_attn_plan* p, int* route) {
  if (!p || !route) return FCONV_E_NULL;
  *route = (p->d.training ? p->bwd_tc : p->fwd_tc) ? FCONV_ATTN_TC : FCONV_ATTN_SIMPLE;
  return FCONV_OK;
}

fconv_status fconv_attn_forward_workspace(const fconv_attn_plan* p, size_t* bytes) {
  if (!p || !bytes) return FCONV_E_NULL;
  *bytes = p->fwd_ws;
  return FCONV_OK;
}

fconv_status fconv_attn_backward_workspace(const fconv_attn_plan* p, size_t* bytes) {
  if (!p || !bytes) return FCONV_E_NULL;
  *bytes = p->bwd_ws;
  return FCONV_OK;
}

fconv_status fconv_attn_forward(const fconv_attn_plan* p, const void* q, const void* k,
                                const void* v, const int32_t* q_lens, const int32_t* kv_lens,
                                void* out, float* lse, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_attn_desc& d = p->d;
  const fconv_status st = attn_inputs(d, q, k, v, q_lens, kv_lens);
  if (st != FCONV_OK) return st;
  if (d.batch * d.len_q == 0) return FCONV_OK;
  if (!out) return FCONV_E_NULL;
  if (misaligned(out, type_size(d.dtype)) || misaligned(lse, 4) || misaligned(workspace, 16))
    return FCONV_E_ALIGNMENT;
  if (out == q || out == k || out == v || out == lse || out == q_lens || out == kv_lens)
    return FCONV_E_ALIAS;
  if (p->fwd_ws && (!workspace || workspace_bytes < p->fwd_ws)) return FCONV_E_WORKSPACE;
  AttnArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_lens = q_lens;
  a.kv_lens = kv_lens;
  a.o = out;
  a.lse = lse;
  a.ws = workspace;
  if (p->fwd_tc) {
    if (!misaligned(q, 16) && !misaligned(k, 16) && !misaligned(v, 16) && !misaligned(out, 16))
      return done(launch_attn_tc_forward(d, p->sms, a, (cudaStream_t)stream));
    if (p->want == FCONV_ATTN_TC) return FCONV_E_ALIGNMENT;
  }
  return done(launch_attn_simple_forward(d, a, (cudaStream_t)stream));
}

fconv_status fconv_attn_backward(const fconv_attn_plan* p, const void* dout, const void* q,
                                 const void* k, const void* v, const void* out, const float* lse,
                                 const int32_t* q_lens, const int32_t* kv_lens, void* dq,
                                 void* dk, void* dv, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_attn_desc& d = p->d;
  if (!d.training) return FCONV_E_UNSUPPORTED;
  const fconv_status st = attn_inputs(d, q, k, v, q_lens, kv_lens);
  if (st != FCONV_OK) return st;
  const bool nq = d.batch * d.len_q > 0, nk = d.batch * d.len_k > 0;
  if (!nq && !nk) return FCONV_OK;
  if ((nq && (!dout || !out || !lse || !dq)) || (nk && (!dk || !dv))) return FCONV_E_NULL;
  const size_t e = type_size(d.dtype);
  if (misaligned(dout, e) || misaligned(out, e) || misaligned(dq, e) || misaligned(dk, e) ||
      misaligned(dv, e) || misaligned(lse, 4) || misaligned(workspace, 16))
    return FCONV_E_ALIGNMENT;
  const void* in[] = {dout, q, k, v, out, lse, q_lens, kv_lens};
  const void* outs[] = {dq, dk, dv};
  for (int i = 0; i < 3; ++i) {
    for (const void* x : in)
      if (outs[i] && outs[i] == x) return FCONV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return FCONV_E_ALIAS;
  }
  if (p->bwd_ws && (!workspace || workspace_bytes < p->bwd_ws)) return FCONV_E_WORKSPACE;
  AttnArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.dout = dout;
  a.q_lens = q_lens;
  a.kv_lens = kv_lens;
  a.lse = const_cast<float*>(lse);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.ws = workspace;
  if (p->bwd_tc) {
    bool whole = true;
    for (const void* x : {dout, q, k, v, out, (const void*)dq, (const void*)dk, (const void*)dv})
      whole = whole && !misaligned(x, 16);
    if (whole) return done(launch_attn_tc_backward(d, p->sms, a, (cudaStream_t)stream));
    if (p->want == FCONV_ATTN_TC) return FCONV_E_ALIGNMENT;
  }
  return done(launch_attn_simple_backward(d, a, (cudaStream_t)stream));
}

void fconv_attn_destroy(fconv_attn_plan* p) { delete p; }

}  // extern "C"
