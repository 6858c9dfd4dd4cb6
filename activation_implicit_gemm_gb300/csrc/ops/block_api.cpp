// C ABI and planner of the head norms with rotation and of the gated feed-forward block
// (include/fconv_ops.h). As in ops_api.cpp every rule is checked before anything is launched.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "api_common.h"

using namespace fconv::ops;

struct fconv_norm_rope_plan {
  fconv_norm_rope_desc d;
  int sms;
  size_t workspace;
};
struct fconv_mlp_plan {
  fconv_mlp_desc d;
  int sms;
  int want;
  size_t saved;           // bytes of g and u
  size_t fwd_ws, bwd_ws;  // bwd_ws without room for g and u
};

namespace {

fconv_status check_norm_rope(const fconv_norm_rope_desc& d) {
  if (!known_type(d.dtype) || !known_type(d.param_dtype) ||
      (d.param_dtype != d.dtype && d.param_dtype != FCONV_F32))
    return FCONV_E_UNSUPPORTED;
  if (!small(d.batch, 0) || !small(d.len, 0) || !small(d.heads_q, 1) || !small(d.heads_k, 0) ||
      !small(d.head_dim, 1) || (d.axes > 0 && d.pos_batch != 1 && d.pos_batch != d.batch))
    return FCONV_E_EXTENT;
  if (d.axes < 0 || d.axes > 3 || d.pairing < FCONV_ROPE_INTERLEAVED ||
      d.pairing > FCONV_ROPE_HALF_PER_AXIS || d.pos_type < FCONV_POS_I32 ||
      d.pos_type > FCONV_POS_F32 || !(d.eps > 0.0f) || !std::isfinite(d.eps))
    return FCONV_E_ATTR_VALUE;
  int64_t pairs = 0;
  for (int i = 0; i < d.axes; ++i) {
    if (!small(d.section[i], 0)) return FCONV_E_ATTR_VALUE;
    pairs += d.section[i];
  }
  if (pairs > d.head_dim / 2) return FCONV_E_EXTENT;
  if (d.has_k_weight && !d.heads_k) return FCONV_E_BIAS_SHAPE;
  const int64_t eq[3] = {d.batch, d.len, d.heads_q}, ek[3] = {d.batch, d.len, d.heads_k};
  // a training plan's outputs are dq and dk
  if (!strides_ok(d.q_stride, eq, d.head_dim, false) ||
      !strides_ok(d.q_out_stride, eq, d.head_dim, !d.training) ||
      (d.training && !strides_ok(d.dq_stride, eq, d.head_dim, true)))
    return FCONV_E_STRIDE;
  if (d.heads_k && (!strides_ok(d.k_stride, ek, d.head_dim, false) ||
                    !strides_ok(d.k_out_stride, ek, d.head_dim, !d.training) ||
                    (d.training && !strides_ok(d.dk_stride, ek, d.head_dim, true))))
    return FCONV_E_STRIDE;
  if (d.head_dim > kNormRopeMostDim || d.heads_q + d.heads_k > 65535 ||
      d.batch * d.len > INT_MAX / 32)  // 32 lanes a token at most
    return FCONV_E_UNSUPPORTED;
  return FCONV_OK;
}

// What the forward and the backward pass of the head norms share.
fconv_status norm_rope_inputs(const fconv_norm_rope_desc& d, const void* q, const void* k,
                              const void* w, const void* kw, const void* positions,
                              const float* inv_freq) {
  if (d.batch * d.len > 0 && (!q || (d.heads_k && !k) || (d.axes && (!positions || !inv_freq))))
    return FCONV_E_NULL;
  if ((d.has_weight && !w) || (d.has_k_weight && !kw)) return FCONV_E_NULL;
  if ((!d.has_weight && w) || (!d.has_k_weight && kw)) return FCONV_E_BIAS_SHAPE;
  if ((!d.heads_k && k) || (!d.axes && (positions || inv_freq))) return FCONV_E_EXTENT;
  const size_t e = type_size(d.dtype), pe = type_size(d.param_dtype);
  if (misaligned(q, e) || misaligned(k, e) || misaligned(w, pe) || misaligned(kw, pe) ||
      misaligned(positions, d.pos_type == FCONV_POS_I64 ? 8 : 4) || misaligned(inv_freq, 4))
    return FCONV_E_ALIGNMENT;
  return FCONV_OK;
}

bool known_gate(int act) {
  return act == FCONV_ACT_NONE || act == FCONV_ACT_RELU || act == FCONV_ACT_SIGMOID ||
         act == FCONV_ACT_QUICKGELU || act == FCONV_ACT_GELU || act == FCONV_ACT_FASTGELU;
}

fconv_status check_mlp(const fconv_mlp_desc& d) {
  if (!known_type(d.dtype)) return FCONV_E_UNSUPPORTED;
  if (!small(d.tokens, 0) || !small(d.features, 1) || !small(d.hidden, 1) ||
      !small(d.out_features, 1))
    return FCONV_E_EXTENT;
  if (!known_gate(d.activation)) return FCONV_E_ACTIVATION;
  if (d.activation == FCONV_ACT_QUICKGELU && !std::isfinite(d.alpha)) return FCONV_E_ATTR_VALUE;
  for (int64_t s : {d.x_stride, d.gate_stride, d.up_stride, d.down_stride})
    if (s < 0) return FCONV_E_STRIDE;
  if (d.tokens > 1 && d.y_stride < d.out_features) return FCONV_E_STRIDE;
  if (d.training && (d.dy_stride < 0 || (d.tokens > 1 && d.dx_stride < d.features)))
    return FCONV_E_STRIDE;
  // what a grid or a buffer of any product could need
  const double widest = (double)(d.features > d.out_features ? d.features : d.out_features);
  const double rows = (double)d.tokens / 32 + 1, hidden = (double)d.hidden / 32 + 1;
  if (rows * hidden > INT_MAX / 2 || rows * (widest / 32 + 1) > INT_MAX / 2 ||
      hidden * (widest / 32 + 1) > INT_MAX / 2)
    return FCONV_E_UNSUPPORTED;
  return FCONV_OK;
}

size_t whole(size_t bytes) { return (bytes + 255) / 256 * 256; }

// The larger one of what the routes of a plan need.
size_t mlp_workspace(const fconv_mlp_plan& p, bool backward) {
  const size_t simple = mlp_simple_workspace(p.d, backward, p.sms);
  const size_t tc =
      p.want == FCONV_MLP_SIMPLE ? 0 : mlp_tc_workspace(p.d, backward, p.sms);
  return whole(simple > tc ? simple : tc);
}

fconv_status mlp_inputs(const fconv_mlp_desc& d, const void* x, const void* w_gate,
                        const void* w_up, const void* w_down, const void* b_gate,
                        const void* b_up) {
  if ((d.tokens && !x) || !w_gate || !w_up || !w_down || (d.has_b_gate && !b_gate) ||
      (d.has_b_up && !b_up))
    return FCONV_E_NULL;
  if ((!d.has_b_gate && b_gate) || (!d.has_b_up && b_up)) return FCONV_E_BIAS_SHAPE;
  const size_t e = type_size(d.dtype);
  for (const void* p : {x, w_gate, w_up, w_down, b_gate, b_up})
    if (misaligned(p, e)) return FCONV_E_ALIGNMENT;
  return FCONV_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------- head norms with rotation

fconv_status fconv_norm_rope_plan_create(const fconv_norm_rope_desc* desc, int device,
                                         fconv_norm_rope_plan** out) {
  const fconv_status st = new_plan(desc, device, check_norm_rope, out);
  if (st == FCONV_OK && (*out)->d.training)
    (*out)->workspace = norm_rope_workspace((*out)->d, (*out)->sms);
  return st;
}

fconv_status fconv_norm_rope_workspace_size(const fconv_norm_rope_plan* p, size_t* bytes) {
  if (!p || !bytes) return FCONV_E_NULL;
  *bytes = p->workspace;
  return FCONV_OK;
}

fconv_status fconv_norm_rope_forward(const fconv_norm_rope_plan* p, const void* q, const void* k,
                                     const void* weight, const void* k_weight,
                                     const void* positions, const float* inv_freq, void* q_out,
                                     void* k_out, void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_norm_rope_desc& d = p->d;
  if (d.training) return FCONV_E_UNSUPPORTED;
  const fconv_status st = norm_rope_inputs(d, q, k, weight, k_weight, positions, inv_freq);
  if (st != FCONV_OK) return st;
  if (d.batch * d.len == 0) return FCONV_OK;
  if (!q_out || (d.heads_k && !k_out)) return FCONV_E_NULL;
  if (!d.heads_k && k_out) return FCONV_E_EXTENT;
  const size_t e = type_size(d.dtype);
  if (misaligned(q_out, e) || misaligned(k_out, e)) return FCONV_E_ALIGNMENT;
  if ((q_out == q && !same_strides(d.q_stride, d.q_out_stride)) ||
      (k && k_out == k && !same_strides(d.k_stride, d.k_out_stride)) || (k && q_out == k) ||
      (k && (k_out == q || k_out == q_out)))
    return FCONV_E_ALIAS;
  for (const void* in : {weight, k_weight, positions, (const void*)inv_freq})
    if (in && (q_out == in || k_out == in)) return FCONV_E_ALIAS;
  NormRopeArgs a{};
  a.q = q;
  a.k = k;
  a.w = weight;
  a.kw = k_weight;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.k_out = k_out;
  return done(launch_norm_rope_forward(d, p->sms, a, (cudaStream_t)stream));
}

fconv_status fconv_norm_rope_backward(const fconv_norm_rope_plan* p, const void* dq_out,
                                      const void* dk_out, const void* q, const void* k,
                                      const void* weight, const void* k_weight,
                                      const void* positions, const float* inv_freq, void* dq,
                                      void* dk, void* dweight, void* dk_weight, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_norm_rope_desc& d = p->d;
  if (!d.training) return FCONV_E_UNSUPPORTED;
  const fconv_status st = norm_rope_inputs(d, q, k, weight, k_weight, positions, inv_freq);
  if (st != FCONV_OK) return st;
  if (d.batch * d.len > 0 && (!dq_out || !dq || (d.heads_k && (!dk_out || !dk)))) return FCONV_E_NULL;
  if (!d.heads_k && (dk_out || dk)) return FCONV_E_EXTENT;
  if ((!d.has_weight && dweight) || (!d.has_k_weight && dk_weight)) return FCONV_E_BIAS_SHAPE;
  const size_t e = type_size(d.dtype), pe = type_size(d.param_dtype);
  if (misaligned(dq_out, e) || misaligned(dk_out, e) || misaligned(dq, e) || misaligned(dk, e) ||
      misaligned(dweight, pe) || misaligned(dk_weight, pe) || misaligned(workspace, 16))
    return FCONV_E_ALIGNMENT;
  if ((dq && dq == dq_out && !same_strides(d.dq_stride, d.q_out_stride)) ||
      (dk && dk == dk_out && !same_strides(d.dk_stride, d.k_out_stride)) ||
      (dq && dq == dk_out) || (dk && dk == dq_out))
    return FCONV_E_ALIAS;
  const void* in[] = {q, k, weight, k_weight, positions, inv_freq};
  const void* outs[] = {dq, dk, dweight, dk_weight};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    for (const void* x : in)
      if (outs[i] == x) return FCONV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (outs[i] == outs[j]) return FCONV_E_ALIAS;
    if (i >= 2 && (outs[i] == dq_out || outs[i] == dk_out)) return FCONV_E_ALIAS;
  }
  const bool sums = dweight || dk_weight;
  if (sums && (!workspace || workspace_bytes < p->workspace)) return FCONV_E_WORKSPACE;
  NormRopeArgs a{};
  a.q = q;
  a.k = k;
  a.w = weight;
  a.kw = k_weight;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.q_out = dq_out;
  a.k_out = dk_out;
  a.dq = dq;
  a.dk = dk;
  a.dw = dweight;
  a.dkw = dk_weight;
  a.ws = sums ? (float*)workspace : nullptr;
  return done(launch_norm_rope_backward(d, p->sms, a, (cudaStream_t)stream));
}

void fconv_norm_rope_destroy(fconv_norm_rope_plan* p) { delete p; }

// ------------------------------------------------------------- gated feed-forward block

fconv_status fconv_mlp_plan_create(const fconv_mlp_desc* desc, int device, int route,
                                   fconv_mlp_plan** out) {
  const fconv_status st = new_plan(desc, device, check_mlp, out);
  if (st != FCONV_OK) return st;
  fconv_mlp_plan* p = *out;
  const fconv_mlp_desc& d = p->d;
  if (route < FCONV_MLP_AUTO || route > FCONV_MLP_TC) {
    delete p;
    *out = nullptr;
    return FCONV_E_UNSUPPORTED;
  }
  p->want = route;
  p->saved = mlp_saved_bytes(d);
  p->fwd_ws = mlp_workspace(*p, false);
  if (d.training) p->bwd_ws = mlp_workspace(*p, true);
  return FCONV_OK;
}

fconv_status fconv_mlp_plan_route(const fconv_mlp_plan* p, int* route) {
  if (!p || !route) return FCONV_E_NULL;
  *route = p->want == FCONV_MLP_SIMPLE ? FCONV_MLP_SIMPLE : FCONV_MLP_TC;
  return FCONV_OK;
}

fconv_status fconv_mlp_forward_workspace(const fconv_mlp_plan* p, size_t* bytes) {
  if (!p || !bytes) return FCONV_E_NULL;
  *bytes = p->fwd_ws;
  return FCONV_OK;
}

fconv_status fconv_mlp_backward_workspace(const fconv_mlp_plan* p, size_t* bytes) {
  if (!p || !bytes) return FCONV_E_NULL;
  *bytes = p->bwd_ws ? p->bwd_ws + p->saved : 0;
  return FCONV_OK;
}

fconv_status fconv_mlp_saved_size(const fconv_mlp_plan* p, size_t* bytes) {
  if (!p || !bytes) return FCONV_E_NULL;
  *bytes = p->saved;
  return FCONV_OK;
}

fconv_status fconv_mlp_forward(const fconv_mlp_plan* p, const void* x, const void* w_gate,
                               const void* w_up, const void* w_down, const void* b_gate,
                               const void* b_up, const void* b_down, void* y, float* saved,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_mlp_desc& d = p->d;
  const fconv_status st = mlp_inputs(d, x, w_gate, w_up, w_down, b_gate, b_up);
  if (st != FCONV_OK) return st;
  if (d.has_b_down && !b_down) return FCONV_E_NULL;
  if (!d.has_b_down && b_down) return FCONV_E_BIAS_SHAPE;
  if (d.tokens == 0) return FCONV_OK;
  if (!y) return FCONV_E_NULL;
  const size_t e = type_size(d.dtype);
  if (misaligned(y, e) || misaligned(b_down, e) || misaligned(saved, 16) ||
      misaligned(workspace, 16))
    return FCONV_E_ALIGNMENT;
  for (const void* in : {x, w_gate, w_up, w_down, b_gate, b_up, b_down})
    if (in && (y == in || saved == in)) return FCONV_E_ALIAS;
  if (y == saved) return FCONV_E_ALIAS;
  if (!workspace || workspace_bytes < p->fwd_ws) return FCONV_E_WORKSPACE;
  MlpArgs a{};
  a.x = x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.w_down = w_down;
  a.b_gate = b_gate;
  a.b_up = b_up;
  a.b_down = b_down;
  a.y = y;
  a.saved = saved;
  a.ws = workspace;
  if (p->want != FCONV_MLP_SIMPLE) {
    if (mlp_tc_supported(d, a, false))
      return done(launch_mlp_tc_forward(d, p->sms, a, (cudaStream_t)stream));
    if (p->want == FCONV_MLP_TC) return FCONV_E_ALIGNMENT;
  }
  return done(launch_mlp_simple_forward(d, a, (cudaStream_t)stream));
}

fconv_status fconv_mlp_backward(const fconv_mlp_plan* p, const void* dy, const void* x,
                                const void* w_gate, const void* w_up, const void* w_down,
                                const void* b_gate, const void* b_up, const float* saved, void* dx,
                                void* dw_gate, void* dw_up, void* dw_down, void* db_gate,
                                void* db_up, void* db_down, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!p) return FCONV_E_NULL;
  const fconv_mlp_desc& d = p->d;
  if (!d.training) return FCONV_E_UNSUPPORTED;
  const fconv_status st = mlp_inputs(d, x, w_gate, w_up, w_down, b_gate, b_up);
  if (st != FCONV_OK) return st;
  if (d.tokens && !dy) return FCONV_E_NULL;
  if ((!d.has_b_gate && db_gate) || (!d.has_b_up && db_up) || (!d.has_b_down && db_down))
    return FCONV_E_BIAS_SHAPE;
  const void* in[] = {dy, x, w_gate, w_up, w_down, b_gate, b_up, saved};
  void* outs[] = {dx, dw_gate, dw_up, dw_down, db_gate, db_up, db_down};
  const size_t e = type_size(d.dtype);
  if (misaligned(dy, e) || misaligned(saved, 16) || misaligned(workspace, 16))
    return FCONV_E_ALIGNMENT;
  for (int i = 0; i < 7; ++i) {
    if (misaligned(outs[i], e)) return FCONV_E_ALIGNMENT;
    if (!outs[i]) continue;
    for (const void* x : in)
      if (outs[i] == x) return FCONV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (outs[i] == outs[j]) return FCONV_E_ALIAS;
  }
  if (!workspace || workspace_bytes < p->bwd_ws + (saved ? 0 : p->saved)) return FCONV_E_WORKSPACE;
  MlpArgs a{};
  a.x = x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.w_down = w_down;
  a.b_gate = b_gate;
  a.b_up = b_up;
  a.dy = dy;
  a.dx = d.tokens ? dx : nullptr;
  a.dw_gate = dw_gate;
  a.dw_up = dw_up;
  a.dw_down = dw_down;
  a.db_gate = db_gate;
  a.db_up = db_up;
  a.db_down = db_down;
  a.saved = saved ? const_cast<float*>(saved) : (float*)((char*)workspace + p->bwd_ws);
  a.remake = !saved;
  a.ws = workspace;
  if (p->want != FCONV_MLP_SIMPLE && d.tokens > 0) {  // no tokens: zeros, by the other route
    if (mlp_tc_supported(d, a, true))
      return done(launch_mlp_tc_backward(d, p->sms, a, (cudaStream_t)stream));
    if (p->want == FCONV_MLP_TC) return FCONV_E_ALIGNMENT;
  }
  return done(launch_mlp_simple_backward(d, p->sms, a, (cudaStream_t)stream));
}

void fconv_mlp_destroy(fconv_mlp_plan* p) { delete p; }

}  // extern "C"
