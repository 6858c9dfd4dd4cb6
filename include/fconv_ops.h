/*
 * fconv_ops.h -- C ABI of the token-side operators in libfconv.so: layer norm, rotary
 * positions with several axes, and attention, each with its gradient.
 *
 * They follow the conventions of fconv.h: a descriptor is validated by *_plan_create before
 * anything is allocated or launched; a plan owns only host state; the caller owns every tensor
 * and the workspace; a run checks its pointers and the workspace, then enqueues on the given
 * stream (a cudaStream_t; NULL = legacy default) and returns; on any error detected on the
 * host nothing is launched and no output is written. No call aborts the process. A plan may be
 * used from several streams at once as long as each call has a workspace of its own.
 *
 * Every sum, softmax statistic and norm is held in f32; each output is rounded once. Beyond that
 * only attention in f16 and bf16 rounds: on FCONV_ATTN_TC its probabilities and its score gradients
 * are 16-bit operands of the products that follow, and on either route the gradient's delta comes
 * from out as it was rounded. With FCONV_ATTN_TC its outputs are off by 1.2 to 1.5 times their own
 * rounding, dq and dk over a few dozen keys by up to 1.8 times. Results do not depend on the order
 * in which blocks run: there are no floating-point atomics.
 */
#ifndef FCONV_OPS_H_
#define FCONV_OPS_H_

#include "fconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The text of any status, those of fconv.h included. */
const char* fconv_ops_status_string(int status);

/* Synchronise `stream`, then read and clear the error word that these operators' kernels set
 * when a bounded wait gives up: FCONV_OK, FCONV_E_DEVICE_TIMEOUT or FCONV_E_CUDA. */
fconv_status fconv_ops_check_device(void* stream);

/* ------------------------------------------------------------------------- layer norm
 * x is (outer, channels, inner), contiguous; every vector of `channels` values is normalised:
 *   y = (x - mean) * rstd * w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 * inner = 1 is the row form (the last axis of token rows); inner > 1 the channels-first form
 * (N, C, D1..Dn with inner = D1*..*Dn). w and b have `channels` values of param_dtype, which
 * is dtype or FCONV_F32; both are optional. mean and rstd are f32 (outer, inner).
 * outer may be 0 (nothing to do; the gradients of w and b are then zero). */
typedef struct {
  int dtype;       /* x, y, dy, dx: FCONV_F32, FCONV_F16 or FCONV_BF16 */
  int param_dtype; /* w, b, dw, db: dtype or FCONV_F32 */
  int64_t outer, channels, inner;
  int has_weight, has_bias;
  float eps; /* finite and > 0 */
} fconv_norm_desc;
typedef struct fconv_norm_plan fconv_norm_plan;

fconv_status fconv_norm_plan_create(const fconv_norm_desc* desc, int device,
                                    fconv_norm_plan** out);
/* Workspace of the backward pass (partial sums of dw and db); the forward pass needs none. */
fconv_status fconv_norm_workspace_size(const fconv_norm_plan* plan, size_t* bytes);
/* mean and rstd may be NULL (inference); y may be x. */
fconv_status fconv_norm_forward(const fconv_norm_plan* plan, const void* x, const void* w,
                                const void* b, void* y, float* mean, float* rstd, void* stream);
/* dx = rstd * (g - mean(g) - xhat * mean(g * xhat)), g = dy * w, xhat = (x - mean) * rstd;
 * dw = sum(dy * xhat) and db = sum(dy) over outer and inner. dw and db may be NULL (not
 * wanted); dw needs has_weight, db needs has_bias. dx may be dy. */
fconv_status fconv_norm_backward(const fconv_norm_plan* plan, const void* dy, const void* x,
                                 const void* w, const float* mean, const float* rstd, void* dx,
                                 void* dw, void* db, void* workspace, size_t workspace_bytes,
                                 void* stream);
void fconv_norm_destroy(fconv_norm_plan* plan);

/* ------------------------------------------------------- rotary positions, several axes
 * q is (batch, len, heads_q, head_dim) and k (batch, len, heads_k, head_dim) with any strides
 * of their first three axes (in elements) and the last axis contiguous; heads_k = 0 for q
 * alone. A token has a position on each of `axes` axes (1 to 3: e.g. time, height, width).
 * The pairs of a head are split into sections, one per axis: pair p of section a turns by
 *   angle = positions[b, t, a] * inv_freq[p]
 *   (u, v) -> (u cos - v sin, v cos + u sin)        inverse: (u cos + v sin, v cos - u sin)
 * and elements past the last pair are copied. The inverse is the gradient's pass: it takes
 * dq', dk' to dq, dk. Angles are reduced modulo 2 pi with the error of the product corrected, so
 * long positions keep their precision, up to 2^53. */
typedef enum {
  FCONV_ROPE_INTERLEAVED = 0,   /* pair p is elements (2p, 2p + 1) */
  FCONV_ROPE_HALF = 1,          /* pair p is elements (p, p + pairs) */
  FCONV_ROPE_HALF_PER_AXIS = 2  /* section a of n pairs starting at pair s: (s + p, s + p + n) */
} fconv_rope_pairing;
typedef enum {
  FCONV_POS_I32 = 0,
  FCONV_POS_I64 = 1,
  FCONV_POS_F32 = 2
} fconv_rope_postype;
typedef struct {
  int dtype;
  int64_t batch, len, heads_q, heads_k, head_dim;
  int64_t q_stride[3], k_stride[3];       /* of (batch, token, head), in elements */
  int64_t q_out_stride[3], k_out_stride[3];
  int axes;                               /* 1..3 */
  int64_t section[3];                     /* pairs per axis; their sum <= head_dim / 2 */
  int pairing, pos_type;
  int64_t pos_batch;                      /* 1 (shared) or batch: positions (pos_batch, len, axes),
                                             contiguous */
  int inverse;
} fconv_rope_desc;
typedef struct fconv_rope_plan fconv_rope_plan;

fconv_status fconv_rope_plan_create(const fconv_rope_desc* desc, int device,
                                    fconv_rope_plan** out);
/* inv_freq: f32, one per pair. q_out may be q with the same strides (in place), likewise k;
 * outputs must not overlap the inputs in any other way. k and k_out are NULL iff heads_k = 0. */
fconv_status fconv_rope_run(const fconv_rope_plan* plan, const void* q, const void* k,
                            const void* positions, const float* inv_freq, void* q_out,
                            void* k_out, void* stream);
void fconv_rope_destroy(fconv_rope_plan* plan);

/* ---------------------------------------------------------------------------- attention
 * q, out, dout, dq: (batch, len_q, heads_q, head_dim); k, v, dk, dv: (batch, len_k, heads_kv,
 * head_dim); any strides of the first three axes (in elements; 0 on an input broadcasts), the
 * last axis contiguous. heads_q is a multiple of heads_kv: head h reads key head
 * h / (heads_q / heads_kv). head_dim 1..256.
 *   s = scale * q k^T,  p = softmax(s) over the keys a query sees,  out = p v,
 *   lse = log(sum(exp(s)))                                (f32, (batch, heads_q, len_q))
 * q_lens and kv_lens (int32 (batch), each optional) hold the valid tokens of each sequence,
 * clamped to [0, len]; tokens past them take no part, whatever they hold (NaN included).
 * causal: query i sees key j iff j <= i + (kv_len - q_len), so the last query sees every key.
 * A query that sees no key (or lies past q_len) has out 0, lse -inf and zero gradient.
 * A non-finite key or value that lies inside kv_len and is hidden from a query only by the
 * causal order can reach that query. Scores that come out as -inf (keys of f32's or bf16's lowest
 * value, say) have probability 0, and a row that has no others counts as seeing no key; on
 * FCONV_ATTN_TC such a key's value must still give a finite product with dout. */
typedef struct {
  int dtype;
  int64_t batch, len_q, len_k, heads_q, heads_kv, head_dim;
  int64_t q_stride[3], k_stride[3], v_stride[3], out_stride[3]; /* (batch, token, head) */
  int64_t dout_stride[3], dq_stride[3], dk_stride[3], dv_stride[3]; /* backward only */
  float scale; /* finite and > 0 */
  int causal, has_q_lens, has_kv_lens;
  int training; /* 1: the plan also runs the backward pass */
} fconv_attn_desc;
typedef enum {
  FCONV_ATTN_AUTO = 0,
  FCONV_ATTN_SIMPLE = 1, /* every type, head_dim, stride: warp-level tensor instructions in split
                            f32 */
  FCONV_ATTN_TC = 2      /* tcgen05 tensor cores: f16 and bf16, head_dim a multiple of 8 up to
                            128, 16-byte strides and addresses */
} fconv_attn_route;
typedef struct fconv_attn_plan fconv_attn_plan;

/* route: FCONV_ATTN_AUTO, or one that must run the request (else FCONV_E_UNSUPPORTED). */
fconv_status fconv_attn_plan_create(const fconv_attn_desc* desc, int device, int route,
                                    fconv_attn_plan** out);
/* The route of a call whose device addresses are 16-byte aligned, of the backward pass in a
 * training plan (a call with others runs on FCONV_ATTN_SIMPLE, unless the plan was made for
 * FCONV_ATTN_TC: then it is refused with FCONV_E_ALIGNMENT). */
fconv_status fconv_attn_plan_route(const fconv_attn_plan* plan, int* route);
fconv_status fconv_attn_forward_workspace(const fconv_attn_plan* plan, size_t* bytes);
fconv_status fconv_attn_backward_workspace(const fconv_attn_plan* plan, size_t* bytes);
/* lse may be NULL (inference). out must not overlap an input. */
fconv_status fconv_attn_forward(const fconv_attn_plan* plan, const void* q, const void* k,
                                const void* v, const int32_t* q_lens, const int32_t* kv_lens,
                                void* out, float* lse, void* workspace, size_t workspace_bytes,
                                void* stream);
/* out and lse are the forward pass's. Gradients of tokens past their lengths are zero. dq, dk
 * and dv must not overlap each other or an input. */
fconv_status fconv_attn_backward(const fconv_attn_plan* plan, const void* dout, const void* q,
                                 const void* k, const void* v, const void* out, const float* lse,
                                 const int32_t* q_lens, const int32_t* kv_lens, void* dq,
                                 void* dk, void* dv, void* workspace, size_t workspace_bytes,
                                 void* stream);
void fconv_attn_destroy(fconv_attn_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* FCONV_OPS_H_ */
