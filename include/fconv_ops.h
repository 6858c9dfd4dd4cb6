/*
 * fconv_ops.h -- C ABI of the token-side operators in libfconv.so: layer norm, rotary
 * positions with several axes (alone, or with the norm of each head), attention, and the gated
 * feed-forward block, each with its gradient.
 *
 * They follow the conventions of fconv.h: a descriptor is validated by *_plan_create before
 * anything is allocated or launched; a plan owns only host state; the caller owns every tensor
 * and the workspace; a run checks its pointers and the workspace, then enqueues on the given
 * stream (a cudaStream_t; NULL = legacy default) and returns; on any error detected on the
 * host nothing is launched and no output is written. No call aborts the process. A plan may be
 * used from several streams at once as long as each call has a workspace of its own.
 *
 * Every sum, softmax statistic and norm is held in f32; each output is rounded once. Beyond that
 * two operators round in f16 and bf16. Attention on FCONV_ATTN_TC: its probabilities and its score
 * gradients are 16-bit operands of the products that follow, and on either route the gradient's
 * delta comes from out as it was rounded. With FCONV_ATTN_TC its outputs are off by 1.2 to 1.5 times
 * their own rounding, dq and dk over a few dozen keys by up to 1.8 times. The gated feed-forward
 * block: its hidden values and their gradients, as its section says. Results do not depend on the
 * order in which blocks run: there are no floating-point atomics.
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

/* ------------------------------------------- norm of each head, with rotary positions
 * Every head of q (batch, len, heads_q, head_dim) and k (batch, len, heads_k, head_dim) is divided
 * by its root mean square, multiplied by a weight of head_dim values and turned by its token's
 * position, in one pass:
 *   n = x * r,  r = 1 / sqrt(mean(x^2) + eps),  z = n * w,  y = z turned as by fconv_rope_run
 * Strides and positions are those of fconv_rope_desc; axes = 0 leaves the rotation out (positions
 * and inv_freq are then NULL). Weights have param_dtype, which is dtype or FCONV_F32; q and k have
 * one each, both optional. heads_k = 0 for q alone. head_dim 1..512. The squares are summed in f32:
 * a head whose sum passes the type (values of f32 and bf16 past about 1e18) comes out as zeros, its
 * gradient as zeros or NaN. */
typedef struct {
  int dtype, param_dtype;
  int64_t batch, len, heads_q, heads_k, head_dim;
  int64_t q_stride[3], k_stride[3];         /* of (batch, token, head), in elements */
  int64_t q_out_stride[3], k_out_stride[3]; /* forward: y; backward: y's gradient */
  int64_t dq_stride[3], dk_stride[3];       /* backward: x's gradient */
  int has_weight, has_k_weight;
  float eps; /* finite and > 0 */
  int axes;  /* 0..3 */
  int64_t section[3];
  int pairing, pos_type;
  int64_t pos_batch;
  int training; /* 1: the plan is of the backward pass */
} fconv_norm_rope_desc;
typedef struct fconv_norm_rope_plan fconv_norm_rope_plan;

fconv_status fconv_norm_rope_plan_create(const fconv_norm_rope_desc* desc, int device,
                                         fconv_norm_rope_plan** out);
/* Workspace of the backward pass where a weight's gradient is wanted. */
fconv_status fconv_norm_rope_workspace_size(const fconv_norm_rope_plan* plan, size_t* bytes);
/* q_out may be q with the same strides (in place), likewise k. */
fconv_status fconv_norm_rope_forward(const fconv_norm_rope_plan* plan, const void* q,
                                     const void* k, const void* weight, const void* k_weight,
                                     const void* positions, const float* inv_freq, void* q_out,
                                     void* k_out, void* stream);
/* q and k are the forward pass's inputs; r is made again from them. dq may be dq_out with the same
 * strides, likewise dk. dweight and dk_weight are sums over batch, tokens and heads, of
 * param_dtype; they may be NULL (not wanted). */
fconv_status fconv_norm_rope_backward(const fconv_norm_rope_plan* plan, const void* dq_out,
                                      const void* dk_out, const void* q, const void* k,
                                      const void* weight, const void* k_weight,
                                      const void* positions, const float* inv_freq, void* dq,
                                      void* dk, void* dweight, void* dk_weight, void* workspace,
                                      size_t workspace_bytes, void* stream);
void fconv_norm_rope_destroy(fconv_norm_rope_plan* plan);

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

/* ---------------------------------------------------------- gated feed-forward block
 *   g = x w_gate^T + b_gate,  u = x w_up^T + b_up,  h = act(g) * u,  y = h w_down^T + b_down
 * x is (tokens, features), w_gate and w_up (hidden, features), w_down (out_features, hidden), y
 * (tokens, out_features); all with contiguous rows a stride (in elements) apart, so that gate and
 * up may be halves of one packed weight. Biases are contiguous, each optional, and of dtype.
 * act is one of FCONV_ACT_NONE, RELU, SIGMOID, GELU (erf), FASTGELU (tanh) and QUICKGELU
 * (v * sigmoid(alpha v); alpha = 1 is SiLU). With no tokens the weights' gradients are zero.
 * g and u are f32; in f16 and bf16 h, and in the backward pass the gradients of g and u, are rounded
 * to dtype once as operands of the next product: in f16 they overflow past 65504 and lose bits under
 * 6e-5. The 16-bit outputs are off by about 1.4 times their own rounding, over a few dozen hidden
 * values by up to 1.8 in single calls. The forward pass of up to 32 tokens (but on FCONV_MLP_SIMPLE)
 * keeps h to 2^-16 of itself (f16: 2^-22, 2^-36 under 6e-5, up to 65504) and rounds y alone. 16-bit
 * sums on tensor cores lose up to 1e-4 of themselves where all terms have one sign, however long.
 * In f32 nothing is rounded to fewer bits (operands are split into parts that add up to them), but
 * that values under 2^-110 may lose their last parts and an infinity may come out as NaN. */
typedef struct {
  int dtype;
  int64_t tokens, features, hidden, out_features;
  int64_t x_stride, y_stride, gate_stride, up_stride, down_stride;
  int64_t dy_stride, dx_stride; /* backward only; weights' gradients are contiguous */
  int has_b_gate, has_b_up, has_b_down;
  int activation; /* fconv_act */
  float alpha;    /* of QUICKGELU */
  int training;   /* 1: the plan also runs the backward pass */
} fconv_mlp_desc;
typedef enum {
  FCONV_MLP_AUTO = 0,
  FCONV_MLP_SIMPLE = 1, /* one warp-level kernel for every call */
  FCONV_MLP_TC = 2      /* tcgen05 tensor cores, and a kernel that streams the weights for the
                           forward pass of up to 32 tokens. f32, and tensors whose rows do not
                           start on 16 bytes, are copied into the workspace first. */
} fconv_mlp_route;
typedef struct fconv_mlp_plan fconv_mlp_plan;

/* route: FCONV_MLP_AUTO, or one that must run the request (else FCONV_E_UNSUPPORTED). */
fconv_status fconv_mlp_plan_create(const fconv_mlp_desc* desc, int device, int route,
                                   fconv_mlp_plan** out);
/* The route of a call with tokens whose device addresses are 16-byte aligned. One with others runs
 * on FCONV_MLP_SIMPLE if TMA had to read them where they are, unless the plan was made for
 * FCONV_MLP_TC: then FCONV_E_ALIGNMENT. */
fconv_status fconv_mlp_plan_route(const fconv_mlp_plan* plan, int* route);
fconv_status fconv_mlp_forward_workspace(const fconv_mlp_plan* plan, size_t* bytes);
fconv_status fconv_mlp_backward_workspace(const fconv_mlp_plan* plan, size_t* bytes);
/* Bytes of `saved`: g and u in f32, in an order of the library's own. */
fconv_status fconv_mlp_saved_size(const fconv_mlp_plan* plan, size_t* bytes);
/* saved may be NULL (inference, or a backward pass that makes g and u again). y must not be an
 * input. */
fconv_status fconv_mlp_forward(const fconv_mlp_plan* plan, const void* x, const void* w_gate,
                               const void* w_up, const void* w_down, const void* b_gate,
                               const void* b_up, const void* b_down, void* y, float* saved,
                               void* workspace, size_t workspace_bytes, void* stream);
/* saved is a forward pass's of the same x, w_gate, w_up and biases, or NULL: g and u are then made
 * again from these. Every gradient may be NULL (not wanted). */
fconv_status fconv_mlp_backward(const fconv_mlp_plan* plan, const void* dy, const void* x,
                                const void* w_gate, const void* w_up, const void* w_down,
                                const void* b_gate, const void* b_up, const float* saved, void* dx,
                                void* dw_gate, void* dw_up, void* dw_down, void* db_gate,
                                void* db_up, void* db_down, void* workspace,
                                size_t workspace_bytes, void* stream);
void fconv_mlp_destroy(fconv_mlp_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* FCONV_OPS_H_ */
