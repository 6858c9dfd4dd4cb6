// Internal interface between the token-side operators' planner (ops_api.cpp) and their
// CUDA launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../../include/fconv_ops.h"

namespace fconv {
namespace ops {

// Launchers return a cudaError_t as int (0 = success).

struct NormArgs {
  const void* x;
  const void* dy;
  const void* w;
  const void* b;
  void* y;  // y, or dx
  void* dw;
  void* db;
  float* mean;
  float* rstd;
  float* ws;
};
int launch_norm_forward(const fconv_norm_desc& d, int sms, const NormArgs& a, cudaStream_t s);
int launch_norm_backward(const fconv_norm_desc& d, int sms, const NormArgs& a, cudaStream_t s);
size_t norm_workspace(const fconv_norm_desc& d, int sms);
int read_and_clear_norm_error(cudaStream_t s, unsigned* value);

struct RopeArgs {
  const void* q;
  const void* k;
  const void* pos;
  const float* inv_freq;
  void* q_out;
  void* k_out;
};
int launch_rope(const fconv_rope_desc& d, int sms, const RopeArgs& a, cudaStream_t s);

struct NormRopeArgs {
  const void* q;
  const void* k;
  const void* w;
  const void* kw;
  const void* pos;
  const float* inv_freq;
  const void* q_out;  // written by the forward pass, the incoming gradient of the backward pass
  const void* k_out;
  void* dq;  // backward
  void* dk;
  void* dw;
  void* dkw;
  float* ws;  // null: no weight's gradient is wanted
};
constexpr int kNormRopeMostDim = 512;
int launch_norm_rope_forward(const fconv_norm_rope_desc& d, int sms, const NormRopeArgs& a,
                             cudaStream_t s);
int launch_norm_rope_backward(const fconv_norm_rope_desc& d, int sms, const NormRopeArgs& a,
                              cudaStream_t s);
size_t norm_rope_workspace(const fconv_norm_rope_desc& d, int sms);

struct MlpArgs {
  const void* x;
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  const void* b_gate;
  const void* b_up;
  const void* b_down;
  void* y;
  const void* dy;  // backward
  void* dx;
  void* dw_gate;
  void* dw_up;
  void* dw_down;
  void* db_gate;
  void* db_up;
  void* db_down;
  float* saved;  // g and u, or null
  bool remake;   // backward: make g and u first
  void* ws;
};
size_t mlp_saved_bytes(const fconv_mlp_desc& d);
size_t mlp_simple_workspace(const fconv_mlp_desc& d, bool backward, int sms);
int launch_mlp_simple_forward(const fconv_mlp_desc& d, const MlpArgs& a, cudaStream_t s);
int launch_mlp_simple_backward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s);
// Tensor-core route (k_mlp_tc.cu): whether it takes the addresses of a call, its workspace.
bool mlp_tc_supported(const fconv_mlp_desc& d, const MlpArgs& a, bool backward);
size_t mlp_tc_workspace(const fconv_mlp_desc& d, bool backward, int sms);
int launch_mlp_tc_forward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s);
int launch_mlp_tc_backward(const fconv_mlp_desc& d, int sms, const MlpArgs& a, cudaStream_t s);
int read_and_clear_mlp_error(cudaStream_t s, unsigned* value);
// Its products for up to kMlpFewTokens tokens (k_mlp_few.cu); h has rows of h_row elements of the
// call's type (gated: may be null), in 16-bit types twice, its second part h_plane elements on.
constexpr int kMlpFewTokens = 32;
int launch_mlp_few_gated(const fconv_mlp_desc& d, const MlpArgs& a, void* h, int64_t h_row,
                         int64_t h_plane, cudaStream_t s);
int launch_mlp_few_down(const fconv_mlp_desc& d, const MlpArgs& a, const void* h, int64_t h_row,
                        int64_t h_plane, cudaStream_t s);

// Tensors copied into rows of whole 16-byte units, f32 as three bf16 planes (k_mlp_prep.cu).
struct PrepItem {
  const void* src;
  void* dst;
  int64_t rows, cols, src_row, dst_row, plane;  // elements
};
struct PrepArgs {
  PrepItem m[5];
  int count;
};
int launch_mlp_prep(int dtype, const PrepArgs& a, cudaStream_t s);

// Column sums of up to three matrices with the same rows (those without `out` are left out), of
// dtype or, with `planes`, of f32 as three bf16 planes. `early`: the launch before it has waited for
// what made the matrices.
struct SumsArgs {
  const void* p;
  int64_t row, cols, plane;  // strides of rows and planes in elements
  void* out;
};
size_t column_sums_workspace(const int64_t cols[3], int sms);
int launch_column_sums(int dtype, bool planes, bool early, const SumsArgs m[3], int64_t rows,
                       float* part, int sms, cudaStream_t s);

struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* out;  // backward
  const void* dout;
  const int32_t* q_lens;
  const int32_t* kv_lens;
  void* o;  // forward
  float* lse;
  void* dq;
  void* dk;
  void* dv;
  void* ws;
};
// The route without tcgen05: warp-level tensor instructions, for head lengths up to 128 in
// k_attn_mma.cu and beyond in k_attn_mma_wide.cu.
int launch_attn_wide_forward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s);
int launch_attn_wide_backward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s);
int launch_attn_simple_forward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s);
int launch_attn_simple_backward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s);
size_t attn_simple_backward_workspace(const fconv_attn_desc& d);

// Tensor-core route (k_attn_tc_*.cu): addresses must be 16-byte aligned.
bool attn_tc_supported(const fconv_attn_desc& d);
size_t attn_tc_forward_workspace(const fconv_attn_desc& d, int sms);
int launch_attn_tc_forward(const fconv_attn_desc& d, int sms, const AttnArgs& a, cudaStream_t s);
int read_and_clear_attn_forward_error(cudaStream_t s, unsigned* value);
bool attn_tc_backward_supported(const fconv_attn_desc& d);
size_t attn_tc_backward_workspace(const fconv_attn_desc& d, int sms);
int launch_attn_tc_backward(const fconv_attn_desc& d, int sms, const AttnArgs& a, cudaStream_t s);
int read_and_clear_attn_backward_error(cudaStream_t s, unsigned* value);

// Lets a kernel use more shared memory than the default 48 KB; asks the runtime once for each
// (kernel, device, larger size).
int allow_smem(const void* kernel, size_t bytes);

// Whether a launch's block count fits the grid's first axis.
inline bool grid_ok(long long blocks) { return blocks > 0 && blocks <= 0x7fffffffLL; }

}  // namespace ops
}  // namespace fconv
