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
