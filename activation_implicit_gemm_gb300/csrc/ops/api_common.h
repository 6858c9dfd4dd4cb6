// Checks and plan making that the C entry points of the token-side operators share.
#pragma once

#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <new>
#include <utility>

#include "ops_internal.h"

namespace fconv {
namespace ops {
namespace {

inline int device_sms(int device) {
  int dev = device, sms = 0;
  if ((dev < 0 && cudaGetDevice(&dev) != cudaSuccess) ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0) {
    cudaGetLastError();
    return 152;  // no device here: plan for a GB300
  }
  return sms;
}

inline bool known_type(int t) { return t == FCONV_F32 || t == FCONV_F16 || t == FCONV_BF16; }
inline bool small(int64_t v, int64_t least) { return v >= least && v <= INT_MAX / 2; }
inline bool misaligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
inline size_t type_size(int t) { return t == FCONV_F32 ? 4 : 2; }

// Strides of an input: none negative. Of an output also: no two elements at one address, for
// which each axis must step past all that the axes of smaller steps span.
inline bool strides_ok(const int64_t st[3], const int64_t ext[3], int64_t last, bool output) {
  int64_t s[4] = {1, st[0], st[1], st[2]}, e[4] = {last, ext[0], ext[1], ext[2]};
  for (int i = 1; i < 4; ++i)
    if (s[i] < 0) return false;
  if (!output) return true;
  for (int i = 1; i < 4; ++i)
    for (int j = i; j > 1 && s[j] < s[j - 1]; --j) {
      std::swap(s[j], s[j - 1]);
      std::swap(e[j], e[j - 1]);
    }
  int64_t span = 0;
  for (int i = 0; i < 4; ++i) {
    if (e[i] <= 1) continue;
    if (s[i] <= span) return false;
    span += s[i] * (e[i] - 1);
  }
  return true;
}

inline bool same_strides(const int64_t a[3], const int64_t b[3]) {
  return a[0] == b[0] && a[1] == b[1] && a[2] == b[2];
}

inline fconv_status done(int err) {
  if (err == 0) return FCONV_OK;
  cudaGetLastError();  // reported here, not by the caller's next check
  return FCONV_E_CUDA;
}

template <typename Plan, typename Desc>
fconv_status new_plan(const Desc* desc, int device, fconv_status (*check)(const Desc&),
                      Plan** out) {
  if (!out) return FCONV_E_NULL;
  *out = nullptr;
  if (!desc) return FCONV_E_NULL;
  const fconv_status st = check(*desc);
  if (st != FCONV_OK) return st;
  Plan* p = new (std::nothrow) Plan();
  if (!p) return FCONV_E_NOMEM;
  p->d = *desc;
  p->sms = device_sms(device);
  *out = p;
  return FCONV_OK;
}

}  // namespace
}  // namespace ops
}  // namespace fconv
