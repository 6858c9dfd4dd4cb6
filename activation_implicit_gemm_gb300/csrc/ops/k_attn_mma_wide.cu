// The split-f32 attention kernels (attn_mma.cuh) for head lengths from 129 to 256: one block an
// SM, and in the gradient kernels shorter tiles of what is walked.
#include "attn_mma.cuh"

namespace fconv {
namespace ops {
namespace {

template <typename T, bool BWD>
int by_type(const fconv_attn_desc& d, const Geom& g, const AttnArgs& a, cudaStream_t s) {
  if constexpr (sizeof(T) == 4) {
    if (whole_rows(d, a))
      return BWD ? backward_t<T, 32, true>(g, a, s) : forward_t<T, 32, true>(g, a, s);
  }
  return BWD ? backward_t<T, 32, false>(g, a, s) : forward_t<T, 32, false>(g, a, s);
}

}  // namespace

int launch_attn_wide_forward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s) {
  const Geom g = geom_of(d, a);
#define FCONV_M(T) return by_type<T, false>(d, g, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

int launch_attn_wide_backward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s) {
  const Geom g = geom_of(d, a);
#define FCONV_M(T) return by_type<T, true>(d, g, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
