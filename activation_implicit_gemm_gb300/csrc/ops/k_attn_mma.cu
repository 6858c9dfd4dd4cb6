// The split-f32 attention kernels (attn_mma.cuh) for head lengths up to 128, and the dispatch of
// the route.
#include "attn_mma.cuh"

namespace fconv {
namespace ops {
namespace {

// NT: 8-column tiles of head_dim in registers, fitted for f32 rows of whole 16-byte units, the
// most for the rest.
template <typename T, bool BWD>
int by_size(const fconv_attn_desc& d, const Geom& g, const AttnArgs& a, cudaStream_t s) {
#define FCONV_RUN(NT, VEC) \
  return BWD ? backward_t<T, NT, VEC>(g, a, s) : forward_t<T, NT, VEC>(g, a, s)
  if constexpr (sizeof(T) == 4) {
    if (whole_rows(d, a)) {
      if (g.Dp <= 64) FCONV_RUN(8, true);
      if (g.Dp <= 96) FCONV_RUN(12, true);
      FCONV_RUN(16, true);
    }
  }
  FCONV_RUN(16, false);
#undef FCONV_RUN
}

}  // namespace

size_t attn_simple_backward_workspace(const fconv_attn_desc& d) {
  return (size_t)d.batch * (size_t)d.heads_q * (size_t)d.len_q * sizeof(float);
}

int launch_attn_simple_forward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s) {
  const Geom g = geom_of(d, a);
  if (g.B * g.Lq == 0) return 0;
  if (g.D > 128) return launch_attn_wide_forward(d, a, s);
#define FCONV_M(T) return by_size<T, false>(d, g, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

int launch_attn_simple_backward(const fconv_attn_desc& d, const AttnArgs& a, cudaStream_t s) {
  const Geom g = geom_of(d, a);
  if (g.D > 128) return launch_attn_wide_backward(d, a, s);
#define FCONV_M(T) return by_size<T, true>(d, g, a, s)
  FCONV_OPS_TYPE(d.dtype, FCONV_M)
#undef FCONV_M
}

}  // namespace ops
}  // namespace fconv
