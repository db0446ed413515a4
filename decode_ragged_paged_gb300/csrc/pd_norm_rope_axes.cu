// pd_norm_rope_axes.cu -- the norm and rotation's kernels for positions with several axes.
#include "pd_norm_rope.cuh"

namespace pd {

cudaError_t launch_norm_rope_axes(const NormRopeParams& p, int32_t elem_size, int32_t vec, unsigned grid,
                                  cudaStream_t stream) {
  return launch_norm_rope_form<true>(p, elem_size, vec, grid, stream);
}

}  // namespace pd
