// Residual addition with layer norm, forward: norm_fwd.cuh.
#include "norm_fwd.cuh"

namespace moe {

cudaError_t launch_add_layer_norm(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s) {
  return drawn_at(p) ? launch_add_layer_norm_at(p, dtype, res_dtype, vec, s)
                     : fwd_launch<true, false>(p, dtype, res_dtype, vec, s);
}

}  // namespace moe
