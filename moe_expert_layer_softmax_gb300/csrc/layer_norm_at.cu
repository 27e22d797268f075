// Residual addition with layer norm, forward, dropout's offset with a part on the
// device: norm_fwd.cuh.
#include "norm_fwd.cuh"

namespace moe {

cudaError_t launch_add_layer_norm_at(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s) {
  return fwd_launch<true, true>(p, dtype, res_dtype, vec, s);
}

}  // namespace moe
