// Backward of the residual addition with the root-mean-square norm, dropout's offset with a part on the
// device: norm_bwd.cuh.
#include "norm_bwd.cuh"

namespace moe {

cudaError_t launch_add_norm_bwd_at(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw, cudaStream_t s) {
  return bwd_launch<false, true>(p, dtype, res_dtype, vec, dw, nullptr, s);
}

}  // namespace moe
