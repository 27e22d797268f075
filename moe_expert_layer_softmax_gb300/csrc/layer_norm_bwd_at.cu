// Backward of the residual addition with layer norm, dropout's offset with a part on the
// device: norm_bwd.cuh.
#include "norm_bwd.cuh"

namespace moe {

cudaError_t launch_add_layer_norm_bwd_at(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw, float* db,
                                         cudaStream_t s) {
  return bwd_launch<true, true>(p, dtype, res_dtype, vec, dw, db, s);
}

}  // namespace moe
