// Backward of the residual addition with layer norm: norm_bwd.cuh.
#include "norm_bwd.cuh"

namespace moe {

cudaError_t launch_add_layer_norm_bwd(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw, float* db,
                                      cudaStream_t s) {
  return drawn_at(p) ? launch_add_layer_norm_bwd_at(p, dtype, res_dtype, vec, dw, db, s)
                     : bwd_launch<true, false>(p, dtype, res_dtype, vec, dw, db, s);
}

}  // namespace moe
