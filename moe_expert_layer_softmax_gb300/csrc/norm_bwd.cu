// Backward of the residual addition with the root-mean-square norm: norm_bwd.cuh.
#include "norm_bwd.cuh"

namespace moe {

cudaError_t launch_add_norm_bwd(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw,
                                cudaStream_t s) {
  return drawn_at(p) ? launch_add_norm_bwd_at(p, dtype, res_dtype, vec, dw, s)
                     : bwd_launch<false, false>(p, dtype, res_dtype, vec, dw, nullptr, s);
}

}  // namespace moe
