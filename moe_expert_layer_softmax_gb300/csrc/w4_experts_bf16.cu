// The SwiGLU experts on 4-bit weights for bf16 activations and scales: w4_experts.cuh.
#include "w4_experts.cuh"

namespace moe {

cudaError_t launch_experts_w4_bf16(const ExpertsW4Params& p, cudaStream_t s) {
  return experts_group<__nv_bfloat16>(p.group, p, s);
}

}  // namespace moe
