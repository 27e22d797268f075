// The SwiGLU experts on 4-bit weights for fp16 activations and scales: w4_experts.cuh.
#include "w4_experts.cuh"

namespace moe {

cudaError_t launch_experts_w4_f16(const ExpertsW4Params& p, cudaStream_t s) {
  return experts_group<__half>(p.group, p, s);
}

}  // namespace moe
