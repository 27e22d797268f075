// Internal launch interface of the layer for a few tokens (few.cu), called by its C
// entry point (api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

constexpr int kFewMaxRoutes = MOE_FEW_MAX_TOKENS * 32;   // top_k <= 32

struct FewTensors {
  const void *x, *w_router, *w_gate, *w_up, *w_down;
};

// The routes by experts, from the up kernel to the down kernel (in the workspace).
struct FewLists {
  int32_t n_act;
  uint16_t base[258];
  uint8_t act[256];
  uint8_t tok[kFewMaxRoutes];
  float gate[kFewMaxRoutes];
};

struct FewParams {
  int T, d, E, k, f;
  const float* bias;     // [T, E] or NULL
  float* logits;         // [T, E] or NULL (written with a router)
  int32_t* topk_idx;     // [T, k]: written with a router, else read
  float* gates;
  void* act;             // bf16 [T k, 2, f]: a rounded, and the rest
  void* out;
  int32_t* err;
  FewLists* lists;
  // set by the launcher
  bool router;
  int t_pad, router_bytes, router_stages, part_at;
};

cudaError_t launch_few(const FewParams& p, const FewTensors& w, cudaStream_t s);

}  // namespace moe
