// Internal launch interface of the kernels around the layer (norm.cu, w4.cu),
// called by their C entry points (api_block.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "block.cuh"

namespace moe {

struct AddNormParams {
  int64_t rows, rows_pad;   // rows_pad: rows up to a whole 128-row tile (8-bit output)
  int32_t d;
  int32_t group;            // threads of a row group (set by the launcher)
  float inv_d;
  bool w_f32, x_f16;
  const void* x;
  int64_t ld_x;
  const void* residual;
  int64_t ld_residual;
  const void* weight;
  void* h;
  int64_t ld_h;
  void* y;
  int64_t ld_y;
  float* rstd;
  uint8_t* y_q;
  uint8_t* y_scales;
  void* y_dq;
  DropRng rng;
  float eps;
};

struct AddNormBwdParams {
  int64_t rows;
  int32_t d;
  int32_t group;
  float inv_d;
  bool w_f32, x_f16;
  const void* dy;
  int64_t ld_dy;
  const void* h;
  int64_t ld_h;
  const void* dres;
  int64_t ld_dres;
  const float* rstd;
  const void* weight;
  void* dh;
  int64_t ld_dh;
  void* dx;
  int64_t ld_dx;
  float* partial;
  DropRng rng;
};

struct DropoutParams {
  int64_t rows;
  int32_t cols;
  int32_t group;   // lanes of a row (set by the launcher)
  const void* x;
  int64_t ld_x;
  void* y;
  int64_t ld_y;
  DropRng rng;
};

constexpr int kNormMaxWidth = 32768;     // 1024 threads, four groups of eight columns each
constexpr int kNormPartialRows = 1024;   // most blocks of the backward: rows of partial weight gradients

// vec: neighbouring columns that an access takes, 8, 2 or 1 (block.cuh, V)
cudaError_t launch_add_norm(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s);
cudaError_t launch_add_norm_bwd(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw,
                                cudaStream_t s);
cudaError_t launch_dropout(const DropoutParams& p, int dtype, int vec, cudaStream_t s);

// ---------------------------------------------------------------- 4-bit weights
constexpr int kW4MaxColumns = 1 << 18;   // K, d and f: stages of a block's share count in 32 bits

struct ExpertsW4Params {
  int32_t T, d, E, k, f, group;
  const void* x;
  int64_t ld_x;
  const int32_t* topk_idx;
  const float* gates;
  const uint8_t *gate_q, *up_q, *down_q;
  const void *gate_s, *up_s, *down_s;
  void* out;
  int64_t ld_out;
  void* act;       // workspace: gated activations of each route: fp32 [T*k, f], or two bf16 parts [2][T*k, f]
  float* y;        // workspace (more than one token): product of each route [T*k, d]
  int32_t* err;
};

cudaError_t launch_quantize_w4(int64_t rows, int K, int group, int dtype, const void* src,
                               uint8_t* q, void* scales, cudaStream_t s);
cudaError_t launch_dequantize_w4(int64_t rows, int K, int group, int dtype, const uint8_t* q,
                                 const void* scales, float* out, cudaStream_t s);
cudaError_t launch_matvec_w4(int M, int N, int K, int group, int dtype, const void* x, int64_t ld_x,
                             const uint8_t* q, const void* scales, void* y, int64_t ld_y,
                             cudaStream_t s);
cudaError_t launch_experts_w4_bf16(const ExpertsW4Params& p, cudaStream_t s);
cudaError_t launch_experts_w4_f16(const ExpertsW4Params& p, cudaStream_t s);

}  // namespace moe
