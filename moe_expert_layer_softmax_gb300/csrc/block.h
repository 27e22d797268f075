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
  const void* bias;         // layer norm, nullable
  void* h;
  int64_t ld_h;
  void* y;
  int64_t ld_y;
  float* mean;              // layer norm, nullable
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
  const float* mean;   // layer norm
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
cudaError_t launch_add_layer_norm(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s);
cudaError_t launch_add_layer_norm_bwd(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw, float* db,
                                      cudaStream_t s);
// The same with dropout whose offset has a part on the device.
cudaError_t launch_add_norm_at(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s);
cudaError_t launch_add_norm_bwd_at(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw, cudaStream_t s);
cudaError_t launch_add_layer_norm_at(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s);
cudaError_t launch_add_layer_norm_bwd_at(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw, float* db,
                                         cudaStream_t s);
cudaError_t launch_dropout(const DropoutParams& p, int dtype, int vec, cudaStream_t s);

// ---------------------------------------------------------------- AdamW
constexpr int kStateBlock = 128;    // values that share a scale of the 8-bit states
constexpr int kAdamwFew = 16, kAdamwMost = 224;   // tensors of a launch's table, short and long

struct AdamwTensor {
  void* param;
  const void* grad;
  float* master;
  void *m, *v;
  float *m_scale, *v_scale;
  int64_t numel;
  uint32_t first;   // block that it begins with
  uint32_t vec;     // vector accesses: pointers on 16-byte boundaries, codes on 8 (scales: any)
};

struct AdamwScalars {
  float beta1, one_beta1, beta2, one_beta2, eps;
  float root_scale, decay, rate;   // 1 / sqrt(1 - b2^t), 1 - lr wd, lr / (1 - b1^t)
};

struct AdamwParams {
  int n, first_tensor;   // tensors of this launch, and those of the call before them
  int turns;             // chunks that a block takes one after the other
  bool narrow;           // eps and 1 / sqrt(1 - b2^t) where the divisor stays within 2^-60 .. 2^60
  AdamwScalars s;
  const float* grad_scale;
  const float* lr_dev;
  const int64_t* step_dev;
  const uint64_t* offset_dev;   // nullable: added to the offset o1 : o0
  double lr, beta1, beta2, weight_decay, c1;   // c1: 1 - b1^t of the host's t
  uint32_t k0, k1, o0, o1;
};

int64_t adamw_blocks(int64_t numel, int turns);   // blocks of a tensor, each of so many chunks
int adamw_turns(int64_t chunks, bool small);               // of a block of a launch of so many chunks
cudaError_t launch_adamw(const AdamwTensor* t, const AdamwParams& p, int param_dtype, int grad_dtype, bool master,
                         bool small, int64_t blocks, cudaStream_t s);

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
