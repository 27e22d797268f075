// C entry points of the operators around the layer: residual addition with the
// root-mean-square norm, dropout, 4-bit weights.  Argument validation and
// launches only; declarations and documentation: include/moe.h.
#include <cmath>

#include "moe.h"
#include "block.h"
#include "kernels.h"

namespace moe {

namespace {

bool is_dtype(int t) { return t == MOE_DT_BF16 || t == MOE_DT_F16 || t == MOE_DT_F32; }
int size_of(int t) { return t == MOE_DT_F32 ? 4 : 2; }

bool on_boundary(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

bool ready() {
  const DeviceInfo* i = device_info();
  return i != nullptr && i->ready;
}

// A matrix operand: present, on an element boundary, rows that do not overlap.
int check_matrix(const void* p, int64_t ld, int64_t cols, int dtype) {
  if (p == nullptr || ld < cols) return MOE_ERR_INVALID;
  return on_boundary(p, size_of(dtype)) ? MOE_OK : MOE_ERR_ALIGN;
}

// The largest access (columns: 8, 2 or 1, at most `most`) that every row of a
// matrix takes: eight columns from a 16-byte boundary, or a pair from its own.
int row_access(const void* p, int64_t ld, int64_t rows, int dtype, int most = 8) {
  if (p == nullptr) return most;
  const int64_t size = size_of(dtype), stride = rows == 1 ? 0 : ld * size;
  if (most == 8 && (!on_boundary(p, 16) || stride % 16 != 0)) most = 2;
  if (most == 2 && (!on_boundary(p, 2 * size) || stride % (2 * size) != 0)) most = 1;
  return most;
}
int width_access(int32_t d) { return d % 8 == 0 ? 8 : d % 2 == 0 ? 2 : 1; }

// p in [0, 1]; the keep probability is a multiple of 2^-16.
int make_rng(float p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev, DropRng* g) {
  if (!(p >= 0.0f && p <= 1.0f)) return MOE_ERR_INVALID;
  g->k0 = (uint32_t)seed;
  g->k1 = (uint32_t)(seed >> 32);
  g->o0 = (uint32_t)offset;
  g->o1 = (uint32_t)(offset >> 32);
  g->offset_dev = offset_dev;
  if (!on_boundary(offset_dev, 8)) return MOE_ERR_ALIGN;
  g->threshold = (uint32_t)std::floor((double)p * 65536.0 + 0.5);
  g->scale = g->threshold < 65536u ? (float)(65536.0 / (65536.0 - g->threshold)) : 0.0f;
  return MOE_OK;
}

int check_norm_types(int64_t rows, int32_t d, int dtype, int res_dtype, int w_dtype) {
  if (rows < 0 || d < 1 || !is_dtype(dtype) || !is_dtype(res_dtype) || !is_dtype(w_dtype))
    return MOE_ERR_INVALID;
  if (res_dtype != dtype && res_dtype != MOE_DT_F32) return MOE_ERR_INVALID;
  if (w_dtype != dtype && w_dtype != MOE_DT_F32) return MOE_ERR_INVALID;
  if (d > kNormMaxWidth || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_w4(int64_t rows, int32_t K, int32_t group, int dtype) {
  if (rows < 0 || K < 1 || (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16)) return MOE_ERR_INVALID;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
  if (K % group != 0 || K > kW4MaxColumns) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

#define MOE_TRY(expr)              \
  do {                             \
    int _rc = (expr);              \
    if (_rc != MOE_OK) return _rc; \
  } while (0)

// present and on a 16-byte boundary
#define MOE_BUFFER(p)                                 \
  do {                                                \
    if ((p) == nullptr) return MOE_ERR_INVALID;       \
    if (!on_boundary((p), 16)) return MOE_ERR_ALIGN;  \
  } while (0)

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

int check_experts(int32_t T, int32_t d, int32_t E, int32_t k, int32_t f, int32_t group) {
  if (T < 0 || d < 1 || E < 1 || k < 1 || f < 1) return MOE_ERR_INVALID;
  if (d % 128 != 0 || f % 128 != 0 || E > 256 || k > 32) return MOE_ERR_UNSUPPORTED;
  if (d > kW4MaxColumns || f > kW4MaxColumns) return MOE_ERR_UNSUPPORTED;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)T * k > MOE_W4_MAX_ROUTES) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Checks and parameters of either norm's forward; without rows p.rows
// stays zero and nothing is launched.  The layer norm's bias and mean may be NULL.
template <typename Args>
int add_norm_params(const Args* a, const uint64_t* offset_dev, const void* bias, float* mean, AddNormParams& p, int& vec) {
  MOE_TRY(check_norm_types(a->rows, a->d, a->dtype, a->res_dtype, a->w_dtype));
  MOE_TRY(make_rng(a->p, a->seed, a->offset, offset_dev, &p.rng));
  if (!(a->eps >= 0.0f) || std::isinf(a->eps)) return MOE_ERR_INVALID;
  if (a->rows == 0) return MOE_OK;
  MOE_TRY(check_matrix(a->x, a->ld_x, a->d, a->dtype));
  if (a->residual) MOE_TRY(check_matrix(a->residual, a->ld_residual, a->d, a->res_dtype));
  if (a->weight == nullptr) return MOE_ERR_INVALID;
  if (!on_boundary(a->weight, size_of(a->w_dtype))) return MOE_ERR_ALIGN;
  if (a->h) {
    MOE_TRY(check_matrix(a->h, a->ld_h, a->d, a->res_dtype));
  } else if (a->residual || p.rng.threshold) {
    return MOE_ERR_INVALID;   // the stream that the norm and the backward read
  }
  if (a->rstd && !on_boundary(a->rstd, 4)) return MOE_ERR_ALIGN;
  if (mean && !on_boundary(mean, 4)) return MOE_ERR_ALIGN;
  if (bias && !on_boundary(bias, size_of(a->w_dtype))) return MOE_ERR_ALIGN;
  vec = row_access(a->x, a->ld_x, a->rows, a->dtype, width_access(a->d));
  vec = row_access(a->residual, a->ld_residual, a->rows, a->res_dtype, vec);
  vec = row_access(a->h, a->ld_h, a->rows, a->res_dtype, vec);
  vec = row_access(a->weight, 0, 1, a->w_dtype, vec);
  vec = row_access(bias, 0, 1, a->w_dtype, vec);
  p.rows_pad = a->rows;
  if (a->y_q) {
    // codes and scales for whole 128-row tiles, 128-column scale atoms
    if (a->dtype != MOE_DT_BF16 || a->d % 128 != 0) return MOE_ERR_UNSUPPORTED;
    if (a->y != nullptr || a->y_scales == nullptr) return MOE_ERR_INVALID;
    MOE_BUFFER(a->y_q);
    MOE_BUFFER(a->y_scales);
    if (a->y_dq) MOE_BUFFER(a->y_dq);
    if (vec != 8) return MOE_ERR_ALIGN;
    p.rows_pad = (a->rows + kTileM - 1) / kTileM * kTileM;
  } else {
    if (a->y_scales || a->y_dq) return MOE_ERR_INVALID;
    MOE_TRY(check_matrix(a->y, a->ld_y, a->d, a->dtype));
    vec = row_access(a->y, a->ld_y, a->rows, a->dtype, vec);
  }
  if (!ready()) return MOE_ERR_NOT_INIT;
  p.rows = a->rows; p.d = a->d; p.inv_d = 1.0f / (float)a->d;
  p.w_f32 = a->w_dtype == MOE_DT_F32; p.x_f16 = a->dtype == MOE_DT_F16;
  p.x = a->x; p.ld_x = a->ld_x;
  p.residual = a->residual; p.ld_residual = a->ld_residual;
  p.weight = a->weight;
  p.bias = bias;
  p.mean = mean;
  p.h = a->h; p.ld_h = a->ld_h;
  p.y = a->y; p.ld_y = a->ld_y;
  p.rstd = a->rstd;
  p.y_q = a->y_q; p.y_scales = a->y_scales; p.y_dq = a->y_dq;
  p.eps = a->eps;
  return MOE_OK;
}

// The same for the backward.
template <typename Args>
int add_norm_bwd_params(const Args* a, const float* mean, bool sums, void* ws, AddNormBwdParams& p, int& vec) {
  MOE_TRY(check_matrix(a->dy, a->ld_dy, a->d, a->dtype));
  MOE_TRY(check_matrix(a->h, a->ld_h, a->d, a->res_dtype));
  if (a->dres) MOE_TRY(check_matrix(a->dres, a->ld_dres, a->d, a->res_dtype));
  if (a->dh) MOE_TRY(check_matrix(a->dh, a->ld_dh, a->d, a->res_dtype));
  if (a->dx) MOE_TRY(check_matrix(a->dx, a->ld_dx, a->d, a->dtype));
  if (a->rstd == nullptr || a->weight == nullptr) return MOE_ERR_INVALID;
  if (!on_boundary(a->rstd, 4) || !on_boundary(a->weight, size_of(a->w_dtype))) return MOE_ERR_ALIGN;
  if (sums) MOE_BUFFER(ws);
  if (!ready()) return MOE_ERR_NOT_INIT;
  vec = row_access(a->dy, a->ld_dy, a->rows, a->dtype, width_access(a->d));
  vec = row_access(a->h, a->ld_h, a->rows, a->res_dtype, vec);
  vec = row_access(a->dres, a->ld_dres, a->rows, a->res_dtype, vec);
  vec = row_access(a->dh, a->ld_dh, a->rows, a->res_dtype, vec);
  vec = row_access(a->dx, a->ld_dx, a->rows, a->dtype, vec);
  vec = row_access(a->weight, 0, 1, a->w_dtype, vec);
  p.rows = a->rows; p.d = a->d; p.inv_d = 1.0f / (float)a->d;
  p.w_f32 = a->w_dtype == MOE_DT_F32; p.x_f16 = a->dtype == MOE_DT_F16;
  p.dy = a->dy; p.ld_dy = a->ld_dy;
  p.h = a->h; p.ld_h = a->ld_h;
  p.dres = a->dres; p.ld_dres = a->ld_dres;
  p.mean = mean; p.rstd = a->rstd; p.weight = a->weight;
  p.dh = a->dh; p.ld_dh = a->ld_dh;
  p.dx = a->dx; p.ld_dx = a->ld_dx;
  p.partial = sums ? static_cast<float*>(ws) : nullptr;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int moe_add_norm(const moe_add_norm_args_t* a, void* stream) { return moe_add_norm_at(a, nullptr, stream); }

int moe_add_norm_at(const moe_add_norm_args_t* a, const uint64_t* offset_dev, void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID;
  AddNormParams p = {};
  int vec = 0;
  MOE_TRY(add_norm_params(a, offset_dev, nullptr, nullptr, p, vec));
  if (p.rows == 0) return MOE_OK;
  return launch_add_norm(p, a->dtype, a->res_dtype, vec, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_add_layer_norm(const moe_add_layer_norm_args_t* a, void* stream) {
  return moe_add_layer_norm_at(a, nullptr, stream);
}

int moe_add_layer_norm_at(const moe_add_layer_norm_args_t* a, const uint64_t* offset_dev, void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID;
  AddNormParams p = {};
  int vec = 0;
  MOE_TRY(add_norm_params(a, offset_dev, a->bias, a->mean, p, vec));
  if (p.rows == 0) return MOE_OK;
  return launch_add_layer_norm(p, a->dtype, a->res_dtype, vec, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_add_norm_bwd_workspace_size(int64_t rows, int32_t d, size_t* ws_bytes) {
  if (rows < 0 || d < 1 || ws_bytes == nullptr) return MOE_ERR_INVALID;
  if (d > kNormMaxWidth || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  *ws_bytes = round256((size_t)(rows < kNormPartialRows ? rows : kNormPartialRows) * d * 4);
  return MOE_OK;
}

int moe_add_norm_bwd(const moe_add_norm_bwd_args_t* a, void* ws, void* stream) {
  return moe_add_norm_bwd_at(a, ws, nullptr, stream);
}

int moe_add_norm_bwd_at(const moe_add_norm_bwd_args_t* a, void* ws, const uint64_t* offset_dev, void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID;
  MOE_TRY(check_norm_types(a->rows, a->d, a->dtype, a->res_dtype, a->w_dtype));
  AddNormBwdParams p = {};
  MOE_TRY(make_rng(a->p, a->seed, a->offset, offset_dev, &p.rng));
  if (!a->dh && !a->dx && !a->dw) return MOE_ERR_INVALID;
  if (a->dw && !on_boundary(a->dw, 4)) return MOE_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) {   // an empty sum
    if (a->dw && cudaMemsetAsync(a->dw, 0, (size_t)a->d * 4, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  int vec = 0;
  MOE_TRY(add_norm_bwd_params(a, nullptr, a->dw != nullptr, ws, p, vec));
  return launch_add_norm_bwd(p, a->dtype, a->res_dtype, vec, a->dw, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_add_layer_norm_bwd_workspace_size(int64_t rows, int32_t d, size_t* ws_bytes) {
  if (rows < 0 || d < 1 || ws_bytes == nullptr) return MOE_ERR_INVALID;
  if (d > kNormMaxWidth || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  *ws_bytes = round256((size_t)(rows < kNormPartialRows ? rows : kNormPartialRows) * d * 8);
  return MOE_OK;
}

int moe_add_layer_norm_bwd(const moe_add_layer_norm_bwd_args_t* a, void* ws, void* stream) {
  return moe_add_layer_norm_bwd_at(a, ws, nullptr, stream);
}

int moe_add_layer_norm_bwd_at(const moe_add_layer_norm_bwd_args_t* a, void* ws, const uint64_t* offset_dev, void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID;
  MOE_TRY(check_norm_types(a->rows, a->d, a->dtype, a->res_dtype, a->w_dtype));
  AddNormBwdParams p = {};
  MOE_TRY(make_rng(a->p, a->seed, a->offset, offset_dev, &p.rng));
  if (!a->dh && !a->dx && !a->dw && !a->db) return MOE_ERR_INVALID;
  if ((a->dw && !on_boundary(a->dw, 4)) || (a->db && !on_boundary(a->db, 4))) return MOE_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) {   // empty sums
    for (float* sum : {a->dw, a->db})
      if (sum && cudaMemsetAsync(sum, 0, (size_t)a->d * 4, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (a->mean == nullptr) return MOE_ERR_INVALID;
  if (!on_boundary(a->mean, 4)) return MOE_ERR_ALIGN;
  int vec = 0;
  MOE_TRY(add_norm_bwd_params(a, a->mean, a->dw || a->db, ws, p, vec));
  return launch_add_layer_norm_bwd(p, a->dtype, a->res_dtype, vec, a->dw, a->db, st) == cudaSuccess ? MOE_OK
                                                                                                    : MOE_ERR_CUDA;
}

int moe_dropout(int64_t rows, int32_t cols, int32_t dtype, const void* x, int64_t ld_x, void* y,
                int64_t ld_y, float prob, uint64_t seed, uint64_t offset, void* stream) {
  return moe_dropout_at(rows, cols, dtype, x, ld_x, y, ld_y, prob, seed, offset, nullptr, stream);
}

int moe_dropout_at(int64_t rows, int32_t cols, int32_t dtype, const void* x, int64_t ld_x, void* y, int64_t ld_y,
                   float prob, uint64_t seed, uint64_t offset, const uint64_t* offset_dev, void* stream) {
  if (rows < 0 || cols < 1 || !is_dtype(dtype)) return MOE_ERR_INVALID;
  if (rows > INT32_MAX || cols > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  DropoutParams p = {};
  MOE_TRY(make_rng(prob, seed, offset, offset_dev, &p.rng));
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_matrix(x, ld_x, cols, dtype));
  MOE_TRY(check_matrix(y, ld_y, cols, dtype));
  if (!ready()) return MOE_ERR_NOT_INIT;
  p.rows = rows; p.cols = cols;
  p.x = x; p.ld_x = ld_x;
  p.y = y; p.ld_y = ld_y;
  const int vec = row_access(y, ld_y, rows, dtype, row_access(x, ld_x, rows, dtype, width_access(cols)));
  return launch_dropout(p, dtype, vec, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_adamw(const moe_adamw_args_t* a, void* stream) { return moe_adamw_at(a, nullptr, stream); }

int moe_adamw_at(const moe_adamw_args_t* a, const uint64_t* offset_dev, void* stream) {
  if (a == nullptr || a->n_tensors < 0) return MOE_ERR_INVALID;
  if (!is_dtype(a->param_dtype) || !is_dtype(a->grad_dtype)) return MOE_ERR_INVALID;
  if (a->grad_dtype != a->param_dtype && a->grad_dtype != MOE_DT_F32) return MOE_ERR_INVALID;
  if (a->state_bits != 32 && a->state_bits != 8) return MOE_ERR_INVALID;
  if (!(a->beta1 >= 0.0 && a->beta1 < 1.0) || !(a->beta2 >= 0.0 && a->beta2 < 1.0)) return MOE_ERR_INVALID;
  if (!(a->eps >= 0.0) || std::isinf(a->eps) || !(a->weight_decay >= 0.0) || std::isinf(a->weight_decay))
    return MOE_ERR_INVALID;
  if (!a->lr_dev && (!(a->lr >= 0.0) || std::isinf(a->lr))) return MOE_ERR_INVALID;
  if (!a->step_dev && a->step < 1) return MOE_ERR_INVALID;
  if (!on_boundary(a->grad_scale, 4) || !on_boundary(a->lr_dev, 4) || !on_boundary(a->step_dev, 8)) return MOE_ERR_ALIGN;
  if (!on_boundary(offset_dev, 8)) return MOE_ERR_ALIGN;
  if (a->n_tensors == 0) return MOE_OK;
  if (a->tensors == nullptr) return MOE_ERR_INVALID;
  if (a->n_tensors > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  const bool small = a->state_bits == 8;
  bool master = false;   // of the tensors that are not empty
  for (int i = 0; i < a->n_tensors && !master; ++i) master = a->tensors[i].numel > 0 && a->tensors[i].master != nullptr;
  const int ps = size_of(a->param_dtype), gs = size_of(a->grad_dtype);
  int64_t total = 0;
  for (int i = 0; i < a->n_tensors; ++i) {   // all of them before the first launch
    const moe_adamw_tensor_t& t = a->tensors[i];
    if (t.numel < 0) return MOE_ERR_INVALID;
    if (t.numel > (int64_t(1) << 34)) return MOE_ERR_UNSUPPORTED;
    if (t.numel == 0) continue;
    if ((t.master != nullptr) != master) return MOE_ERR_INVALID;
    if (!t.param || !t.grad || !t.m || !t.v || (small && (!t.m_scale || !t.v_scale))) return MOE_ERR_INVALID;
    if (!on_boundary(t.param, ps) || !on_boundary(t.grad, gs) || !on_boundary(t.master, 4)) return MOE_ERR_ALIGN;
    if (!small && (!on_boundary(t.m, 4) || !on_boundary(t.v, 4))) return MOE_ERR_ALIGN;
    if (small && (!on_boundary(t.m_scale, 4) || !on_boundary(t.v_scale, 4))) return MOE_ERR_ALIGN;
    total += adamw_blocks(t.numel, 1);
  }
  if (total == 0) return MOE_OK;
  // without a copy in 32 bits: fp32 itself, or bf16 with drawn rounding
  if (master ? a->param_dtype == MOE_DT_F32 : a->param_dtype == MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
  if (total > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (!ready()) return MOE_ERR_NOT_INIT;
  AdamwParams p = {};
  p.s.beta1 = (float)a->beta1; p.s.one_beta1 = (float)(1.0 - a->beta1);
  p.s.beta2 = (float)a->beta2; p.s.one_beta2 = (float)(1.0 - a->beta2);
  p.s.eps = (float)a->eps;
  // 1 / sqrt(1 - b2^t) is at most 1 / sqrt(1 - b2), whatever t
  p.narrow = a->eps >= 0x1p-60 && a->eps <= 1.0 && 1.0 - a->beta2 >= 0x1p-16;
  p.lr = a->lr; p.beta1 = a->beta1; p.beta2 = a->beta2; p.weight_decay = a->weight_decay;
  if (!a->step_dev) {
    p.c1 = 1.0 - std::pow(a->beta1, (double)a->step);
    p.s.root_scale = (float)(1.0 / std::sqrt(1.0 - std::pow(a->beta2, (double)a->step)));
  }
  if (!a->step_dev && !a->lr_dev) {
    p.s.decay = (float)(1.0 - a->lr * a->weight_decay);
    p.s.rate = (float)(a->lr / p.c1);
  }
  p.grad_scale = a->grad_scale; p.lr_dev = a->lr_dev; p.step_dev = a->step_dev; p.offset_dev = offset_dev;
  p.k0 = (uint32_t)a->seed; p.k1 = (uint32_t)(a->seed >> 32);
  p.o0 = (uint32_t)a->offset; p.o1 = (uint32_t)(a->offset >> 32);
  AdamwTensor list[kAdamwMost];
  for (int i = 0; i < a->n_tensors;) {
    int64_t blocks = 0, chunks = 0;
    p.first_tensor = i;
    for (int j = i; j < a->n_tensors && j < i + kAdamwMost; ++j) chunks += adamw_blocks(a->tensors[j].numel, 1);
    p.turns = adamw_turns(chunks, small);
    for (p.n = 0; p.n < kAdamwMost && i < a->n_tensors; ++i, ++p.n) {
      const moe_adamw_tensor_t& t = a->tensors[i];
      AdamwTensor& e = list[p.n];
      e.param = t.param; e.grad = t.grad; e.master = t.master; e.m = t.m; e.v = t.v;
      e.m_scale = t.m_scale; e.v_scale = t.v_scale;
      e.numel = t.numel;
      e.first = (uint32_t)blocks;
      e.vec = on_boundary(t.param, 16) && on_boundary(t.grad, 16) && on_boundary(t.master, 16) &&
              on_boundary(t.m, small ? 8 : 16) && on_boundary(t.v, small ? 8 : 16);
      blocks += adamw_blocks(t.numel, p.turns);
    }
    if (blocks == 0) continue;
    if (launch_adamw(list, p, a->param_dtype, a->grad_dtype, master, small, blocks, static_cast<cudaStream_t>(stream)) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

int moe_quantize_w4(int64_t rows, int32_t K, int32_t group, int32_t dtype, const void* src,
                    uint8_t* q, void* scales, void* stream) {
  MOE_TRY(check_w4(rows, K, group, dtype));
  if (rows == 0) return MOE_OK;
  MOE_BUFFER(src); MOE_BUFFER(q); MOE_BUFFER(scales);
  if (rows * (int64_t)(K / 8) > (int64_t)INT32_MAX * 256) return MOE_ERR_UNSUPPORTED;
  if (!ready()) return MOE_ERR_NOT_INIT;
  return launch_quantize_w4(rows, K, group, dtype, src, q, scales,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_dequantize_w4(int64_t rows, int32_t K, int32_t group, int32_t dtype, const uint8_t* q,
                      const void* scales, float* out, void* stream) {
  MOE_TRY(check_w4(rows, K, group, dtype));
  if (rows == 0) return MOE_OK;
  MOE_BUFFER(q); MOE_BUFFER(scales); MOE_BUFFER(out);
  if (rows * (int64_t)(K / 8) > (int64_t)INT32_MAX * 256) return MOE_ERR_UNSUPPORTED;
  if (!ready()) return MOE_ERR_NOT_INIT;
  return launch_dequantize_w4(rows, K, group, dtype, q, scales, out,
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_matvec_w4(int32_t M, int32_t N, int32_t K, int32_t group, int32_t dtype, const void* x,
                  int64_t ld_x, const uint8_t* q, const void* scales, void* y, int64_t ld_y,
                  void* stream) {
  if (M < 0 || N < 1) return MOE_ERR_INVALID;
  MOE_TRY(check_w4(N, K, group, dtype));
  if (N > 16 * 65535) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  MOE_BUFFER(x); MOE_BUFFER(q); MOE_BUFFER(scales);
  if (ld_x < K) return MOE_ERR_INVALID;
  if (M > 1 && ld_x % 8 != 0) return MOE_ERR_ALIGN;   // rows of x are read 16 bytes at a time
  MOE_TRY(check_matrix(y, ld_y, N, dtype));
  if (!ready()) return MOE_ERR_NOT_INIT;
  return launch_matvec_w4(M, N, K, group, dtype, x, ld_x, q, scales, y, ld_y,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_experts_w4_workspace_size(int32_t T, int32_t d, int32_t E, int32_t k, int32_t f,
                                  size_t* ws_bytes) {
  MOE_TRY(check_experts(T, d, E, k, f, 128));
  if (ws_bytes == nullptr) return MOE_ERR_INVALID;
  const size_t R = (size_t)T * k;
  *ws_bytes = 256 + round256(R * f * 4) + round256(R * d * 4);
  return MOE_OK;
}

int moe_experts_w4(const moe_experts_w4_args_t* a, void* ws, void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID;
  MOE_TRY(check_experts(a->T, a->d_model, a->n_experts, a->top_k, a->d_ff, a->group));
  if (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16) return MOE_ERR_INVALID;
  if (a->T == 0) return MOE_OK;
  MOE_BUFFER(a->x); MOE_BUFFER(a->topk_idx); MOE_BUFFER(a->gates);
  MOE_BUFFER(a->gate_q); MOE_BUFFER(a->up_q); MOE_BUFFER(a->down_q);
  MOE_BUFFER(a->gate_s); MOE_BUFFER(a->up_s); MOE_BUFFER(a->down_s);
  MOE_BUFFER(a->out); MOE_BUFFER(ws);
  if (!ready()) return MOE_ERR_NOT_INIT;
  const size_t R = (size_t)a->T * a->top_k;
  ExpertsW4Params p = {};
  p.T = a->T; p.d = a->d_model; p.E = a->n_experts; p.k = a->top_k; p.f = a->d_ff;
  p.group = a->group;
  p.x = a->x; p.ld_x = a->d_model;
  p.topk_idx = a->topk_idx; p.gates = a->gates;
  p.gate_q = a->gate_q; p.up_q = a->up_q; p.down_q = a->down_q;
  p.gate_s = a->gate_s; p.up_s = a->up_s; p.down_s = a->down_s;
  p.out = a->out; p.ld_out = a->d_model;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.err = reinterpret_cast<int32_t*>(w);
  p.act = w + 256;
  p.y = reinterpret_cast<float*>(w + 256 + round256(R * a->d_ff * 4));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == MOE_DT_BF16 ? launch_experts_w4_bf16(p, st) : launch_experts_w4_f16(p, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
