// Residual addition with the root-mean-square norm, its backward, and dropout
// (sm_103a).
//
//   u = dropout(x)                      (u = x without dropout)
//   h = residual + u, rounded to the stream's type
//   r = (mean(h^2) + eps)^(-1/2),  y = h r w
// The norm is that of the rounded h: it is what the backward gets, so forward
// and backward see the same values.  y leaves in the activations' type, or as
// E4M3 codes with one E8M0 scale per 32 columns (rounded once, from the 32-bit
// y), optionally with the values the codes stand for.  With g = w dy:
//   dh = dres + r (g - h r^2 mean(g h)),  dx = dropout'(dh),  dw = sum dy h r.
//
// Every kernel here is bound by HBM: one read and one write of each matrix.  A
// row stays in registers between the pass that sums it and the pass that
// writes it.  Sums are taken in a fixed order (no atomics).
#include "block.cuh"
#include "block.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kNormThreads = 256;      // threads of a block whose row group is smaller
constexpr int kNormMaxThreads = 1024;

MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum over the G consecutive threads of a row group (G a power of two >= 32),
// the same value in every thread.  `red` has one float per warp; every thread
// of the block calls this.
MOE_DEV float group_sum(float v, int G, float* red) {
  v = warp_sum(v);
  if (G == 32) return v;
  __syncthreads();   // the previous use of red has been read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int w0 = (threadIdx.x / G) * (G >> 5);
  float s = 0.0f;
  for (int i = 0; i < (G >> 5); ++i) s += red[w0 + i];
  return s;
}

template <bool VEC>
MOE_DEV void load_weight8(const void* w, bool w_f32, bool w_f16, int c, int d, float* f) {
  if (w_f32) {
    widen8(load8<float, VEC>(static_cast<const float*>(w), c, d), f);
  } else if (w_f16) {
    widen8(load8<__half, VEC>(static_cast<const __half*>(w), c, d), f);
  } else {
    widen8(load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w), c, d), f);
  }
}

// One row group of G threads per row; each thread holds NV groups of eight
// columns.  MX: codes, scales and (dq) their values instead of y; rows at or
// past `rows` are the padding of the last 128-row tile.
template <typename TX, typename TR, bool MX, bool VEC, int NV>
__global__ void __launch_bounds__(kNormMaxThreads) add_norm_kernel(AddNormParams p) {
  pdl_begin();
  __shared__ float red[kNormMaxThreads / 32];
  const int G = p.group;
  const int lane = threadIdx.x & (G - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
  const int d = p.d;
  const bool live = row < p.rows;
  float h[NV][8];
  float ss = 0.0f;
  if (live) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.ld_x;
    const TR* res = p.residual ? static_cast<const TR*>(p.residual) + row * p.ld_residual : nullptr;
    Raw8<TX> xr[NV];
    Raw8<TR> rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * 8;
      if (c < d) {
        xr[i] = load8<TX, VEC>(x, c, d);
        if (res) rr[i] = load8<TR, VEC>(res, c, d);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * 8;
      if (c < d) {
        widen8(xr[i], h[i]);
        if (p.rng.threshold) drop8(h[i], c, (uint32_t)row, p.rng);
        if (res) {
          float f[8];
          widen8(rr[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += f[j];
        }
        if (p.h) {
          const Raw8<TR> hr = narrow8<TR>(h[i]);
          store8<TR, VEC>(static_cast<TR*>(p.h) + row * p.ld_h, c, d, hr);
          widen8(hr, h[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
      }
    }
  }
  ss = group_sum(ss, G, red);
  const float rstd = __frsqrt_rn(ss / (float)d + p.eps);
  if (live && lane == 0 && p.rstd) p.rstd[row] = rstd;
  if (!MX) {
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * 8;
      if (c < d) {
        float w[8];
        load_weight8<VEC>(p.weight, p.w_f32, sizeof(TX) == 2 && p.x_f16, c, d, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = (h[i][j] * w[j]) * rstd;
        store8<TX, VEC>(static_cast<TX*>(p.y) + row * p.ld_y, c, d, narrow8<TX>(h[i]));
      }
    }
  } else {
    // d is a multiple of 128: the four lanes of a 32-column block are all live
    // or all past the row's end
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * 8;
      float amax = 0.0f;
      if (c < d && live) {
        float w[8];
        load_weight8<VEC>(p.weight, p.w_f32, false, c, d, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[i][j] = (h[i][j] * w[j]) * rstd;
          amax = fmaxf(amax, fabsf(h[i][j]));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if (c < d && row < p.rows_pad) {
        const int s = mx_scale_exp(amax);
        uint2 q = make_uint2(0, 0);
        if (live) {
          const float inv = exp2i(-s);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = h[i][j] * inv;
          q = e4m3x8(v);
        }
        *reinterpret_cast<uint2*>(p.y_q + row * d + c) = q;
        if ((lane & 3) == 0) p.y_scales[sf_offset(row, c >> 5, d >> 5)] = (uint8_t)(s + 127);
        if (p.y_dq) {
          const float up = exp2i(s);
          float v[8];
          e4m3x2_to_f32(q.x, v[0], v[1]);
          e4m3x2_to_f32(q.x >> 16, v[2], v[3]);
          e4m3x2_to_f32(q.y, v[4], v[5]);
          e4m3x2_to_f32(q.y >> 16, v[6], v[7]);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= up;
          store8<__nv_bfloat16, true>(static_cast<__nv_bfloat16*>(p.y_dq) + row * d, c, d,
                                      narrow8<__nv_bfloat16>(v));
        }
      }
    }
  }
}

// Backward: a fixed grid of blocks takes the rows in turn and keeps the weight
// gradient of its rows in registers; the partial sums of the row groups go to
// `partial` [gridDim.x * groups per block, d].
template <typename TX, typename TR, bool VEC, int NV>
__global__ void __launch_bounds__(kNormMaxThreads) add_norm_bwd_kernel(AddNormBwdParams p) {
  pdl_begin();
  __shared__ float red[kNormMaxThreads / 32];
  const int G = p.group;
  const int lane = threadIdx.x & (G - 1);
  const int per_block = blockDim.x / G;
  const int d = p.d;
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  for (int64_t row0 = (int64_t)blockIdx.x * per_block; row0 < p.rows;
       row0 += (int64_t)gridDim.x * per_block) {
    const int64_t row = row0 + threadIdx.x / G;
    const bool live = row < p.rows;
    float r = 0.0f, dot = 0.0f;
    Raw8<TX> dyr[NV];
    Raw8<TR> hr[NV], dr[NV];
    if (live) {
      const TX* dy = static_cast<const TX*>(p.dy) + row * p.ld_dy;
      const TR* h = static_cast<const TR*>(p.h) + row * p.ld_h;
      const TR* dres = p.dres ? static_cast<const TR*>(p.dres) + row * p.ld_dres : nullptr;
      r = p.rstd[row];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * G) * 8;
        if (c < d) {
          dyr[i] = load8<TX, VEC>(dy, c, d);
          hr[i] = load8<TR, VEC>(h, c, d);
          if (dres) dr[i] = load8<TR, VEC>(dres, c, d);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * G) * 8;
        if (c < d) {
          float w[8], a[8], b[8];
          load_weight8<VEC>(p.weight, p.w_f32, sizeof(TX) == 2 && p.x_f16, c, d, w);
          widen8(dyr[i], a);
          widen8(hr[i], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float ah = a[j] * b[j];
            dw[i][j] = fmaf(ah, r, dw[i][j]);
            dot = fmaf(ah, w[j], dot);
          }
        }
      }
    }
    dot = group_sum(dot, G, red);
    if (live && (p.dh || p.dx)) {
      const float k = r * r * (dot / (float)d);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * G) * 8;
        if (c < d) {
          float w[8], a[8], b[8];
          load_weight8<VEC>(p.weight, p.w_f32, sizeof(TX) == 2 && p.x_f16, c, d, w);
          widen8(dyr[i], a);
          widen8(hr[i], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] = r * (a[j] * w[j] - b[j] * k);
          if (p.dres) {
            widen8(dr[i], b);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] += b[j];
          }
          if (p.dh) store8<TR, VEC>(static_cast<TR*>(p.dh) + row * p.ld_dh, c, d, narrow8<TR>(a));
          if (p.dx) {
            if (p.rng.threshold) drop8(a, c, (uint32_t)row, p.rng);
            store8<TX, VEC>(static_cast<TX*>(p.dx) + row * p.ld_dx, c, d, narrow8<TX>(a));
          }
        }
      }
    }
  }
  if (p.partial) {
    float* out = p.partial + ((int64_t)blockIdx.x * per_block + threadIdx.x / G) * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < d) out[c + j] = dw[i][j];
    }
  }
}

// dw[c] = sum of the partial rows, 32 columns a block: 8 warps take every
// eighth row, their sums are added in warp order.
__global__ void __launch_bounds__(256) add_norm_dw_kernel(const float* __restrict__ partial,
                                                          int n_partial, int d,
                                                          float* __restrict__ dw) {
  pdl_begin();
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.0f;
  if (c < d)
    for (int i = warp; i < n_partial; i += 8) acc += partial[(int64_t)i * d + c];
  s[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < d) {
    float sum = 0.0f;
    for (int i = 0; i < 8; ++i) sum += s[i][lane];
    dw[c] = sum;
  }
}

// y = dropout(x): blocks of 32 x 8 threads, a thread takes eight columns of a row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(DropoutParams p) {
  pdl_begin();
  const int64_t stride_r = (int64_t)gridDim.y * 8;
  for (int64_t row = (int64_t)blockIdx.y * 8 + threadIdx.y; row < p.rows; row += stride_r) {
    const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
    T* y = static_cast<T*>(p.y) + row * p.ld_y;
    for (int64_t c = ((int64_t)blockIdx.x * 32 + threadIdx.x) * 8; c < p.cols;
         c += (int64_t)gridDim.x * 256) {
      float f[8];
      widen8(load8<T, VEC>(x, (int)c, p.cols), f);
      if (p.rng.threshold) drop8(f, (int)c, (uint32_t)row, p.rng);
      store8<T, VEC>(y, (int)c, p.cols, narrow8<T>(f));
    }
  }
}

// Threads of a row group and groups of eight columns each holds.  Two groups a
// thread where the row allows it; a power of two of at least a warp.
void row_split(int d, int* group, int* nv) {
  const int g8 = (d + 7) / 8;
  int G = 32;
  while (G < kNormMaxThreads && G * 2 < g8) G *= 2;
  int n = 1;
  while (n * G < g8) n *= 2;
  *group = G;
  *nv = n;
}

template <typename TX, typename TR, bool MX, bool VEC>
cudaError_t fwd_nv(const AddNormParams& p, int nv, cudaStream_t s) {
  const int threads = p.group < kNormThreads ? kNormThreads : p.group;
  const int64_t per = threads / p.group;
  const dim3 grid((unsigned)(((MX ? p.rows_pad : p.rows) + per - 1) / per));
  switch (nv) {
    case 1: return launch_pdl(add_norm_kernel<TX, TR, MX, VEC, 1>, grid, dim3(threads), 0, s, p);
    case 2: return launch_pdl(add_norm_kernel<TX, TR, MX, VEC, 2>, grid, dim3(threads), 0, s, p);
    default: return launch_pdl(add_norm_kernel<TX, TR, MX, VEC, 4>, grid, dim3(threads), 0, s, p);
  }
}

template <typename TX, typename TR>
cudaError_t fwd_vec(const AddNormParams& p, bool vec, int nv, cudaStream_t s) {
  return vec ? fwd_nv<TX, TR, false, true>(p, nv, s) : fwd_nv<TX, TR, false, false>(p, nv, s);
}

template <typename TX, typename TR, bool VEC>
cudaError_t bwd_nv(const AddNormBwdParams& p, int blocks, int threads, int nv, cudaStream_t s) {
  switch (nv) {
    case 1: return launch_pdl(add_norm_bwd_kernel<TX, TR, VEC, 1>, dim3(blocks), dim3(threads), 0, s, p);
    case 2: return launch_pdl(add_norm_bwd_kernel<TX, TR, VEC, 2>, dim3(blocks), dim3(threads), 0, s, p);
    default: return launch_pdl(add_norm_bwd_kernel<TX, TR, VEC, 4>, dim3(blocks), dim3(threads), 0, s, p);
  }
}

template <typename TX, typename TR>
cudaError_t bwd_vec(const AddNormBwdParams& p, bool vec, int blocks, int threads, int nv,
                    cudaStream_t s) {
  return vec ? bwd_nv<TX, TR, true>(p, blocks, threads, nv, s)
             : bwd_nv<TX, TR, false>(p, blocks, threads, nv, s);
}

// Rows of partial weight gradients: row groups of the backward's grid, at most
// kNormPartialRows and never more than there are rows.
void bwd_grid(int64_t rows, int group, int* blocks, int* threads) {
  *threads = group < kNormThreads ? kNormThreads : group;
  const int per = *threads / group;
  const int64_t need = (rows + per - 1) / per;
  const int most = kNormPartialRows / per;
  *blocks = (int)(need < most ? need : most);
}

}  // namespace

int64_t norm_partial_rows(int64_t rows, int d) {
  int G, nv, blocks, threads;
  row_split(d, &G, &nv);
  bwd_grid(rows, G, &blocks, &threads);
  return (int64_t)blocks * (threads / G);
}

cudaError_t launch_add_norm(AddNormParams p, int dtype, int res_dtype, bool vec, cudaStream_t s) {
  int nv;
  row_split(p.d, &p.group, &nv);
  const bool same = dtype == res_dtype;
  if (p.y_q) {
    return same ? fwd_nv<__nv_bfloat16, __nv_bfloat16, true, true>(p, nv, s)
                : fwd_nv<__nv_bfloat16, float, true, true>(p, nv, s);
  }
  if (dtype == MOE_DT_BF16)
    return same ? fwd_vec<__nv_bfloat16, __nv_bfloat16>(p, vec, nv, s)
                : fwd_vec<__nv_bfloat16, float>(p, vec, nv, s);
  if (dtype == MOE_DT_F16)
    return same ? fwd_vec<__half, __half>(p, vec, nv, s) : fwd_vec<__half, float>(p, vec, nv, s);
  return fwd_vec<float, float>(p, vec, nv, s);
}

cudaError_t launch_add_norm_bwd(AddNormBwdParams p, int dtype, int res_dtype, bool vec, float* dw,
                                cudaStream_t s) {
  int nv, blocks, threads;
  row_split(p.d, &p.group, &nv);
  bwd_grid(p.rows, p.group, &blocks, &threads);
  const bool same = dtype == res_dtype;
  cudaError_t e;
  if (dtype == MOE_DT_BF16)
    e = same ? bwd_vec<__nv_bfloat16, __nv_bfloat16>(p, vec, blocks, threads, nv, s)
             : bwd_vec<__nv_bfloat16, float>(p, vec, blocks, threads, nv, s);
  else if (dtype == MOE_DT_F16)
    e = same ? bwd_vec<__half, __half>(p, vec, blocks, threads, nv, s)
             : bwd_vec<__half, float>(p, vec, blocks, threads, nv, s);
  else
    e = bwd_vec<float, float>(p, vec, blocks, threads, nv, s);
  if (e != cudaSuccess || dw == nullptr) return e;
  return launch_pdl(add_norm_dw_kernel, dim3((unsigned)((p.d + 31) / 32)), dim3(256), 0, s,
                    static_cast<const float*>(p.partial), blocks * (threads / p.group), p.d, dw);
}

cudaError_t launch_dropout(const DropoutParams& p, int dtype, bool vec, cudaStream_t s) {
  const int64_t gx = ((int64_t)p.cols + 255) / 256, gy = (p.rows + 7) / 8;
  const dim3 grid((unsigned)(gx < 65535 ? gx : 65535), (unsigned)(gy < 65535 ? gy : 65535));
  const dim3 block(32, 8);
  if (dtype == MOE_DT_BF16)
    return vec ? launch_pdl(dropout_kernel<__nv_bfloat16, true>, grid, block, 0, s, p)
               : launch_pdl(dropout_kernel<__nv_bfloat16, false>, grid, block, 0, s, p);
  if (dtype == MOE_DT_F16)
    return vec ? launch_pdl(dropout_kernel<__half, true>, grid, block, 0, s, p)
               : launch_pdl(dropout_kernel<__half, false>, grid, block, 0, s, p);
  return vec ? launch_pdl(dropout_kernel<float, true>, grid, block, 0, s, p)
             : launch_pdl(dropout_kernel<float, false>, grid, block, 0, s, p);
}

}  // namespace moe
