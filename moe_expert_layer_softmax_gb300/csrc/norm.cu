// Residual addition with the root-mean-square norm (forward) and dropout: the
// formulas and the pipeline are described in norm.cuh.
#include "norm_fwd.cuh"

namespace moe {

namespace {

// y = dropout(x): a warp, or (SMALL, rows up to 64 and 128 columns) 8 or 16 lanes,
// takes eight columns a lane of two rows at a time.  Bound by the generator (16-bit
// types) and HBM (fp32): 16384 x 2048 bf16 25.9 us, 5.2 TB/s; fp32 42.7 us, 6.3 TB/s.  Four
// blocks a multiprocessor leave 64 registers: at most 12 bytes a thread spill.  The branch
// for an offset on the device costs nothing (with and without it 25.9 and 26.0 us).
template <typename T, int V, bool SMALL>
__global__ void __launch_bounds__(256, 4) dropout_kernel(DropoutParams p) {
  __shared__ uint4 xch[V == 8 ? 1 : 256];
  pdl_begin();
  const int L = SMALL ? p.group : 32, lane = threadIdx.x & (L - 1), group = threadIdx.x / L, per = 256 / L * 2;
  const int before = (threadIdx.x & 31) / L * 2;   // rows of the warp's lanes before this one
  auto sync = []() { __syncwarp(); };
  const int64_t step = (int64_t)gridDim.y * per;
  for (int i = blockIdx.x; i * (int64_t)(8 * L) < p.cols; i += gridDim.x) {
    const int c = first_column<V>(i, lane, L);
    const bool in = c < p.cols;
    int64_t row = (int64_t)blockIdx.y * per + group * 2;
    const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
    T* y = static_cast<T*>(p.y) + row * p.ld_y;
    // a warp goes on while its first lanes have a row
    for (; row - before < p.rows; row += step, x += step * p.ld_x, y += step * p.ld_y) {
      const bool one = in && row < p.rows, two = in && row + 1 < p.rows;
      const Raw8<T> raw[2] = {load8_warp<T, V>(x, c, L, p.cols, one),
                              load8_warp<T, V>(x + p.ld_x, c, L, p.cols, two)};
      uint4 numbers[2];
      if (p.rng.threshold) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          numbers[u] = make_uint4((uint32_t)(lane + L * i), (uint32_t)(row + u), 0, 0);
        if (p.rng.offset_dev) draw<true>(numbers, p.rng); else draw<false>(numbers, p.rng);
        if constexpr (V != 8) {
#pragma unroll
          for (int u = 0; u < 2; ++u) exchange_numbers<V>(numbers[u], lane, L, xch + group * L, sync);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float f[8];
        widen8(raw[u], f);
        if (p.rng.threshold) drop8(f, numbers[u], p.rng);
        store8_warp<T, V>(y + u * p.ld_y, c, L, p.cols, narrow8<T>(f), u == 0 ? one : two);
      }
    }
  }
}

}  // namespace

cudaError_t launch_add_norm(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s) {
  return drawn_at(p) ? launch_add_norm_at(p, dtype, res_dtype, vec, s)
                     : fwd_launch<false, false>(p, dtype, res_dtype, vec, s);
}

template <typename T> static cudaError_t dropout_types(const DropoutParams& p, int vec, dim3 grid, cudaStream_t s) {
  const bool small = p.group < 32;
  if (vec == 8)
    return small ? launch_pdl(dropout_kernel<T, 8, true>, grid, dim3(256), 0, s, p)
                 : launch_pdl(dropout_kernel<T, 8, false>, grid, dim3(256), 0, s, p);
  if (vec == 2)
    return small ? launch_pdl(dropout_kernel<T, 2, true>, grid, dim3(256), 0, s, p)
                 : launch_pdl(dropout_kernel<T, 2, false>, grid, dim3(256), 0, s, p);
  return small ? launch_pdl(dropout_kernel<T, 1, true>, grid, dim3(256), 0, s, p)
               : launch_pdl(dropout_kernel<T, 1, false>, grid, dim3(256), 0, s, p);
}

cudaError_t launch_dropout(const DropoutParams& args, int dtype, int vec, cudaStream_t s) {
  DropoutParams p = args;
  p.group = p.cols <= 64 ? 8 : p.cols <= 128 ? 16 : 32;
  // four blocks a multiprocessor, all of them there at once (one block more than
  // that costs a second round: 3.4 and 5.0 TB/s at 768 columns); as many rows a
  // block as that leaves
  const int per = 256 / p.group * 2;
  const int64_t chunks = ((int64_t)p.cols + 255) / 256, most = (int64_t)device_info()->sm_count * 4;
  const int64_t gx = chunks < 65535 ? chunks : 65535, need = (p.rows + per - 1) / per;
  int64_t gy = gx < most ? most / gx : 1;
  gy = gy < need ? gy : need;
  const dim3 grid((unsigned)gx, (unsigned)(gy < 65535 ? gy : 65535));
  if (dtype == MOE_DT_BF16) return dropout_types<__nv_bfloat16>(p, vec, grid, s);
  if (dtype == MOE_DT_F16) return dropout_types<__half>(p, vec, grid, s);
  return dropout_types<float>(p, vec, grid, s);
}

}  // namespace moe
