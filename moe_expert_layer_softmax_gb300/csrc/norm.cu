// Residual addition with the root-mean-square norm (forward) and dropout: the
// formulas and the pipeline are described in norm.cuh.
#include "norm.cuh"

namespace moe {

namespace {

// One row group per row; each thread holds NV times eight columns.  MX: codes,
// scales and (dq) their values instead of y; the rows from `rows` on are the
// padding of the last 128-row tile.  Measured: 8192 x 2048 bf16 23.7 us (5.7 TB/s),
// bound by HBM and, at 60% of the issue slots, by waits between instructions; 8
// bits, dropout, 32768 x 4096 238 us (5.1 TB/s), 65% of the issue slots.
template <typename TX, typename TR, bool MX, int V, bool RING, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, norm_blocks(RING, NV, MAXT)) add_norm_kernel(AddNormParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[2][kNormMaxThreads / 32];
  __shared__ uint4 xch[V == 8 ? 1 : MAXT];
  using Ring = RowRing<8 * (sizeof(TX) + sizeof(TR)), NV>;
  constexpr int XP = sizeof(TX) / 2, RP = sizeof(TR) / 2;   // 16-byte pieces of eight columns
  pdl_begin();
  const RowGroup<NV == 1> rg(p.group);
  const int G = rg.G, lane = rg.lane, d = p.d;
  auto sync = [&]() { rg.sync(); };
  float w[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first_column<V>(i, lane, G);
    load_weight8<V>(p.weight, p.w_f32, sizeof(TX) == 2 && p.x_f16, c, G, d, w[i]);
  }
  const int64_t step = (int64_t)gridDim.x * rg.per;
  int64_t row = (int64_t)blockIdx.x * rg.per + rg.group;
  Ring ring(smem, G);
  // RING: where the next row to copy starts
  const TX* cx = static_cast<const TX*>(p.x) + row * p.ld_x;
  const TR* cr = p.residual ? static_cast<const TR*>(p.residual) + row * p.ld_residual : nullptr;
  int64_t copy_row = row;
  auto copy = [&]() {
    if (copy_row < p.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        ring.put(i * XP, cx, (lane + i * G) * 8, d);
        if (cr) ring.put(NV * XP + i * RP, cr, (lane + i * G) * 8, d);
      }
      cx += step * p.ld_x;
      if (cr) cr += step * p.ld_residual;
      copy_row += step;
    }
    ring.ahead = ring.next(ring.ahead);
    cp_async_commit();
  };
  if constexpr (RING) {
#pragma unroll 1
    for (int i = 0; i < Ring::kDepth - 1; ++i) copy();
  }
  // without a ring: the next row, on its way in registers
  constexpr bool AHEAD = !RING && NV == 1 && MAXT < kNormMaxThreads;
  Raw8<TX> ax = {};
  Raw8<TR> ar = {};
  auto fetch = [&](int64_t at) {
    const int c = first_column<V>(0, lane, G);
    const bool in = c < d && at < p.rows;
    ax = load8_warp<TX, V>(static_cast<const TX*>(p.x) + at * p.ld_x, c, G, d, in);
    if (cr) ar = load8_warp<TR, V>(static_cast<const TR*>(p.residual) + at * p.ld_residual, c, G, d, in);
  };
  if constexpr (AHEAD) fetch(row);
  // a warp goes on while its first group has a row
  for (int turn = 0; row - rg.before() < p.rows; row += step, turn ^= 1) {
    const bool live = NV > 1 || row < p.rows;
    float h[NV][8];
    if constexpr (RING) {
      __syncwarp();   // every lane has read the slot that is filled now
      copy();
      cp_async_wait<Ring::kDepth - 1>();
      __syncwarp();
    }
    uint4 numbers[NV];
    if (p.rng.threshold) drop_numbers<V>(numbers, lane, G, (uint32_t)row, p.rng, xch + rg.group * G, sync);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<V>(i, lane, G);
      const bool in = c < d && live;
      Raw8<TX> xr = {};
      Raw8<TR> rr = {};
      if constexpr (RING) {
        xr = ring.template get<TX>(i * XP);
        if (cr) rr = ring.template get<TR>(NV * XP + i * RP);
      } else if constexpr (AHEAD) {
        xr = ax;
        rr = ar;
        fetch(row + step);
      } else {
        xr = load8_warp<TX, V>(static_cast<const TX*>(p.x) + row * p.ld_x, c, G, d, in);
        if (cr) rr = load8_warp<TR, V>(static_cast<const TR*>(p.residual) + row * p.ld_residual, c, G, d, in);
      }
      widen8(xr, h[i]);
      if (p.rng.threshold) drop8(h[i], numbers[i], p.rng);
      if (cr) {
        float f[8];
        widen8(rr, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += f[j];
      }
      if (p.h) {
        const Raw8<TR> hr = narrow8<TR>(h[i]);
        store8_warp<TR, V>(static_cast<TR*>(p.h) + row * p.ld_h, c, G, d, hr, in);
        widen8(hr, h[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
    if constexpr (RING) ring.slot = ring.next(ring.slot);
    ss = rg.sum(ss, red[turn]);
    const float rstd = inv_sqrt(fmaf(ss, p.inv_d, p.eps));
    if (lane == 0 && p.rstd && live) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<V>(i, lane, G);
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = (h[i][j] * w[i][j]) * rstd;
        if (MX) amax = fmaxf(amax, fabsf(h[i][j]));
      }
      if constexpr (!MX) {
        store8_warp<TX, V>(static_cast<TX*>(p.y) + row * p.ld_y, c, G, d, narrow8<TX>(h[i]), c < d && live);
      } else {
        // d is a multiple of 128: the 16 lanes of four 32-column blocks are all
        // within the row or all past its end
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int s = mx_scale_exp(amax);
        // the scales of four neighbouring blocks are four neighbouring bytes
        uint32_t four = (uint32_t)(s + 127) << (8 * ((lane >> 2) & 3));
        four |= __shfl_xor_sync(0xffffffffu, four, 4);
        four |= __shfl_xor_sync(0xffffffffu, four, 8);
        if (c < d && live) {
          const float inv = exp2i(-s);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = h[i][j] * inv;
          const uint2 q = e4m3x8(v);
          *reinterpret_cast<uint2*>(p.y_q + row * d + c) = q;
          if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.y_scales + sf_offset(row, c >> 5, d >> 5)) = four;
          if (p.y_dq) {
            const float up = exp2i(s);
            e4m3x2_to_f32(q.x, v[0], v[1]);
            e4m3x2_to_f32(q.x >> 16, v[2], v[3]);
            e4m3x2_to_f32(q.y, v[4], v[5]);
            e4m3x2_to_f32(q.y >> 16, v[6], v[7]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= up;
            store8<__nv_bfloat16, 8>(static_cast<__nv_bfloat16*>(p.y_dq) + row * d, c, 1, d,
                                        narrow8<__nv_bfloat16>(v));
          }
        }
      }
    }
  }
  if constexpr (MX) {   // the padding: zero codes, scale 2^0
    if (row - step >= p.rows) row -= step;   // it went on with its warp
    for (; row < p.rows_pad; row += step) {
      for (int c = lane * 8; c < d; c += G * 8) {
        *reinterpret_cast<uint2*>(p.y_q + row * d + c) = make_uint2(0, 0);
        if ((c & 31) == 0) p.y_scales[sf_offset(row, c >> 5, d >> 5)] = 127;
        if (p.y_dq) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y_dq) + row * d + c) = make_uint4(0, 0, 0, 0);
      }
    }
  }
}

// y = dropout(x): a warp, or (SMALL, rows up to 64 and 128 columns) 8 or 16 lanes,
// takes eight columns a lane of two rows at a time.  Bound by the generator (16-bit
// types) and HBM (fp32): 16384 x 2048 bf16 26.6 us, 5.0 TB/s; fp32 5.7 TB/s.  Four
// blocks a multiprocessor leave 64 registers: with vector loads 12 to 40 bytes a thread
// spill (fp32 12, fp16 20, bf16 40; without them at most 12).
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
          numbers[u] = make_uint4((uint32_t)(lane + L * i), (uint32_t)(row + u), p.rng.o0, p.rng.o1);
        philox4x32_10(numbers, p.rng.k0, p.rng.k1);
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

template <typename TX, typename TR, bool MX, int V, bool RING, int NV, int MAXT>
cudaError_t fwd_run(const AddNormParams& p, int threads, cudaStream_t s) {
  auto* kernel = &add_norm_kernel<TX, TR, MX, V, RING, NV, MAXT>;
  constexpr int ring = RING ? RowRing<8 * (sizeof(TX) + sizeof(TR)), NV>::kBytes : 0;
  if constexpr (RING) {
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kernel), MAXT * ring);
    if (e != cudaSuccess) return e;
  }
  constexpr int planned = norm_blocks(RING, NV, MAXT);
  int resident = norm_resident(planned, MAXT, threads, ring);
  // Where the ring leaves room for one block and not two, two rounds of blocks all
  // the same when each has many rows and no numbers to draw.  Measured in one and in
  // two rounds (us): fp32, 8192 columns, 600 rows 14.9 and 17.8, 2000 rows 42.7 and
  // 42.7, 8192 rows 176 and 166; with dropout 16.2 and 19.0, 44.9 and 45.8, 162 and 164.
  if (resident < planned * MAXT / threads && p.rng.threshold == 0 && p.rows > (int64_t)device_info()->sm_count * 13)
    resident = planned * MAXT / threads;
  const int blocks = row_blocks(MX ? p.rows_pad : p.rows, p.group, threads, resident);
  return launch_pdl(kernel, dim3(blocks), dim3(threads), (size_t)threads * ring, s, p);
}

// Rows up to 8192 columns come through the ring of 256 threads, up to 16384 (but
// where both matrices are fp32) of 512; wider ones are read as they are needed.
// A thread holds two groups of eight columns, more where the threads need it (rows
// without vector loads: one), for the 8-bit output three or four.  Measured at 32768
// x 4096 (8-bit, dropout) 243 us with four, 266 with two; at 8192 x 2048 (bf16) 26
// with four, 24 with two.
template <typename TX, typename TR, bool MX, int V>
cudaError_t fwd_types(const AddNormParams& p, cudaStream_t s) {
  constexpr bool wide = V == 8 && RowRing<8 * (sizeof(TX) + sizeof(TR)), 4>::kFits512;
  AddNormParams q = p;
  if constexpr (V == 8) {
    RowSplit split(p.d, !MX || p.d <= 512 ? 2 : 3, 4, kNormThreads);
    q.group = split.group;
    if (split.group) {
      const int threads = split.threads();
      if (split.nv == 1) return fwd_run<TX, TR, MX, 8, true, 1, kNormThreads>(q, threads, s);
      if (split.nv == 2) return fwd_run<TX, TR, MX, 8, true, 2, kNormThreads>(q, threads, s);
      if (split.nv == 3) return fwd_run<TX, TR, MX, 8, true, 3, kNormThreads>(q, threads, s);
      return fwd_run<TX, TR, MX, 8, true, 4, kNormThreads>(q, threads, s);
    }
    if constexpr (wide) {
      split = RowSplit(p.d, 3, 4, 512);
      q.group = split.group;
      if (split.group)
        return split.nv == 3 ? fwd_run<TX, TR, MX, 8, true, 3, 512>(q, q.group, s)
                             : fwd_run<TX, TR, MX, 8, true, 4, 512>(q, q.group, s);
    }
  } else {
    const RowSplit split(p.d, 1, 1, kNormMaxThreads);
    q.group = split.group;
    if (split.group) {
      const int threads = split.threads();
      if (split.group > 512) return fwd_run<TX, TR, MX, V, false, 1, kNormMaxThreads>(q, threads, s);
      return split.group <= kNormThreads ? fwd_run<TX, TR, MX, V, false, 1, kNormThreads>(q, threads, s)
                                         : fwd_run<TX, TR, MX, V, false, 1, 512>(q, threads, s);
    }
  }
  const RowSplit split(p.d, wide ? 3 : 2, 4, kNormMaxThreads);
  q.group = split.group;
  if constexpr (!wide)
    if (split.nv == 2) return fwd_run<TX, TR, MX, V, false, 2, kNormMaxThreads>(q, q.group, s);
  return split.nv == 3 ? fwd_run<TX, TR, MX, V, false, 3, kNormMaxThreads>(q, q.group, s)
                       : fwd_run<TX, TR, MX, V, false, 4, kNormMaxThreads>(q, q.group, s);
}

template <typename TX, typename TR>
cudaError_t fwd_vec(const AddNormParams& p, int vec, cudaStream_t s) {
  return vec == 8   ? fwd_types<TX, TR, false, 8>(p, s)
         : vec == 2 ? fwd_types<TX, TR, false, 2>(p, s)
                    : fwd_types<TX, TR, false, 1>(p, s);
}

}  // namespace

cudaError_t launch_add_norm(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s) {
  const bool same = dtype == res_dtype;
  if (p.y_q)
    return same ? fwd_types<__nv_bfloat16, __nv_bfloat16, true, 8>(p, s)
                : fwd_types<__nv_bfloat16, float, true, 8>(p, s);
  if (dtype == MOE_DT_BF16)
    return same ? fwd_vec<__nv_bfloat16, __nv_bfloat16>(p, vec, s) : fwd_vec<__nv_bfloat16, float>(p, vec, s);
  if (dtype == MOE_DT_F16)
    return same ? fwd_vec<__half, __half>(p, vec, s) : fwd_vec<__half, float>(p, vec, s);
  return fwd_vec<float, float>(p, vec, s);
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
