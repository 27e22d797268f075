// Residual addition with a norm, forward: the kernel and the choice of its variant,
// for the root-mean-square norm (norm.cu) and the layer norm (layer_norm.cu).  The
// formulas and the pipeline are described in norm.cuh.
#pragma once

#include "norm.cuh"

namespace moe {

namespace {

// One row group per row; each thread holds NV times eight columns.  MX: codes,
// scales and (dq) their values instead of y; the rows from `rows` on are the
// padding of the last 128-row tile.  Measured: 8192 x 2048 bf16 23.7 us (5.7 TB/s),
// bound by HBM and, at 60% of the issue slots, by waits between instructions; 8
// bits, dropout, 32768 x 4096 238 us (5.1 TB/s), 65% of the issue slots.
template <bool LN, bool AT, typename TX, typename TR, bool MX, int V, bool RING, int NV, int MAXT>
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
  // Layer norm.  The bias stays in registers where there is room, or comes from the cache
  // for each row.  With up to 16 columns a thread its arithmetic goes in pairs; pairs of
  // 24 or 32 columns need more registers than there are: 8192 columns in bf16 4.2 TB/s in
  // pairs, 4.7 one by one, 12288 3.6 and 4.0 (but 2048 5.1 and 4.9).
  constexpr bool KEEP = LN && NV <= 2, PAIRS = LN && NV <= 2;
  float bias[KEEP ? NV : 1][8] = {};
  if constexpr (KEEP) {
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        load_weight8<V>(p.bias, p.w_f32, sizeof(TX) == 2 && p.x_f16, first_column<V>(i, lane, G), G, d, bias[i]);
    }
  }
  // layer norm: columns of this warp (of a row), and what the warps tell each other
  __shared__ float4 parts[2][LN ? kNormMaxThreads / 32 : 1];
  float mine = 0.0f, inv_mine = 0.0f;
  if constexpr (LN) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) mine += column_of<V>(first_column<V>(i, lane, G), j, G) < d ? 1.0f : 0.0f;
    mine = rg.part(mine);
    inv_mine = mine > 0.0f ? 1.0f / mine : 0.0f;
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
    if (p.rng.threshold) drop_numbers<V, AT>(numbers, lane, G, (uint32_t)row, p.rng, xch + rg.group * G, sync);
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
      for (int j = 0; j < 8; ++j) ss = LN ? ss + h[i][j] : fmaf(h[i][j], h[i][j], ss);
    }
    if constexpr (RING) ring.slot = ring.next(ring.slot);
    if constexpr (LN) {
      // the deviations from the warp's mean, then their squares; the warps' are joined
      // with the squares of their means' distances (Chan, Golub, LeVeque 1979): a stream
      // that is far from zero keeps its variance, and one barrier is enough
      const float part = rg.part(ss), near = part * inv_mine;
      float mean, apart = 0.0f;
      if constexpr (PAIRS) {
        Two squares(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = first_column<V>(i, lane, G);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            Two t = sum(Two(h[i][j], h[i][j + 1]), Two(-near, -near));
            if (V != 8 || c >= d) {   // places past the row's end: none
              const float2 q = t.get();
              t = Two(column_of<V>(c, j, G) < d ? q.x : 0.0f, column_of<V>(c, j + 1, G) < d ? q.y : 0.0f);
            }
            squares = fma(t, t, squares);
          }
        }
        const float2 q = squares.get();
        apart = q.x + q.y;
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = first_column<V>(i, lane, G);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float t = column_of<V>(c, j, G) < d ? h[i][j] - near : 0.0f;
            apart = fmaf(t, t, apart);
          }
        }
      }
      ss = rg.join(part, near, rg.part(apart), mine, p.inv_d, parts[turn], mean);
      if (lane == 0 && p.mean && live) p.mean[row] = mean;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          if constexpr (PAIRS) {
            const float2 t = sum(Two(h[i][j], h[i][j + 1]), Two(-mean, -mean)).get();
            h[i][j] = t.x;
            h[i][j + 1] = t.y;
          } else {
            h[i][j] -= mean;
            h[i][j + 1] -= mean;
          }
        }
    } else {
      ss = rg.sum(ss, red[turn]);
    }
    const float rstd = inv_sqrt(fmaf(ss, p.inv_d, p.eps));
    if (lane == 0 && p.rstd && live) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<V>(i, lane, G);
      float amax = 0.0f;
      float b[8];
      if constexpr (LN && !KEEP) {
        if (p.bias) {
          load_weight8<V>(p.bias, p.w_f32, sizeof(TX) == 2 && p.x_f16, c, G, d, b);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] = 0.0f;
        }
      }
      if constexpr (LN) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float* f = KEEP ? bias[KEEP ? i : 0] : b;
          if constexpr (PAIRS) {
            const Two n = mul(Two(h[i][j], h[i][j + 1]), Two(rstd, rstd));
            const float2 t = fma(n, Two(w[i][j], w[i][j + 1]), Two(f[j], f[j + 1])).get();
            h[i][j] = t.x;
            h[i][j + 1] = t.y;
          } else {
            h[i][j] = fmaf(h[i][j] * rstd, w[i][j], f[j]);
            h[i][j + 1] = fmaf(h[i][j + 1] * rstd, w[i][j + 1], f[j + 1]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (!LN) h[i][j] = (h[i][j] * w[i][j]) * rstd;
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

template <bool LN, bool AT, typename TX, typename TR, bool MX, int V, bool RING, int NV, int MAXT>
cudaError_t fwd_run(const AddNormParams& p, int threads, cudaStream_t s) {
  auto* kernel = &add_norm_kernel<LN, AT, TX, TR, MX, V, RING, NV, MAXT>;
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
// without vector loads: one); with RMS norm and 8-bit output three or four.  Measured there
// at 32768 x 4096 with dropout 243 us with four, 266 with two; at 8192 x 2048 (bf16) 26
// with four, 24 with two.  The layer norm takes two for either output: the pairs of its
// arithmetic need their registers (above: KEEP, PAIRS).
template <bool LN, bool AT, typename TX, typename TR, bool MX, int V>
cudaError_t fwd_types(const AddNormParams& p, cudaStream_t s) {
  constexpr bool wide = V == 8 && RowRing<8 * (sizeof(TX) + sizeof(TR)), 4>::kFits512;
  AddNormParams q = p;
  if constexpr (V == 8) {
    RowSplit split(p.d, LN || !MX || p.d <= 512 ? 2 : 3, 4, kNormThreads);
    q.group = split.group;
    if (split.group) {
      const int threads = split.threads();
      if (split.nv == 1) return fwd_run<LN, AT, TX, TR, MX, 8, true, 1, kNormThreads>(q, threads, s);
      if (split.nv == 2) return fwd_run<LN, AT, TX, TR, MX, 8, true, 2, kNormThreads>(q, threads, s);
      if (split.nv == 3) return fwd_run<LN, AT, TX, TR, MX, 8, true, 3, kNormThreads>(q, threads, s);
      return fwd_run<LN, AT, TX, TR, MX, 8, true, 4, kNormThreads>(q, threads, s);
    }
    if constexpr (wide) {
      split = RowSplit(p.d, 3, 4, 512);
      q.group = split.group;
      if (split.group)
        return split.nv == 3 ? fwd_run<LN, AT, TX, TR, MX, 8, true, 3, 512>(q, q.group, s)
                             : fwd_run<LN, AT, TX, TR, MX, 8, true, 4, 512>(q, q.group, s);
    }
  } else {
    const RowSplit split(p.d, 1, 1, kNormMaxThreads);
    q.group = split.group;
    if (split.group) {
      const int threads = split.threads();
      if (split.group > 512) return fwd_run<LN, AT, TX, TR, MX, V, false, 1, kNormMaxThreads>(q, threads, s);
      return split.group <= kNormThreads ? fwd_run<LN, AT, TX, TR, MX, V, false, 1, kNormThreads>(q, threads, s)
                                         : fwd_run<LN, AT, TX, TR, MX, V, false, 1, 512>(q, threads, s);
    }
  }
  const RowSplit split(p.d, wide ? 3 : 2, 4, kNormMaxThreads);
  q.group = split.group;
  if constexpr (!wide)
    if (split.nv == 2) return fwd_run<LN, AT, TX, TR, MX, V, false, 2, kNormMaxThreads>(q, q.group, s);
  return split.nv == 3 ? fwd_run<LN, AT, TX, TR, MX, V, false, 3, kNormMaxThreads>(q, q.group, s)
                       : fwd_run<LN, AT, TX, TR, MX, V, false, 4, kNormMaxThreads>(q, q.group, s);
}

template <bool LN, bool AT, typename TX, typename TR>
cudaError_t fwd_vec(const AddNormParams& p, int vec, cudaStream_t s) {
  return vec == 8   ? fwd_types<LN, AT, TX, TR, false, 8>(p, s)
         : vec == 2 ? fwd_types<LN, AT, TX, TR, false, 2>(p, s)
                    : fwd_types<LN, AT, TX, TR, false, 1>(p, s);
}

// The entry of either norm: a kernel for the types and the access.
template <bool LN, bool AT> cudaError_t fwd_launch(const AddNormParams& p, int dtype, int res_dtype, int vec, cudaStream_t s) {
  const bool same = dtype == res_dtype;
  if (p.y_q)
    return same ? fwd_types<LN, AT, __nv_bfloat16, __nv_bfloat16, true, 8>(p, s)
                : fwd_types<LN, AT, __nv_bfloat16, float, true, 8>(p, s);
  if (dtype == MOE_DT_BF16)
    return same ? fwd_vec<LN, AT, __nv_bfloat16, __nv_bfloat16>(p, vec, s)
                : fwd_vec<LN, AT, __nv_bfloat16, float>(p, vec, s);
  if (dtype == MOE_DT_F16)
    return same ? fwd_vec<LN, AT, __half, __half>(p, vec, s) : fwd_vec<LN, AT, __half, float>(p, vec, s);
  return fwd_vec<LN, AT, float, float>(p, vec, s);
}

}  // namespace

}  // namespace moe
