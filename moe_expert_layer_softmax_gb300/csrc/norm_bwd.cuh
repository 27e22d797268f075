// Residual addition with a norm, backward: the kernels and the choice of their
// variant, for the root-mean-square norm (norm_bwd.cu) and the layer norm
// (layer_norm_bwd.cu).  The formulas and the pipeline are described in norm.cuh.
#pragma once

#include "norm.cuh"

namespace moe {

namespace {

// Rows that take no vector loads: whether the next one is fetched into registers
// (two blocks a multiprocessor then, three otherwise).  Measured with and without,
// TB/s: 1001 columns bf16 3.0 and 2.6, on an fp32 stream 5.0 and 4.1; 1002 columns
// on an fp32 stream 4.8 and 4.2, but bf16 throughout 2.2 and 2.95.
template <typename TR, int V, bool RING, int NV, int MAXT>
constexpr bool kNextInRegisters = !RING && NV == 1 && MAXT < kNormMaxThreads && !(V == 2 && sizeof(TR) == 2);

// Backward: the weight gradient of a block's rows stays in registers; one row of
// partial sums a block goes to `partial` [gridDim.x, d].  Measured: 8192 x 2048
// bf16 33.2 us (5.05 TB/s; 4 us of it the sum of the partial rows), 32768 x 4096 on
// an fp32 stream with dropout 317 us (6.8 TB/s, a plain copy's rate).
template <bool LN, bool AT, typename TX, typename TR, int V, bool RING, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, norm_blocks(RING || kNextInRegisters<TR, V, RING, NV, MAXT>, NV, MAXT)) add_norm_bwd_kernel(AddNormBwdParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[2][kNormMaxThreads / 32], red2[2][LN ? kNormMaxThreads / 32 : 4];
  // drop numbers that change hands; at the end the sums of the row groups
  // (eight floats a thread and NV, in the ring where there is one; only blocks of
  // kNormThreads have groups)
  __shared__ uint4 xch[RING ? 1 : MAXT <= kNormThreads ? MAXT * 2 * NV : V == 8 ? 1 : MAXT];
  using Ring = RowRing<8 * (sizeof(TX) + 2 * sizeof(TR)), NV>;
  constexpr int XP = sizeof(TX) / 2, RP = sizeof(TR) / 2;   // 16-byte pieces of eight columns
  pdl_begin();
  const RowGroup<NV == 1> rg(p.group);
  const int G = rg.G, lane = rg.lane, d = p.d;
  auto sync = [&]() { rg.sync(); };
  float w[NV][8], dw[NV][8];
  Two db[LN ? NV : 1][4], dwp[LN ? NV : 1][4];   // layer norm: in pairs
  if constexpr (LN) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) db[i][j] = dwp[i][j] = Two(0.0f, 0.0f);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first_column<V>(i, lane, G);
    load_weight8<V>(p.weight, p.w_f32, sizeof(TX) == 2 && p.x_f16, c, G, d, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * rg.per;
  int64_t row = (int64_t)blockIdx.x * rg.per + rg.group;
  Ring ring(smem, G);
  // RING: where the next row to copy starts
  const TX* cy = static_cast<const TX*>(p.dy) + row * p.ld_dy;
  const TR* ch = static_cast<const TR*>(p.h) + row * p.ld_h;
  const TR* cd = p.dres ? static_cast<const TR*>(p.dres) + row * p.ld_dres : nullptr;
  int64_t copy_row = row;
  auto copy = [&]() {
    if (copy_row < p.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * G) * 8;
        ring.put(i * XP, cy, c, d);
        ring.put(NV * XP + i * RP, ch, c, d);
        if (cd) ring.put(NV * (XP + RP) + i * RP, cd, c, d);
      }
      cy += step * p.ld_dy;
      ch += step * p.ld_h;
      if (cd) cd += step * p.ld_dres;
      copy_row += step;
    }
    ring.ahead = ring.next(ring.ahead);
    cp_async_commit();
  };
  if constexpr (RING) {
#pragma unroll 1
    for (int i = 0; i < Ring::kDepth - 1; ++i) copy();
  }
  float rn = row < p.rows ? p.rstd[row] : 0.0f;
  float mn = LN && row < p.rows ? p.mean[row] : 0.0f;
  // without a ring: the next row, on its way in registers
  constexpr bool AHEAD = kNextInRegisters<TR, V, RING, NV, MAXT>;
  Raw8<TX> ay = {};
  Raw8<TR> ah = {}, ad = {}, dr0 = {};
  auto fetch = [&](int64_t at) {
    const int c = first_column<V>(0, lane, G);
    const bool in = c < d && at < p.rows;
    ay = load8_warp<TX, V>(static_cast<const TX*>(p.dy) + at * p.ld_dy, c, G, d, in);
    ah = load8_warp<TR, V>(static_cast<const TR*>(p.h) + at * p.ld_h, c, G, d, in);
    if (cd) ad = load8_warp<TR, V>(static_cast<const TR*>(p.dres) + at * p.ld_dres, c, G, d, in);
  };
  if constexpr (AHEAD) fetch(row);
  // a warp goes on while its first group has a row; one without adds zeros
  for (int turn = 0; row - rg.before() < p.rows; row += step, turn ^= 1) {
    const bool live = NV > 1 || row < p.rows;
    Raw8<TX> yr[NV] = {};
    Raw8<TR> hr[NV] = {};
    // a group without a row multiplies its zeros by zeros
    const float r = LN && !live ? 0.0f : rn, mean = LN && live ? mn : 0.0f;
    if (row + step < p.rows) {
      rn = p.rstd[row + step];
      if constexpr (LN) mn = p.mean[row + step];
    }
    if constexpr (RING) {
      __syncwarp();   // every lane has read the slot that is filled now
      copy();
      cp_async_wait<Ring::kDepth - 1>();
      __syncwarp();
    }
    float dot = 0.0f;
    Two dots(0.0f, 0.0f), sums(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<V>(i, lane, G);
      if constexpr (RING) {
        if (live) {
          yr[i] = ring.template get<TX>(i * XP);
          hr[i] = ring.template get<TR>(NV * XP + i * RP);
        }
      } else if constexpr (AHEAD) {
        yr[i] = ay;
        hr[i] = ah;
        dr0 = ad;
        fetch(row + step);
      } else {
        yr[i] = load8_warp<TX, V>(static_cast<const TX*>(p.dy) + row * p.ld_dy, c, G, d, c < d && live);
        hr[i] = load8_warp<TR, V>(static_cast<const TR*>(p.h) + row * p.ld_h, c, G, d, c < d && live);
      }
      float a[8], b[8];
      widen8(yr[i], a);
      widen8(hr[i], b);
      if constexpr (LN) {   // sums of g = w dy and of g (h - mean)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Two y(a[2 * j], a[2 * j + 1]), c = sum(Two(b[2 * j], b[2 * j + 1]), Two(-mean, -mean));
          const Two g = mul(y, Two(w[i][2 * j], w[i][2 * j + 1]));
          dwp[i][j] = fma(mul(y, Two(r, r)), c, dwp[i][j]);
          db[i][j] = sum(db[i][j], y);
          sums = sum(sums, g);
          dots = fma(g, c, dots);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float ah = a[j] * b[j];
          dw[i][j] = fmaf(ah, r, dw[i][j]);
          dot = fmaf(ah, w[i][j], dot);
        }
      }
    }
    float k, mg = 0.0f;
    if constexpr (LN) {
      const float2 s = sums.get(), t = dots.get();
      mg = s.x + s.y;
      dot = t.x + t.y;
      rg.sum2(mg, dot, red[turn], red2[turn]);
      mg *= p.inv_d;
      k = r * (r * (dot * p.inv_d));
    } else {
      dot = rg.sum(dot, red[turn]);
      k = r * r * (dot * p.inv_d);
    }
    uint4 numbers[NV];
    if (p.dx && p.rng.threshold)
      drop_numbers<V, AT>(numbers, lane, G, (uint32_t)row, p.rng, xch + rg.group * G, sync);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<V>(i, lane, G);
      const bool in = c < d && live;
      float a[8], b[8];
      if constexpr (LN && RING) {   // again, and not in registers past the barrier
        if (live) {
          yr[i] = ring.template get<TX>(i * XP);
          hr[i] = ring.template get<TR>(NV * XP + i * RP);
        }
      }
      widen8(yr[i], a);
      widen8(hr[i], b);
      if constexpr (LN) {   // r (g - mean(g) - (h - mean) r^2 mean(g (h - mean)))
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Two c = sum(Two(b[2 * j], b[2 * j + 1]), Two(-mean, -mean));
          const Two g = fma(Two(a[2 * j], a[2 * j + 1]), Two(w[i][2 * j], w[i][2 * j + 1]), Two(-mg, -mg));
          const float2 o = mul(fma(c, Two(-k, -k), g), Two(r, r)).get();
          a[2 * j] = o.x;
          a[2 * j + 1] = o.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = r * (a[j] * w[i][j] - b[j] * k);
      }
      if (cd) {
        Raw8<TR> dr = {};
        if constexpr (RING)
          dr = ring.template get<TR>(NV * (XP + RP) + i * RP);
        else if constexpr (AHEAD)
          dr = dr0;
        else
          dr = load8_warp<TR, V>(static_cast<const TR*>(p.dres) + row * p.ld_dres, c, G, d, in);
        widen8(dr, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += b[j];
      }
      if (p.dh) store8_warp<TR, V>(static_cast<TR*>(p.dh) + row * p.ld_dh, c, G, d, narrow8<TR>(a), in);
      if (p.dx) {
        if (p.rng.threshold) drop8(a, numbers[i], p.rng);
        store8_warp<TX, V>(static_cast<TX*>(p.dx) + row * p.ld_dx, c, G, d, narrow8<TX>(a), in);
      }
    }
    if constexpr (RING) ring.slot = ring.next(ring.slot);
  }
  if (!p.partial) return;
  // a row of the workspace: dw, with layer norm db behind it
  float* out = p.partial + (int64_t)blockIdx.x * d * (LN ? 2 : 1);
  auto write = [&](const float (&v)[NV][8], float* out) {
    if (rg.per > 1) {   // the row groups' sums, added in their order
      float* all = RING ? reinterpret_cast<float*>(smem) : reinterpret_cast<float*>(xch);
      const int width = G * NV * 8;
      cp_async_wait<0>();
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) all[rg.group * width + column_of<V>(first_column<V>(i, lane, G), j, G)] = v[i][j];
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += blockDim.x) {
        float s = 0.0f;
        for (int g = 0; g < rg.per; ++g) s += all[g * width + c];
        out[c] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = first_column<V>(i, lane, G);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (column_of<V>(c, j, G) < d) out[column_of<V>(c, j, G)] = v[i][j];
      }
    }
  };
  if constexpr (LN) {
    float db_[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 s = dwp[i][j].get(), t = db[i][j].get();
        dw[i][2 * j] = s.x; dw[i][2 * j + 1] = s.y;
        db_[i][2 * j] = t.x; db_[i][2 * j + 1] = t.y;
      }
    write(dw, out);
    write(db_, out + d);
  } else {
    write(dw, out);
  }
}

// dw[c] = sum of the partial rows, 32 columns a block: 32 warps take every
// 32nd row, their sums are added in warp order.  Columns from `split` on are db's;
// either of the two may be missing.
__global__ void __launch_bounds__(1024) add_norm_dw_kernel(const float* __restrict__ partial, int n_partial, int d,
                                                           int split, float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float s[32][33];
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int i = warp; i < n_partial; i += 32) acc += partial[(int64_t)i * d + c];
  }
  s[warp][lane] = acc;
  __syncthreads();
  const float sum = warp_sum(s[lane][warp]);   // column `warp` of the 32
  const int column = blockIdx.x * 32 + warp;
  if (lane == 0 && column < d) {
    if (column < split) {
      if (dw) dw[column] = sum;
    } else if (db) {
      db[column - split] = sum;
    }
  }
}

template <bool LN, bool AT, typename TX, typename TR, int V, bool RING, int NV, int MAXT>
cudaError_t bwd_run(const AddNormBwdParams& p, int threads, int* blocks, cudaStream_t s) {
  auto* kernel = &add_norm_bwd_kernel<LN, AT, TX, TR, V, RING, NV, MAXT>;
  constexpr int ring = RING ? RowRing<8 * (sizeof(TX) + 2 * sizeof(TR)), NV>::kBytes : 0;
  if constexpr (RING) {
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kernel), MAXT * ring);
    if (e != cudaSuccess) return e;
  }
  constexpr int most = norm_blocks(RING || kNextInRegisters<TR, V, RING, NV, MAXT>, NV, MAXT);
  *blocks = row_blocks(p.rows, p.group, threads, norm_resident(most, MAXT, threads, ring));
  if (*blocks > kNormPartialRows) *blocks = kNormPartialRows;   // rows of the workspace
  return launch_pdl(kernel, dim3(*blocks), dim3(threads), (size_t)threads * ring, s, p);
}

// Rows up to 8192 columns (512 threads; 16384 where both matrices are 16 bits)
// come through the ring; wider ones are read as they are needed.
template <bool LN, bool AT, typename TX, typename TR, int V>
cudaError_t bwd_types(const AddNormBwdParams& p, int* blocks, cudaStream_t s) {
  constexpr bool wide = V == 8 && RowRing<8 * (sizeof(TX) + 2 * sizeof(TR)), 4>::kFits512;
  AddNormBwdParams q = p;
  RowSplit split = V == 8 ? RowSplit(p.d, 2, wide ? 4 : 2, 512) : RowSplit(p.d, 1, 1, kNormMaxThreads);
  q.group = split.group;
  if (split.group) {
    const int threads = split.threads();
    if constexpr (wide) {
      if (split.nv == 3) return bwd_run<LN, AT, TX, TR, V, true, 3, 512>(q, threads, blocks, s);
      if (split.nv == 4) return bwd_run<LN, AT, TX, TR, V, true, 4, 512>(q, threads, blocks, s);
    }
    if constexpr (V == 8) {
      if (split.nv == 2 && split.group <= kNormThreads)
        return bwd_run<LN, AT, TX, TR, V, true, 2, kNormThreads>(q, threads, blocks, s);
      return split.nv == 1 ? bwd_run<LN, AT, TX, TR, V, true, 1, kNormThreads>(q, threads, blocks, s)
                           : bwd_run<LN, AT, TX, TR, V, true, 2, 512>(q, threads, blocks, s);
    } else {
      if (split.group > 512) return bwd_run<LN, AT, TX, TR, V, false, 1, kNormMaxThreads>(q, threads, blocks, s);
      return split.group <= kNormThreads ? bwd_run<LN, AT, TX, TR, V, false, 1, kNormThreads>(q, threads, blocks, s)
                                         : bwd_run<LN, AT, TX, TR, V, false, 1, 512>(q, threads, blocks, s);
    }
  }
  split = RowSplit(p.d, wide ? 3 : 2, 4, kNormMaxThreads);
  q.group = split.group;
  if constexpr (!wide)
    if (split.nv == 2) return bwd_run<LN, AT, TX, TR, V, false, 2, kNormMaxThreads>(q, q.group, blocks, s);
  return split.nv == 3 ? bwd_run<LN, AT, TX, TR, V, false, 3, kNormMaxThreads>(q, q.group, blocks, s)
                       : bwd_run<LN, AT, TX, TR, V, false, 4, kNormMaxThreads>(q, q.group, blocks, s);
}

template <bool LN, bool AT, typename TX, typename TR>
cudaError_t bwd_vec(const AddNormBwdParams& p, int vec, int* blocks, cudaStream_t s) {
  return vec == 8   ? bwd_types<LN, AT, TX, TR, 8>(p, blocks, s)
         : vec == 2 ? bwd_types<LN, AT, TX, TR, 2>(p, blocks, s)
                    : bwd_types<LN, AT, TX, TR, 1>(p, blocks, s);
}

// The entry of either norm: a kernel for the types and the access, and the sum of
// the blocks' weight (and bias) gradients.
template <bool LN, bool AT>
cudaError_t bwd_launch(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw, float* db, cudaStream_t s) {
  const bool same = dtype == res_dtype;
  int blocks = 0;
  cudaError_t e;
  if (dtype == MOE_DT_BF16)
    e = same ? bwd_vec<LN, AT, __nv_bfloat16, __nv_bfloat16>(p, vec, &blocks, s)
             : bwd_vec<LN, AT, __nv_bfloat16, float>(p, vec, &blocks, s);
  else if (dtype == MOE_DT_F16)
    e = same ? bwd_vec<LN, AT, __half, __half>(p, vec, &blocks, s) : bwd_vec<LN, AT, __half, float>(p, vec, &blocks, s);
  else
    e = bwd_vec<LN, AT, float, float>(p, vec, &blocks, s);
  if (e != cudaSuccess || p.partial == nullptr) return e;
  const int width = LN ? 2 * p.d : p.d;
  return launch_pdl(add_norm_dw_kernel, dim3((unsigned)((width + 31) / 32)), dim3(1024), 0, s,
                    static_cast<const float*>(p.partial), blocks, width, p.d, dw, db);
}

}  // namespace

}  // namespace moe
