// Backward of the residual addition with the root-mean-square norm: the formulas
// and the pipeline are described in norm.cuh.
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
template <typename TX, typename TR, int V, bool RING, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, norm_blocks(RING || kNextInRegisters<TR, V, RING, NV, MAXT>, NV, MAXT)) add_norm_bwd_kernel(AddNormBwdParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[2][kNormMaxThreads / 32];
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
    const float r = rn;
    if (row + step < p.rows) rn = p.rstd[row + step];
    if constexpr (RING) {
      __syncwarp();   // every lane has read the slot that is filled now
      copy();
      cp_async_wait<Ring::kDepth - 1>();
      __syncwarp();
    }
    float dot = 0.0f;
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
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float ah = a[j] * b[j];
        dw[i][j] = fmaf(ah, r, dw[i][j]);
        dot = fmaf(ah, w[i][j], dot);
      }
    }
    dot = rg.sum(dot, red[turn]);
    const float k = r * r * (dot * p.inv_d);
    uint4 numbers[NV];
    if (p.dx && p.rng.threshold)
      drop_numbers<V>(numbers, lane, G, (uint32_t)row, p.rng, xch + rg.group * G, sync);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<V>(i, lane, G);
      const bool in = c < d && live;
      float a[8], b[8];
      widen8(yr[i], a);
      widen8(hr[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = r * (a[j] * w[i][j] - b[j] * k);
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
  float* out = p.partial + (int64_t)blockIdx.x * d;
  if (rg.per > 1) {   // the row groups' sums, added in their order
    float* all = RING ? reinterpret_cast<float*>(smem) : reinterpret_cast<float*>(xch);
    const int width = G * NV * 8;
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) all[rg.group * width + column_of<V>(first_column<V>(i, lane, G), j, G)] = dw[i][j];
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
        if (column_of<V>(c, j, G) < d) out[column_of<V>(c, j, G)] = dw[i][j];
    }
  }
}

// dw[c] = sum of the partial rows, 32 columns a block: 32 warps take every
// 32nd row, their sums are added in warp order.
__global__ void __launch_bounds__(1024) add_norm_dw_kernel(const float* __restrict__ partial,
                                                           int n_partial, int d,
                                                           float* __restrict__ dw) {
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
  if (lane == 0 && blockIdx.x * 32 + warp < d) dw[blockIdx.x * 32 + warp] = sum;
}

template <typename TX, typename TR, int V, bool RING, int NV, int MAXT>
cudaError_t bwd_run(const AddNormBwdParams& p, int threads, int* blocks, cudaStream_t s) {
  auto* kernel = &add_norm_bwd_kernel<TX, TR, V, RING, NV, MAXT>;
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
template <typename TX, typename TR, int V>
cudaError_t bwd_types(const AddNormBwdParams& p, int* blocks, cudaStream_t s) {
  constexpr bool wide = V == 8 && RowRing<8 * (sizeof(TX) + 2 * sizeof(TR)), 4>::kFits512;
  AddNormBwdParams q = p;
  RowSplit split = V == 8 ? RowSplit(p.d, 2, wide ? 4 : 2, 512) : RowSplit(p.d, 1, 1, kNormMaxThreads);
  q.group = split.group;
  if (split.group) {
    const int threads = split.threads();
    if constexpr (wide) {
      if (split.nv == 3) return bwd_run<TX, TR, V, true, 3, 512>(q, threads, blocks, s);
      if (split.nv == 4) return bwd_run<TX, TR, V, true, 4, 512>(q, threads, blocks, s);
    }
    if constexpr (V == 8) {
      if (split.nv == 2 && split.group <= kNormThreads)
        return bwd_run<TX, TR, V, true, 2, kNormThreads>(q, threads, blocks, s);
      return split.nv == 1 ? bwd_run<TX, TR, V, true, 1, kNormThreads>(q, threads, blocks, s)
                           : bwd_run<TX, TR, V, true, 2, 512>(q, threads, blocks, s);
    } else {
      if (split.group > 512) return bwd_run<TX, TR, V, false, 1, kNormMaxThreads>(q, threads, blocks, s);
      return split.group <= kNormThreads ? bwd_run<TX, TR, V, false, 1, kNormThreads>(q, threads, blocks, s)
                                         : bwd_run<TX, TR, V, false, 1, 512>(q, threads, blocks, s);
    }
  }
  split = RowSplit(p.d, wide ? 3 : 2, 4, kNormMaxThreads);
  q.group = split.group;
  if constexpr (!wide)
    if (split.nv == 2) return bwd_run<TX, TR, V, false, 2, kNormMaxThreads>(q, q.group, blocks, s);
  return split.nv == 3 ? bwd_run<TX, TR, V, false, 3, kNormMaxThreads>(q, q.group, blocks, s)
                       : bwd_run<TX, TR, V, false, 4, kNormMaxThreads>(q, q.group, blocks, s);
}

template <typename TX, typename TR>
cudaError_t bwd_vec(const AddNormBwdParams& p, int vec, int* blocks, cudaStream_t s) {
  return vec == 8   ? bwd_types<TX, TR, 8>(p, blocks, s)
         : vec == 2 ? bwd_types<TX, TR, 2>(p, blocks, s)
                    : bwd_types<TX, TR, 1>(p, blocks, s);
}

}  // namespace

cudaError_t launch_add_norm_bwd(const AddNormBwdParams& p, int dtype, int res_dtype, int vec, float* dw,
                                cudaStream_t s) {
  const bool same = dtype == res_dtype;
  int blocks = 0;
  cudaError_t e;
  if (dtype == MOE_DT_BF16)
    e = same ? bwd_vec<__nv_bfloat16, __nv_bfloat16>(p, vec, &blocks, s)
             : bwd_vec<__nv_bfloat16, float>(p, vec, &blocks, s);
  else if (dtype == MOE_DT_F16)
    e = same ? bwd_vec<__half, __half>(p, vec, &blocks, s) : bwd_vec<__half, float>(p, vec, &blocks, s);
  else
    e = bwd_vec<float, float>(p, vec, &blocks, s);
  if (e != cudaSuccess || dw == nullptr) return e;
  return launch_pdl(add_norm_dw_kernel, dim3((unsigned)((p.d + 31) / 32)), dim3(1024), 0, s,
                    static_cast<const float*>(p.partial), blocks, p.d, dw);
}

}  // namespace moe
