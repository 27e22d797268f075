// 4-bit weights with group scales (sm_103a): quantiser, products with a few
// vectors, and the SwiGLU experts of a few tokens.
//
//   W[n, k] = (code[n, k] - 8) * scale[n, k / G],   G = 32, 64 or 128
// Two codes a byte, the even column in the low nibble; row-major, so one row of
// K columns is K/2 contiguous bytes.
//
// Bound by the weights' bytes: every weight is read once and used for a handful
// of tokens.  The products run on mma.sync m16n8k16 with 16 weight rows as A and
// eight tokens as B: the tensor core only has to keep up with HBM here, and the
// fragment form lets each lane turn its own 4-bit words into operands without
// shared memory.  The sum over k may visit columns in any order as long as A
// and B agree, so a lane's fragment columns are simply those of the words it
// loaded.  Products of a group are exact integers times activations, summed in
// fp32; the group's scale multiplies the fp32 sum.
#include "block.cuh"
#include "block.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kW4Warps = 8;   // warps of a block; they split K

// ------------------------------------------------------------------ fragments
template <typename T> struct MmaT;
template <> struct MmaT<__nv_bfloat16> {
  // 128 + code is exact in bf16 (0x4300 = 128); 136 = 128 + 8
  static MOE_DEV uint32_t widen(uint32_t nibbles) {
    uint32_t v = (nibbles & 0x000F000Fu) | 0x43004300u;
    __nv_bfloat162 h = *reinterpret_cast<__nv_bfloat162*>(&v);
    h = __hsub2(h, __floats2bfloat162_rn(136.0f, 136.0f));
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static MOE_DEV void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};
template <> struct MmaT<__half> {
  // 1024 + code is exact in fp16 (0x6400 = 1024); 1032 = 1024 + 8
  static MOE_DEV uint32_t widen(uint32_t nibbles) {
    uint32_t v = (nibbles & 0x000F000Fu) | 0x64006400u;
    __half2 h = *reinterpret_cast<__half2*>(&v);
    h = __hsub2(h, __floats2half2_rn(1032.0f, 1032.0f));
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static MOE_DEV void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

template <int W> struct Words { uint32_t w[W]; };
template <int W> MOE_DEV Words<W> load_words(const uint32_t* p) {
  Words<W> r;
  if constexpr (W == 4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
    r.w[0] = __ldg(p);
  }
  return r;
}

// One group of 32 W columns of 16 weight rows (this lane's words of rows g and
// g + 8) times NT tiles of eight vectors.  xp[j]: this lane's vector of tile j
// at the lane's first column of the group, or NULL (a vector that is not there).
template <typename T, int W, int NT>
MOE_DEV void group_mma(const Words<W>& wa, const Words<W>& wb, const T* const* xp, int64_t col,
                       float (*c)[4]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {   // columns (q, q + 4) of the word's eight
      a[q] = MmaT<T>::widen(wa.w[i] >> (4 * q));
      b[q] = MmaT<T>::widen(wb.w[i] >> (4 * q));
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (xp[j]) x = __ldg(reinterpret_cast<const uint4*>(xp[j] + col) + i);
      const uint32_t x04 = __byte_perm(x.x, x.z, 0x5410), x15 = __byte_perm(x.x, x.z, 0x7632);
      const uint32_t x26 = __byte_perm(x.y, x.w, 0x5410), x37 = __byte_perm(x.y, x.w, 0x7632);
      MmaT<T>::mma(c[j], a[0], b[0], a[1], b[1], x04, x15);
      MmaT<T>::mma(c[j], a[2], b[2], a[3], b[3], x26, x37);
    }
  }
}

// 16 weight rows (ra, rb: this lane's rows g and g + 8; sa, sb their scales)
// times NT tiles of vectors over the groups first, first + step, ... < groups.
template <typename T, typename S, int W, int NT>
MOE_DEV void rows_product(const uint32_t* ra, const uint32_t* rb, const S* sa, const S* sb,
                          const T* const* xp, int first, int step, int groups, float (*acc)[4]) {
  constexpr int U = 4;
  const int t = threadIdx.x & 3;
  for (int q0 = first; q0 < groups; q0 += step * U) {
    Words<W> wa[U], wb[U];
    float fa[U], fb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + u * step;
      if (q < groups) {
        wa[u] = load_words<W>(ra + (int64_t)q * (4 * W) + t * W);
        wb[u] = load_words<W>(rb + (int64_t)q * (4 * W) + t * W);
        fa[u] = Elem<S>::to_f(sa[q]);
        fb[u] = Elem<S>::to_f(sb[q]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + u * step;
      if (q < groups) {
        float c[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) c[j][i] = 0.0f;
        group_mma<T, W, NT>(wa[u], wb[u], xp, (int64_t)q * (32 * W) + t * (8 * W), c);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[j][0] = fmaf(fa[u], c[j][0], acc[j][0]);
          acc[j][1] = fmaf(fa[u], c[j][1], acc[j][1]);
          acc[j][2] = fmaf(fb[u], c[j][2], acc[j][2]);
          acc[j][3] = fmaf(fb[u], c[j][3], acc[j][3]);
        }
      }
    }
  }
}

// Accumulators of all warps to shared memory: red[warp][tile][row 16][vector 8].
template <int NT>
MOE_DEV void store_partials(float (*acc)[4], float (*red)[NT][16][8]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    *reinterpret_cast<float2*>(&red[warp][j][g][2 * t]) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(&red[warp][j][g + 8][2 * t]) = make_float2(acc[j][2], acc[j][3]);
  }
}

// ------------------------------------------------------------------ matvec
template <typename T, int W, int NT>
__global__ void __launch_bounds__(kW4Warps * 32) matvec_w4_kernel(
    int M, int N, int K, const T* __restrict__ x, int64_t ld_x, const uint8_t* __restrict__ wq,
    const T* __restrict__ ws, T* __restrict__ y, int64_t ld_y) {
  pdl_begin();
  __shared__ float red[kW4Warps][NT][16][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int m0 = blockIdx.x * (8 * NT);
  const int64_t n0 = (int64_t)blockIdx.y * 16;
  const int groups = K / (32 * W);
  // rows past N read row N - 1 and are not written
  const int64_t na = min(n0 + g, (int64_t)N - 1), nb = min(n0 + g + 8, (int64_t)N - 1);
  const T* xp[NT];
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int m = m0 + j * 8 + g;
    xp[j] = m < M ? x + m * ld_x : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
  }
  rows_product<T, T, W, NT>(reinterpret_cast<const uint32_t*>(wq + na * (K / 2)),
                            reinterpret_cast<const uint32_t*>(wq + nb * (K / 2)), ws + na * groups,
                            ws + nb * groups, xp, warp, kW4Warps, groups, acc);
  store_partials<NT>(acc, red);
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 128; i += kW4Warps * 32) {
    const int row = i & 15, col = i >> 4;   // col: vector within the block's 8 NT
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kW4Warps; ++w) s += red[w][col >> 3][row][col & 7];
    if (m0 + col < M && n0 + row < N) y[(m0 + col) * ld_y + n0 + row] = Elem<T>::from_f(s);
  }
  (void)t;
}

// ------------------------------------------------------------------ experts
// The routes of expert e, in `list`; returns their count.  Every thread calls.
MOE_DEV int gather_routes(const int32_t* idx, int R, int e, int32_t* list, int32_t* count) {
  if (threadIdx.x == 0) *count = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < R; r += blockDim.x)
    if (idx[r] == e) list[atomicAdd(count, 1)] = r;   // the order changes no result
  __syncthreads();
  return *count;
}

// The expert of grid row y: expert y, or (fewer routes than experts) the expert
// of route y when no earlier route has it.  -1: nothing to do.
MOE_DEV int block_expert(const int32_t* idx, int R, int E, int y) {
  if (R >= E) return y;
  const int e = idx[y];
  if (e < 0 || e >= E) return -1;
  for (int r = 0; r < y; ++r)
    if (idx[r] == e) return -1;
  return e;
}

// act[route] = silu(W_gate x) * (W_up x) as two bf16 parts (high, low): eight
// columns of d_ff a block; the fragment's rows are eight gate rows and the
// same eight up rows, so both products of a value meet in one lane's column.
template <typename T, int W, int NT>
__global__ void __launch_bounds__(kW4Warps * 32) experts_w4_up_kernel(ExpertsW4Params p) {
  pdl_begin();
  extern __shared__ int32_t list[];
  __shared__ float red[kW4Warps][NT][16][8];
  __shared__ int32_t count;
  const int R = p.T * p.k;
  const int e = block_expert(p.topk_idx, R, p.E, blockIdx.y);
  if (e < 0) return;
  const int n = gather_routes(p.topk_idx, R, e, list, &count);
  if (n == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2;
  const int groups = p.d / (32 * W);
  const int f0 = blockIdx.x * 8;
  const int64_t row = (int64_t)e * p.f + f0 + g;
  const uint32_t* ra = reinterpret_cast<const uint32_t*>(p.gate_q + row * (p.d / 2));
  const uint32_t* rb = reinterpret_cast<const uint32_t*>(p.up_q + row * (p.d / 2));
  const T* sa = static_cast<const T*>(p.gate_s) + row * groups;
  const T* sb = static_cast<const T*>(p.up_s) + row * groups;
  const T* x = static_cast<const T*>(p.x);
  __nv_bfloat16* hi = static_cast<__nv_bfloat16*>(p.act);
  __nv_bfloat16* lo = hi + (int64_t)R * p.f;
  for (int m0 = 0; m0 < n; m0 += 8 * NT) {
    const T* xp[NT];
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int m = m0 + j * 8 + g;
      xp[j] = m < n ? x + (int64_t)(list[m] / p.k) * p.ld_x : nullptr;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    }
    rows_product<T, T, W, NT>(ra, rb, sa, sb, xp, warp, kW4Warps, groups, acc);
    __syncthreads();   // the previous round of red has been read
    store_partials<NT>(acc, red);
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 64; i += kW4Warps * 32) {
      const int col = i >> 3, r8 = i & 7;
      if (m0 + col < n) {
        float h = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < kW4Warps; ++w) {
          h += red[w][col >> 3][r8][col & 7];
          u += red[w][col >> 3][r8 + 8][col & 7];
        }
        const float a = h / (1.0f + expf(-h)) * u;
        const __nv_bfloat16 ah = __float2bfloat16_rn(a);
        const int64_t at = (int64_t)list[m0 + col] * p.f + f0 + r8;
        hi[at] = ah;
        lo[at] = __float2bfloat16_rn(a - __bfloat162float(ah));
      }
    }
  }
}

// y[route] = gate * W_down act: 16 columns of d a block.  The two bf16 parts
// of the activations keep 16 bits of them, so storing them costs no accuracy
// beside the bf16 result.
template <typename S, int W, int NT>
__global__ void __launch_bounds__(kW4Warps * 32) experts_w4_down_kernel(ExpertsW4Params p) {
  pdl_begin();
  extern __shared__ int32_t list[];
  __shared__ float red[kW4Warps][NT][16][8];
  __shared__ int32_t count;
  const int R = p.T * p.k;
  const int e = block_expert(p.topk_idx, R, p.E, blockIdx.y);
  if (e < 0) return;
  const int n = gather_routes(p.topk_idx, R, e, list, &count);
  if (n == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2;
  const int groups = p.f / (32 * W);
  const int d0 = blockIdx.x * 16;
  const int64_t row = (int64_t)e * p.d + d0 + g;
  const uint32_t* ra = reinterpret_cast<const uint32_t*>(p.down_q + row * (p.f / 2));
  const uint32_t* rb = ra + (int64_t)8 * (p.f / 8);
  const S* sa = static_cast<const S*>(p.down_s) + row * groups;
  const S* sb = sa + (int64_t)8 * groups;
  const __nv_bfloat16* hi = static_cast<const __nv_bfloat16*>(p.act);
  for (int m0 = 0; m0 < n; m0 += 4 * NT) {
    // vectors of tile j: the high parts of four routes and their low parts
    const __nv_bfloat16* xp[NT];
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int m = m0 + j * 4 + (g & 3);
      xp[j] = m < n ? hi + ((int64_t)(g >> 2) * R + list[m]) * p.f : nullptr;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    }
    rows_product<__nv_bfloat16, S, W, NT>(ra, rb, sa, sb, xp, warp, kW4Warps, groups, acc);
    __syncthreads();
    store_partials<NT>(acc, red);
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 64; i += kW4Warps * 32) {
      const int col = i >> 4, r16 = i & 15;   // col: route within the block's 4 NT
      if (m0 + col < n) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kW4Warps; ++w)
          s += red[w][col >> 2][r16][col & 3] + red[w][col >> 2][r16][(col & 3) + 4];
        const int r = list[m0 + col];
        p.y[(int64_t)r * p.d + d0 + r16] = s * p.gates[r];
      }
    }
  }
}

// out[t] = sum of the routes' outputs in j order; a route without an expert
// (-1) adds nothing, an expert id out of range is reported and adds nothing.
template <typename T>
__global__ void __launch_bounds__(256) experts_w4_join_kernel(ExpertsW4Params p) {
  pdl_begin();
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int t = blockIdx.y;
  if (c >= p.d) return;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < p.k; ++j) {
    const int r = t * p.k + j;
    const int e = p.topk_idx[r];
    if (e >= 0 && e < p.E) {
      const float4 v = *reinterpret_cast<const float4*>(p.y + (int64_t)r * p.d + c);
      a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
    } else if (e != -1 && c == 0) {
      raise_error(p.err, MOE_DEVERR_BOUNDS);
    }
  }
  T* out = static_cast<T*>(p.out) + t * p.ld_out + c;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = Elem<T>::from_f(a[i]);
}

// ------------------------------------------------------------------ quantiser
// A thread takes eight columns, G / 8 lanes a group: scale = max|w| / 7 rounded
// to the weights' type, code = w / scale rounded to nearest even, plus 8.
template <typename T>
__global__ void __launch_bounds__(256) quantize_w4_kernel(int64_t n8, int group,
                                                          const T* __restrict__ src,
                                                          uint32_t* __restrict__ q,
                                                          T* __restrict__ scales) {
  pdl_begin();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int lanes = group / 8;
  float v[8];
  float amax = 0.0f;
  if (i < n8) {
    widen8(load8<T, true>(src + i * 8, 0, 8), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
  }
  for (int off = 1; off < lanes; off <<= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (i >= n8) return;
  const T st = Elem<T>::from_f(amax / 7.0f);
  const float s = Elem<T>::to_f(st);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float z = s > 0.0f ? rintf(v[j] / s) : 0.0f;
    w |= (uint32_t)((int)fminf(fmaxf(z, -8.0f), 7.0f) + 8) << (4 * j);
  }
  q[i] = w;
  if (i % lanes == 0) scales[i / lanes] = st;
}

template <typename T>
__global__ void __launch_bounds__(256) dequantize_w4_kernel(int64_t n8, int group,
                                                            const uint32_t* __restrict__ q,
                                                            const T* __restrict__ scales,
                                                            float4* __restrict__ out) {
  pdl_begin();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const uint32_t w = q[i];
  const float s = Elem<T>::to_f(scales[i / (group / 8)]);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)((int)((w >> (4 * j)) & 15u) - 8) * s;
  out[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
  out[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename T, int W>
cudaError_t matvec_nt(int M, int N, int K, const void* x, int64_t ld_x, const uint8_t* q,
                      const void* sc, void* y, int64_t ld_y, cudaStream_t s) {
  const int nt = M <= 8 ? 1 : M <= 16 ? 2 : 4;
  const dim3 grid((unsigned)((M + 8 * nt - 1) / (8 * nt)), (unsigned)((N + 15) / 16));
  const dim3 block(kW4Warps * 32);
  const T *xt = static_cast<const T*>(x), *st = static_cast<const T*>(sc);
  T* yt = static_cast<T*>(y);
  if (nt == 1)
    return launch_pdl(matvec_w4_kernel<T, W, 1>, grid, block, 0, s, M, N, K, xt, ld_x, q, st, yt, ld_y);
  if (nt == 2)
    return launch_pdl(matvec_w4_kernel<T, W, 2>, grid, block, 0, s, M, N, K, xt, ld_x, q, st, yt, ld_y);
  return launch_pdl(matvec_w4_kernel<T, W, 4>, grid, block, 0, s, M, N, K, xt, ld_x, q, st, yt, ld_y);
}

template <typename T, int W>
cudaError_t experts_nt(const ExpertsW4Params& p, cudaStream_t s) {
  const int R = p.T * p.k;
  const unsigned gy = (unsigned)(R < p.E ? R : p.E);
  const size_t smem = (size_t)R * 4;
  const dim3 block(kW4Warps * 32);
  cudaError_t e;
  if (p.T <= 8)
    e = launch_pdl(experts_w4_up_kernel<T, W, 1>, dim3(p.f / 8, gy), block, smem, s, p);
  else
    e = launch_pdl(experts_w4_up_kernel<T, W, 2>, dim3(p.f / 8, gy), block, smem, s, p);
  if (e != cudaSuccess) return e;
  if (p.T <= 4)
    e = launch_pdl(experts_w4_down_kernel<T, W, 1>, dim3(p.d / 16, gy), block, smem, s, p);
  else
    e = launch_pdl(experts_w4_down_kernel<T, W, 2>, dim3(p.d / 16, gy), block, smem, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(experts_w4_join_kernel<T>, dim3((p.d + 1023) / 1024, p.T), dim3(256), 0, s, p);
}

template <typename T>
cudaError_t experts_group(const ExpertsW4Params& p, cudaStream_t s) {
  if (p.group == 32) return experts_nt<T, 1>(p, s);
  if (p.group == 64) return experts_nt<T, 2>(p, s);
  return experts_nt<T, 4>(p, s);
}

template <typename T>
cudaError_t matvec_group(int M, int N, int K, int group, const void* x, int64_t ld_x,
                         const uint8_t* q, const void* sc, void* y, int64_t ld_y, cudaStream_t s) {
  if (group == 32) return matvec_nt<T, 1>(M, N, K, x, ld_x, q, sc, y, ld_y, s);
  if (group == 64) return matvec_nt<T, 2>(M, N, K, x, ld_x, q, sc, y, ld_y, s);
  return matvec_nt<T, 4>(M, N, K, x, ld_x, q, sc, y, ld_y, s);
}

}  // namespace

cudaError_t launch_quantize_w4(int64_t rows, int K, int group, int dtype, const void* src,
                               uint8_t* q, void* scales, cudaStream_t s) {
  const int64_t n8 = rows * (K / 8);
  const dim3 grid((unsigned)((n8 + 255) / 256));
  uint32_t* qw = reinterpret_cast<uint32_t*>(q);
  if (dtype == MOE_DT_BF16)
    return launch_pdl(quantize_w4_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, n8, group,
                      static_cast<const __nv_bfloat16*>(src), qw, static_cast<__nv_bfloat16*>(scales));
  return launch_pdl(quantize_w4_kernel<__half>, grid, dim3(256), 0, s, n8, group,
                    static_cast<const __half*>(src), qw, static_cast<__half*>(scales));
}

cudaError_t launch_dequantize_w4(int64_t rows, int K, int group, int dtype, const uint8_t* q,
                                 const void* scales, float* out, cudaStream_t s) {
  const int64_t n8 = rows * (K / 8);
  const dim3 grid((unsigned)((n8 + 255) / 256));
  const uint32_t* qw = reinterpret_cast<const uint32_t*>(q);
  float4* o = reinterpret_cast<float4*>(out);
  if (dtype == MOE_DT_BF16)
    return launch_pdl(dequantize_w4_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, n8, group, qw,
                      static_cast<const __nv_bfloat16*>(scales), o);
  return launch_pdl(dequantize_w4_kernel<__half>, grid, dim3(256), 0, s, n8, group, qw,
                    static_cast<const __half*>(scales), o);
}

cudaError_t launch_matvec_w4(int M, int N, int K, int group, int dtype, const void* x, int64_t ld_x,
                             const uint8_t* q, const void* scales, void* y, int64_t ld_y,
                             cudaStream_t s) {
  return dtype == MOE_DT_BF16
             ? matvec_group<__nv_bfloat16>(M, N, K, group, x, ld_x, q, scales, y, ld_y, s)
             : matvec_group<__half>(M, N, K, group, x, ld_x, q, scales, y, ld_y, s);
}

cudaError_t launch_experts_w4(const ExpertsW4Params& p, int dtype, cudaStream_t s) {
  return dtype == MOE_DT_BF16 ? experts_group<__nv_bfloat16>(p, s) : experts_group<__half>(p, s);
}

}  // namespace moe
