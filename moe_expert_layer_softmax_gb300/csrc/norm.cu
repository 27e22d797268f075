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
// row stays in registers between the pass that sums it and the pass that writes
// it.  A fixed grid takes the rows in turn; where a thread holds eight columns,
// the rows to come (one or three, kept at 48 KB or more a multiprocessor) are on
// their way into shared memory, each thread copying and reading its own pieces,
// so that the pipeline needs no barrier and no registers.  Sums are taken in a
// fixed order (no atomics).
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
// the same value in every thread.  `red`: one float per warp, another array in
// turn for the next call, so that one barrier is enough.  Every thread calls.
MOE_DEV float group_sum(float v, int G, float* red) {
  v = warp_sum(v);
  if (G == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int n = G >> 5;   // <= 32
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < n ? red[(threadIdx.x / G) * n + lane] : 0.0f);
}

template <bool VEC>
MOE_DEV void load_weight8(const void* w, bool w_f32, bool w_f16, int c, int G, int d, float* f) {
  if (w_f32) {
    widen8(load8<float, VEC>(static_cast<const float*>(w), c, G, d), f);
  } else if (w_f16) {
    widen8(load8<__half, VEC>(static_cast<const __half*>(w), c, G, d), f);
  } else {
    widen8(load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w), c, G, d), f);
  }
}

// A thread's pieces (eight columns of each of up to three matrices) of the rows
// to come: cp.async into slots of its own.  Slots are laid out piece by piece
// (16 bytes a thread), so that neighbouring threads touch neighbouring banks.
// Two rows where a thread's pieces are large, else four: 96 KB at 512 threads.
template <int BYTES> struct RowRing {
  static constexpr int kDepth = BYTES <= 48 ? 4 : 2;
  static constexpr int kPieces = BYTES / 16;
  uint32_t mine;     // slot 0, piece 0
  uint32_t piece;    // bytes between pieces
  uint32_t slot;     // bytes: the next one to read
  MOE_DEV explicit RowRing(void* smem)
      : mine(smem_u32(smem) + threadIdx.x * 16), piece(blockDim.x * 16), slot(0) {}
  MOE_DEV uint32_t size() const { return piece * kPieces; }
  MOE_DEV uint32_t after(uint32_t at, int rows) const {
    at += rows * size();
    return at >= kDepth * size() ? at - kDepth * size() : at;
  }
  template <typename T> MOE_DEV static void put(uint32_t at, uint32_t piece, const T* from) {
    constexpr int n = sizeof(T) / 2;
#pragma unroll
    for (int i = 0; i < n; ++i) cp_async16(at + i * piece, reinterpret_cast<const uint8_t*>(from) + i * 16);
  }
  template <typename T> MOE_DEV static Raw8<T> get(uint32_t at, uint32_t piece) {
    Raw8<T> r;
    uint4* q = reinterpret_cast<uint4*>(&r);
    constexpr int n = sizeof(T) / 2;
#pragma unroll
    for (int i = 0; i < n; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w) : "r"(at + i * piece));
    return r;
  }
};

// One row group of G threads per row; each thread holds NV times eight columns.
// MX: codes, scales and (dq) their values instead of y; rows at or past `rows`
// are the padding of the last 128-row tile.
template <typename TX, typename TR, bool MX, bool VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, VEC ? 1024 / MAXT : 1) add_norm_kernel(AddNormParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr bool RING = VEC && NV == 1;
  using Ring = RowRing<8 * (sizeof(TX) + sizeof(TR))>;
  __shared__ float red[2][kNormMaxThreads / 32];
  __shared__ uint4 xch[VEC ? 1 : MAXT];
  pdl_begin();
  const int G = p.group;
  const int lane = threadIdx.x & (G - 1);
  const int per = blockDim.x / G, group = threadIdx.x / G;
  const int d = p.d;
  float w[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first_column<VEC>(i, lane, G);
    if (c < d) load_weight8<VEC>(p.weight, p.w_f32, sizeof(TX) == 2 && p.x_f16, c, G, d, w[i]);
  }
  auto sync = [&]() {
    if (G == 32) __syncwarp(); else __syncthreads();
  };
  const int64_t last = MX ? p.rows_pad : p.rows, step = (int64_t)gridDim.x * per;
  int64_t row0 = (int64_t)blockIdx.x * per;
  Ring ring(smem);
  const int c0 = lane * 8;
  auto copy = [&](int64_t row, uint32_t slot) {
    if (row < p.rows && c0 < d) {
      const uint32_t at = ring.mine + slot;
      Ring::put(at, ring.piece, static_cast<const TX*>(p.x) + row * p.ld_x + c0);
      if (p.residual)
        Ring::put(at + sizeof(TX) / 2 * ring.piece, ring.piece, static_cast<const TR*>(p.residual) + row * p.ld_residual + c0);
    }
    cp_async_commit();
  };
  if constexpr (RING) {
    for (int i = 0; i < Ring::kDepth - 1; ++i) copy(row0 + group + i * step, i * ring.size());
  }
  for (int turn = 0; row0 < last; row0 += step, turn ^= 1) {
    const int64_t row = row0 + group;
    const bool live = row < p.rows;
    float h[NV][8];
    Raw8<TX> xr[NV];
    Raw8<TR> rr[NV];
    if constexpr (RING) {
      copy(row + (Ring::kDepth - 1) * step, ring.after(ring.slot, Ring::kDepth - 1));
      cp_async_wait<Ring::kDepth - 1>();
      const uint32_t at = ring.mine + ring.slot;
      xr[0] = Ring::template get<TX>(at, ring.piece);
      if (p.residual) rr[0] = Ring::template get<TR>(at + sizeof(TX) / 2 * ring.piece, ring.piece);
      ring.slot = ring.after(ring.slot, 1);
    } else if (live) {
      const TX* x = static_cast<const TX*>(p.x) + row * p.ld_x;
      const TR* res = static_cast<const TR*>(p.residual) + row * p.ld_residual;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = first_column<VEC>(i, lane, G);
        if (c < d) {
          xr[i] = load8<TX, VEC>(x, c, G, d);
          if (p.residual) rr[i] = load8<TR, VEC>(res, c, G, d);
        }
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<VEC>(i, lane, G);
      uint4 numbers;
      if (p.rng.threshold) numbers = drop_numbers_of<VEC>(i, lane, G, (uint32_t)row, p.rng, xch + group * G, sync);
      if (c < d && live) {
        widen8(xr[i], h[i]);
        if (p.rng.threshold) drop8(h[i], numbers, p.rng);
        if (p.residual) {
          float f[8];
          widen8(rr[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += f[j];
        }
        if (p.h) {
          const Raw8<TR> hr = narrow8<TR>(h[i]);
          store8<TR, VEC>(static_cast<TR*>(p.h) + row * p.ld_h, c, G, d, hr);
          widen8(hr, h[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
      }
    }
    ss = group_sum(ss, G, red[turn]);
    const float rstd = __frsqrt_rn(ss / (float)d + p.eps);
    if (live && lane == 0 && p.rstd) p.rstd[row] = rstd;
    if (!MX) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = first_column<VEC>(i, lane, G);
        if (c < d && live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] = (h[i][j] * w[i][j]) * rstd;
          store8<TX, VEC>(static_cast<TX*>(p.y) + row * p.ld_y, c, G, d, narrow8<TX>(h[i]));
        }
      }
    } else {
      // d is a multiple of 128: the four lanes of a 32-column block are all live
      // or all past the row's end
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = first_column<VEC>(i, lane, G);
        float amax = 0.0f;
        if (c < d && live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h[i][j] = (h[i][j] * w[i][j]) * rstd;
            amax = fmaxf(amax, fabsf(h[i][j]));
          }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int s = mx_scale_exp(amax);
        // the scales of four neighbouring blocks are four neighbouring bytes
        uint32_t four = (uint32_t)(s + 127) << (8 * ((lane >> 2) & 3));
        four |= __shfl_xor_sync(0xffffffffu, four, 4);
        four |= __shfl_xor_sync(0xffffffffu, four, 8);
        if (c < d && row < last) {
          uint2 q = make_uint2(0, 0);
          if (live) {
            const float inv = exp2i(-s);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = h[i][j] * inv;
            q = e4m3x8(v);
          }
          *reinterpret_cast<uint2*>(p.y_q + row * d + c) = q;
          if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.y_scales + sf_offset(row, c >> 5, d >> 5)) = four;
          if (p.y_dq) {
            const float up = exp2i(s);
            float v[8];
            e4m3x2_to_f32(q.x, v[0], v[1]);
            e4m3x2_to_f32(q.x >> 16, v[2], v[3]);
            e4m3x2_to_f32(q.y, v[4], v[5]);
            e4m3x2_to_f32(q.y >> 16, v[6], v[7]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= up;
            store8<__nv_bfloat16, true>(static_cast<__nv_bfloat16*>(p.y_dq) + row * d, c, 1, d,
                                        narrow8<__nv_bfloat16>(v));
          }
        }
      }
    }
  }
}

// Backward: the weight gradient of a block's rows stays in registers; one row of
// partial sums a block goes to `partial` [gridDim.x, d].
template <typename TX, typename TR, bool VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, VEC ? 1024 / MAXT : 1) add_norm_bwd_kernel(AddNormBwdParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr bool RING = VEC && NV == 1;
  using Ring = RowRing<8 * (sizeof(TX) + 2 * sizeof(TR))>;
  __shared__ float red[2][kNormMaxThreads / 32];
  __shared__ uint4 xch[MAXT];
  pdl_begin();
  const int G = p.group;
  const int lane = threadIdx.x & (G - 1);
  const int per = blockDim.x / G, group = threadIdx.x / G;
  const int d = p.d;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first_column<VEC>(i, lane, G);
    if (c < d) load_weight8<VEC>(p.weight, p.w_f32, sizeof(TX) == 2 && p.x_f16, c, G, d, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  auto sync = [&]() {
    if (G == 32) __syncwarp(); else __syncthreads();
  };
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t row0 = (int64_t)blockIdx.x * per;
  Ring ring(smem);
  const int c0 = lane * 8;
  auto copy = [&](int64_t row, uint32_t slot) {
    if (row < p.rows && c0 < d) {
      const uint32_t at = ring.mine + slot;
      Ring::put(at, ring.piece, static_cast<const TX*>(p.dy) + row * p.ld_dy + c0);
      Ring::put(at + sizeof(TX) / 2 * ring.piece, ring.piece, static_cast<const TR*>(p.h) + row * p.ld_h + c0);
      if (p.dres)
        Ring::put(at + (sizeof(TX) + sizeof(TR)) / 2 * ring.piece, ring.piece,
                  static_cast<const TR*>(p.dres) + row * p.ld_dres + c0);
    }
    cp_async_commit();
  };
  if constexpr (RING) {
    for (int i = 0; i < Ring::kDepth - 1; ++i) copy(row0 + group + i * step, i * ring.size());
  }
  float rn = row0 + group < p.rows ? p.rstd[row0 + group] : 0.0f;
  for (int turn = 0; row0 < p.rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + group;
    const bool live = row < p.rows;
    Raw8<TX> yr[NV];
    Raw8<TR> hr[NV], dr[NV];
    const float r = rn;
    if (row + step < p.rows) rn = p.rstd[row + step];
    if constexpr (RING) {
      copy(row + (Ring::kDepth - 1) * step, ring.after(ring.slot, Ring::kDepth - 1));
      cp_async_wait<Ring::kDepth - 1>();
      const uint32_t at = ring.mine + ring.slot;
      yr[0] = Ring::template get<TX>(at, ring.piece);
      hr[0] = Ring::template get<TR>(at + sizeof(TX) / 2 * ring.piece, ring.piece);
      if (p.dres) dr[0] = Ring::template get<TR>(at + (sizeof(TX) + sizeof(TR)) / 2 * ring.piece, ring.piece);
      ring.slot = ring.after(ring.slot, 1);
    } else if (live) {
      const TX* dy = static_cast<const TX*>(p.dy) + row * p.ld_dy;
      const TR* h = static_cast<const TR*>(p.h) + row * p.ld_h;
      const TR* dres = static_cast<const TR*>(p.dres) + row * p.ld_dres;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = first_column<VEC>(i, lane, G);
        if (c < d) {
          yr[i] = load8<TX, VEC>(dy, c, G, d);
          hr[i] = load8<TR, VEC>(h, c, G, d);
          if (p.dres) dr[i] = load8<TR, VEC>(dres, c, G, d);
        }
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<VEC>(i, lane, G);
      if (c < d && live) {
        float a[8], b[8];
        widen8(yr[i], a);
        widen8(hr[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float ah = a[j] * b[j];
          dw[i][j] = fmaf(ah, r, dw[i][j]);
          dot = fmaf(ah, w[i][j], dot);   // columns past d hold zeros
        }
      }
    }
    dot = group_sum(dot, G, red[turn]);
    if (!p.dh && !p.dx) continue;
    const float k = r * r * (dot / (float)d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<VEC>(i, lane, G);
      uint4 numbers;
      if (p.dx && p.rng.threshold) numbers = drop_numbers_of<VEC>(i, lane, G, (uint32_t)row, p.rng, xch + group * G, sync);
      if (c < d && live) {
        float a[8], b[8];
        widen8(yr[i], a);
        widen8(hr[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = r * (a[j] * w[i][j] - b[j] * k);
        if (p.dres) {
          widen8(dr[i], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] += b[j];
        }
        if (p.dh) store8<TR, VEC>(static_cast<TR*>(p.dh) + row * p.ld_dh, c, G, d, narrow8<TR>(a));
        if (p.dx) {
          if (p.rng.threshold) drop8(a, numbers, p.rng);
          store8<TX, VEC>(static_cast<TX*>(p.dx) + row * p.ld_dx, c, G, d, narrow8<TX>(a));
        }
      }
    }
  }
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * d;
  const int cs = column_step<VEC>(G);
  if (per > 1) {   // NV is 1: the row groups' sums, added in their order
    float* all = reinterpret_cast<float*>(xch);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) all[group * 8 * G + first_column<VEC>(0, lane, G) + j * cs] = dw[0][j];
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
      float s = 0.0f;
      for (int g = 0; g < per; ++g) s += all[g * 8 * G + c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<VEC>(i, lane, G);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j * cs < d) out[c + j * cs] = dw[i][j];
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

// y = dropout(x): a warp takes 256 columns of two rows at a time.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(DropoutParams p) {
  __shared__ uint4 xch[VEC ? 1 : 256];
  pdl_begin();
  constexpr int U = 2;
  const int lane = threadIdx.x;
  auto sync = []() { __syncwarp(); };
  for (int64_t row = ((int64_t)blockIdx.y * 8 + threadIdx.y) * U; row < p.rows; row += (int64_t)gridDim.y * 8 * U) {
    const int n = (int)min((int64_t)U, p.rows - row);
    for (int64_t i = blockIdx.x; i * 256 < p.cols; i += gridDim.x) {
      const int c = first_column<VEC>((int)i, lane, 32);
      Raw8<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < n && c < p.cols)
          raw[u] = load8<T, VEC>(static_cast<const T*>(p.x) + (row + u) * p.ld_x, c, 32, p.cols);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= n) break;
        float f[8];
        uint4 numbers;
        if (p.rng.threshold)
          numbers = drop_numbers_of<VEC>((int)i, lane, 32, (uint32_t)(row + u), p.rng, xch + (VEC ? 0 : threadIdx.y * 32), sync);
        if (c < p.cols) {
          widen8(raw[u], f);
          if (p.rng.threshold) drop8(f, numbers, p.rng);
          store8<T, VEC>(static_cast<T*>(p.y) + (row + u) * p.ld_y, c, 32, p.cols, narrow8<T>(f));
        }
      }
    }
  }
}

// Threads of a row group, a power of two of at least a warp, and how many times
// eight columns each holds: one as far as a block goes.
void row_split(int d, int* group, int* nv) {
  const int g8 = (d + 7) / 8;
  int G = 32;
  while (G < kNormMaxThreads && G < g8) G *= 2;
  int n = 1;
  while (n * G < g8) n *= 2;
  *group = G;
  *nv = n;
}

// Blocks: enough row groups for every row, or kNormThreadsPerSm threads a
// multiprocessor.
constexpr int kNormThreadsPerSm = 1024;
void row_grid(int64_t rows, int group, int* blocks, int* threads) {
  *threads = group < kNormThreads ? kNormThreads : group;
  const int per = *threads / group;
  const int64_t need = (rows + per - 1) / per;
  const int64_t most = (int64_t)device_info()->sm_count * (kNormThreadsPerSm / *threads);
  *blocks = (int)(need < most ? need : most);
}

// p = NULL: raise the kernel's shared memory limit.
template <typename P, typename F>
cudaError_t run_rows(F* kernel, const P* p, int64_t rows, int ring_bytes, int depth, cudaStream_t s) {
  if (p == nullptr)
    return ring_bytes == 0 ? cudaSuccess
                           : cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  kNormMaxThreads * ring_bytes * depth);
  int blocks, threads;
  row_grid(rows, p->group, &blocks, &threads);
  return launch_pdl(kernel, dim3(blocks), dim3(threads), (size_t)threads * ring_bytes * depth, s, *p);
}

template <typename TX, typename TR, bool MX, bool VEC, int NV, int MAXT>
cudaError_t fwd_run(const AddNormParams* p, cudaStream_t s) {
  constexpr int bytes = VEC && NV == 1 ? 8 * (sizeof(TX) + sizeof(TR)) : 0;
  return run_rows(&add_norm_kernel<TX, TR, MX, VEC, NV, MAXT>, p, p ? (MX ? p->rows_pad : p->rows) : 0, bytes,
                  RowRing<8 * (sizeof(TX) + sizeof(TR))>::kDepth, s);
}
template <typename TX, typename TR, bool VEC, int NV, int MAXT>
cudaError_t bwd_run(const AddNormBwdParams* p, cudaStream_t s) {
  constexpr int bytes = VEC && NV == 1 ? 8 * (sizeof(TX) + 2 * sizeof(TR)) : 0;
  return run_rows(&add_norm_bwd_kernel<TX, TR, VEC, NV, MAXT>, p, p ? p->rows : 0, bytes,
                  RowRing<8 * (sizeof(TX) + 2 * sizeof(TR))>::kDepth, s);
}

template <typename TX, typename TR, bool MX, bool VEC>
cudaError_t fwd_nv(const AddNormParams* p, int nv, cudaStream_t s) {
  if (p == nullptr) {
    const cudaError_t e = fwd_run<TX, TR, MX, VEC, 1, 512>(p, s);
    return e == cudaSuccess ? fwd_run<TX, TR, MX, VEC, 1, 1024>(p, s) : e;
  }
  if (nv == 1) return p->group <= 512 ? fwd_run<TX, TR, MX, VEC, 1, 512>(p, s) : fwd_run<TX, TR, MX, VEC, 1, 1024>(p, s);
  return nv == 2 ? fwd_run<TX, TR, MX, VEC, 2, 1024>(p, s) : fwd_run<TX, TR, MX, VEC, 4, 1024>(p, s);
}
template <typename TX, typename TR, bool VEC>
cudaError_t bwd_nv(const AddNormBwdParams* p, int nv, cudaStream_t s) {
  if (p == nullptr) {
    const cudaError_t e = bwd_run<TX, TR, VEC, 1, 512>(p, s);
    return e == cudaSuccess ? bwd_run<TX, TR, VEC, 1, 1024>(p, s) : e;
  }
  if (nv == 1) return p->group <= 512 ? bwd_run<TX, TR, VEC, 1, 512>(p, s) : bwd_run<TX, TR, VEC, 1, 1024>(p, s);
  return nv == 2 ? bwd_run<TX, TR, VEC, 2, 1024>(p, s) : bwd_run<TX, TR, VEC, 4, 1024>(p, s);
}

template <typename TX, typename TR>
cudaError_t fwd_vec(const AddNormParams* p, bool vec, int nv, cudaStream_t s) {
  return vec ? fwd_nv<TX, TR, false, true>(p, nv, s) : fwd_nv<TX, TR, false, false>(p, nv, s);
}
template <typename TX, typename TR>
cudaError_t bwd_vec(const AddNormBwdParams* p, bool vec, int nv, cudaStream_t s) {
  return vec ? bwd_nv<TX, TR, true>(p, nv, s) : bwd_nv<TX, TR, false>(p, nv, s);
}

template <typename TX, typename TR> cudaError_t init_types() {
  const cudaError_t e = fwd_vec<TX, TR>(nullptr, true, 1, nullptr);
  return e == cudaSuccess ? bwd_vec<TX, TR>(nullptr, true, 1, nullptr) : e;
}

}  // namespace

cudaError_t norm_init() {
  cudaError_t e = init_types<__nv_bfloat16, __nv_bfloat16>();
  if (e == cudaSuccess) e = init_types<__nv_bfloat16, float>();
  if (e == cudaSuccess) e = init_types<__half, __half>();
  if (e == cudaSuccess) e = init_types<__half, float>();
  if (e == cudaSuccess) e = init_types<float, float>();
  if (e == cudaSuccess) e = fwd_nv<__nv_bfloat16, __nv_bfloat16, true, true>(nullptr, 1, nullptr);
  if (e == cudaSuccess) e = fwd_nv<__nv_bfloat16, float, true, true>(nullptr, 1, nullptr);
  return e;
}

cudaError_t launch_add_norm(AddNormParams p, int dtype, int res_dtype, bool vec, cudaStream_t s) {
  int nv;
  row_split(p.d, &p.group, &nv);
  const bool same = dtype == res_dtype;
  if (p.y_q) {
    return same ? fwd_nv<__nv_bfloat16, __nv_bfloat16, true, true>(&p, nv, s)
                : fwd_nv<__nv_bfloat16, float, true, true>(&p, nv, s);
  }
  if (dtype == MOE_DT_BF16)
    return same ? fwd_vec<__nv_bfloat16, __nv_bfloat16>(&p, vec, nv, s)
                : fwd_vec<__nv_bfloat16, float>(&p, vec, nv, s);
  if (dtype == MOE_DT_F16)
    return same ? fwd_vec<__half, __half>(&p, vec, nv, s) : fwd_vec<__half, float>(&p, vec, nv, s);
  return fwd_vec<float, float>(&p, vec, nv, s);
}

cudaError_t launch_add_norm_bwd(AddNormBwdParams p, int dtype, int res_dtype, bool vec, float* dw,
                                cudaStream_t s) {
  int nv, blocks, threads;
  row_split(p.d, &p.group, &nv);
  row_grid(p.rows, p.group, &blocks, &threads);
  const bool same = dtype == res_dtype;
  cudaError_t e;
  if (dtype == MOE_DT_BF16)
    e = same ? bwd_vec<__nv_bfloat16, __nv_bfloat16>(&p, vec, nv, s)
             : bwd_vec<__nv_bfloat16, float>(&p, vec, nv, s);
  else if (dtype == MOE_DT_F16)
    e = same ? bwd_vec<__half, __half>(&p, vec, nv, s) : bwd_vec<__half, float>(&p, vec, nv, s);
  else
    e = bwd_vec<float, float>(&p, vec, nv, s);
  if (e != cudaSuccess || dw == nullptr) return e;
  return launch_pdl(add_norm_dw_kernel, dim3((unsigned)((p.d + 31) / 32)), dim3(1024), 0, s,
                    static_cast<const float*>(p.partial), blocks, p.d, dw);
}

cudaError_t launch_dropout(const DropoutParams& p, int dtype, bool vec, cudaStream_t s) {
  const int64_t gx = ((int64_t)p.cols + 255) / 256, gy = (p.rows + 15) / 16;
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
