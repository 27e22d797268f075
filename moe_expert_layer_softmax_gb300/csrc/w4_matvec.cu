// Products of a few vectors with 4-bit weights (sm_103a): y[m, n] = sum_k x[m, k]
// W[n, k].  How the weights are streamed, and what bounds it: w4.cuh.  Measured
// back to back from HBM: one vector and 4096 x 4096 5.8 us (8.9 MB, 1.5 TB/s;
// about 4 us of it start and end of the kernel), 20011 x 2048 8.5, 4096 x 14336
// 11.8 us (2.6 TB/s); eight vectors 6.8, 10.7 and 15.1 us; 64 vectors 19, 41 and
// 74 us.
#include "w4.cuh"

namespace moe {

namespace {

struct MatvecArgs {
  int M, N, K;
  const void* x;
  int64_t ld_x;
  const uint8_t* q;
  const void* sc;
  void* y;
  int64_t ld_y;
  int seg_tiles;   // most tiles of a segment (shared memory of the parts)
};

// Rows past N repeat row N - 1 and are not written.
template <typename S, int W> struct MatvecRows {
  const uint8_t* q;
  const S* sc;
  int64_t n0;
  int N, K, groups;
  MOE_DEV RowPtr operator()(int tile, int, int stage) const {
    const int lane = threadIdx.x & 31;
    const int64_t base = n0 + tile * 16, last = N - 1;
    RowPtr r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.row[i] = q + min(base + (lane >> 3) + 4 * i, last) * (K / 2) + (int64_t)stage * 64 + (lane & 7) * 16;
    r.s = reinterpret_cast<const uint8_t*>(sc + min(base + (lane & 15), last) * groups + stage * (4 / W));
    return r;
  }
  MOE_DEV void scales(int tile, const S** a, const S** b) const {
    const int g = (threadIdx.x & 31) >> 2;
    const int64_t base = n0 + tile * 16, last = N - 1;
    *a = sc + min(base + g, last) * groups;
    *b = sc + min(base + g + 8, last) * groups;
  }
};

template <typename T, int W, int NT, XSource XS, bool FULL>
__global__ void __launch_bounds__(kW4Threads, 1) matvec_w4_kernel(MatvecArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_begin();
  const uint32_t rings = smem_u32(smem);
  float* parts = reinterpret_cast<float*>(smem + kRingsBytes);
  const int g = (threadIdx.x & 31) >> 2;
  const int all = (a.N + 15) / 16, stages = (a.K + 127) / 128;
  StagedAt at;
  at.x = rings + kRingsBytes + (a.seg_tiles + kW4Warps) * NT * 512;
  at.low = 0;
  at.stride = staged_stride(a.K);
  at.table = at.x + a.M * at.stride;
  const int first = (int)((int64_t)blockIdx.x * all / gridDim.x);
  const int last = (int)((int64_t)(blockIdx.x + 1) * all / gridDim.x);
  const T* x = static_cast<const T*>(a.x);
  const T* sc = static_cast<const T*>(a.sc);
  T* y = static_cast<T*>(a.y);
  for (int t0 = first; t0 < last; t0 += a.seg_tiles) {
    const int tiles = min(last - t0, a.seg_tiles);
    const MatvecRows<T, W> rows = {a.q, sc, (int64_t)t0 * 16, a.N, a.K, a.K / (32 * W)};
    for (int m0 = 0; m0 < a.M; m0 += 8 * NT) {
      Segment<T, T, W, NT, false, XS, FULL, false, 8 * NT, MatvecRows<T, W>> seg(
          rings, rows, tiles, 1, stages, a.K, sc + (int64_t)a.N * rows.groups);
      seg.start();
      const int here = min(a.M - m0, 8 * NT);   // kStaged: all of them
      Vectors<T, NT> v;
      if constexpr (XS == kStaged) {
        if (t0 == first) stage_vectors<T, W, false, 8>(at, here, a.K, [&](int m) { return x + m * a.ld_x; });
        __syncthreads();
        staged_at(v, at, here);
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j) v.x[j] = x + (m0 + min(j * 8 + g, here - 1)) * a.ld_x;
      }
      seg.finish(v, (here + 7) / 8, parts);
      __syncthreads();
      for (int i = threadIdx.x; i < tiles * here * 16; i += kW4Threads) {
        const int row = i & 15, tile = (i >> 4) / here, col = (i >> 4) - tile * here;
        const int64_t n = (int64_t)(t0 + tile) * 16 + row;
        if (n < a.N) {
          const PartRange w(tile, tiles, (stages + 1) / 2);
          y[(m0 + col) * a.ld_y + n] = Elem<T>::from_f(
              sum_parts(parts, NT * 128, tile, w, (col >> 3) * 128 + row * 8 + (col & 7)));
        }
      }
      __syncthreads();
    }
  }
}

// Staged vectors and the factors of eight for each stage.
int64_t staged_bytes(int M, int K) { return (int64_t)M * staged_stride(K) + (int64_t)K / 128 * 32; }

// Most tiles of a block.
int share_of(int N) {
  const int all = (N + 15) / 16, sms = device_info()->sm_count;
  return (all + sms - 1) / sms;
}

template <typename T, int W, int NT, XSource XS, bool FULL>
cudaError_t matvec_launch(const MatvecArgs& a, cudaStream_t s) {
  const int all = (a.N + 15) / 16, sms = device_info()->sm_count;
  const int x_bytes = XS == kStaged ? (int)staged_bytes(a.M, a.K) : 0;
  const int room = (kSmemMost - kRingsBytes - x_bytes) / (NT * 512) - kW4Warps;
  const int share = share_of(a.N);
  MatvecArgs args = a;
  args.seg_tiles = share < room ? share : room;
  const size_t smem = kRingsBytes + (size_t)(args.seg_tiles + kW4Warps) * NT * 512 + x_bytes;
  static SmemLimit limit;
  return launch_w4(limit, &matvec_w4_kernel<T, W, NT, XS, FULL>, dim3(all < sms ? all : sms), smem, 0, s, args);
}

// Vectors are staged (whole stages only) where each block has a tile for every
// vector that it stages, and they leave room for the parts of eight tiles;
// otherwise they are read where they are, sixteen a pass over the weights or, of
// more than that, 32 (64 vectors, sixteen and 32 a pass: 4096 x 4096 24.3 and 19.1,
// 20011 x 2048 48.5 and 40.8, 4096 x 14336 79.6 and 74.3 us; 17 vectors 12.0 and
// 10.0, 21.5 and 17.9, 31.6 and 31.1).
// Measured, staged and read (us): 4096 x 4096, two tiles a block: 5.8 and 6.0
// with one vector, 7.2 and 6.4 with four, 9.1 and 6.8 with eight; 20011 x 2048, nine
// tiles: 8.5 and 9.7 with one, 10.7 and 12.1 with eight (in groups of 32 9.7 and 10.2,
// 11.9 and 11.6); staged rounds of sixteen, when last tried, 15.9 and 14.1.
template <typename T, int W, bool FULL>
cudaError_t matvec_nt(const MatvecArgs& a, cudaStream_t s) {
  if constexpr (FULL) {
    if (a.M <= 8 && a.M <= share_of(a.N) && staged_bytes(a.M, a.K) <= kSmemMost - kRingsBytes - (8 + kW4Warps) * 512)
      return matvec_launch<T, W, 1, kStaged, FULL>(a, s);
  }
  return a.M > 16 ? matvec_launch<T, W, 4, kNatural, FULL>(a, s) : matvec_launch<T, W, 2, kNatural, FULL>(a, s);
}

template <typename T> cudaError_t matvec_group(int group, const MatvecArgs& a, cudaStream_t s) {
  const bool full = a.K % 128 == 0;
  if (group == 32) return full ? matvec_nt<T, 1, true>(a, s) : matvec_nt<T, 1, false>(a, s);
  if (group == 64) return full ? matvec_nt<T, 2, true>(a, s) : matvec_nt<T, 2, false>(a, s);
  return matvec_nt<T, 4, true>(a, s);
}

}  // namespace

cudaError_t launch_matvec_w4(int M, int N, int K, int group, int dtype, const void* x, int64_t ld_x,
                             const uint8_t* q, const void* scales, void* y, int64_t ld_y,
                             cudaStream_t s) {
  const MatvecArgs a = {M, N, K, x, ld_x, q, scales, y, ld_y, 0};
  return dtype == MOE_DT_BF16 ? matvec_group<__nv_bfloat16>(group, a, s) : matvec_group<__half>(group, a, s);
}

}  // namespace moe
