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
// The least a call costs is one read and one write of each matrix.  A row stays in
// registers between the pass that sums it and the pass that writes it.  A fixed
// grid takes the rows in turn while the rows to come (one to three) are on their
// way into shared memory, each thread copying and reading its own pieces, so that
// the pipeline needs no barrier and no registers: 512 threads a multiprocessor
// keep 50 to 130 KB in flight.  A thread holds 16 columns (rows up to 256: 8; the
// 8-bit output and wide rows: up to 32), so that what a row costs beside its
// elements (the sums over threads, the square root, addresses) is shared: with
// eight columns a thread the 8192 x 2048 forward took 294 instructions per eight
// columns and 28.5 us, bound by issue.  A row has a group of 8, 16 or any multiple
// of 32 threads: with whole warps alone rows of 64 columns ran at 1.8 TB/s, with
// powers of two alone 768 columns left a quarter of the lanes idle.  Rows that
// take no vector loads are read by elements or pairs, neighbours by neighbours, one
// group of columns a thread (two spilled: 1001 columns in fp32 4.3 and 5.6 TB/s),
// the next row on its way in registers (6.1).
// Sums are taken in a fixed order (no atomics).
//
// Measured (TB/s of HBM against a copy's 6.7; bf16 matrices, bf16 stream / fp32
// stream, without dropout): forward 64 to 8192 columns 5.4-6.5 / 5.5-6.4, 12288
// and 16384 5.6-5.9 / 5.7; backward 5.4-6.2 / 5.7-6.4, 12288 4.2 / 3.0.  With
// dropout the generator adds its instructions: bf16 stream 4.3-6.0, fp32 stream
// 5.3-6.5.  8-bit output, 4096 columns: 4.95 / 6.0, with dropout 4.05 / 5.5.  Wider
// rows than a ring holds 3.3-4.5 forward, 1.4-3.4 backward; other widths up to 4096
// in bf16 2.1-3.2, on an fp32 stream 3.3-5.2, in fp32 4.7-6.8, up to 8192 1.7-3.0,
// 2.6-4.3 and 3.2-5.8 (with 1024 threads; 512 with twice the columns spilled: 4999
// columns in fp32 3.2 and 4.1 forward, 2.3 and 3.2 backward).
#pragma once

#include "block.cuh"
#include "block.h"
#include "kernels.h"

namespace moe {

constexpr int kNormThreads = 256;      // threads of a block whose row group is not larger
constexpr int kNormMaxThreads = 1024;
// Blocks of kNormThreads on a multiprocessor: with a ring by registers and shared
// memory, without one as many as hide the loads.
constexpr int norm_blocks(bool ring, int nv, int most) {
  return most > kNormThreads ? 1 : ring || nv > 1 ? 2 : 3;
}
constexpr int kNormRingBytes = 96 * 1024;   // of a block

MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The threads of a block form groups of G, one a row: a multiple of 32, or (SMALL)
// 8 or 16.
template <bool SMALL> struct RowGroup {
  int G, lane, group, per;
  MOE_DEV explicit RowGroup(int G_)
      : G(G_), lane(threadIdx.x % G_), group(threadIdx.x / G_), per(blockDim.x / G_) {}
  // Groups that start earlier in the same warp.
  MOE_DEV int before() const { return SMALL ? (threadIdx.x & 31) / min(G, 32) : 0; }
  MOE_DEV void sync() const {
    if (G <= 32) __syncwarp(); else bar_sync(1 + group, G);
  }
  // Sum over the group, the same value in every thread.  `red`: a float for each
  // warp of the block, another array in turn for the next call (so that one
  // barrier is enough).
  MOE_DEV float sum(float v, float* red) const {
    if (!SMALL || G >= 32) {
      v = warp_sum(v);
    } else {
      for (int off = G >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    }
    if (G <= 32) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    bar_sync(1 + group, G);
    const int n = G >> 5;
    const float* from = red + group * n;
    float s = 0.0f;
    if (n & 3) {
      for (int i = 0; i < n; ++i) s += from[i];
    } else {
      for (int i = 0; i < n; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(from + i);
        s += (q.x + q.y) + (q.z + q.w);
      }
    }
    return s;
  }
};

// 1 / sqrt(v) to about an ulp: the approximation and one Newton step.
MOE_DEV float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  // zero, infinity and NaN: the approximation is the answer
  if (!(v > 0.0f) || !(v < INFINITY)) return r;
  return fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
}

template <int V>
MOE_DEV void load_weight8(const void* w, bool w_f32, bool w_f16, int c, int G, int d, float* f) {
  if (c >= d) {   // columns past the row's end: zeros all through
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
  } else if (w_f32) {
    widen8(load8<float, V>(static_cast<const float*>(w), c, G, d), f);
  } else if (w_f16) {
    widen8(load8<__half, V>(static_cast<const __half*>(w), c, G, d), f);
  } else {
    widen8(load8<__nv_bfloat16, V>(static_cast<const __nv_bfloat16*>(w), c, G, d), f);
  }
}

// The pieces (16 bytes) of the rows to come: cp.async into slots, BYTES for eight
// columns of up to three matrices, NV times.  Slots are laid out piece by piece
// (16 bytes a thread), so that neighbouring threads touch neighbouring banks.  A
// thread copies and reads its own pieces; where eight columns are two pieces
// (fp32) a warp (or a smaller group) copies its pieces as they follow one another,
// which fills whole sectors, and each lane reads its two: piece q lies at place q
// ^ (q >> 3 & 1), so that eight lanes' reads miss each other's banks.
template <int BYTES, int NV> struct RowRing {
  static constexpr int kFit = kNormRingBytes / (kNormThreads * BYTES * NV);
  static constexpr int kDepth = kFit < 2 ? 2 : kFit > 4 ? 4 : kFit;
  static constexpr int kBytes = BYTES * NV * kDepth;   // a thread
  static constexpr bool kFits512 = kFit >= 2;          // 512 threads' rings, in twice kNormRingBytes
  uint32_t mine, warp;   // slot 0, piece 0: this thread's, that of lane 0
  uint32_t piece;        // bytes between pieces
  uint32_t slot;         // bytes: the next one to read
  uint32_t ahead;        // bytes: the next one to fill
  int width_;            // NV = 1: groups may be smaller than a warp
  MOE_DEV RowRing(void* smem, int G)
      : mine(smem_u32(smem) + threadIdx.x * 16), piece(blockDim.x * 16), slot(0), ahead(0), width_(G < 32 ? G : 32) {
    warp = mine - lane() * 16;
  }
  // Threads of a warp, or of a smaller group, and this one among them.
  MOE_DEV int width() const { return NV == 1 ? width_ : 32; }
  MOE_DEV int lane() const { return threadIdx.x & (width() - 1); }
  MOE_DEV uint32_t next(uint32_t at) const {
    at += piece * (BYTES / 16 * NV);
    return at == piece * (BYTES / 16 * NV) * kDepth ? 0 : at;
  }
  // Copy columns c .. c + 7 of a row of d to piece `at` of the slot that is
  // filled (c a multiple of 8; columns from d on become zeros).
  template <typename T> MOE_DEV void put(int at, const T* row, int c, int d) const {
    if constexpr (sizeof(T) == 2) {
      const bool in = c < d;
      cp_async16(mine + ahead + at * piece, row + (in ? c : 0), in ? 16 : 0);
    } else {
      const int lane = this->lane(), first = c - lane * 8;   // of lane 0
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int q = lane + width() * i;
        const bool in = first + q * 4 < d;
        cp_async16(warp + ahead + (at + i) * piece + (lane ^ (q >> 3 & 1)) * 16, row + (in ? first + q * 4 : 0), in ? 16 : 0);
      }
    }
  }
  // This thread's eight columns at piece `at` of the slot that is read.
  template <typename T> MOE_DEV Raw8<T> get(int at) const {
    Raw8<T> r;
    uint4* q = reinterpret_cast<uint4*>(&r);
    if constexpr (sizeof(T) == 2) {
      load(mine + slot + at * piece, q[0]);
    } else {
      const int lane = this->lane();
      const uint32_t from = warp + slot + (at + (2 * lane >= width())) * piece;
      const int first = (2 * lane & (width() - 1)) ^ (lane >> 2 & 1);
      load(from + first * 16, q[0]);
      load(from + (first ^ 1) * 16, q[1]);
    }
    return r;
  }
  MOE_DEV static void load(uint32_t at, uint4& x) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at));
  }
};

// Threads of a row group (8, 16 or a multiple of 32) and how many times eight
// columns each holds: as few as `least` and up to `most`, so that the group is no
// larger than `limit` and the fewest places stay empty; group 0: it does not fit.
struct RowSplit {
  int group, nv;
  RowSplit(int d, int least, int most, int limit) : group(0), nv(1) {
    const int g8 = (d + 7) / 8;
    if (g8 <= 32) {
      group = g8 <= 8 ? 8 : g8 <= 16 ? 16 : 32;
      return;
    }
    for (int n = least; n <= most; ++n) {
      const int g = ((g8 + n - 1) / n + 31) / 32 * 32;
      if (g > limit || (group && g * n > group * nv)) continue;
      if (group && least < 3) break;   // the fewest columns a thread that fit
      group = g;
      nv = n;
    }
  }
  // Threads of a block: whole groups in kNormThreads, or a larger one.
  int threads() const { return group > kNormThreads ? group : kNormThreads / group * group; }
};

// Blocks of `threads` that stay on a multiprocessor: what the registers are for
// (`blocks` of `maxt` threads) and, with a ring of `ring` bytes a thread, what the
// shared memory has room for (four groups of columns of two fp32 matrices: a ring of
// up to 128 KB, one block and not two).
constexpr int kSmShared = 228 * 1024;
constexpr int kBlockShared = 1024 + 512;   // beside the ring: what the system keeps, and the static arrays
constexpr int norm_resident(int blocks, int maxt, int threads, int ring) {
  const int by_threads = blocks * maxt / threads, by_shared = kSmShared / (threads * ring + kBlockShared);
  return ring && by_shared < by_threads ? by_shared : by_threads;
}

// Blocks: enough row groups for every row, or as many as stay on the device,
// `resident` on a multiprocessor.
inline int row_blocks(int64_t rows, int group, int threads, int resident) {
  const int per = threads / group;
  const int64_t need = (rows + per - 1) / per, most = (int64_t)device_info()->sm_count * resident;
  return (int)(need < most ? need : most);
}

}  // namespace moe
