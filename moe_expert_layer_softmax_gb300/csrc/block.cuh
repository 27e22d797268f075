// Device helpers shared by the kernels around the layer (norm, dropout, 4-bit
// weights): groups of eight columns in any element type, and the counter-based
// generator of the dropout.
#pragma once

#include "common.cuh"

namespace moe {

// ------------------------------------------------------------------ element types
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static MOE_DEV float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
  static MOE_DEV __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
  static MOE_DEV float to_f(__half v) { return __half2float(v); }
  static MOE_DEV __half from_f(float v) { return __float2half_rn(v); }
};
template <> struct Elem<float> {
  static MOE_DEV float to_f(float v) { return v; }
  static MOE_DEV float from_f(float v) { return v; }
};

// Eight neighbouring columns as they lie in memory (16 or 32 bytes).
template <typename T> struct alignas(16) Raw8 { T v[8]; };

template <typename T> MOE_DEV void widen8(const Raw8<T>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = Elem<T>::to_f(r.v[i]);
}
template <typename T> MOE_DEV Raw8<T> narrow8(const float* f) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = Elem<T>::from_f(f[i]);
  return r;
}

// Eight values of a row that one of `G` neighbouring threads holds.  V = 8: the
// columns [8 l, 8 l + 8), one or two 16-byte accesses (rows on 16-byte boundaries,
// whole groups).  V = 2: the pairs of columns 2 l, 2 (l + G), 2 (l + 2 G) and 2 (l +
// 3 G) (an even width, rows on a pair's boundary); V = 1: the columns l, l + G, ... l
// + 7 G.  Narrow accesses, but neighbouring threads touch neighbouring ones; columns
// at or past d read as zero and are not written.  `l` counts from a multiple of G (V
// = 8) or of 8 G columns.
template <int V> MOE_DEV int first_column(int i, int lane, int G) {
  return V == 8 ? (lane + i * G) * 8 : i * 8 * G + lane * V;
}
// Column of value j of those that start at c.
template <int V> MOE_DEV int column_of(int c, int j, int G) { return c + j / V * (V * G) + j % V; }

// A pair of columns as one word (16-bit types) or two.
template <typename T> struct PairOf { using type = uint32_t; };
template <> struct PairOf<float> { using type = uint2; };

template <typename T, int V> MOE_DEV Raw8<T> load8(const T* row, int c, int G, int d) {
  Raw8<T> r;
  if constexpr (V == 8) {
    constexpr int n = sizeof(Raw8<T>) / 16;
    uint4* q = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < n; ++i) q[i] = *(reinterpret_cast<const uint4*>(row + c) + i);
  } else if constexpr (V == 2) {
    using P = typename PairOf<T>::type;
    P* q = reinterpret_cast<P*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = column_of<V>(c, 2 * i, G);
      q[i] = at < d ? *reinterpret_cast<const P*>(row + at) : P{};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = c + j * G < d ? row[c + j * G] : Elem<T>::from_f(0.0f);
  }
  return r;
}
template <typename T, int V> MOE_DEV void store8(T* row, int c, int G, int d, const Raw8<T>& r) {
  if constexpr (V == 8) {
    constexpr int n = sizeof(Raw8<T>) / 16;
    const uint4* q = reinterpret_cast<const uint4*>(&r);
#pragma unroll
    for (int i = 0; i < n; ++i) *(reinterpret_cast<uint4*>(row + c) + i) = q[i];
  } else if constexpr (V == 2) {
    using P = typename PairOf<T>::type;
    const P* q = reinterpret_cast<const P*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = column_of<V>(c, 2 * i, G);
      if (at < d) *reinterpret_cast<P*>(row + at) = q[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j * G < d) row[c + j * G] = r.v[j];
  }
}

// The same for a whole warp whose lanes hold neighbouring groups of eight columns
// (V = 8; each lane calls, `in`: its group is part of the row).  Eight fp32 values
// are two 16-byte accesses; lanes go in pairs, so that each access of the pair
// fills a 32-byte sector instead of two half sectors.
template <typename T, int V> MOE_DEV Raw8<T> load8_warp(const T* row, int c, int G, int d, bool in) {
  Raw8<T> r = {};
  if constexpr (V == 8 && sizeof(T) == 4) {
    const bool odd = threadIdx.x & 1;
    const bool other = __shfl_xor_sync(0xffffffffu, (int)in, 1);
    const T* even = row + (odd ? c - 8 : c);   // the pair's sixteen columns
    uint4 a = {}, b = {};
    if (odd ? other : in) a = *(reinterpret_cast<const uint4*>(even) + odd);
    if (odd ? in : other) b = *(reinterpret_cast<const uint4*>(even) + 2 + odd);
    // even lanes keep a and take the odd lane's a; odd lanes keep b and take b
    uint4 give = odd ? a : b, got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
    got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
    got.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
    got.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
    uint4* q = reinterpret_cast<uint4*>(&r);
    q[0] = odd ? got : a;
    q[1] = odd ? b : got;
  } else {
    if (in) r = load8<T, V>(row, c, G, d);
  }
  return r;
}
template <typename T, int V> MOE_DEV void store8_warp(T* row, int c, int G, int d, const Raw8<T>& r, bool in) {
  if constexpr (V == 8 && sizeof(T) == 4) {
    const bool odd = threadIdx.x & 1;
    const bool other = __shfl_xor_sync(0xffffffffu, (int)in, 1);
    T* even = row + (odd ? c - 8 : c);
    const uint4* q = reinterpret_cast<const uint4*>(&r);
    const uint4 give = odd ? q[0] : q[1];
    uint4 got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
    got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
    got.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
    got.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
    if (odd ? other : in) *(reinterpret_cast<uint4*>(even) + odd) = odd ? got : q[0];
    if (odd ? in : other) *(reinterpret_cast<uint4*>(even) + 2 + odd) = odd ? q[1] : got;
  } else {
    if (in) store8<T, V>(row, c, G, d, r);
  }
}

// ------------------------------------------------------------------ asynchronous copies
MOE_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// bytes: 16, or 0 for zeros in place of the source
MOE_DEV void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
MOE_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> MOE_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------ dropout
// Keep mask of the dropout, a pure function of (seed, offset, row, column):
// Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel Random
// Numbers: As Easy as 1, 2, 3", SC 2011) with the seed as its 64-bit key and the
// counter (column / 8, row, offset low, offset high).  One evaluation gives 128
// bits: sixteen for each of eight neighbouring columns, so the generator costs a
// quarter of what 32 bits a value in every fourth call would.  A column is kept
// when its number is at least `threshold` = p 2^16 rounded; the kept values are
// multiplied by 2^16 / (2^16 - threshold), the inverse of the exact keep
// probability, so the expectation is exact although p has 16 bits.
struct DropRng {
  uint32_t k0, k1, o0, o1;
  uint32_t threshold;   // 0: keep everything
  float scale;
};

// Philox of N counters at once: the rounds' keys are made once.
template <int N> MOE_DEV void philox4x32_10(uint4 (&c)[N], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint64_t a = (uint64_t)c[n].x * 0xD2511F53u;
      const uint64_t b = (uint64_t)c[n].z * 0xCD9E8D57u;
      c[n] = make_uint4((uint32_t)(b >> 32) ^ c[n].y ^ k0, (uint32_t)b,
                        (uint32_t)(a >> 32) ^ c[n].w ^ k1, (uint32_t)a);
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// Drop and scale eight values by their numbers.  Dropped places become zero
// whatever they held (a NaN there does not survive).
MOE_DEV void drop8(float* f, const uint4& r, const DropRng& g) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  // A half-word is compared in the upper half of a word: (w >> 16) >= t is w > t
  // 2^16 - 1.  `limit` is that, 0xFFFFFFFF (nothing is above) where t is 65536.
  const uint32_t limit = (g.threshold << 16) - 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = (w[i] << 16) > limit ? f[2 * i] * g.scale : 0.0f;
    f[2 * i + 1] = w[i] > limit ? f[2 * i + 1] * g.scale : 0.0f;
  }
}

// Numbers change hands: each of G threads has made those of eight neighbouring
// columns, 8 G in a row, and gets those of the columns that it holds (V = 2, 1).
// `xch`: G entries of the group's own; `sync`: a barrier of the G threads at least.
template <int V, typename Sync>
MOE_DEV void exchange_numbers(uint4& r, int lane, int G, uint4* xch, Sync sync) {
  sync();   // the previous numbers have been read
  xch[lane] = r;
  sync();
  if constexpr (V == 2) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(xch);
    r = make_uint4(w[lane], w[lane + G], w[lane + 2 * G], w[lane + 3 * G]);
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(xch);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (uint32_t)h[2 * j * G + lane] | (uint32_t)h[(2 * j + 1) * G + lane] << 16;
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The numbers of a thread's N times eight values of a row: groups lane, lane +
// G, ... of neighbouring columns (V = 8), or the columns first_column() says.
template <int V, int N, typename Sync>
MOE_DEV void drop_numbers(uint4 (&r)[N], int lane, int G, uint32_t row, const DropRng& g, uint4* xch, Sync sync) {
#pragma unroll
  for (int n = 0; n < N; ++n) r[n] = make_uint4((uint32_t)(lane + n * G), row, g.o0, g.o1);
  philox4x32_10(r, g.k0, g.k1);
  if constexpr (V != 8) {
#pragma unroll
    for (int n = 0; n < N; ++n) exchange_numbers<V>(r[n], lane, G, xch, sync);
  }
}

}  // namespace moe
