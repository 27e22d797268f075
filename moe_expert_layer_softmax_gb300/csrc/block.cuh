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

// Load / store columns [c, c + 8) of a row.  VEC: whole groups on 16-byte
// boundaries; otherwise element by element, columns at or past d read as zero
// and are not written.
template <typename T, bool VEC> MOE_DEV Raw8<T> load8(const T* row, int c, int d) {
  Raw8<T> r;
  if constexpr (VEC) {
    constexpr int n = sizeof(Raw8<T>) / 16;
    uint4* q = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < n; ++i) q[i] = *(reinterpret_cast<const uint4*>(row + c) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = c + i < d ? row[c + i] : Elem<T>::from_f(0.0f);
  }
  return r;
}
template <typename T, bool VEC> MOE_DEV void store8(T* row, int c, int d, const Raw8<T>& r) {
  if constexpr (VEC) {
    constexpr int n = sizeof(Raw8<T>) / 16;
    const uint4* q = reinterpret_cast<const uint4*>(&r);
#pragma unroll
    for (int i = 0; i < n; ++i) *(reinterpret_cast<uint4*>(row + c) + i) = q[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < d) row[c + i] = r.v[i];
  }
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

MOE_DEV uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c.x * 0xD2511F53u;
    const uint64_t b = (uint64_t)c.z * 0xCD9E8D57u;
    c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b,
                   (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// Drop and scale columns [c, c + 8) of `row` (c a multiple of 8).  Dropped
// places become zero whatever they held (a NaN there does not survive).
MOE_DEV void drop8(float* f, int c, uint32_t row, const DropRng& g) {
  const uint4 r = philox4x32_10(make_uint4((uint32_t)c >> 3, row, g.o0, g.o1), g.k0, g.k1);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = (w[i] & 0xFFFFu) >= g.threshold ? f[2 * i] * g.scale : 0.0f;
    f[2 * i + 1] = (w[i] >> 16) >= g.threshold ? f[2 * i + 1] * g.scale : 0.0f;
  }
}

}  // namespace moe
