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

// Eight values of a row that one of `G` neighbouring threads holds.  VEC: the
// columns [8 l, 8 l + 8), one or two 16-byte accesses (rows on 16-byte boundaries,
// whole groups).  Otherwise the columns l, l + G, ... l + 7 G: single elements,
// but neighbouring threads touch neighbouring ones; columns at or past d read as
// zero and are not written.  `l` counts from a multiple of G (VEC) or of 8 G.
template <bool VEC> MOE_DEV int first_column(int i, int lane, int G) {
  return VEC ? (lane + i * G) * 8 : i * 8 * G + lane;
}
template <bool VEC> MOE_DEV int column_step(int G) { return VEC ? 1 : G; }

template <typename T, bool VEC> MOE_DEV Raw8<T> load8(const T* row, int c, int G, int d) {
  Raw8<T> r;
  if constexpr (VEC) {
    constexpr int n = sizeof(Raw8<T>) / 16;
    uint4* q = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < n; ++i) q[i] = *(reinterpret_cast<const uint4*>(row + c) + i);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = c + j * G < d ? row[c + j * G] : Elem<T>::from_f(0.0f);
  }
  return r;
}
template <typename T, bool VEC> MOE_DEV void store8(T* row, int c, int G, int d, const Raw8<T>& r) {
  if constexpr (VEC) {
    constexpr int n = sizeof(Raw8<T>) / 16;
    const uint4* q = reinterpret_cast<const uint4*>(&r);
#pragma unroll
    for (int i = 0; i < n; ++i) *(reinterpret_cast<uint4*>(row + c) + i) = q[i];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j * G < d) row[c + j * G] = r.v[j];
  }
}

// ------------------------------------------------------------------ asynchronous copies
MOE_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// The eight numbers of columns [8 group, 8 group + 8) of a row.
MOE_DEV uint4 drop_numbers(uint32_t group, uint32_t row, const DropRng& g) {
  return philox4x32_10(make_uint4(group, row, g.o0, g.o1), g.k0, g.k1);
}

// Drop and scale eight values by those numbers.  Dropped places become zero
// whatever they held (a NaN there does not survive).
MOE_DEV void drop8(float* f, const uint4& r, const DropRng& g) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  // a half-word is compared in the upper half of a word: (w >> 16) >= t is w >=
  // t << 16, and t = 65536 (drop everything) has scale 0 and is taken apart
  const uint32_t t = g.threshold << 16;
  if (g.threshold > 0xFFFFu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.0f;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = (w[i] << 16) >= t ? f[2 * i] * g.scale : 0.0f;
    f[2 * i + 1] = w[i] >= t ? f[2 * i + 1] * g.scale : 0.0f;
  }
}

// The numbers of a thread's eight values: its own where they are neighbouring
// columns; where they are G apart, each of the G threads makes those of eight
// neighbouring columns and they change hands in shared memory (`xch`: G entries
// of the group's own; `sync` is a barrier of the G threads at least, called
// twice).
template <bool VEC, typename Sync>
MOE_DEV uint4 drop_numbers_of(int i, int lane, int G, uint32_t row, const DropRng& g, uint4* xch, Sync sync) {
  const uint4 r = drop_numbers((uint32_t)(lane + i * G), row, g);
  if constexpr (VEC) {
    return r;
  } else {
    sync();   // the previous numbers have been read
    xch[lane] = r;
    sync();
    const uint16_t* h = reinterpret_cast<const uint16_t*>(xch);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (uint32_t)h[2 * j * G + lane] | (uint32_t)h[(2 * j + 1) * G + lane] << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace moe
