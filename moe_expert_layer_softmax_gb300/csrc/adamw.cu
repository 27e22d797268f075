// AdamW over many tensors in one launch (sm_103a).
//
//   g = grad * grad_scale
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g g,  root = sqrt(v)
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) * (m / (root / sqrt(1 - b2^t) + eps))
// Every product, sum, quotient and root is rounded to 32 bits by itself, in this
// order (no contraction): a step can be repeated bit for bit by any program that
// does the same.
//
// States in 8 bits: E4M3 codes with one fp32 scale (largest magnitude / 448) for
// 128 neighbouring values.  The second moment is held as its root, which halves its
// range in powers of two: 448 / 2^-9 of the codes is then 2^36 of v in a block.  A
// state that moves by a few per cent a step (1 - b2 = 0.001) would stand still if it
// were rounded to the nearest of steps of 6 to 12 per cent; it is rounded up with the
// probability of its remainder instead, by 16 bits of the generator that the dropout
// uses, so that its mean is right.  A root above zero is never held as zero: a first
// moment beside it that was rounded up would otherwise be divided by eps alone.
// Parameters in bf16 without an fp32 copy are rounded in the same way, for the same
// reason: a step of lr is often less than half of theirs.
//
// The least that a step costs is one read of the gradient and one read and one write
// of everything else.  A block takes 2048 neighbouring values at a time, a thread eight,
// all loads issued before the first is used.  Measured on 201 M values, fp32 gradients:
// bf16 with fp32 copies and 32-bit states (30 bytes a value) 847 us, 7.1 TB/s, HBM; bf16
// alone with 8-bit states (12 bytes) 621 us, 3.9 TB/s: 85 instructions a value, a fifth of
// them the generator's (without it 512 us with one chunk a block, when the whole took 666),
// fill 67 % of the issue slots; in the rest the warps wait for loads, which a thread issues
// for its next chunk only when it is done with this one (registers for both cost a block of
// four and gave nothing).  Scalar products and roots took 753 us there, the compiler's
// division and root and a rounding by conversions 908.
// Values whose moments are zero (a gradient that has always been zero: experts that never
// had a token) take the roots and quotients one by one: an eighth of the values 671 us, all
// of them 1029; gradients of zero beside moments that are not 628.
#include "block.cuh"
#include "block.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamChunk = kAdamThreads * 8;   // values of a block's turn: whole scale blocks

template <int N> struct AdamwList {
  AdamwTensor t[N];   // `first` ascending, behind the last one in use: the end
  AdamwParams p;
};

// Sums of pairs, one by one: a packed product and a packed sum after it came out as one
// fused operation (CUDA 13.0), rounded once and not twice.
MOE_DEV float2 add(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }

// Correctly rounded roots and quotients of pairs from the hardware's approximations by
// the iterations of P. Markstein ("Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990): a Newton step on the reciprocal
// (root), then the residual of the quotient (square), which is exact, decides the last
// bit.  For v in [2^-100, 2^100], |m| in [2^-60, 2^60] and n in -[2^-60, 2^60], where
// nothing on the way leaves the normal range.  Compared with __fsqrt_rn on every
// mantissa of both parities, the reciprocal with __frcp_rn on every mantissa (then the
// quotient is right by Markstein's theorem), 2.5e10 quotients with __fdiv_rn: no difference.
// tests/test_gpu_adamw_ranges.py repeats the roots, the reciprocals and 7e7 quotients.
MOE_DEV Two roots(float2 v) {
  float x, y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(v.x));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v.y));
  const Two a(x, y), g = mul(Two(v), a), h = mul(a, Two(-0.5f, -0.5f)), r = fma(g, h, Two(0.5f, 0.5f));
  const Two g1 = fma(g, r, g), h1 = fma(h, r, h);
  const float2 q = g1.get();
  return fma(Two(fmaf(q.x, q.x, -v.x), fmaf(q.y, q.y, -v.y)), h1, g1);
}
// m / -n
MOE_DEV Two quotients(Two m, float2 n) {
  float x, y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(-n.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-n.y));
  const Two a(x, y), d(n), b = fma(fma(d, a, Two(1.0f, 1.0f)), a, a), q = mul(m, b);
  return fma(fma(d, q, m), b, q);
}

// b^t in double, by squaring.
MOE_DEV double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

// The constants of a step whose rate or number is on the device: two threads, one for
// those of the first moment and one for that of the second (64-bit arithmetic is slow).
MOE_DEV void device_scalars(const AdamwParams& p, AdamwScalars& s) {
  const bool second = threadIdx.x & 1;
  double c = second ? 0.0 : p.c1;
  if (p.step_dev) c = 1.0 - power(second ? p.beta2 : p.beta1, *p.step_dev);
  if (!second) {
    const double lr = p.lr_dev ? (double)*p.lr_dev : p.lr;
    s.decay = (float)(1.0 - lr * p.weight_decay);
    s.rate = (float)(lr / c);
  } else {
    s.root_scale = p.step_dev ? (float)(1.0 / sqrt(c)) : p.s.root_scale;
  }
}

// Eight values from `at`; behind `n` zeros.
template <typename T> MOE_DEV Raw8<T> fetch8(const T* p, int64_t at, int64_t n, bool vec) {
  if (vec) return load8<T, 8>(p + at, 0, 1, 8);
  Raw8<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.v[j] = at + j < n ? p[at + j] : Elem<T>::from_f(0.0f);
  return r;
}
template <typename T> MOE_DEV void put8(T* p, int64_t at, int64_t n, bool vec, const Raw8<T>& r) {
  if (vec) return store8<T, 8>(p + at, 0, 1, 8, r);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (at + j < n) p[at + j] = r.v[j];
}

// Number j (16 bits) of the eight that a counter gives, and the same times 16.
MOE_DEV uint32_t number_of(const uint4& r, int j) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  return j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
}
MOE_DEV uint32_t number16_of(const uint4& r, int j) { return number_of(r, j) << 4; }

// The largest and the smallest magnitude of eight values; a NaN goes through to both.
MOE_DEV void magnitudes(const float* x, float& most, float& least) {
  most = least = fabsf(x[0]);
#pragma unroll
  for (int j = 1; j < 7; j += 2) {
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(most) : "f"(most), "f"(fabsf(x[j])), "f"(fabsf(x[j + 1])));
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(least) : "f"(least), "f"(fabsf(x[j])), "f"(fabsf(x[j + 1])));
  }
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(most) : "f"(most), "f"(fabsf(x[7])));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(least) : "f"(least), "f"(fabsf(x[7])));
}

// Eight values to codes with the scale of the 16 lanes' 128 values; the scale is
// returned.  `most`, `least`: the magnitudes() of the eight.  An infinity or a NaN
// becomes a NaN and takes no part in the scale.  ROOT: nothing is below zero, and what is
// above it does not become zero.
//
// A magnitude z = |x| 448 / top goes up to the next code where its remainder, in units of
// the codes' distance, is at least 1 - r / 2^16: the upper three bits of the mantissa
// stay, and adding r at the upper sixteen of the twenty others carries into them exactly
// then.  (Past 448 the conversion saturates.)  Below 2^-6 the distance is 2^-9, that of
// the values from 2^-6 on: such values are moved there and back, cut off to steps of
// 2^-29, which leaves the comparison with multiples of 2^-25 as it is.  Few warps hold
// one: the others take none of these steps.
template <bool ROOT> MOE_DEV float quantize8(const float* x, float most, float least, const uint4& numbers, uint2& codes) {
  float top = most;
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, top, off);
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(top) : "f"(top), "f"(other));
  }
  const bool odd = __any_sync(0xffffffffu, !(top < INFINITY));
  if (odd) {   // the largest finite one (every lane takes part)
    top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]) < INFINITY ? fabsf(x[j]) : 0.0f);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  }
  const bool some = top >= 0x1p-100f;   // smaller values have no inverse in 32 bits
  const float inv = some ? __fmul_rn(448.0f, __frcp_rn(top)) : 0.0f;
  const Two inv2(inv, inv);
  float z[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 p = mul(Two(x[j], x[j + 1]), inv2).get();
    z[j] = p.x;
    z[j + 1] = p.y;
  }
  if (odd || __any_sync(0xffffffffu, __fmul_rn(least, inv) < 0x1p-6f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(z[j]), shift = a < 0x1p-6f ? 0x1p-6f : 0.0f;
      float q = __uint_as_float((__float_as_uint(__fadd_rz(a, shift)) + number16_of(numbers, j)) & 0xFFF00000u) - shift;
      if (ROOT && a > 0.0f) q = fmaxf(q, 0x1p-9f);
      z[j] = fabsf(x[j]) < INFINITY ? copysignf(q, x[j]) : NAN;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t bits = __float_as_uint(z[j]), up = (bits & 0x7FFFFFFFu) + number16_of(numbers, j);
      z[j] = __uint_as_float(ROOT ? (bits + number16_of(numbers, j)) & 0xFFF00000u : (up & 0x7FF00000u) | (bits & 0x80000000u));
    }
  }
  codes = e4m3x8(z);
  return some ? __fmul_rn(top, 1.0f / 448.0f) : 0.0f;
}

// The values of eight codes, or (SQUARE) their squares.
template <bool SQUARE> MOE_DEV void widen_codes(const uint2& q, float scale, float* f) {
  e4m3x2_to_f32(q.x, f[0], f[1]);
  e4m3x2_to_f32(q.x >> 16, f[2], f[3]);
  e4m3x2_to_f32(q.y, f[4], f[5]);
  e4m3x2_to_f32(q.y >> 16, f[6], f[7]);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    Two t = mul(Two(f[j], f[j + 1]), Two(scale, scale));
    if (SQUARE) t = mul(t, t);
    const float2 p = t.get();
    f[j] = p.x;
    f[j + 1] = p.y;
  }
}

// TP, TG: types of parameters and gradients; MASTER: the fp32 copy is what is
// stepped, the parameter its rounding; SMALL: states in 8 bits.  AT: part of the numbers'
// offset lies on the device (a kernel of its own: as a branch it cost every call with
// 8-bit states 1 %, 627 and 633 us).
template <int N, typename TP, typename TG, bool MASTER, bool SMALL, bool AT>
__global__ void __launch_bounds__(kAdamThreads, 4) adamw_kernel(const __grid_constant__ AdamwList<N> list) {
  constexpr bool DRAWN = !MASTER && sizeof(TP) == 2;   // parameters rounded by the generator
  __shared__ AdamwScalars shared;
  pdl_begin();
  const AdamwParams& p = list.p;
  AdamwScalars s = p.s;
  if (p.lr_dev || p.step_dev) {
    if (threadIdx.x < 2) device_scalars(p, shared);
    __syncthreads();
    s.decay = shared.decay;
    s.rate = shared.rate;
    s.root_scale = shared.root_scale;
  }
  uint32_t o0 = p.o0, o1 = p.o1;
  if constexpr (AT) {
    const uint64_t offset = ((uint64_t)o1 << 32 | o0) + *p.offset_dev;
    o0 = (uint32_t)offset;
    o1 = (uint32_t)(offset >> 32);
  }
  // the tensor of this block: the last one that begins at or before it
  int lo = 0, hi = p.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (list.t[mid].first <= blockIdx.x) lo = mid; else hi = mid;
  }
  const AdamwTensor& t = list.t[lo];
  const int64_t n = t.numel;
  int64_t at = (int64_t)(blockIdx.x - t.first) * p.turns * kAdamChunk + threadIdx.x * 8;
#pragma unroll 1
  for (int turn = 0; turn < p.turns && at - (int)threadIdx.x * 8 < n; ++turn, at += kAdamChunk) {
    const bool vec = t.vec && at + 8 <= n;
    const bool live = at < n;
    const int64_t block = at / kStateBlock;

    float g[8], w[8], m[8], v[8];
    {
      const Raw8<TG> gr = fetch8(static_cast<const TG*>(t.grad), at, n, vec);
      Raw8<float> wm;
      Raw8<TP> wp;
      if constexpr (MASTER)
        wm = fetch8<float>(t.master, at, n, vec);
      else
        wp = fetch8(static_cast<const TP*>(t.param), at, n, vec);
      if constexpr (SMALL) {
        uint2 mq = {}, vq = {};
        float ms = 0.0f, vs = 0.0f;
        if (live) {
          ms = t.m_scale[block];
          vs = t.v_scale[block];
        }
        const uint8_t *mc = static_cast<const uint8_t*>(t.m), *vc = static_cast<const uint8_t*>(t.v);
        if (vec) {
          mq = *reinterpret_cast<const uint2*>(mc + at);
          vq = *reinterpret_cast<const uint2*>(vc + at);
        } else {
          uint32_t mw[2] = {}, vw[2] = {};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (at + j < n) {
              mw[j >> 2] |= (uint32_t)mc[at + j] << (8 * (j & 3));
              vw[j >> 2] |= (uint32_t)vc[at + j] << (8 * (j & 3));
            }
          }
          mq = make_uint2(mw[0], mw[1]);
          vq = make_uint2(vw[0], vw[1]);
        }
        widen_codes<false>(mq, ms, m);
        widen_codes<true>(vq, vs, v);
      } else {
        widen8(fetch8<float>(static_cast<const float*>(t.m), at, n, vec), m);
        widen8(fetch8<float>(static_cast<const float*>(t.v), at, n, vec), v);
      }
      widen8(gr, g);
      if constexpr (MASTER) widen8(wm, w); else widen8(wp, w);
    }
    if (p.grad_scale) {
      const float scale = *p.grad_scale;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(g[j], scale);
    }
    const Two beta1(s.beta1, s.beta1), one_beta1(s.one_beta1, s.one_beta1), beta2(s.beta2, s.beta2),
        one_beta2(s.one_beta2, s.one_beta2);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const Two gg(g[j], g[j + 1]);
      const float2 mm = add(mul(Two(m[j], m[j + 1]), beta1).get(), mul(gg, one_beta1).get());
      const float2 vv = add(mul(Two(v[j], v[j + 1]), beta2).get(), mul(mul(gg, gg), one_beta2).get());
      m[j] = mm.x; m[j + 1] = mm.y;
      v[j] = vv.x; v[j + 1] = vv.y;
    }
    float root[8], m_most, m_least, v_most, v_least, r_most, r_least;   // (roots have the order of their squares)
    magnitudes(m, m_most, m_least);
    magnitudes(v, v_most, v_least);
    // the divisor, root * root_scale + eps, below zero: what quotients() takes
    const Two root_scale(-s.root_scale, -s.root_scale), decay(s.decay, s.decay), rate(-s.rate, -s.rate);
    const float2 eps = make_float2(-s.eps, -s.eps);
    if (p.narrow && v_least >= 0x1p-100f && v_most <= 0x1p100f && m_least >= 0x1p-60f && m_most <= 0x1p60f) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const Two rt = roots(make_float2(v[j], v[j + 1]));
        const Two q = quotients(Two(m[j], m[j + 1]), add(mul(rt, root_scale).get(), eps));
        const float2 ww = add(mul(Two(w[j], w[j + 1]), decay).get(), mul(q, rate).get()), rr = rt.get();
        root[j] = rr.x; root[j + 1] = rr.y;
        w[j] = ww.x; w[j + 1] = ww.y;
      }
      if constexpr (SMALL) {
        const float2 r = roots(make_float2(v_most, v_least)).get();
        r_most = r.x;
        r_least = r.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        root[j] = __fsqrt_rn(v[j]);
        const float d = __fadd_rn(__fmul_rn(root[j], s.root_scale), s.eps);
        w[j] = __fadd_rn(__fmul_rn(w[j], s.decay), -__fmul_rn(__fdiv_rn(m[j], d), s.rate));
      }
      r_most = __fsqrt_rn(v_most);
      r_least = __fsqrt_rn(v_least);
    }
    uint4 numbers[3];
    if constexpr (SMALL || DRAWN) {
      // the place's counter: its group of eight, the tensor and what is rounded
      const uint32_t tensor = 4u * (uint32_t)(p.first_tensor + lo), group = (uint32_t)(at >> 3);
      constexpr int from = SMALL ? 0 : 2, count = (SMALL ? 2 : 0) + (DRAWN ? 1 : 0);
      uint4 c[count];
#pragma unroll
      for (int i = 0; i < count; ++i) c[i] = make_uint4(group, tensor + from + i, o0, o1);
      philox4x32_10(c, p.k0, p.k1);
#pragma unroll
      for (int i = 0; i < count; ++i) numbers[from + i] = c[i];
    }
    if constexpr (SMALL) {
      uint2 mq, vq;
      const float ms = quantize8<false>(m, m_most, m_least, numbers[0], mq);
      const float vs = quantize8<true>(root, r_most, r_least, numbers[1], vq);
      if (live && (threadIdx.x & 15) == 0) {
        t.m_scale[block] = ms;
        t.v_scale[block] = vs;
      }
      uint8_t *mc = static_cast<uint8_t*>(t.m), *vc = static_cast<uint8_t*>(t.v);
      if (vec) {
        *reinterpret_cast<uint2*>(mc + at) = mq;
        *reinterpret_cast<uint2*>(vc + at) = vq;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (at + j < n) {
            mc[at + j] = (uint8_t)((j < 4 ? mq.x : mq.y) >> (8 * (j & 3)));
            vc[at + j] = (uint8_t)((j < 4 ? vq.x : vq.y) >> (8 * (j & 3)));
          }
        }
      }
    } else {
      put8(static_cast<float*>(t.m), at, n, vec, narrow8<float>(m));
      put8(static_cast<float*>(t.v), at, n, vec, narrow8<float>(v));
    }
    if constexpr (MASTER) put8(t.master, at, n, vec, narrow8<float>(w));
    if constexpr (DRAWN) {
      // the upper 16 bits are what bf16 keeps; not finite: as it is
      uint32_t words[4];
      float most, least;
      magnitudes(w, most, least);
      if (most < INFINITY) {
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          words[j >> 1] = __byte_perm(__float_as_uint(w[j]) + number_of(numbers[2], j),
                                      __float_as_uint(w[j + 1]) + number_of(numbers[2], j + 1), 0x7632);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          uint32_t lo = __float_as_uint(w[j]), hi = __float_as_uint(w[j + 1]);
          if (fabsf(w[j]) < INFINITY) lo += number_of(numbers[2], j);
          if (fabsf(w[j + 1]) < INFINITY) hi += number_of(numbers[2], j + 1);
          words[j >> 1] = __byte_perm(lo, hi, 0x7632);
        }
      }
      Raw8<TP> out;
      *reinterpret_cast<uint4*>(&out) = make_uint4(words[0], words[1], words[2], words[3]);
      put8(static_cast<TP*>(t.param), at, n, vec, out);
    } else {
      put8(static_cast<TP*>(t.param), at, n, vec, narrow8<TP>(w));
    }
  }
}

template <int N, typename TP, typename TG, bool MASTER>
cudaError_t adamw_bits(const AdamwTensor* t, const AdamwParams& p, bool small, int64_t blocks, cudaStream_t s) {
  AdamwList<N> list;
  for (int i = 0; i < p.n; ++i) list.t[i] = t[i];
  list.p = p;
  const dim3 grid((unsigned)blocks), threads(kAdamThreads);
  if (small)
    return p.offset_dev ? launch_pdl(adamw_kernel<N, TP, TG, MASTER, true, true>, grid, threads, 0, s, list)
                        : launch_pdl(adamw_kernel<N, TP, TG, MASTER, true, false>, grid, threads, 0, s, list);
  if constexpr (!MASTER && sizeof(TP) == 2) {   // bf16 alone: its rounding draws numbers
    if (p.offset_dev) return launch_pdl(adamw_kernel<N, TP, TG, MASTER, false, true>, grid, threads, 0, s, list);
  }
  return launch_pdl(adamw_kernel<N, TP, TG, MASTER, false, false>, grid, threads, 0, s, list);
}

// A launch's table lies in its arguments: a short one where it does.
template <typename TP, typename TG, bool MASTER>
cudaError_t adamw_table(const AdamwTensor* t, const AdamwParams& p, bool small, int64_t blocks, cudaStream_t s) {
  return p.n <= kAdamwFew ? adamw_bits<kAdamwFew, TP, TG, MASTER>(t, p, small, blocks, s)
                          : adamw_bits<kAdamwMost, TP, TG, MASTER>(t, p, small, blocks, s);
}

}  // namespace

int64_t adamw_blocks(int64_t numel, int turns) {
  return (numel + (int64_t)kAdamChunk * turns - 1) / ((int64_t)kAdamChunk * turns);
}

// With states in 8 bits a block takes up to eight chunks, as long as there are two blocks
// for each that is resident (four a multiprocessor).  Measured on 201 M values with one,
// two, four, eight and sixteen: 697, 687, 647, 621, 620 us, with rate and step number on
// the device 919, 750, 691, 649, 634; with states in 32 bits 846, 859, 887, 891, 892.
int adamw_turns(int64_t chunks, bool small) {
  const int64_t most = chunks / ((int64_t)device_info()->sm_count * 8);
  return !small || most < 1 ? 1 : most < 8 ? (int)most : 8;
}

cudaError_t launch_adamw(const AdamwTensor* t, const AdamwParams& p, int param_dtype, int grad_dtype, bool master,
                         bool small, int64_t blocks, cudaStream_t s) {
  const bool g32 = grad_dtype == MOE_DT_F32;
  if (param_dtype == MOE_DT_F32) return adamw_table<float, float, false>(t, p, small, blocks, s);
  if (param_dtype == MOE_DT_F16)
    return g32 ? adamw_table<__half, float, true>(t, p, small, blocks, s)
               : adamw_table<__half, __half, true>(t, p, small, blocks, s);
  if (master)
    return g32 ? adamw_table<__nv_bfloat16, float, true>(t, p, small, blocks, s)
               : adamw_table<__nv_bfloat16, __nv_bfloat16, true>(t, p, small, blocks, s);
  return g32 ? adamw_table<__nv_bfloat16, float, false>(t, p, small, blocks, s)
             : adamw_table<__nv_bfloat16, __nv_bfloat16, false>(t, p, small, blocks, s);
}

}  // namespace moe
