// Quantiser and its inverse of 4-bit weights with group scales (sm_103a); the
// format is described in w4.cuh.  One read and one write.  The quantiser is bound by
// issue (85% of the slots): 297 instructions for eight columns, most of them the
// divisions, 2.1-2.4 TB/s (4096 x 4096 20.0 us, 131072 x 4096 573 us, bf16,
// groups of 128); the inverse by the fp32 values that it writes, 4.3-5.2 TB/s (17.4
// and 466 us).
#include "block.cuh"
#include "block.h"
#include "kernels.h"

namespace moe {

namespace {

// ------------------------------------------------------------------ quantiser
// A thread takes eight columns, G / 8 lanes a group: scale = max|w| / 7 rounded
// to the weights' type, code = w / scale rounded to nearest even, plus 8.  The
// maximum is that of the bits of |w|, which order as the values do, infinity above
// all numbers and NaN above infinity: a group with either gets a NaN for its scale
// (no scale stands for it, and a number would hide it).
template <typename T>
__global__ void __launch_bounds__(256) quantize_w4_kernel(int64_t n8, int group,
                                                          const T* __restrict__ src,
                                                          uint32_t* __restrict__ q,
                                                          T* __restrict__ scales) {
  pdl_begin();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int lanes = group / 8;
  float v[8];
  uint32_t two = 0;   // the maxima of even and odd columns
  if (i < n8) {
    const Raw8<T> r = load8<T, 8>(src + i * 8, 0, 1, 8);
    const uint32_t* pair = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int j = 0; j < 4; ++j) two = __vmaxu2(two, pair[j] & 0x7FFF7FFFu);
    widen8(r, v);
  }
  for (int off = 1; off < lanes; off <<= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, off));
  if (i >= n8) return;
  const uint16_t top = (uint16_t)max(two & 0xFFFFu, two >> 16);
  const float amax = Elem<T>::to_f(*reinterpret_cast<const T*>(&top));
  const T st = Elem<T>::from_f((amax < INFINITY ? amax : NAN) / 7.0f);
  const float s = Elem<T>::to_f(st);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int z = s > 0.0f ? __float2int_rn(v[j] / s) : 0;   // scale zero or NaN: code 8
    w |= (uint32_t)(min(max(z, -8), 7) + 8) << (4 * j);
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

}  // namespace moe
