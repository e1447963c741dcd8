// Device helpers of the microscaled (MX) formats: 32 consecutive columns of a
// row share one power-of-two scale (e8m0: byte s stands for 2^(s - 127), 255
// for NaN) and hold e4m3 (8-bit) or e2m1 (4-bit) codes.
//
// Scale rules, on the bits of the block's largest magnitude `amax`:
//   e2m1  2^(floor(log2 amax) - 2): the block's exponent maps onto e2m1's
//         largest (4 = 2^2); magnitudes above 6 saturate (the conversion of
//         the OCP Microscaling Formats specification v1.0, section 6.3)
//   e4m3  the smallest power of two with amax / scale <= 448, one more than
//         the same rule gives when amax's mantissa is above 1.75: nothing
//         saturates, and the step lost is the format's own exponent range
// A block of zeros (and any amax too small for its scale) takes 2^-127; a
// block that holds an infinity or a NaN takes the NaN scale and zero codes.
// Multiplying by the inverse scale is exact up to values that round to zero,
// so the codes are the correctly rounded (ties to even) quotients.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

// Lets the next kernel of the stream start its set-up as soon as every CTA of
// this grid has started (it still waits for this grid's end in pdl_wait).
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

namespace mx {

constexpr int kBlock = 32;   // columns of one scale
constexpr int kPad = 128;    // rows are padded to a multiple of this many columns
constexpr uint32_t kInfBits = 0x7f800000u;

__host__ __device__ __forceinline__ int padded(int K) { return (K + kPad - 1) / kPad * kPad; }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// e8m0 byte of a block with largest magnitude bits `amax` (E2M1: 4-bit codes)
template <bool E2M1>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= kInfBits) return 255u;
  const int e = (int)(amax >> 23);  // biased; 0 for zero and subnormals
  const int s = E2M1 ? e - 2 : e - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(s, 0);
}
// 1 / scale (exact; scale bytes are at most 252 here, 0 for the NaN scale so
// that its codes come out zero)
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// value of a scale byte
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}

// A zero inverse scale marks a block with a non-finite value: 0 * inf is NaN,
// so its values are replaced before the conversion.
__device__ __forceinline__ float scaled(float v, float inv) { return inv == 0.0f ? 0.0f : v * inv; }
__device__ __forceinline__ void scale8(float (&v)[8], float inv) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= inv;
  if (inv == 0.0f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}
// eight values, already divided by their scale, as e4m3 codes (column order)
__device__ __forceinline__ uint2 e4m3x8(const float (&q)[8]) {
  return make_uint2(e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16),
                    e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16));
}
__device__ __forceinline__ uint32_t e2m1x8(const float (&q)[8]) {
  return e2m1x2(q[0], q[1]) | (e2m1x2(q[2], q[3]) << 8) | (e2m1x2(q[4], q[5]) << 16) |
         (e2m1x2(q[6], q[7]) << 24);
}

// Eight consecutive elements of a row as float, columns c0 .. c0 + 7 of n
// (zeros past the end); VEC: the eight are whole and 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* __restrict__ p, int c0, int n, float (&v)[8]) {
  if constexpr (VEC) {
    if (c0 < n) {
      if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p + c0);
        const float4 b = *reinterpret_cast<const float4*>(p + c0 + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      } else {
        constexpr bool F16 = std::is_same<T, __half>::value;
        const uint4 u = *reinterpret_cast<const uint4*>(p + c0);
        v[0] = lo16<F16>(u.x); v[1] = hi16<F16>(u.x); v[2] = lo16<F16>(u.y); v[3] = hi16<F16>(u.y);
        v[4] = lo16<F16>(u.z); v[5] = hi16<F16>(u.z); v[6] = lo16<F16>(u.w); v[7] = hi16<F16>(u.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + i < n ? Elem<T>::to_f(p[c0 + i]) : 0.0f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* __restrict__ p, int c0, int n, const float (&v)[8]) {
  if constexpr (VEC) {
    if (c0 < n) {
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p + c0) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + c0 + 4) = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        constexpr bool F16 = std::is_same<T, __half>::value;
        *reinterpret_cast<uint4*>(p + c0) = make_uint4(pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]),
                                                       pack2<F16>(v[4], v[5]), pack2<F16>(v[6], v[7]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < n) p[c0 + i] = Elem<T>::from_f(v[i]);
  }
}

}  // namespace mx
}  // namespace moe
