// Rows to microscaled floats and back (mx_dev.cuh holds the formats and their
// scale rules).  One pass: eight consecutive columns a thread, so four
// neighbouring lanes own a 32-column block and agree on its scale with two
// shuffles.  Bound by HBM: a bf16 element moves 2 bytes in and 17/16 (e4m3)
// or 17/32 (e2m1) out.
#include <algorithm>
#include <type_traits>

#include "mx_dev.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// item i of the grid: columns 8 (i % ipr) .. of row i / ipr, ipr = Kp / 8 (a
// multiple of 16, so a block's four lanes never straddle two rows)
template <typename T, bool E2M1, bool VEC>
__global__ void __launch_bounds__(kThreads)
    mx_quantize_kernel(const T* __restrict__ x, int64_t stride, uint32_t items, int K, int Kp,
                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  pdl_wait();
  const uint32_t ipr = (uint32_t)Kp / 8;
  const uint32_t step = gridDim.x * kThreads;
  // the lanes of a warp leave the loop together: items is a multiple of 16
  // and a block is four lanes, so a shuffle's partners are in or out as one
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < items; i += step) {
    const uint32_t row = i / ipr;
    const int c0 = (int)(i - row * ipr) * 8;
    float v[8];
    mx::load8<T, VEC>(x + (int64_t)row * stride, c0, K, v);
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, mx::abs_bits(v[j]));
    const uint32_t mask = 0xfu << (threadIdx.x & 28);
    amax = max(amax, __shfl_xor_sync(mask, amax, 1));
    amax = max(amax, __shfl_xor_sync(mask, amax, 2));
    const uint32_t byte = mx::scale_byte<E2M1>(amax);
    const float inv = mx::inv_scale(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = mx::scaled(v[j], inv);
    if constexpr (E2M1)
      reinterpret_cast<uint32_t*>(codes)[i] = mx::e2m1x8(v);
    else
      reinterpret_cast<uint2*>(codes)[i] = mx::e4m3x8(v);
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
  }
}

template <typename T, bool E2M1, bool VEC>
__global__ void __launch_bounds__(kThreads)
    mx_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                         uint32_t items, int K, int Kp, T* __restrict__ out) {
  pdl_wait();
  const uint32_t ipr = (uint32_t)Kp / 8;
  const uint32_t step = gridDim.x * kThreads;
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < items; i += step) {
    const uint32_t row = i / ipr;
    const int c0 = (int)(i - row * ipr) * 8;
    if (c0 >= K) continue;
    const float s = mx::scale_value(scales[i >> 2]);
    float v[8];
    if constexpr (E2M1) {
      const uint32_t q = reinterpret_cast<const uint32_t*>(codes)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(q >> (8 * j)), __NV_E2M1);
        const float2 f = __half22float2(h);
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
    } else {
      const uint2 q = reinterpret_cast<const uint2*>(codes)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = j < 2 ? q.x : q.y;
        const __half2 h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w >> (16 * (j & 1))), __NV_E4M3);
        const float2 f = __half22float2(h);
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
    }
    mx::store8<T, VEC>(out + (int64_t)row * K, c0, K, v);
  }
}

// at most one resident round of CTAs (a grid-stride loop takes the rest)
int grid_for(const void* kernel, uint32_t items) {
  const long long want = ((long long)items + kThreads - 1) / kThreads;
  return (int)std::min<long long>(want, (long long)num_sms() * resident_ctas(kernel, kThreads));
}

template <typename T, bool E2M1, bool VEC>
cudaError_t quantize(const void* x, int64_t rows, int K, int64_t stride, void* codes,
                     void* scales, cudaStream_t s) {
  const int Kp = mx::padded(K);
  const uint32_t items = (uint32_t)(rows * (Kp / 8));
  auto kern = mx_quantize_kernel<T, E2M1, VEC>;
  cudaError_t e = launch_pdl(kern, dim3(grid_for((const void*)kern, items)), dim3(kThreads), 0, s,
                             static_cast<const T*>(x), stride, items, K, Kp,
                             static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
  count_launch();
  return e;
}
template <typename T, bool E2M1, bool VEC>
cudaError_t dequantize(const void* codes, const void* scales, int64_t rows, int K, void* out,
                       cudaStream_t s) {
  const int Kp = mx::padded(K);
  const uint32_t items = (uint32_t)(rows * (Kp / 8));
  auto kern = mx_dequantize_kernel<T, E2M1, VEC>;
  cudaError_t e = launch_pdl(kern, dim3(grid_for((const void*)kern, items)), dim3(kThreads), 0, s,
                             static_cast<const uint8_t*>(codes),
                             static_cast<const uint8_t*>(scales), items, K, Kp,
                             static_cast<T*>(out));
  count_launch();
  return e;
}

template <typename T>
cudaError_t quantize_t(const void* x, int64_t rows, int K, int64_t stride, int fmt, bool vec,
                       void* codes, void* scales, cudaStream_t s) {
  if (fmt == MOE_MX_E2M1)
    return vec ? quantize<T, true, true>(x, rows, K, stride, codes, scales, s)
               : quantize<T, true, false>(x, rows, K, stride, codes, scales, s);
  return vec ? quantize<T, false, true>(x, rows, K, stride, codes, scales, s)
             : quantize<T, false, false>(x, rows, K, stride, codes, scales, s);
}
template <typename T>
cudaError_t dequantize_t(const void* codes, const void* scales, int64_t rows, int K, int fmt,
                         bool vec, void* out, cudaStream_t s) {
  if (fmt == MOE_MX_E2M1)
    return vec ? dequantize<T, true, true>(codes, scales, rows, K, out, s)
               : dequantize<T, true, false>(codes, scales, rows, K, out, s);
  return vec ? dequantize<T, false, true>(codes, scales, rows, K, out, s)
             : dequantize<T, false, false>(codes, scales, rows, K, out, s);
}

}  // namespace

cudaError_t launch_mx_quantize(const void* x, int64_t rows, int K, int64_t stride, moe_dtype dt,
                               int fmt, void* codes, void* scales, cudaStream_t s) {
  const int64_t per16 = dt == MOE_F32 ? 4 : 8;  // elements of 16 bytes
  const bool vec = K % 8 == 0 && stride % per16 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  if (dt == MOE_F32) return quantize_t<float>(x, rows, K, stride, fmt, vec, codes, scales, s);
  if (dt == MOE_F16) return quantize_t<__half>(x, rows, K, stride, fmt, vec, codes, scales, s);
  return quantize_t<__nv_bfloat16>(x, rows, K, stride, fmt, vec, codes, scales, s);
}

cudaError_t launch_mx_dequantize(const void* codes, const void* scales, int64_t rows, int K,
                                 int fmt, moe_dtype dt, void* out, cudaStream_t s) {
  const bool vec = K % 8 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  if (dt == MOE_F32) return dequantize_t<float>(codes, scales, rows, K, fmt, vec, out, s);
  if (dt == MOE_F16) return dequantize_t<__half>(codes, scales, rows, K, fmt, vec, out, s);
  return dequantize_t<__nv_bfloat16>(codes, scales, rows, K, fmt, vec, out, s);
}

}  // namespace moe
