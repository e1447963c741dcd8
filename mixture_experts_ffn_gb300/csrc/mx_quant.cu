// Rows to microscaled floats and back (mx_dev.cuh holds the formats and their
// scale rules).  One pass: eight consecutive columns a thread, so four
// neighbouring lanes own a 32-column block and agree on its scale with two
// shuffles.  Bound by HBM: a bf16 element moves 2 bytes in and 33/32 (e4m3)
// or 17/32 (e2m1) out.  184320 x 2880 bf16: to e2m1 242 us, to e4m3 271, back
// from e2m1 236, from e4m3 263 (5.5 to 6.1 TB/s); the next item's load is issued
// before an item is converted (4% faster), four items a thread in flight were
// slower (by 30%).
#include <algorithm>
#include <type_traits>

#include "mx_dev.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Item i: columns 8 (i % ipr) .. of row i / ipr, ipr = Kp / 8 (a multiple of
// 16, so a block's four lanes never straddle two rows).  A thread's next item
// is a grid's width on: row and column advance by fixed amounts, so the loop
// divides nothing (6% of the time to e2m1).
struct Walk {
  uint32_t i, row, col, ipr, step, drow, dcol;
  __device__ __forceinline__ explicit Walk(uint32_t ipr_) {
    ipr = ipr_;
    i = blockIdx.x * kThreads + threadIdx.x;
    step = gridDim.x * kThreads;
    row = i / ipr;
    col = i - row * ipr;
    drow = step / ipr;
    dcol = step - drow * ipr;
  }
  __device__ __forceinline__ void next() {
    i += step;
    row += drow;
    col += dcol;
    if (col >= ipr) {
      col -= ipr;
      ++row;
    }
  }
};

// Largest magnitude of a 16-byte vector of bfloat16, as float bits: the bits
// of a magnitude order as the magnitudes do, two at a time.
__device__ __forceinline__ uint32_t amax_bf16x8(const uint4& u) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
  return max(a & 0xffff0000u, a << 16);
}

template <typename T, bool E2M1, bool VEC>
__global__ void __launch_bounds__(kThreads)
    mx_quantize_kernel(const T* __restrict__ x, int64_t stride, uint32_t items, int K, int Kp,
                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  pdl_launch();
  pdl_wait();
  // the lanes of a warp leave the loop together: items is a multiple of 16
  // and a block is four lanes, so a shuffle's partners are in or out as one
  const uint32_t mask = 0xfu << (threadIdx.x & 28);
  auto finish = [&](uint32_t i, float (&v)[8], uint32_t amax) {
    amax = max(amax, __shfl_xor_sync(mask, amax, 1));
    amax = max(amax, __shfl_xor_sync(mask, amax, 2));
    const uint32_t byte = mx::scale_byte<E2M1>(amax);
    mx::scale8(v, mx::inv_scale(byte));
    if constexpr (E2M1)
      reinterpret_cast<uint32_t*>(codes)[i] = mx::e2m1x8(v);
    else
      reinterpret_cast<uint2*>(codes)[i] = mx::e4m3x8(v);
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
  };
  Walk w((uint32_t)Kp / 8);
  if constexpr (VEC && sizeof(T) == 2) {
    // the next item's 16 bytes are in flight while this one is converted
    auto fetch = [&]() {
      const int c0 = (int)w.col * 8;
      return w.i < items && c0 < K
                 ? __ldcs(reinterpret_cast<const uint4*>(x + (int64_t)w.row * stride + c0))
                 : make_uint4(0, 0, 0, 0);
    };
    uint4 next = fetch();
    while (w.i < items) {
      const uint4 u = next;
      const uint32_t i = w.i;
      w.next();
      next = fetch();
      constexpr bool F16 = std::is_same<T, __half>::value;
      float v[8] = {lo16<F16>(u.x), hi16<F16>(u.x), lo16<F16>(u.y), hi16<F16>(u.y),
                    lo16<F16>(u.z), hi16<F16>(u.z), lo16<F16>(u.w), hi16<F16>(u.w)};
      uint32_t amax = 0;
      if constexpr (F16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, mx::abs_bits(v[j]));
      } else {
        amax = amax_bf16x8(u);
      }
      finish(i, v, amax);
    }
  } else {
    for (; w.i < items; w.next()) {
      float v[8];
      mx::load8<T, VEC>(x + (int64_t)w.row * stride, (int)w.col * 8, K, v);
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, mx::abs_bits(v[j]));
      finish(w.i, v, amax);
    }
  }
}

template <typename T, bool E2M1, bool VEC>
__global__ void __launch_bounds__(kThreads)
    mx_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                         uint32_t items, int K, int Kp, T* __restrict__ out) {
  pdl_launch();
  pdl_wait();
  Walk w((uint32_t)Kp / 8);
  uint2 next = make_uint2(0, 0);
  uint32_t next_byte = 0;
  auto fetch = [&]() {  // the next item's codes and scale, in flight while this one is converted
    if (w.i >= items) return;
    if constexpr (E2M1)
      next.x = __ldcs(reinterpret_cast<const uint32_t*>(codes) + w.i);
    else
      next = __ldcs(reinterpret_cast<const uint2*>(codes) + w.i);
    next_byte = scales[w.i >> 2];
  };
  fetch();
  while (w.i < items) {
    const uint2 q = next;
    const float s = mx::scale_value(next_byte);
    const int c0 = (int)w.col * 8;
    T* o = out + (int64_t)w.row * K;
    w.next();
    fetch();
    if (c0 >= K) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __half2 h;
      if constexpr (E2M1)
        h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(q.x >> (8 * j)), __NV_E2M1);
      else
        h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)((j < 2 ? q.x : q.y) >> (16 * (j & 1))), __NV_E4M3);
      const float2 f = __half22float2(h);
      v[2 * j] = f.x * s;
      v[2 * j + 1] = f.y * s;
    }
    mx::store8<T, VEC>(o, c0, K, v);
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
