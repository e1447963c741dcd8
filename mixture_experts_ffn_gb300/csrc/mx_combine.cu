// The weighted combine of the microscaled layer: out[t] = sum_k w[t, k] *
// y[row of route (t, k)], from the down product's float32 rows, in ascending k
// and rounded once.  Keeping y in float32 leaves the layer a single rounding
// of its output (error 1.7e-3 of the result in bfloat16; 2.4e-3 with y rounded
// too) for 2 more bytes a value of y: 2048 x 4 routes of 2880 columns, 94 MB,
// mostly stay inside the L2.  Bound by that traffic: y once in, out once.
#include <algorithm>
#include <type_traits>

#include "mx_dev.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 8;  // routes whose rows are in flight together

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads)
    mx_combine_kernel(const float* __restrict__ y, const float* __restrict__ w,
                      const int32_t* __restrict__ r2r, int Tn, int K, int H, int M,
                      T* __restrict__ out) {
  pdl_launch();
  pdl_wait();
  const int nvec = H / VEC;
  const long long items = (long long)Tn * nvec, step = (long long)gridDim.x * kThreads;
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < items; i += step) {
    const int t = (int)(i / nvec), v = (int)(i - (long long)t * nvec);
    float acc[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += kGroup) {
      int row[kGroup];
      float wk[kGroup], q[kGroup][VEC];
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        const bool in = k0 + j < K;
        row[j] = in ? __ldg(r2r + (size_t)t * K + k0 + j) : -1;
        wk[j] = in ? __ldg(w + (size_t)t * K + k0 + j) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        // a route without a row (an expert id out of range) adds nothing
        const bool ok = row[j] >= 0 && row[j] < M;
        const float* src = y + (size_t)(ok ? row[j] : 0) * H + (size_t)v * VEC;
        if constexpr (VEC == 4) {
          const float4 f = ok ? __ldg(reinterpret_cast<const float4*>(src)) : make_float4(0, 0, 0, 0);
          q[j][0] = f.x; q[j][1] = f.y; q[j][2] = f.z; q[j][3] = f.w;
        } else {
          q[j][0] = ok ? __ldg(src) : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[c] = fmaf(wk[j], q[j][c], acc[c]);
    }
    T* dst = out + (size_t)t * H + (size_t)v * VEC;
    if constexpr (VEC == 4) {
      constexpr bool F16 = std::is_same<T, __half>::value;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack2<F16>(acc[0], acc[1]), pack2<F16>(acc[2], acc[3]));
    } else {
      dst[0] = Elem<T>::from_f(acc[0]);
    }
  }
}

template <typename T, int VEC>
cudaError_t go(const float* y, const float* w, const int32_t* r2r, int T_, int K, int H, void* out,
               cudaStream_t s) {
  auto kern = mx_combine_kernel<T, VEC>;
  const long long items = (long long)T_ * (H / VEC);
  const long long cap = (long long)num_sms() * resident_ctas((const void*)kern, kThreads);
  const int grid =
      (int)std::max<long long>(1, std::min<long long>(cap, (items + kThreads - 1) / kThreads));
  cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kThreads), 0, s, y, w, r2r, T_, K, H, T_ * K,
                             static_cast<T*>(out));
  count_launch();
  return e;
}

}  // namespace

cudaError_t launch_mx_combine(const float* y, const float* w, const int32_t* route_to_row, int T,
                              int K, int H, moe_dtype dt, void* out, cudaStream_t s) {
  const bool vec = H % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 7) == 0;
  if (dt == MOE_F16)
    return vec ? go<__half, 4>(y, w, route_to_row, T, K, H, out, s)
               : go<__half, 1>(y, w, route_to_row, T, K, H, out, s);
  return vec ? go<__nv_bfloat16, 4>(y, w, route_to_row, T, K, H, out, s)
             : go<__nv_bfloat16, 1>(y, w, route_to_row, T, K, H, out, s);
}

}  // namespace moe
