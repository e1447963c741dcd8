// Gradient of the weighted combine (moe_combine): with route r = t K + k in row
// row = route_to_row[r] and out[t] = c sum_k w[r] y[row],
//   d_y[row] = c w[r] d_out[t],   d_w[r] = c <d_out[t], y[row]>.
// One pass over y and d_out: a route's products with d_out[t] and its scaled
// copy come from the same registers.  Bound by HBM: y read, d_y written.
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// A warp takes a route; its lanes walk the row.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const T* __restrict__ d_out, const T* __restrict__ y,
                            const float* __restrict__ w, const int32_t* __restrict__ route_to_row,
                            int M, int K, int H, float scale, T* __restrict__ d_y,
                            float* __restrict__ d_w) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kThreads / 32);
  for (int r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < M; r += warps) {
    const int row = route_to_row[r];
    const bool ok = row >= 0 && row < M;
    float dot = 0.0f;
    if (ok) {
      const T* d = d_out + (size_t)(r / K) * H;
      const size_t at = (size_t)row * H;
      const float f = d_y ? scale * w[r] : 0.0f;
      for (int h = lane; h < H; h += 32) {
        const float v = Elem<T>::to_f(d[h]);
        if (d_w) dot = fmaf(v, Elem<T>::to_f(y[at + h]), dot);
        if (d_y) d_y[at + h] = Elem<T>::from_f(f * v);
      }
    }
    if (d_w) {
      dot = warp_sum(dot);
      if (lane == 0) d_w[r] = scale * dot;
    }
  }
}

template <typename T>
cudaError_t launch_t(const void* d_out, const void* y, const float* w, const int32_t* r2r, int M,
                     int K, int H, float scale, void* d_y, float* d_w, cudaStream_t s) {
  const auto kern = combine_backward_kernel<T>;
  const long long want = ((long long)M + kThreads / 32 - 1) / (kThreads / 32);
  const long long cap = (long long)num_sms() * resident_ctas((const void*)kern, kThreads);
  const cudaError_t e =
      launch_pdl(kern, dim3((unsigned)std::min(want, cap)), dim3(kThreads), 0, s,
                 static_cast<const T*>(d_out), static_cast<const T*>(y), w, r2r, M, K, H, scale,
                 static_cast<T*>(d_y), d_w);
  count_launch();
  return e;
}

}  // namespace

cudaError_t launch_combine_backward(const void* d_out, const void* y, const float* w,
                                    const int32_t* route_to_row, int T, int K, int H, moe_dtype dt,
                                    float scale, void* d_y, float* d_w, cudaStream_t s) {
  const int M = T * K;
  if (M == 0) return cudaSuccess;
  if (dt == MOE_BF16)
    return launch_t<__nv_bfloat16>(d_out, y, w, route_to_row, M, K, H, scale, d_y, d_w, s);
  if (dt == MOE_F16)
    return launch_t<__half>(d_out, y, w, route_to_row, M, K, H, scale, d_y, d_w, s);
  return launch_t<float>(d_out, y, w, route_to_row, M, K, H, scale, d_y, d_w, s);
}

}  // namespace moe
