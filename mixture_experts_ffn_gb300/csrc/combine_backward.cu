// Gradient of the weighted combine (moe_combine): with route r = t K + k in row
// row = route_to_row[r] and out[t] = c sum_k w[r] y[row],
//   d_y[row] = c w[r] d_out[t],   d_w[r] = c <d_out[t], y[row]>.
// One pass over y and d_out: a route's products with d_out[t] and its scaled
// copy come from the same registers.  Bound by HBM: y read, d_y written (8192 tokens,
// top-8, 7168 columns, bf16: 311 us, 6.4 TB/s; the sum of the rows in permute.cu 166 us,
// 6.4 TB/s; a plain copy of as much as y here 276 us, 6.8 TB/s).
#include <algorithm>
#include <type_traits>

#include "mx_dev.cuh"

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
  const long long warps = gridDim.x * (kThreads / 32);
  for (long long r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < M; r += warps) {
    const int row = route_to_row[r];
    const bool ok = row >= 0 && row < M;
    float dot = 0.0f;
    if (ok) {
      const T* d = d_out + (size_t)((int)r / K) * H;
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

// 16 bytes of a row as floats.
template <typename T>
struct Chunk {
  static constexpr int N = 16 / sizeof(T);
  static __device__ __forceinline__ void get(const uint4& q, float (&v)[N]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 4) {
        v[i] = __uint_as_float(u[i]);
      } else {
        constexpr bool F16 = std::is_same<T, __half>::value;
        v[2 * i] = lo16<F16>(u[i]);
        v[2 * i + 1] = hi16<F16>(u[i]);
      }
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[N]) {
    if constexpr (N == 4) {
      return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                        __float_as_uint(v[3]));
    } else {
      constexpr bool F16 = std::is_same<T, __half>::value;
      return make_uint4(pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]), pack2<F16>(v[4], v[5]),
                        pack2<F16>(v[6], v[7]));
    }
  }
};

// LANES threads a route (a warp, or the whole CTA where routes are few), 16 bytes a
// thread, four of them in flight from each row.  Rows a multiple of 16 bytes, all
// 16-byte aligned.  The K routes of a token are neighbouring warps', so d_out[t]
// comes from the L1 cache but once.
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads)
    combine_backward_vec(const uint4* __restrict__ d_out, const uint4* __restrict__ y,
                         const float* __restrict__ w, const int32_t* __restrict__ route_to_row,
                         int M, int K, int n, float scale, uint4* __restrict__ d_y,
                         float* __restrict__ d_w) {
  constexpr int U = 4, N = Chunk<T>::N;
  __shared__ float part[kThreads / 32];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % LANES;
  const long long groups = gridDim.x * (kThreads / LANES);
  for (long long r = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES; r < M; r += groups) {
    const int row = route_to_row[r];
    float dot[U] = {};
    if (row >= 0 && row < M) {
      const uint4* d = d_out + (size_t)((int)r / K) * n;
      const uint4* src = y + (size_t)row * n;
      uint4* dst = d_y + (size_t)row * n;
      const float f = d_y ? scale * w[r] : 0.0f;
      for (int c0 = lane; c0 < n; c0 += U * LANES) {
        uint4 dq[U], yq[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int c = c0 + j * LANES;
          dq[j] = yq[j] = make_uint4(0, 0, 0, 0);
          if (c < n) {
            dq[j] = __ldg(d + c);
            if (d_w) yq[j] = __ldcs(src + c);
          }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int c = c0 + j * LANES;
          float dv[N], yv[N];
          Chunk<T>::get(dq[j], dv);
          Chunk<T>::get(yq[j], yv);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot[j] = fmaf(dv[i], yv[i], dot[j]);
            dv[i] *= f;
          }
          if (d_y && c < n) dst[c] = Chunk<T>::put(dv);
        }
      }
    }
    if (d_w) {
      float sum = warp_sum((dot[0] + dot[1]) + (dot[2] + dot[3]));
      if constexpr (LANES > 32) {
        __syncthreads();  // the last route's sums were read
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) sum += part[i];
      }
      if (lane == 0) d_w[r] = scale * sum;
    }
  }
}

template <typename T>
cudaError_t launch_t(const void* d_out, const void* y, const float* w, const int32_t* r2r, int M,
                     int K, int H, float scale, void* d_y, float* d_w, cudaStream_t s) {
  const auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  if ((size_t)H * sizeof(T) % 16 == 0 && a16(d_out) && a16(y) && a16(d_y)) {
    // a CTA each for few routes, so that eight warps share a row's latency: 24 routes of
    // 7168 columns 2.2 us against 5.5 with a warp each, 1024 of them 5.5 and 8.6; 2048 of
    // 2880 columns 7.5 and 6.0
    const bool few = M < 8 * num_sms();
    const auto kern = few ? combine_backward_vec<T, kThreads> : combine_backward_vec<T, 32>;
    const long long want = few ? M : ((long long)M + kThreads / 32 - 1) / (kThreads / 32);
    const long long cap = (long long)num_sms() * resident_ctas((const void*)kern, kThreads);
    const cudaError_t e = launch_pdl(
        kern, dim3((unsigned)std::min(want, cap)), dim3(kThreads), 0, s,
        static_cast<const uint4*>(d_out), static_cast<const uint4*>(y), w, r2r, M, K,
        (int)((size_t)H * sizeof(T) / 16), scale, static_cast<uint4*>(d_y), d_w);
    count_launch();
    return e;
  }
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
