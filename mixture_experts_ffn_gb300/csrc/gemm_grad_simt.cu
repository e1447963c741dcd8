// Gradients of a grouped product out = a w_e^T + b_e over the expert-segmented
// row layout, in float32 FMA (float32 operands, and shapes that the tensor-core
// kernels cannot address):
//   d_a[m, k] = sum_n d[m, n] w_e[n, k]           (m in expert e's segment)
//   d_w_e[n, k] = sum_{m in e} d[m, n] a[m, k],   d_b_e[n] = sum_{m in e} d[m, n]
// Both are C = X Y with Y read along its rows; X is read along its rows for d_a
// and along its columns for d_w.  Tile 64 x 128 outputs, 16 terms of the sum a
// step, 4 x 8 outputs a thread; the next step's operands are in registers while
// a step is summed.  Bound by the float32 pipes (and, for d_w of few rows, by
// writing d_w).
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int GM = 64, GN = 128, GK = 16;
constexpr int kThreads = 256;

// X(i, q): output row i, term q.  Row i of the tile, i < mi valid, and terms
// q < nq: element i * ldx + q (d_a) or q * ldx + i (d_w) of x.
template <typename T, bool WGRAD>
__device__ __forceinline__ void grad_tile(const T* __restrict__ x, size_t ldx, int mi,
                                          const T* __restrict__ y, size_t ldy, int nj, int nq,
                                          T* __restrict__ c, size_t ldc,
                                          float (&Xs)[GK][GM + 4], float (&Ys)[GK][GN + 4]) {
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float acc[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  float xr[4], yr[8];
  auto fetch = [&](int q0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int idx = tid + r * kThreads;
      const int i = WGRAD ? idx & 63 : idx >> 4, q = q0 + (WGRAD ? idx >> 6 : idx & 15);
      xr[r] = i < mi && q < nq ? Elem<T>::to_f(x[WGRAD ? q * ldx + i : i * ldx + q]) : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int idx = tid + r * kThreads;
      const int j = idx & 127, q = q0 + (idx >> 7);
      yr[r] = j < nj && q < nq ? Elem<T>::to_f(y[q * ldy + j]) : 0.0f;
    }
  };
  fetch(0);
  for (int q0 = 0; q0 < nq; q0 += GK) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int idx = tid + r * kThreads;
      if (WGRAD) Xs[idx >> 6][idx & 63] = xr[r];
      else Xs[idx & 15][idx >> 4] = xr[r];
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int idx = tid + r * kThreads;
      Ys[idx >> 7][idx & 127] = yr[r];
    }
    __syncthreads();
    if (q0 + GK < nq) fetch(q0 + GK);
#pragma unroll
    for (int q = 0; q < GK; ++q) {
      const float4 xv = *reinterpret_cast<const float4*>(&Xs[q][ty * 4]);
      const float4 y0 = *reinterpret_cast<const float4*>(&Ys[q][tx * 4]);
      const float4 y1 = *reinterpret_cast<const float4*>(&Ys[q][64 + tx * 4]);
      const float xa[4] = {xv.x, xv.y, xv.z, xv.w};
      const float ya[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(xa[i], ya[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (ty * 4 + i >= mi) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = (j >> 2) * 64 + tx * 4 + (j & 3);
      if (col < nj) c[(size_t)(ty * 4 + i) * ldc + col] = Elem<T>::from_f(acc[i][j]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    dgrad_simt_kernel(const T* __restrict__ d, const T* __restrict__ w,
                      const int32_t* __restrict__ seg_end, int M, int N, int K, int E,
                      T* __restrict__ d_a) {
  __shared__ float Xs[GK][GM + 4], Ys[GK][GN + 4];
  __shared__ int prefix[kMaxExperts + 1];
  __shared__ int scan_tmp[33];
  pdl_wait();
  const int n_tiles = (K + GN - 1) / GN;
  const int total = build_tile_prefix(seg_end, E, M, GM, n_tiles, prefix, scan_tmp);
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const SegTile st = decode_tile(tile, prefix, seg_end, E, M, GM, n_tiles);
    const int k0 = st.n_idx * GN;
    grad_tile<T, false>(d + (size_t)st.m0 * N, N, st.m_end - st.m0,
                        w + (size_t)st.e * N * K + k0, K, K - k0, N,
                        d_a + (size_t)st.m0 * K + k0, K, Xs, Ys);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    wgrad_simt_kernel(const T* __restrict__ d, const T* __restrict__ a,
                      const int32_t* __restrict__ seg_end, int M, int N, int K, int E,
                      T* __restrict__ d_w) {
  __shared__ float Xs[GK][GM + 4], Ys[GK][GN + 4];
  pdl_wait();
  const long long tn = (N + GM - 1) / GM, tk = (K + GN - 1) / GN;
  for (long long tile = blockIdx.x; tile < tn * tk * E; tile += gridDim.x) {
    const int e = (int)(tile / (tn * tk));
    const long long in = tile - e * (tn * tk);
    const int n0 = (int)(in / tk) * GM, k0 = (int)(in % tk) * GN;
    int lo, hi;
    seg_bounds(seg_end, e, M, 0, lo, hi);
    grad_tile<T, true>(d + (size_t)lo * N + n0, N, N - n0, a + (size_t)lo * K + k0, K, K - k0,
                       hi - lo, d_w + ((size_t)e * N + n0) * K + k0, K, Xs, Ys);
  }
}

// Column sums of d over every expert's rows: a CTA takes 32 columns of an
// expert, its warps the rows in turn, and the warps' sums are added in order.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    bias_grad_kernel(const T* __restrict__ d, const int32_t* __restrict__ seg_end, int M, int N,
                     T* __restrict__ d_bias) {
  __shared__ float part[kThreads / 32][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.y, n = blockIdx.x * 32 + lane;
  int lo, hi;
  seg_bounds(seg_end, e, M, 0, lo, hi);
  float sum = 0.0f;
  if (n < N)
    for (int m = lo + warp; m < hi; m += kThreads / 32) sum += Elem<T>::to_f(d[(size_t)m * N + n]);
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && n < N) {
    for (int i = 1; i < kThreads / 32; ++i) sum += part[i][lane];
    d_bias[(size_t)e * N + n] = Elem<T>::from_f(sum);
  }
}

template <typename T>
cudaError_t dgrad_t(const void* d, const void* w, const int32_t* seg_end, int M, int N, int K,
                    int E, void* d_a, cudaStream_t s) {
  const long long tiles = (long long)((M + GM - 1) / GM + E) * ((K + GN - 1) / GN);
  const auto kern = dgrad_simt_kernel<T>;
  const long long cap = (long long)num_sms() * resident_ctas((const void*)kern, kThreads);
  const cudaError_t e = launch_pdl(kern, dim3((unsigned)std::min(tiles, cap)), dim3(kThreads), 0,
                                   s, static_cast<const T*>(d), static_cast<const T*>(w), seg_end,
                                   M, N, K, E, static_cast<T*>(d_a));
  count_launch();
  return e;
}
template <typename T>
cudaError_t wgrad_t(const void* d, const void* a, const int32_t* seg_end, int M, int N, int K,
                    int E, void* d_w, cudaStream_t s) {
  const long long tiles = (long long)((N + GM - 1) / GM) * ((K + GN - 1) / GN) * E;
  const auto kern = wgrad_simt_kernel<T>;
  const long long cap = (long long)num_sms() * resident_ctas((const void*)kern, kThreads);
  const cudaError_t e = launch_pdl(kern, dim3((unsigned)std::min(tiles, cap)), dim3(kThreads), 0,
                                   s, static_cast<const T*>(d), static_cast<const T*>(a), seg_end,
                                   M, N, K, E, static_cast<T*>(d_w));
  count_launch();
  return e;
}
template <typename T>
cudaError_t bias_t(const void* d, const int32_t* seg_end, int M, int N, int E, void* d_bias,
                   cudaStream_t s) {
  const cudaError_t e = launch_pdl(bias_grad_kernel<T>, dim3((N + 31) / 32, E), dim3(kThreads), 0,
                                   s, static_cast<const T*>(d), seg_end, M, N,
                                   static_cast<T*>(d_bias));
  count_launch();
  return e;
}

}  // namespace

cudaError_t launch_dgrad_simt(const void* d, const void* w, const int32_t* seg_end, int M, int N,
                              int K, int E, moe_dtype dt, void* d_a, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  if (dt == MOE_BF16) return dgrad_t<__nv_bfloat16>(d, w, seg_end, M, N, K, E, d_a, s);
  if (dt == MOE_F16) return dgrad_t<__half>(d, w, seg_end, M, N, K, E, d_a, s);
  return dgrad_t<float>(d, w, seg_end, M, N, K, E, d_a, s);
}

cudaError_t launch_wgrad_simt(const void* d, const void* a, const int32_t* seg_end, int M, int N,
                              int K, int E, moe_dtype dt, void* d_w, cudaStream_t s) {
  if (dt == MOE_BF16) return wgrad_t<__nv_bfloat16>(d, a, seg_end, M, N, K, E, d_w, s);
  if (dt == MOE_F16) return wgrad_t<__half>(d, a, seg_end, M, N, K, E, d_w, s);
  return wgrad_t<float>(d, a, seg_end, M, N, K, E, d_w, s);
}

cudaError_t launch_bias_grad(const void* d, const int32_t* seg_end, int M, int N, int E,
                             moe_dtype dt, void* d_bias, cudaStream_t s) {
  if (dt == MOE_BF16) return bias_t<__nv_bfloat16>(d, seg_end, M, N, E, d_bias, s);
  if (dt == MOE_F16) return bias_t<__half>(d, seg_end, M, N, E, d_bias, s);
  return bias_t<float>(d, seg_end, M, N, E, d_bias, s);
}

}  // namespace moe
