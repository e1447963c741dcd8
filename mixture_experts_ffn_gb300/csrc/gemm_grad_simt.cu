// Gradients of a grouped product out = a w_e^T + b_e over the expert-segmented
// row layout, in float32 FMA (float32 operands, and shapes that the tensor-core
// kernels cannot address):
//   d_a[m, k] = sum_n d[m, n] w_e[n, k]           (m in expert e's segment)
//   d_w_e[n, k] = sum_{m in e} d[m, n] a[m, k],   d_b_e[n] = sum_{m in e} d[m, n]
// Both are C = X Y with Y read along its rows; X is read along its rows for d_a
// and along its columns for d_w.  256 threads a tile; the next step's operands are
// in registers while a step is summed.  Bound by the float32 pipes where tiles are
// many (38 TFLOP/s at 1024 rows an expert, 2048 x 2048, half the pipes' rate; the
// library's product 52: a step of 16 terms lies between two barriers, with scalar loads
// and 12 shared-memory values to 32 FMAs a thread), by the latency of a tile's steps
// where they are few, hence two tiles (pick_tile).  One expert of 2048 rows, 1024 x 1024:
// rows 127 us, weights 146, the library's products 78 and 79; 32 experts of 64, 512 x
// 512: 53 and 36, one library product an expert 450 and 135.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// BM x BN outputs, BM / 16 x BN / 16 of them a thread, BK terms of the sum a step.
template <int BM_, int BN_, int BK_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, BK = BK_, TM = BM / 16, TN = BN / 16;
  static constexpr int XR = BM * BK / kThreads, YR = BN * BK / kThreads;
  struct Shared {
    float x[BK][BM + 4], y[BK][BN + 4];
  };
};
// T consecutive values (T = 2, 4), or two runs of four half a tile apart (T = 8)
template <int T, int B>
__device__ __forceinline__ void take(const float* row, int t, float (&v)[T]) {
  if constexpr (T == 2) {
    const float2 a = *reinterpret_cast<const float2*>(row + 2 * t);
    v[0] = a.x; v[1] = a.y;
  } else {
#pragma unroll
    for (int h = 0; h < T / 4; ++h) {
      const float4 a = *reinterpret_cast<const float4*>(row + h * (B / 2) + 4 * t);
      v[4 * h] = a.x; v[4 * h + 1] = a.y; v[4 * h + 2] = a.z; v[4 * h + 3] = a.w;
    }
  }
}
template <int T, int B>
__device__ __forceinline__ int place(int t, int i) {
  return T == 2 ? 2 * t + i : 4 * t + (i & 3) + (i >> 2) * (B / 2);
}

// X(i, q): output row i, term q.  Row i of the tile, i < mi valid, and terms
// q < nq: element i * ldx + q (d_a) or q * ldx + i (d_w) of x.
template <typename T, bool WGRAD, class G>
__device__ __forceinline__ void grad_tile(const T* __restrict__ x, size_t ldx, int mi,
                                          const T* __restrict__ y, size_t ldy, int nj, int nq,
                                          T* __restrict__ c, size_t ldc, typename G::Shared& sh) {
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float acc[G::TM][G::TN];
#pragma unroll
  for (int i = 0; i < G::TM; ++i)
#pragma unroll
    for (int j = 0; j < G::TN; ++j) acc[i][j] = 0.0f;
  float xr[G::XR], yr[G::YR];
  auto xi = [&](int idx) { return WGRAD ? idx % G::BM : idx / G::BK; };
  auto xq = [&](int idx) { return WGRAD ? idx / G::BM : idx % G::BK; };
  auto fetch = [&](int q0) {
#pragma unroll
    for (int r = 0; r < G::XR; ++r) {
      const int i = xi(tid + r * kThreads), q = q0 + xq(tid + r * kThreads);
      xr[r] = i < mi && q < nq ? Elem<T>::to_f(x[WGRAD ? q * ldx + i : i * ldx + q]) : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < G::YR; ++r) {
      const int idx = tid + r * kThreads, j = idx % G::BN, q = q0 + idx / G::BN;
      yr[r] = j < nj && q < nq ? Elem<T>::to_f(y[q * ldy + j]) : 0.0f;
    }
  };
  fetch(0);
  for (int q0 = 0; q0 < nq; q0 += G::BK) {
#pragma unroll
    for (int r = 0; r < G::XR; ++r) sh.x[xq(tid + r * kThreads)][xi(tid + r * kThreads)] = xr[r];
#pragma unroll
    for (int r = 0; r < G::YR; ++r) {
      const int idx = tid + r * kThreads;
      sh.y[idx / G::BN][idx % G::BN] = yr[r];
    }
    __syncthreads();
    if (q0 + G::BK < nq) fetch(q0 + G::BK);
#pragma unroll 16
    for (int q = 0; q < G::BK; ++q) {
      float xv[G::TM], yv[G::TN];
      take<G::TM, G::BM>(sh.x[q], ty, xv);
      take<G::TN, G::BN>(sh.y[q], tx, yv);
#pragma unroll
      for (int i = 0; i < G::TM; ++i)
#pragma unroll
        for (int j = 0; j < G::TN; ++j) acc[i][j] = fmaf(xv[i], yv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < G::TM; ++i) {
    const int row = place<G::TM, G::BM>(ty, i);
    if (row >= mi) continue;
#pragma unroll
    for (int j = 0; j < G::TN; ++j) {
      const int col = place<G::TN, G::BN>(tx, j);
      if (col < nj) c[(size_t)row * ldc + col] = Elem<T>::from_f(acc[i][j]);
    }
  }
}

template <typename T, class G>
__global__ void __launch_bounds__(kThreads, 2)
    dgrad_simt_kernel(const T* __restrict__ d, const T* __restrict__ w,
                      const int32_t* __restrict__ seg_end, int M, int N, int K, int E,
                      T* __restrict__ d_a) {
  __shared__ __align__(16) typename G::Shared sh;
  __shared__ int prefix[kMaxExperts + 1];
  __shared__ int scan_tmp[33];
  pdl_wait();
  const int n_tiles = (K + G::BN - 1) / G::BN;
  const int total = build_tile_prefix(seg_end, E, M, G::BM, n_tiles, prefix, scan_tmp);
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const SegTile st = decode_tile(tile, prefix, seg_end, E, M, G::BM, n_tiles);
    const int k0 = st.n_idx * G::BN;
    grad_tile<T, false, G>(d + (size_t)st.m0 * N, N, st.m_end - st.m0,
                           w + (size_t)st.e * N * K + k0, K, K - k0, N,
                           d_a + (size_t)st.m0 * K + k0, K, sh);
  }
}

template <typename T, class G>
__global__ void __launch_bounds__(kThreads, 2)
    wgrad_simt_kernel(const T* __restrict__ d, const T* __restrict__ a,
                      const int32_t* __restrict__ seg_end, int M, int N, int K, int E,
                      T* __restrict__ d_w) {
  __shared__ __align__(16) typename G::Shared sh;
  pdl_wait();
  const long long tn = (N + G::BM - 1) / G::BM, tk = (K + G::BN - 1) / G::BN;
  for (long long tile = blockIdx.x; tile < tn * tk * E; tile += gridDim.x) {
    const int e = (int)(tile / (tn * tk));
    const long long in = tile - e * (tn * tk);
    const int n0 = (int)(in / tk) * G::BM, k0 = (int)(in % tk) * G::BN;
    int lo, hi;
    seg_bounds(seg_end, e, M, 0, lo, hi);
    grad_tile<T, true, G>(d + (size_t)lo * N + n0, N, N - n0, a + (size_t)lo * K + k0, K, K - k0,
                          hi - lo, d_w + ((size_t)e * N + n0) * K + k0, K, sh);
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
  if (n < N) {
#pragma unroll 8
    for (int m = lo + warp; m < hi; m += kThreads / 32) sum += Elem<T>::to_f(d[(size_t)m * N + n]);
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && n < N) {
    for (int i = 1; i < kThreads / 32; ++i) sum += part[i][lane];
    d_bias[(size_t)e * N + n] = Elem<T>::from_f(sum);
  }
}

// 64 x 128 outputs a tile where that gives two SMs of five one; where it does not, 32 x
// 32 with four times the terms a step, whose latency then bounds.  2000 rows, 50 x 1000,
// d_w (8 wide tiles): 143 us with the wide tile, 39 with the small one; 3 experts of 100
// rows, 1000 x 1000, d_a (48): 75 and 54; 32 of 64 rows, 2048 x 300 (96): 175 and 213.
// (128 x 128 gains 5 to 12% at 1024 rows an expert and loses as much at 64.)
using Wide = Tile<64, 128, 16>;
using Small = Tile<32, 32, 64>;
template <typename Fn>
cudaError_t pick_tile(long long row_tiles, long long cols, Fn f) {
  if (row_tiles * ((cols + Wide::BN - 1) / Wide::BN) * 5 >= 2 * num_sms()) return f(Wide{});
  return f(Small{});
}

template <typename T>
cudaError_t dgrad_t(const void* d, const void* w, const int32_t* seg_end, int M, int N, int K,
                    int E, void* d_a, cudaStream_t s) {
  // an expert with rows has a tile at least
  const int row_tiles = std::max((M + Wide::BM - 1) / Wide::BM, std::min(E, M));
  return pick_tile(row_tiles, K, [&](auto tile) {
    using G = decltype(tile);
    const long long tiles = ((long long)(M + G::BM - 1) / G::BM + E) * ((K + G::BN - 1) / G::BN);
    const auto kern = dgrad_simt_kernel<T, G>;
    const long long cap = (long long)num_sms() * resident_ctas((const void*)kern, kThreads);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)std::min(tiles, cap)), dim3(kThreads), 0,
                                     s, static_cast<const T*>(d), static_cast<const T*>(w),
                                     seg_end, M, N, K, E, static_cast<T*>(d_a));
    count_launch();
    return e;
  });
}
template <typename T>
cudaError_t wgrad_t(const void* d, const void* a, const int32_t* seg_end, int M, int N, int K,
                    int E, void* d_w, cudaStream_t s) {
  return pick_tile((long long)((N + Wide::BM - 1) / Wide::BM) * E, K, [&](auto tile) {
    using G = decltype(tile);
    const long long tiles =
        (long long)((N + G::BM - 1) / G::BM) * ((K + G::BN - 1) / G::BN) * E;
    const auto kern = wgrad_simt_kernel<T, G>;
    const long long cap = (long long)num_sms() * resident_ctas((const void*)kern, kThreads);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)std::min(tiles, cap)), dim3(kThreads), 0,
                                     s, static_cast<const T*>(d), static_cast<const T*>(a),
                                     seg_end, M, N, K, E, static_cast<T*>(d_w));
    count_launch();
    return e;
  });
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
