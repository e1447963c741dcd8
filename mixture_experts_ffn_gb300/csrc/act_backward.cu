// The activation of a grouped product with an 8-bit checkpoint of its argument,
// and its gradient from that checkpoint.  p holds N1 columns a row, gate and up
// (stacked or interleaved) or one per output; the checkpoint is p as an MX e4m3
// row (mx_dev.cuh), 33/32 bytes a value.
//   silu  a = g s(g) u:      d_g = d u s (1 + g (1 - s)),  d_u = d g s
//   swiglu, G = min(g, limit), U = clamp(u, -limit, limit), s = sigmoid(alpha G),
//         a = G s (U + beta): d_g = d (U + beta) s (1 + alpha G (1 - s)) where
//         g <= limit, d_u = d G s where |u| <= limit, 0 past a clamp
//   gelu  a = g Phi(g) u:    d_g = d u (Phi(g) + g phi(g)), d_u = d g Phi(g)
//   relu  d where p > 0; identity d; gelu and silu without u as d_g with u = 1
// A NaN in p is a NaN in both results (the clamps keep it).  Elementwise; bound
// by HBM.
#include <algorithm>
#include <type_traits>

#include "mx_dev.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct ActArgs {
  int kind, gated, inter, F, N1, Np;
  float limit, alpha, beta;
};

// sigmoid(x) and 1 - sigmoid(x): float32 results take the exact exponential and
// quotient, 16-bit ones the fast forms (within 2^-20 of the value, against 2^-9
// and 2^-12 of the rounding that follows).
template <bool FAST>
__device__ __forceinline__ float sigmoid_t(float x) {
  if constexpr (FAST) return __fdividef(1.0f, 1.0f + __expf(-x));
  else return sigmoidf_(x);
}

// gelu's factor Phi(x); the complementary function keeps its digits for x < 0
__device__ __forceinline__ float phi_cdf(float x) {
  return 0.5f * erfcf(-0.70710678118654752f * x);
}
__device__ __forceinline__ float phi_pdf(float x) {
  return 0.39894228040143268f * expf(-0.5f * x * x);
}

// One gated pair: the activation a, and with d its gradients dg and du.
template <bool FAST>
__device__ __forceinline__ void gated_pair(int kind, float g, float u, float d, const ActArgs& A,
                                           float& a, float& dg, float& du) {
  if (kind == MOE_ACT_GELU_AND_MUL) {
    const float c = phi_cdf(g);
    a = g * c * u;
    dg = d * u * (c + g * phi_pdf(g));
    du = d * (g * c);
    return;
  }
  float G = g, U = u, alpha = 1.0f;
  bool past_g = false, past_u = false;
  if (kind == MOE_ACT_SWIGLU) {
    alpha = A.alpha;
    if (A.limit > 0.0f) {
      past_g = g > A.limit;
      past_u = fabsf(u) > A.limit;
      G = min_nan(g, A.limit);
      U = max_nan(min_nan(u, A.limit), -A.limit);
    }
    U += A.beta;
  }
  const float x = alpha * G;
  const float s = sigmoid_t<FAST>(x);
  const float gs = G * s;
  a = gs * U;
  dg = past_g ? 0.0f : d * U * s * fmaf(x, 1.0f - s, 1.0f);
  du = past_u ? 0.0f : d * gs;
}
// One value of a non-gated kind.
template <bool FAST>
__device__ __forceinline__ void plain_value(int kind, float p, float d, float& a, float& dp) {
  if (kind == MOE_ACT_RELU) {
    a = relu_f(p);
    dp = p != p ? p : p > 0.0f ? d : 0.0f;
  } else if (kind == MOE_ACT_GELU) {
    const float c = phi_cdf(p);
    a = p * c;
    dp = d * (c + p * phi_pdf(p));
  } else if (kind == MOE_ACT_SILU) {
    const float s = sigmoid_t<FAST>(p);
    a = p * s;
    dp = d * s * fmaf(p, 1.0f - s, 1.0f);
  } else {
    a = p;
    dp = d;
  }
}

// rows that hold routes: those below the last segment's end, or all M
__device__ __forceinline__ int live_rows(const int32_t* seg_end, int E, int M) {
  return seg_end ? min(max(seg_end[E - 1], 0), M) : M;
}

// Column of the gate and of the up value of output column j.
__device__ __forceinline__ int gate_col(const ActArgs& A, int j) { return A.inter ? 2 * j : j; }
__device__ __forceinline__ int up_col(const ActArgs& A, int j) {
  return A.inter ? 2 * j + 1 : A.F + j;
}

// Any width and alignment: a warp a row, a lane a column.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    act_checkpoint_any(const T* __restrict__ p, const int32_t* __restrict__ seg_end, int E, int M,
                       ActArgs A, T* __restrict__ out, uint8_t* __restrict__ codes,
                       uint8_t* __restrict__ scales) {
  pdl_wait();
  constexpr bool FAST = sizeof(T) == 2;
  const int lane = threadIdx.x & 31;
  const int rows = live_rows(seg_end, E, M);
  const int warps = gridDim.x * (kThreads / 32);
  for (int m = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); m < rows; m += warps) {
    const T* x = p + (size_t)m * A.N1;
    for (int c0 = 0; c0 < A.Np; c0 += 32) {
      const float v = c0 + lane < A.N1 ? Elem<T>::to_f(x[c0 + lane]) : 0.0f;
      const uint32_t byte =
          mx::scale_byte<false>(__reduce_max_sync(0xffffffffu, mx::abs_bits(v)));
      const float q = mx::scaled(v, mx::inv_scale(byte));
      codes[(size_t)m * A.Np + c0 + lane] = (uint8_t)mx::e4m3x2(q, 0.0f);
      if (lane == 0) scales[((size_t)m * A.Np + c0) >> 5] = (uint8_t)byte;
    }
    if (!out) continue;
    for (int j = lane; j < A.F; j += 32) {
      float a, dg, du;
      if (A.gated)
        gated_pair<FAST>(A.kind, Elem<T>::to_f(x[gate_col(A, j)]), Elem<T>::to_f(x[up_col(A, j)]),
                         0.0f, A, a, dg, du);
      else
        plain_value<FAST>(A.kind, Elem<T>::to_f(x[j]), 0.0f, a, dg);
      out[(size_t)m * A.F + j] = Elem<T>::from_f(a);
    }
  }
}

__device__ __forceinline__ float e4m3_value(uint8_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}

template <typename T, bool MX>
__global__ void __launch_bounds__(kThreads)
    act_backward_any(const void* __restrict__ p, const uint8_t* __restrict__ scales,
                     const T* __restrict__ d_out, const int32_t* __restrict__ seg_end, int E,
                     int M, ActArgs A, T* __restrict__ d_p, T* __restrict__ out) {
  pdl_wait();
  constexpr bool FAST = sizeof(T) == 2;
  const int lane = threadIdx.x & 31;
  const int rows = live_rows(seg_end, E, M);
  const int warps = gridDim.x * (kThreads / 32);
  for (int m = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); m < rows; m += warps) {
    auto value = [&](int c) {
      if constexpr (MX) {
        const size_t at = (size_t)m * A.Np + c;
        return e4m3_value(static_cast<const uint8_t*>(p)[at]) * mx::scale_value(scales[at >> 5]);
      } else {
        return Elem<T>::to_f(static_cast<const T*>(p)[(size_t)m * A.N1 + c]);
      }
    };
    for (int j = lane; j < A.F; j += 32) {
      const float d = Elem<T>::to_f(d_out[(size_t)m * A.F + j]);
      T* dst = d_p + (size_t)m * A.N1;
      float a, dg, du;
      if (A.gated) {
        gated_pair<FAST>(A.kind, value(gate_col(A, j)), value(up_col(A, j)), d, A, a, dg, du);
        dst[gate_col(A, j)] = Elem<T>::from_f(dg);
        dst[up_col(A, j)] = Elem<T>::from_f(du);
      } else {
        plain_value<FAST>(A.kind, value(j), d, a, dg);
        dst[j] = Elem<T>::from_f(dg);
      }
      if (out) out[(size_t)m * A.F + j] = Elem<T>::from_f(a);
    }
  }
}

ActArgs act_args(const moe_act_params& act, int F) {
  ActArgs A;
  A.kind = act.kind;
  A.gated = act_is_gated(act.kind) ? 1 : 0;
  A.inter = act.kind == MOE_ACT_SWIGLU && act.swiglu_fusion == 1 ? 1 : 0;
  A.F = F;
  A.N1 = A.gated ? 2 * F : F;
  A.Np = mx::padded(A.N1);
  A.limit = act.limit;
  A.alpha = act.alpha;
  A.beta = act.beta;
  return A;
}

// CTAs for `rows` rows of one warp each, at most a resident round
int rows_grid(const void* kernel, int rows) {
  const long long want = ((long long)rows + kThreads / 32 - 1) / (kThreads / 32);
  return (int)std::min<long long>(want, (long long)num_sms() * resident_ctas(kernel, kThreads));
}

template <typename T>
cudaError_t checkpoint_t(const void* p, const int32_t* seg_end, int E, int M, const ActArgs& A,
                         void* out, void* codes, void* scales, cudaStream_t s) {
  const auto kern = act_checkpoint_any<T>;
  const cudaError_t e = launch_pdl(kern, dim3(rows_grid((const void*)kern, M)), dim3(kThreads), 0,
                                   s, static_cast<const T*>(p), seg_end, E, M, A,
                                   static_cast<T*>(out), static_cast<uint8_t*>(codes),
                                   static_cast<uint8_t*>(scales));
  count_launch();
  return e;
}
template <typename T, bool MX>
cudaError_t backward_t(const void* p, const void* scales, const void* d_out,
                       const int32_t* seg_end, int E, int M, const ActArgs& A, void* d_p,
                       void* out, cudaStream_t s) {
  const auto kern = act_backward_any<T, MX>;
  const cudaError_t e = launch_pdl(kern, dim3(rows_grid((const void*)kern, M)), dim3(kThreads), 0,
                                   s, p, static_cast<const uint8_t*>(scales),
                                   static_cast<const T*>(d_out), seg_end, E, M, A,
                                   static_cast<T*>(d_p), static_cast<T*>(out));
  count_launch();
  return e;
}

}  // namespace

cudaError_t launch_act_checkpoint(const void* p, const int32_t* seg_end, int E, int M, int F,
                                  moe_dtype dt, const moe_act_params& act, void* out, void* codes,
                                  void* scales, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  const ActArgs A = act_args(act, F);
  if (dt == MOE_BF16)
    return checkpoint_t<__nv_bfloat16>(p, seg_end, E, M, A, out, codes, scales, s);
  if (dt == MOE_F16) return checkpoint_t<__half>(p, seg_end, E, M, A, out, codes, scales, s);
  return checkpoint_t<float>(p, seg_end, E, M, A, out, codes, scales, s);
}

cudaError_t launch_act_backward(const void* p, const void* scales, const void* d_out,
                                const int32_t* seg_end, int E, int M, int F, moe_dtype dt,
                                const moe_act_params& act, void* d_p, void* out, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  const ActArgs A = act_args(act, F);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    return scales ? backward_t<T, true>(p, scales, d_out, seg_end, E, M, A, d_p, out, s)
                  : backward_t<T, false>(p, scales, d_out, seg_end, E, M, A, d_p, out, s);
  };
  if (dt == MOE_BF16) return go(__nv_bfloat16{});
  if (dt == MOE_F16) return go(__half{});
  return go(float{});
}

}  // namespace moe
