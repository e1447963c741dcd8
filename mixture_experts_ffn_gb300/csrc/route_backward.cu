// Gradient of the router (moe_route) with respect to its logits.  With scores
// s_i of the logits z_i, the chosen experts id_k, c = routed_scaling_factor and
// g_k the gradient of topk_weights:
//   renormalised, w_k = c s_k / sum_j s_j =: c v_k:
//     d_z[id_k] += c v_k l_k (g_k - sum_j g_j v_j),  l = dlog s / dz
//     (softmax: 1, since the softmax's own sum cancels in v; sigmoid:
//     sigmoid(-z); sqrt_softplus: sigmoid(z) / (2 softplus(z)))
//   as they are, w_k = c s_k:
//     softmax: d_z[i] = c s_i (sum of g_k over id_k = i - sum_k g_k s_k),
//     others: d_z[id_k] += c g_k s_k l_k.
// Only a softmax whose weights are not renormalised needs more than the K chosen
// logits of a token.  Selection, the correction bias and the groups have no
// gradient.  One warp a token; bound by writing the [T, E] gradients.
#include <algorithm>

#include "mx_dev.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_any(const void* p, size_t i, int dt) {
  if (dt == MOE_F32) return static_cast<const float*>(p)[i];
  if (dt == MOE_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, size_t i, int dt, float v) {
  if (dt == MOE_F32) static_cast<float*>(p)[i] = v;
  else if (dt == MOE_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// log of the score's square for sqrt_softplus and of the score for sigmoid are
// never taken: both scores and their log-derivatives come from e = exp(-|z|).
//   sigmoid:        s = 1 / (1 + exp(-z)),          l = sigmoid(-z)
//   sqrt_softplus:  s = sqrt(max(z, 0) + log1p(e)), l = sigmoid(z) / (2 s^2);
// below z = -80 softplus(z) and sigmoid(z) are both exp(z) to the last bit, so
// l = 1/2 (and exp(z) may underflow).
__device__ __forceinline__ void score_of(int scoring, float z, float& s, float& l) {
  if (scoring == MOE_SCORING_SIGMOID) {
    s = sigmoidf_(z);
    l = sigmoidf_(-z);
  } else {
    const float sp = fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
    s = z < -80.f ? expf(0.5f * z) : sqrtf(sp);
    l = z < -80.f ? 0.5f : sigmoidf_(z) / (2.f * sp);
    if (z != z) s = l = z;  // fmaxf drops a NaN
  }
}

// The calling warp writes zeros over a row of the gradients.
__device__ __forceinline__ void zero_row(void* row, int bytes) {
  const int lane = threadIdx.x & 31;
  if (((reinterpret_cast<uintptr_t>(row) | (uintptr_t)bytes) & 15) == 0) {
    for (int i = lane; i < bytes / 16; i += 32) static_cast<uint4*>(row)[i] = make_uint4(0, 0, 0, 0);
  } else {
    for (int i = lane; i < bytes / 2; i += 32) static_cast<uint16_t*>(row)[i] = 0;
  }
}

// Sum of x over the routes with the calling lane's id, in order (an id may come
// twice): lane j holds the routes j and j + 32 of the token (K <= 64).
__device__ __forceinline__ void same_id_sums(const int (&id)[2], const float (&x)[2], int K,
                                             float (&sum)[2]) {
  sum[0] = sum[1] = 0.f;
  for (int k = 0; k < K; ++k) {
    const int other = __shfl_sync(0xffffffffu, k < 32 ? id[0] : id[1], k & 31);
    const float v = __shfl_sync(0xffffffffu, k < 32 ? x[0] : x[1], k & 31);
    if (other == id[0]) sum[0] += v;
    if (other == id[1]) sum[1] += v;
  }
}

// The gradient is zero but at the chosen experts: all but a softmax whose weights
// are as they are.  The zeros are written while the loads are under way.
__global__ void __launch_bounds__(kThreads)
    route_backward_chosen(const void* __restrict__ logits, const int32_t* __restrict__ ids,
                          const float* __restrict__ d_w, int T, int E, int K, int scoring,
                          int renorm, float rsf, int dt, void* __restrict__ d_logits) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, size = dt == MOE_F32 ? 4 : 2;
  const long long warps = gridDim.x * (kThreads / 32);
  for (long long t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < T; t += warps) {
    const size_t row = (size_t)t * E;
    int id[2];
    float z[2], g[2], s[2] = {}, l[2] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = lane + 32 * q;
      id[q] = k < K ? ids[(size_t)t * K + k] : -1;
      g[q] = k < K ? d_w[(size_t)t * K + k] : 0.f;
    }
    zero_row(static_cast<char*>(d_logits) + row * size, E * size);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (id[q] < 0 || id[q] >= E) id[q] = -1, g[q] = 0.f;  // no expert: takes no part
      z[q] = id[q] >= 0 ? load_any(logits, row + id[q], dt) : -INFINITY;
    }
    const float m = scoring == MOE_SCORING_SOFTMAX ? warp_max(fmaxf(z[0], z[1])) : 0.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (id[q] < 0 || z[q] == -INFINITY) continue;  // a masked expert's score is zero
      if (scoring == MOE_SCORING_SOFTMAX) {
        s[q] = expf(z[q] - m);
        l[q] = 1.f;
      } else {
        score_of(scoring, z[q], s[q], l[q]);
      }
    }
    float mean = 0.f;  // sum_k g_k v_k
    if (renorm) {
      float sum = warp_sum(s[0] + s[1]);
      if (sum < 1e-15f && scoring != MOE_SCORING_SOFTMAX) {
        // Every chosen logit is below -34 (sqrt_softplus -69), where the scores are exp(z)
        // and exp(z / 2) to the last bit and underflow from -89 and -207 on: the same
        // ratios from the differences to the highest.
        const float top = warp_max(fmaxf(z[0], z[1]));
        const float h = scoring == MOE_SCORING_SIGMOID ? 1.f : 0.5f;
#pragma unroll
        for (int q = 0; q < 2; ++q) s[q] = z[q] == -INFINITY ? 0.f : expf(h * (z[q] - top));
        sum = warp_sum(s[0] + s[1]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)  // (no weight where every chosen expert is masked)
        s[q] = id[q] >= 0 && sum != 0.f ? s[q] / sum : 0.f;
      mean = warp_sum(g[0] * s[0] + g[1] * s[1]);
    }
    float x[2], v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) x[q] = id[q] >= 0 ? rsf * s[q] * l[q] * (g[q] - mean) : 0.f;
    same_id_sums(id, x, K, v);
    __syncwarp();  // the chosen experts' values over the zeros
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (id[q] >= 0) store_any(d_logits, row + id[q], dt, v[q]);
  }
}

// Softmax, weights as they are: every expert has a part in the softmax's sum.
// Expert lane + 32 i is in register i (E <= 32 NPL).
template <int NPL>
__global__ void __launch_bounds__(kThreads)
    route_backward_softmax(const void* __restrict__ logits, const int32_t* __restrict__ ids,
                           const float* __restrict__ d_w, int T, int E, int K, float rsf, int dt,
                           void* __restrict__ d_logits) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long warps = gridDim.x * (kThreads / 32);
  for (long long t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < T; t += warps) {
    const size_t row = (size_t)t * E;
    int id[2];
    float g[2], z[NPL];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = lane + 32 * q;
      id[q] = k < K ? ids[(size_t)t * K + k] : -1;
      g[q] = k < K ? d_w[(size_t)t * K + k] : 0.f;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      z[i] = e < E ? load_any(logits, row + e, dt) : -INFINITY;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (id[q] < 0 || id[q] >= E) id[q] = -1, g[q] = 0.f;  // no expert: takes no part
    // the chosen experts' logits again, now from the L1 cache
    float s[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) s[q] = id[q] >= 0 ? load_any(logits, row + id[q], dt) : -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) m = fmaxf(m, z[i]);
    m = warp_max(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      z[i] = z[i] != -INFINITY ? expf(z[i] - m) : 0.f;  // (past E, or masked)
      sum += z[i];
    }
    sum = warp_sum(sum);
    if (sum == 0.f) sum = 1.f;  // every expert is masked: weights and gradients of zero
#pragma unroll
    for (int q = 0; q < 2; ++q)  // (divided also where masked: a NaN of the row is kept)
      s[q] = (s[q] != -INFINITY ? expf(s[q] - m) : 0.f) / sum;
    const float mean = warp_sum(g[0] * s[0] + g[1] * s[1]);  // sum_k g_k s_k
    float v[2];
    same_id_sums(id, g, K, v);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane + 32 * i < E)
        store_any(d_logits, row + lane + 32 * i, dt, rsf * (z[i] / sum) * -mean);
    __syncwarp();  // the chosen experts' values over the others'
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (id[q] >= 0) store_any(d_logits, row + id[q], dt, rsf * s[q] * (v[q] - mean));
  }
}

}  // namespace

cudaError_t launch_route_backward(const void* logits, const int32_t* ids, const float* d_w, int T,
                                  int E, const moe_route_params& p, void* d_logits,
                                  cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const long long want = ((long long)T + kThreads / 32 - 1) / (kThreads / 32);
  auto grid = [&](const void* kern) {
    return dim3((unsigned)std::min(want, (long long)num_sms() * resident_ctas(kern, kThreads)));
  };
  cudaError_t e;
  if (p.scoring == MOE_SCORING_SOFTMAX && !p.renormalize) {
    auto go = [&](auto kern) {
      return launch_pdl(kern, grid((const void*)kern), dim3(kThreads), 0, s, logits, ids, d_w, T, E,
                        (int)p.top_k, p.routed_scaling_factor, (int)p.dtype, d_logits);
    };
    e = E <= 128   ? go(route_backward_softmax<4>)
        : E <= 512 ? go(route_backward_softmax<16>)
                   : go(route_backward_softmax<32>);
  } else {
    e = launch_pdl(route_backward_chosen, grid((const void*)route_backward_chosen), dim3(kThreads),
                   0, s, logits, ids, d_w, T, E, (int)p.top_k, (int)p.scoring,
                   (int)(p.renormalize != 0), p.routed_scaling_factor, (int)p.dtype, d_logits);
  }
  count_launch();
  return e;
}

}  // namespace moe
