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

#include "common.cuh"

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

// Lane j holds the routes j and j + 32 of the token (K <= 64).
__global__ void __launch_bounds__(kThreads)
    route_backward_kernel(const void* __restrict__ logits, const int32_t* __restrict__ ids,
                          const float* __restrict__ d_w, int T, int E, int K, int scoring,
                          int renorm, float rsf, int dt, void* __restrict__ d_logits) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kThreads / 32);
  const bool dense = scoring == MOE_SCORING_SOFTMAX && !renorm;
  for (int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < T; t += warps) {
    const size_t row = (size_t)t * E;
    int id[2];
    float z[2], g[2], s[2], l[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = lane + 32 * q;
      id[q] = k < K ? ids[(size_t)t * K + k] : -1;
      if (id[q] >= E) id[q] = -1;  // an id outside [0, E) takes no part
      const bool in = id[q] >= 0;
      g[q] = in ? d_w[(size_t)t * K + k] : 0.f;
      z[q] = in ? load_any(logits, row + id[q], dt) : -INFINITY;
      s[q] = l[q] = 0.f;
    }
    // scores (softmax: of the chosen experts, or with the whole row's sum)
    float m = 0.f, sum = 0.f;
    if (scoring == MOE_SCORING_SOFTMAX) {
      m = fmaxf(z[0], z[1]);
      if (dense)
        for (int e = lane; e < E; e += 32) m = fmaxf(m, load_any(logits, row + e, dt));
      m = warp_max(m);
      if (dense) {
        for (int e = lane; e < E; e += 32) sum += expf(load_any(logits, row + e, dt) - m);
        sum = warp_sum(sum);
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (id[q] < 0) continue;
      if (scoring == MOE_SCORING_SOFTMAX) {
        s[q] = expf(z[q] - m);
        l[q] = 1.f;
      } else {
        score_of(scoring, z[q], s[q], l[q]);
      }
    }
    if (!dense) sum = renorm ? warp_sum(s[0] + s[1]) : 1.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) s[q] = id[q] >= 0 ? s[q] / sum : 0.f;
    float mean = 0.f;  // sum_k g_k v_k
    if (renorm || dense) {
      mean = (id[0] >= 0 ? g[0] * s[0] : 0.f) + (id[1] >= 0 ? g[1] * s[1] : 0.f);
      mean = warp_sum(mean);
    }
    // a chosen expert's value; the same id twice adds up
    float v[2];
    if (dense) {
      v[0] = g[0];
      v[1] = g[1];
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) v[q] = id[q] >= 0 ? rsf * s[q] * l[q] * (g[q] - mean) : 0.f;
    }
    float add[2] = {0.f, 0.f};
    for (int k = 0; k < K; ++k) {
      const int q = k >> 5;
      const int other = __shfl_sync(0xffffffffu, q ? id[1] : id[0], k & 31);
      const float x = __shfl_sync(0xffffffffu, q ? v[1] : v[0], k & 31);
      if (other == id[0]) add[0] += x;
      if (other == id[1]) add[1] += x;
    }
    for (int e = lane; e < E; e += 32) {
      const float o = dense ? rsf * (expf(load_any(logits, row + e, dt) - m) / sum) * -mean : 0.f;
      store_any(d_logits, row + e, dt, o);
    }
    __syncwarp();  // the row's own values over the others
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (id[q] >= 0)
        store_any(d_logits, row + id[q], dt, dense ? rsf * s[q] * (add[q] - mean) : add[q]);
  }
}

}  // namespace

cudaError_t launch_route_backward(const void* logits, const int32_t* ids, const float* d_w, int T,
                                  int E, const moe_route_params& p, void* d_logits,
                                  cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const long long want = ((long long)T + kThreads / 32 - 1) / (kThreads / 32);
  const long long cap =
      (long long)num_sms() * resident_ctas((const void*)route_backward_kernel, kThreads);
  const cudaError_t e = launch_pdl(route_backward_kernel, dim3((unsigned)std::min(want, cap)),
                                   dim3(kThreads), 0, s, logits, ids, d_w, T, E, (int)p.top_k,
                                   (int)p.scoring, (int)(p.renormalize != 0),
                                   p.routed_scaling_factor, (int)p.dtype, d_logits);
  count_launch();
  return e;
}

}  // namespace moe
