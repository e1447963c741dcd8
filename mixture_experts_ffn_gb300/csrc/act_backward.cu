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
// A NaN in p is a NaN in a (the clamps keep it) and in the gradients that take its value:
// u is not in d_u, nothing in identity's, nor in either past its clamp.  Elementwise, eight
// output columns a thread, the next eight in flight while these are computed (32768 x
// 2880 swiglu gradient 165 -> 153 us, 65536 x 2048 silu checkpoint 196 -> 172).  Bound
// by HBM: these two move 6.2 and 6.3 TB/s.
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

// sigmoid(x): float32 results take the exact exponential and quotient, 16-bit ones
// the fast forms (within (8 + 1.2 |x|) 2^-23 of the value, against 2^-8 and 2^-11
// of the rounding that follows).
template <bool FAST>
__device__ __forceinline__ float sigmoid_t(float x) {
  if constexpr (FAST) return __fdividef(1.0f, 1.0f + __expf(-x));
  else return sigmoidf_(x);
}

// gelu's factors, the normal distribution function c = Phi(x) and density f.
// float32 results: the complementary error function, which keeps its digits for
// x < 0.  16-bit ones: Phi(-|x|) = exp(-x^2 / 2) h(|x|), with h a polynomial of
// t = 1 / (1 + |x| / 5), fitted here (least largest relative error, linear
// programming) to 2^-19 for |x| <= 13, where both factors share the exponential
// (65536 x 2048 bf16: gradient 331 -> 222 us, checkpoint 327 -> 219).
template <bool FAST>
__device__ __forceinline__ void phi(float x, float& c, float& f) {
  if constexpr (FAST) {
    const float e = __expf(-0.5f * x * x);
    const float t = __fdividef(1.0f, fmaf(fabsf(x), 0.2f, 1.0f));
    float h = 0.2790209949016571f;
    h = fmaf(h, t, -0.386553019285202f);
    h = fmaf(h, t, 0.4465286433696747f);
    h = fmaf(h, t, -0.12286803871393204f);
    h = fmaf(h, t, 0.1324034333229065f);
    h = fmaf(h, t, 0.07112088799476624f);
    h = fmaf(h, t, 0.08034771680831909f);
    h *= t * e;
    c = x < 0.0f ? h : 1.0f - h;
    f = 0.39894228040143268f * e;
  } else {
    c = 0.5f * erfcf(-0.70710678118654752f * x);
    f = 0.39894228040143268f * expf(-0.5f * x * x);
  }
}

// One gated pair: the activation a, and with d its gradients dg and du.
template <bool FAST>
__device__ __forceinline__ void gated_pair(int kind, float g, float u, float d, const ActArgs& A,
                                           float& a, float& dg, float& du) {
  if (kind == MOE_ACT_GELU_AND_MUL) {
    float c, f;
    phi<FAST>(g, c, f);
    a = g * c * u;
    dg = d * u * fmaf(g, f, c);
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
    float c, f;
    phi<FAST>(p, c, f);
    a = p * c;
    dp = d * fmaf(p, f, c);
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

// ---------------------------------------------------------------- eight columns a thread
// The shape of p and of the activation, known when compiled.
enum Form { kSilu, kGelu, kSwigluHalves, kSwigluPairs, kPlain };

// Eight consecutive elements as they sit in memory.
template <typename T>
struct Raw8 {
  uint4 q[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {  // read once: first to leave the caches
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[sizeof(T) / 2 - 1].x,
                           q[sizeof(T) / 2 - 1].y, q[sizeof(T) / 2 - 1].z, q[sizeof(T) / 2 - 1].w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
    } else {
      constexpr bool F16 = std::is_same<T, __half>::value;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = lo16<F16>(u[i]);
        v[2 * i + 1] = hi16<F16>(u[i]);
      }
    }
  }
};

// Item i: output columns 8 (i % ipr) .. of row i / ipr; a thread's next item is a
// grid's width on, so the loop divides nothing.
struct Items {
  uint32_t i, row, col, ipr, step, drow, dcol, count;
  __device__ __forceinline__ Items(uint32_t ipr_, uint32_t rows) : ipr(ipr_), count(ipr_ * rows) {
    i = blockIdx.x * kThreads + threadIdx.x;
    step = gridDim.x * kThreads;
    row = i / ipr;
    col = i - row * ipr;
    drow = step / ipr;
    dcol = step - drow * ipr;
  }
  __device__ __forceinline__ bool more() const { return i < count; }
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

// The activation of eight columns, x (and y, the up values) its argument.
template <int FORM, bool FAST>
__device__ __forceinline__ void act8(const float (&x)[8], const float (&y)[8], const float (&d)[8],
                                     const ActArgs& A, float (&a)[8], float (&dx)[8],
                                     float (&dy)[8]) {
  constexpr int KIND = FORM == kSilu   ? MOE_ACT_SILU_AND_MUL
                       : FORM == kGelu ? MOE_ACT_GELU_AND_MUL
                                       : MOE_ACT_SWIGLU;
  if constexpr (FORM != kPlain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) gated_pair<FAST>(KIND, x[i], y[i], d[i], A, a[i], dx[i], dy[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) plain_value<FAST>(A.kind, x[i], d[i], a[i], dx[i]);
  }
}
// (gate, up) pairs of sixteen consecutive columns
__device__ __forceinline__ void unzip(const float (&lo)[8], const float (&hi)[8], float (&x)[8],
                                      float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = lo[2 * i];
    y[i] = lo[2 * i + 1];
    x[4 + i] = hi[2 * i];
    y[4 + i] = hi[2 * i + 1];
  }
}
__device__ __forceinline__ void zip(const float (&x)[8], const float (&y)[8], float (&lo)[8],
                                    float (&hi)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[2 * i] = x[i];
    lo[2 * i + 1] = y[i];
    hi[2 * i] = x[4 + i];
    hi[2 * i + 1] = y[4 + i];
  }
}
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mx::abs_bits(v[i]));
  return m;
}

// F % 32 == 0, p and out 16-byte aligned (other widths, and other starts, go a lane a
// column through act_checkpoint_any: 65536 x 720 silu bf16 218 us, 65536 x 704 here 65;
// 65536 x 360 120, its floor 29).  A 32-column block of the checkpoint is four lanes
// (two when gate and up are interleaved: 16 columns a lane), which agree on its scale
// with shuffles; a block never straddles rows or halves.
template <typename T, int FORM>
__global__ void __launch_bounds__(kThreads)
    act_checkpoint_vec(const T* __restrict__ p, const int32_t* __restrict__ seg_end, int E, int M,
                       ActArgs A, T* __restrict__ out, uint8_t* __restrict__ codes,
                       uint8_t* __restrict__ scales) {
  pdl_launch();
  pdl_wait();
  constexpr bool FAST = sizeof(T) == 2, PAIRS = FORM == kSwigluPairs, ONE = FORM == kPlain;
  const uint32_t mask = 0xfu << (threadIdx.x & 28);
  Items w(A.F / 8, live_rows(seg_end, E, M));
  Raw8<T> r0, r1;
  auto fetch = [&]() {  // the next item's columns, in flight while this one is converted
    if (!w.more()) return;
    const T* src = p + (size_t)w.row * A.N1 + (PAIRS ? 16 : 8) * w.col;
    r0.load(src);
    if constexpr (!ONE) r1.load(src + (PAIRS ? 8 : A.F));
  };
  fetch();
  while (w.more()) {
    float u[8], v[8];
    r0.get(u);
    if constexpr (!ONE) r1.get(v);
    const uint32_t row = w.row, col = w.col;
    w.next();
    fetch();
    // blocks: u and v are one block's (pairs), or u and v of a block each
    uint32_t mu = amax8(u), mv = ONE ? 0 : amax8(v);
    if constexpr (PAIRS) mu = max(mu, mv);
    mu = max(mu, __shfl_xor_sync(mask, mu, 1));
    if constexpr (!PAIRS) mu = max(mu, __shfl_xor_sync(mask, mu, 2));
    const uint32_t bu = mx::scale_byte<false>(mu);
    uint8_t* crow = codes + (size_t)row * A.Np;
    uint8_t* srow = scales + (size_t)row * (A.Np / 32);
    float a[8], s[8], dx[8], dy[8];
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if constexpr (PAIRS) {
      float q[8], t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        q[i] = u[i];
        t[i] = v[i];
      }
      mx::scale8(q, mx::inv_scale(bu));
      mx::scale8(t, mx::inv_scale(bu));
      const uint2 lo = mx::e4m3x8(q), hi = mx::e4m3x8(t);
      *reinterpret_cast<uint4*>(crow + 16 * col) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      if ((threadIdx.x & 1) == 0) srow[col >> 1] = (uint8_t)bu;
      float x[8], y[8];
      unzip(u, v, x, y);
      act8<FORM, FAST>(x, y, zero, A, a, dx, dy);
    } else {
      act8<FORM, FAST>(u, v, zero, A, a, dx, dy);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = u[i];
      mx::scale8(s, mx::inv_scale(bu));
      *reinterpret_cast<uint2*>(crow + 8 * col) = mx::e4m3x8(s);
      if ((threadIdx.x & 3) == 0) srow[col >> 2] = (uint8_t)bu;
      if constexpr (!ONE) {
        mv = max(mv, __shfl_xor_sync(mask, mv, 1));
        mv = max(mv, __shfl_xor_sync(mask, mv, 2));
        const uint32_t bv = mx::scale_byte<false>(mv);
        mx::scale8(v, mx::inv_scale(bv));
        *reinterpret_cast<uint2*>(crow + A.F + 8 * col) = mx::e4m3x8(v);
        if ((threadIdx.x & 3) == 0) srow[(A.F >> 5) + (col >> 2)] = (uint8_t)bv;
      }
    }
    if (out) mx::store8<T, true>(out + (size_t)row * A.F, 8 * col, A.F, a);
    // the blocks past N1, up to the next multiple of 128 columns
    for (uint32_t q = col; q < (uint32_t)(A.Np - A.N1) / 8; q += w.ipr) {
      *reinterpret_cast<uint2*>(crow + A.N1 + 8 * q) = make_uint2(0, 0);
      if ((q & 3) == 0) srow[(A.N1 >> 5) + (q >> 2)] = 0;
    }
  }
}

__device__ __forceinline__ void e4m3_values(const uint2& c, float scale, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)((j < 2 ? c.x : c.y) >> (16 * (j & 1))), __NV_E4M3);
    const float2 f = __half22float2(h);
    v[2 * j] = f.x * scale;
    v[2 * j + 1] = f.y * scale;
  }
}

// F % 8 == 0, p, d_out, d_p and out 16-byte aligned: eight columns, or sixteen
// interleaved ones, lie in one block of the checkpoint.  Four CTAs an SM (64
// registers a thread) gain for silu and SwiGLU (65536 x 2048 silu 218 -> 205 us); the
// other forms lose 1 to 4%.
constexpr int backward_ctas(int form, bool mx) {
  return mx && (form == kSilu || form == kSwigluHalves || form == kSwigluPairs) ? 4 : 1;
}
template <typename T, int FORM, bool MX>
__global__ void __launch_bounds__(kThreads, backward_ctas(FORM, MX))
    act_backward_vec(const void* __restrict__ p, const uint8_t* __restrict__ scales,
                     const T* __restrict__ d_out, const int32_t* __restrict__ seg_end, int E,
                     int M, ActArgs A, T* __restrict__ d_p, T* __restrict__ out) {
  pdl_launch();
  pdl_wait();
  constexpr bool FAST = sizeof(T) == 2, PAIRS = FORM == kSwigluPairs, ONE = FORM == kPlain;
  Items w(A.F / 8, live_rows(seg_end, E, M));
  Raw8<T> rd, r0, r1;      // d_out; p without a checkpoint
  uint2 c0 = {}, c1 = {};  // codes
  uint32_t s0 = 0, s1 = 0;
  auto fetch = [&]() {  // the next item, in flight while this one is computed
    if (!w.more()) return;
    rd.load(d_out + (size_t)w.row * A.F + 8 * w.col);
    const uint32_t at = (PAIRS ? 16 : 8) * w.col;
    if constexpr (MX) {
      const uint8_t* src = static_cast<const uint8_t*>(p) + (size_t)w.row * A.Np + at;
      const uint8_t* sc = scales + (size_t)w.row * (A.Np / 32);
      s0 = sc[at >> 5];
      if constexpr (PAIRS) {
        const uint4 c = __ldcs(reinterpret_cast<const uint4*>(src));
        c0 = make_uint2(c.x, c.y);
        c1 = make_uint2(c.z, c.w);
      } else {
        c0 = __ldcs(reinterpret_cast<const uint2*>(src));
        if constexpr (!ONE) {
          c1 = __ldcs(reinterpret_cast<const uint2*>(src + A.F));
          s1 = sc[(at + A.F) >> 5];
        }
      }
    } else {
      const T* src = static_cast<const T*>(p) + (size_t)w.row * A.N1 + at;
      r0.load(src);
      if constexpr (!ONE) r1.load(src + (PAIRS ? 8 : A.F));
    }
  };
  fetch();
  while (w.more()) {
    float u[8], v[8], d[8], x[8], y[8], a[8];
    rd.get(d);
    if constexpr (MX) {
      e4m3_values(c0, mx::scale_value(s0), u);
      if constexpr (!ONE) e4m3_values(c1, mx::scale_value(PAIRS ? s0 : s1), v);
    } else {
      r0.get(u);
      if constexpr (!ONE) r1.get(v);
    }
    const uint32_t row = w.row, col = w.col;
    w.next();
    fetch();
    T* dst = d_p + (size_t)row * A.N1;
    float dx[8], dy[8];
    if constexpr (PAIRS) {
      unzip(u, v, x, y);
      act8<FORM, FAST>(x, y, d, A, a, dx, dy);
      zip(dx, dy, u, v);
      mx::store8<T, true>(dst, 16 * col, A.N1, u);
      mx::store8<T, true>(dst, 16 * col + 8, A.N1, v);
    } else {
      act8<FORM, FAST>(u, v, d, A, a, dx, dy);
      mx::store8<T, true>(dst, 8 * col, A.N1, dx);
      if constexpr (!ONE) mx::store8<T, true>(dst, A.F + 8 * col, A.N1, dy);
    }
    if (out) mx::store8<T, true>(out + (size_t)row * A.F, 8 * col, A.F, a);
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

// CTAs for the items of M rows, at most a resident round
int items_grid(const void* kernel, int M, int F) {
  const long long want = ((long long)M * (F / 8) + kThreads - 1) / kThreads;
  return (int)std::min<long long>(want, (long long)num_sms() * resident_ctas(kernel, kThreads));
}
bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, int FORM>
cudaError_t checkpoint_form(const void* p, const int32_t* seg_end, int E, int M, const ActArgs& A,
                            void* out, void* codes, void* scales, cudaStream_t s) {
  const auto kern = act_checkpoint_vec<T, FORM>;
  return launch_pdl(kern, dim3(items_grid((const void*)kern, M, A.F)), dim3(kThreads), 0, s,
                    static_cast<const T*>(p), seg_end, E, M, A, static_cast<T*>(out),
                    static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}
template <typename T, int FORM, bool MX>
cudaError_t backward_form(const void* p, const void* scales, const void* d_out,
                          const int32_t* seg_end, int E, int M, const ActArgs& A, void* d_p,
                          void* out, cudaStream_t s) {
  const auto kern = act_backward_vec<T, FORM, MX>;
  return launch_pdl(kern, dim3(items_grid((const void*)kern, M, A.F)), dim3(kThreads), 0, s, p,
                    static_cast<const uint8_t*>(scales), static_cast<const T*>(d_out), seg_end, E,
                    M, A, static_cast<T*>(d_p), static_cast<T*>(out));
}
// f(form) with the form of A as a compile-time constant
template <typename Fn>
cudaError_t with_form(const ActArgs& A, Fn f) {
  if (!A.gated) return f(std::integral_constant<int, kPlain>{});
  if (A.kind == MOE_ACT_SILU_AND_MUL) return f(std::integral_constant<int, kSilu>{});
  if (A.kind == MOE_ACT_GELU_AND_MUL) return f(std::integral_constant<int, kGelu>{});
  if (A.inter) return f(std::integral_constant<int, kSwigluPairs>{});
  return f(std::integral_constant<int, kSwigluHalves>{});
}

template <typename T>
cudaError_t checkpoint_t(const void* p, const int32_t* seg_end, int E, int M, const ActArgs& A,
                         void* out, void* codes, void* scales, cudaStream_t s) {
  if (A.F % 32 == 0 && a16(p) && a16(out)) {
    const cudaError_t e = with_form(A, [&](auto form) {
      return checkpoint_form<T, decltype(form)::value>(p, seg_end, E, M, A, out, codes, scales, s);
    });
    count_launch();
    return e;
  }
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
  if (A.F % 8 == 0 && a16(p) && a16(d_out) && a16(d_p) && a16(out)) {
    const cudaError_t e = with_form(A, [&](auto form) {
      return backward_form<T, decltype(form)::value, MX>(p, scales, d_out, seg_end, E, M, A, d_p,
                                                         out, s);
    });
    count_launch();
    return e;
  }
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
