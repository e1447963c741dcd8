// Residual addition, root-mean-square norm and its 8-bit forms in one pass:
//   h = round(x + r) (or x), y = h * rsqrt(mean(h^2) + eps) * w
// with h and y written in the operand type and y also as e4m3 codes: MX (an
// e8m0 scale per 32 columns) or one float32 scale per 128 columns (what the
// block-scaled FP8 grouped GEMM reads).
//
// The mean is taken over the ROUNDED h, so the result is the norm of the
// residual stream that is stored, and equal to adding first and normalising
// later.  The codes come from the float32 y, not from its rounded copy: one
// rounding instead of two.  Squares are summed in float32, a chain for each of
// a thread's eight columns, then across lanes and warps in a fixed order.
//
// Bound by HBM: x and r in, h, y and the codes out, each once; a row of up to
// 32768 columns stays in registers between the sum and the scaling.  8192 x 7168
// bf16, all outputs: 90 us for 530 MB, 5.9 TB/s, 0.87 of the measured copy rate;
// one row of 7168: 5.3 us, launch latency.  Wider rows have eight groups of eight
// columns a thread, which do not fit the registers of 1024 threads: 1024 x 65536
// takes 351 us (1.7 TB/s), 1024 x 32768 67 (4.5).
#include <algorithm>
#include <type_traits>

#include "mx_dev.cuh"

namespace moe {
namespace {

enum : int { kQuantNone = 0, kQuantMx = 1, kQuantB128 = 2 };

struct NormArgs {
  const void *x, *r, *w;
  void *h, *y;
  uint8_t* codes;
  void* scales;
  int T, H, Hp;
  float eps;
};

// A sum as hi + lo; add keeps the rounding error of hi (Knuth's two-sum).
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  return {s, a.lo + b.lo + ((a.hi - (s - t)) + (b.hi - t))};
}
// Sum over the `warps` warps of a row group (every thread gets it): plain
// float32 inside a warp, whose sum is a small part of the row's, with the
// rounding errors kept across warps, where they would count in full.
__device__ __forceinline__ Two group_sum(float v, float* red, int warps, int warp, int lane) {
  v = warp_sum(v);
  if (warps == 1) return {v, 0.0f};
  if (lane == 0) red[warp] = v;
  __syncthreads();
  int span = 2;  // lanes that hold one copy of all the warps' sums
  while (span < warps) span *= 2;
  const int at = lane & (span - 1);
  Two s{at < warps ? red[at] : 0.0f, 0.0f};
  for (int o = span / 2; o > 0; o >>= 1)
    s = add(s, Two{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
  return s;
}

// 1 / sqrt(sum / n + eps) as hi + lo: one Newton step on rsqrtf's value, its
// residual 1 - m hi^2 taken from the products' exact errors.  An 8-bit code next
// to a tie goes by the last bits of y: with a plain float32 mean and root and two
// rounded products more codes fell on the other side than 64 bits put them.
__device__ __forceinline__ Two inv_root(Two sum, float n, float eps) {
  const float q = sum.hi / n;
  const Two m = add(Two{q, (fmaf(-q, n, sum.hi) + sum.lo) / n}, Two{eps, 0.0f});
  Two r;
  r.hi = rsqrtf(m.hi);
  const float t = m.hi * r.hi;
  const float e = fmaf(-t, r.hi, 1.0f) - (fmaf(m.hi, r.hi, -t) + m.lo * r.hi) * r.hi;
  const float lo = 0.5f * r.hi * e;
  r.lo = isfinite(lo) ? lo : 0.0f;  // m zero, infinite or NaN: hi alone
  return r;
}

// A row is shared by `blockDim.x` threads (one CTA a row), or by one warp
// when WARP_ROW (blockDim.x / 32 rows a CTA); each thread owns ITEMS groups
// of eight columns, consecutive threads owning consecutive groups.
template <typename T, int QUANT, int ITEMS, bool VEC, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 256 : 1024)
    rms_norm_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nthr = WARP_ROW ? 32 : (int)blockDim.x;
  const int t0 = WARP_ROW ? lane : (int)threadIdx.x;
  const int row = WARP_ROW ? (int)(blockIdx.x * (blockDim.x >> 5)) + warp : (int)blockIdx.x;
  pdl_launch();
  pdl_wait();
  if (WARP_ROW && row >= p.T) return;
  const int H = p.H;
  const T* x = static_cast<const T*>(p.x) + (size_t)row * H;
  const T* r = p.r ? static_cast<const T*>(p.r) + (size_t)row * H : nullptr;
  float v[ITEMS][8];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) mx::load8<T, VEC>(x, (t0 + i * nthr) * 8, H, v[i]);
  if (r) {
    float a[ITEMS][8];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) mx::load8<T, VEC>(r, (t0 + i * nthr) * 8, H, a[i]);
    T* h = static_cast<T*>(p.h) + (size_t)row * H;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = Elem<T>::to_f(Elem<T>::from_f(v[i][j] + a[i][j]));
      mx::store8<T, VEC>(h, (t0 + i * nthr) * 8, H, v[i]);
    }
  }
  float ss[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    ss[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) ss[j] = fmaf(v[i][j], v[i][j], ss[j]);
  }
  const float mine = ((ss[0] + ss[1]) + (ss[2] + ss[3])) + ((ss[4] + ss[5]) + (ss[6] + ss[7]));
  const Two sum = group_sum(mine, red, nthr >> 5, warp, lane);
  const Two root = inv_root(sum, (float)H, p.eps);
  T* y = p.y ? static_cast<T*>(p.y) + (size_t)row * H : nullptr;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int item = t0 + i * nthr, c0 = item * 8;
    float w[8];
    mx::load8<T, VEC>(static_cast<const T*>(p.w), c0, H, w);
    uint32_t amax = 0;  // bits of the largest magnitude; a NaN's are above infinity's
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // h * root * w with one rounding: the product's own error rides along
      const float a = v[i][j] * root.hi;
      const float lo = fmaf(v[i][j], root.lo, fmaf(v[i][j], root.hi, -a));
      z[j] = fmaf(a, w[j], lo * w[j]);
      amax = max(amax, mx::abs_bits(z[j]));
    }
    if (amax > mx::kInfBits) {
      // an infinite w or root leaves no error to carry (0 * inf, inf - inf):
      // the product alone, NaN where that is one
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (isnan(z[j])) z[j] = v[i][j] * root.hi * w[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = z[j];
    if (y) mx::store8<T, VEC>(y, c0, H, v[i]);
    if constexpr (QUANT != kQuantNone) {
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if constexpr (QUANT == kQuantMx) {
        const uint32_t byte = mx::scale_byte<false>(amax);
        mx::scale8(v[i], mx::inv_scale(byte));
        if (c0 < p.Hp && (lane & 3) == 0)
          static_cast<uint8_t*>(p.scales)[(size_t)row * (p.Hp / 32) + (item >> 2)] = (uint8_t)byte;
      } else {
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
        // a block with an infinity or a NaN: NaN scale, zero codes
        const bool bad = amax >= mx::kInfBits;
        const float s = fmaxf(__uint_as_float(amax) / 448.0f, 1.17549435e-38f);
        // one quotient a block instead of one a value: a code's argument is
        // then within 2 ulp of y / s
        mx::scale8(v[i], bad ? 0.0f : 1.0f / s);
        if (c0 < p.Hp && (lane & 15) == 0)
          static_cast<float*>(p.scales)[(size_t)row * (p.Hp / 128) + (item >> 4)] =
              bad ? __uint_as_float(0x7fc00000u) : s;
      }
      if (c0 < p.Hp)
        reinterpret_cast<uint2*>(p.codes + (size_t)row * p.Hp)[item] = mx::e4m3x8(v[i]);
    }
  }
}

template <typename T, int QUANT, int ITEMS, bool VEC, bool WARP_ROW>
cudaError_t go(const NormArgs& p, int threads, cudaStream_t s) {
  const int grid = WARP_ROW ? (p.T + threads / 32 - 1) / (threads / 32) : p.T;
  cudaError_t e = launch_pdl(rms_norm_kernel<T, QUANT, ITEMS, VEC, WARP_ROW>, dim3(grid),
                             dim3(threads), 0, s, p);
  count_launch();
  return e;
}

// Threads of a row (bf16, residual, MX out; us, L2 flushed): short rows (up to
// 1024 columns) take a warp each, eight to a CTA (8192 x 256: 15.5, 17.6 with a
// CTA a row).  Longer ones take a CTA each.  Rows for every SM: four groups of
// eight columns a thread keep more bytes in flight per thread (8192 x 7168: 91,
// 140 with one group; 1000 x 2880: 12.4 and 14.4).  Fewer rows than SMs: one
// group a thread shortens the one row's path (one row of 7168: 8.4, 10.4 with
// four; 16 x 2880: 9.3 and 9.4).
template <typename T, int QUANT, bool VEC>
cudaError_t pick(const NormArgs& p, cudaStream_t s) {
  const int items = p.Hp / 8;
  if (items <= 128 && p.T >= 2 * num_sms()) return go<T, QUANT, 4, VEC, true>(p, 256, s);
  const int one = (items + 31) & ~31;
  if (one <= 1024 && p.T < num_sms()) return go<T, QUANT, 1, VEC, false>(p, one, s);
  const int four = ((items + 3) / 4 + 31) & ~31;
  if (four <= 1024) return go<T, QUANT, 4, VEC, false>(p, four, s);
  return go<T, QUANT, 8, VEC, false>(p, ((items + 7) / 8 + 31) & ~31, s);
}
template <typename T>
cudaError_t pick_q(const NormArgs& p, int quant, bool vec, cudaStream_t s) {
  if (quant == MOE_QUANT_MX_E4M3)
    return vec ? pick<T, kQuantMx, true>(p, s) : pick<T, kQuantMx, false>(p, s);
  if (quant == MOE_QUANT_E4M3_BLOCK128)
    return vec ? pick<T, kQuantB128, true>(p, s) : pick<T, kQuantB128, false>(p, s);
  return vec ? pick<T, kQuantNone, true>(p, s) : pick<T, kQuantNone, false>(p, s);
}

}  // namespace

cudaError_t launch_rms_norm(const void* x, const void* residual, const void* weight, int T, int H,
                            moe_dtype dt, float eps, int quant, void* residual_out, void* out,
                            void* codes, void* scales, cudaStream_t s) {
  NormArgs p{x, residual, weight, residual_out, out, static_cast<uint8_t*>(codes), scales, T, H,
             mx::padded(H), eps};
  const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                        reinterpret_cast<uintptr_t>(weight) |
                        reinterpret_cast<uintptr_t>(residual_out) | reinterpret_cast<uintptr_t>(out);
  const bool vec = H % 8 == 0 && (all & 15) == 0;
  if (dt == MOE_F32) return pick_q<float>(p, quant, vec, s);
  if (dt == MOE_F16) return pick_q<__half>(p, quant, vec, s);
  return pick_q<__nv_bfloat16>(p, quant, vec, s);
}

}  // namespace moe
