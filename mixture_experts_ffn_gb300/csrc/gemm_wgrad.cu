// Gradient of a grouped product's weights on SM pairs (tcgen05.mma.cta_group::2):
//   d_w[e, n, k] = sum over the rows m of expert e of d[m, n] a[m, k]
// 16-bit operands and results, float32 accumulators in TMEM.
//
// The sum runs over rows, so both operands are read across their rows: a TMA box
// holds 64 columns (one 128-byte swizzle atom) of 64 rows, and A and B are both
// MN-major.  A pair's tile is 256 n x 256 k; each CTA holds 128 n of d and half of
// the k columns of a: 16 + 16 KB a stage of 64 rows, 6 stages.  A last tile of at
// most 128 k columns is 128 wide (below that an MMA takes no less time).
//
// An expert's rows are few (tens to a thousand) and its tile 128 KB of results, so
// tiles are short and end in a large store: two 256-column accumulators let a
// tile's store overlap the next tile's sum, and two warpgroups drain.
//
// The last stage of an expert reaches into the next expert's rows.  K16 steps past
// its end are not issued; in the last step the rows past the end are cleared in
// both operands (0 times the NaN of a neighbour would be NaN) by a warp of each
// CTA: such a stage's copies complete on a barrier of their own CTA, and the
// clearing warps' arrivals take the place of the copies' on the leader's barrier.
//
// Roles (384 threads per CTA)
//   warp 0 lane 0 : producer
//   warp 1        : TMEM allocation (pair); lane 0 of the leader issues the MMAs
//   warp 2        : clears the rows past an expert's end
//   warps 4..11   : epilogue of the CTA's 128 TMEM lanes, 64 columns at a time
// Tiles go round-robin; an expert without rows gets zeros.  Every wait is bounded
// (2 s); on a timeout the block latches the timeout bit, drains what it issued and
// frees TMEM.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace moe {
namespace {

using namespace tc;

constexpr int BR = 64;                        // rows of a stage
constexpr int BOX_BYTES = 64 * BR * 2;        // 64 columns of 64 rows
constexpr int TN = 256, TK = 256;             // a pair's tile
constexpr int A_BYTES = 2 * BOX_BYTES;        // 128 columns of d
constexpr int B_BYTES = 2 * BOX_BYTES;        // up to 128 columns of a
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 6;
constexpr int TMEM_COLS = 512;
constexpr int EPI_WARPS = 8, EPI_WARP0 = 4;
constexpr int NUM_THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
constexpr int OUT_BYTES_WARP = 32 * 64 * 2;   // 32 rows of 64 columns

struct WgShared {
  uint64_t full[STAGES];   // leader: both CTAs' copies of a stage, or both clearing warps
  uint64_t own[STAGES];    // this CTA's copies of a stage whose rows are cleared
  uint64_t empty[STAGES];  // both: the leader's commit frees the stage
  uint64_t tfull[2];       // both: accumulator ready
  uint64_t tempty[2];      // leader: both CTAs drained the accumulator
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmemBytes =
    (size_t)STAGES * STAGE_BYTES + EPI_WARPS * OUT_BYTES_WARP + sizeof(WgShared) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Tile t: expert e with rows [lo, hi), n0 and k0 its corner, kw its columns (128 or
// 256); `steps` stages.
struct WgTile {
  int e, lo, hi, n0, k0, kw, steps;
};
__device__ __forceinline__ WgTile wg_decode(int t, const int32_t* __restrict__ seg_end, int M,
                                            int K, int tn, int tk) {
  WgTile r;
  const int per = tn * tk;
  r.e = t / per;
  const int in = t - r.e * per;
  r.n0 = (in / tk) * TN;
  r.k0 = (in % tk) * TK;
  r.kw = K - r.k0 > TK / 2 ? TK : TK / 2;
  seg_bounds(seg_end, r.e, M, 0, r.lo, r.hi);
  r.steps = (r.hi - r.lo + BR - 1) / BR;
  return r;
}
// K16 steps of stage s of a tile, and whether its last one has rows to clear
__device__ __forceinline__ int k16_steps(const WgTile& t, int s) {
  return min(4, (t.hi - t.lo - s * BR + 15) >> 4);
}
__device__ __forceinline__ bool has_tail(const WgTile& t) { return ((t.hi - t.lo) & 15) != 0; }

// `n16` (1..4) K16 MMAs of a stage and the commit that frees it in both CTAs.
__device__ __forceinline__ void umma2_rows(uint32_t d_tmem, uint64_t ad, uint64_t bd,
                                           uint32_t idesc, uint32_t accumulate, int n16,
                                           uint32_t bar) {
  constexpr uint32_t S = kMnStep;
  asm volatile(
      "{\n\t.reg .pred p, t, q1, q2, q3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, %4, %4;\n\t"
      "setp.gt.s32 q1, %12, 1;\n\t"
      "setp.gt.s32 q2, %12, 2;\n\t"
      "setp.gt.s32 q3, %12, 3;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@q1 tcgen05.mma.cta_group::2.kind::f16 [%0], %6, %7, %3, t;\n\t"
      "@q2 tcgen05.mma.cta_group::2.kind::f16 [%0], %8, %9, %3, t;\n\t"
      "@q3 tcgen05.mma.cta_group::2.kind::f16 [%0], %10, %11, %3, t;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%5], %13;\n\t}" ::"r"(d_tmem),
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate), "r"(bar), "l"(ad + S), "l"(bd + S),
      "l"(ad + 2 * S), "l"(bd + 2 * S), "l"(ad + 3 * S), "l"(bd + 3 * S), "r"(n16),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int c0, int c1,
                                             int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(su32(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// tm_d: d [M][N], tm_a: a [M][K], boxes {64, 64}; tm_out: d_w [E][N][K], box
// {64, 32, 1}; all with 128-byte swizzle, zeros read and nothing written outside.
template <bool F16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_wgrad_kernel(const __grid_constant__ CUtensorMap tm_d,
                      const __grid_constant__ CUtensorMap tm_a,
                      const __grid_constant__ CUtensorMap tm_out,
                      const int32_t* __restrict__ seg_end, int M, int N, int K, int total, int tn,
                      int tk, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* out_stage = smem + (size_t)STAGES * STAGE_BYTES;
  WgShared* sh = reinterpret_cast<WgShared*>(out_stage + EPI_WARPS * OUT_BYTES_WARP);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  volatile int* abort_flag = &sh->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh->full[s], 2);
      mbar_init(&sh->own[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sh->tfull[a], 1);
      mbar_init(&sh->tempty[a], 2 * 32 * EPI_WARPS);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_d)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_out)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     su32(&sh->tmem_base)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  // everything above overlaps the previous launch; seg_end and the operands are
  // read only after this
  pdl_wait();
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = sh->tmem_base;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  auto decode = [&](int t) { return wg_decode(t, seg_end, M, K, tn, tk); };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------- producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0, own_used = 0, own_phase = 0, last_own = 0, used = 0, used_phase = 0;
      bool ok = true;
      WgTile nx{};
      if (pair < total) nx = decode(pair);
      for (int t = pair; t < total && ok; t += npairs) {
        const WgTile st = nx;  // the next tile's bounds arrive during this one
        if (t + npairs < total) nx = decode(t + npairs);
        const int half = st.kw >> 1;
        const int nb = half / 64;
        const uint32_t tx = (uint32_t)(A_BYTES + nb * BOX_BYTES);
        const int nc = st.n0 + 128 * (int)rank, kc = st.k0 + half * (int)rank;
        for (int s = 0; s < st.steps; ++s) {
          if (!wait_pair(&sh->empty[stage], phase ^ 1u, abort_flag, status)) { ok = false; break; }
          uint8_t* a_dst = smem + (size_t)stage * STAGE_BYTES;
          uint8_t* b_dst = a_dst + A_BYTES;
          uint32_t bar;
          const uint32_t bit = 1u << stage;
          if (s == st.steps - 1 && has_tail(st)) {
            mbar_expect_tx(&sh->own[stage], tx);
            bar = map_to_rank(su32(&sh->own[stage]), rank);
            own_phase = (own_used & bit) ? own_phase ^ bit : own_phase & ~bit;
            own_used |= bit;
            last_own |= bit;
          } else {
            if (leader) {
              mbar_expect_tx(&sh->full[stage], 2 * tx);
              mbar_arrive(&sh->full[stage]);
            }
            bar = map_to_rank(su32(&sh->full[stage]), 0);
            last_own &= ~bit;
          }
          used_phase = (used & bit) ? used_phase ^ bit : used_phase & ~bit;
          used |= bit;
          const int r0 = st.lo + s * BR;
          tma2_2d(a_dst, &tm_d, bar, nc, r0);
          tma2_2d(a_dst + BOX_BYTES, &tm_d, bar, nc + 64, r0);
          tma2_2d(b_dst, &tm_a, bar, kc, r0);
          if (nb == 2) tma2_2d(b_dst + BOX_BYTES, &tm_a, bar, kc + 64, r0);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {  // what is in flight lands before the block exits
        for (int s = 0; s < STAGES; ++s) {
          if (!((used >> s) & 1u)) continue;
          if ((last_own >> s) & 1u) drain_wait(&sh->own[s], (own_phase >> s) & 1u);
          else if (leader) drain_wait(&sh->full[s], (used_phase >> s) & 1u);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------------------------------------- MMA issuer (leader)
      int stage = 0, acc = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true, any = false;
      const uint64_t adesc0 = sw128_mn_desc(su32(smem), BOX_BYTES);
      const uint64_t bdesc0 = sw128_mn_desc(su32(smem + A_BYTES), BOX_BYTES);
      WgTile nx{};
      if (pair < total) nx = decode(pair);
      for (int t = pair; t < total && ok; t += npairs) {
        const WgTile st = nx;
        if (t + npairs < total) nx = decode(t + npairs);
        if (st.steps == 0) continue;
        const uint32_t idesc = idesc_sw(TN, st.kw, F16 ? 1 : 0, true, true);
        if (!wait_pair_tmem(&sh->tempty[acc], aphase ^ 1u, abort_flag, status)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * TK);
        for (int s = 0; s < st.steps; ++s) {
          if (!wait_pair(&sh->full[stage], phase, abort_flag, status)) { ok = false; break; }
          // a clearing warp wrote through the generic proxy, the MMA reads
          // through the async proxy
          if (s == st.steps - 1) fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t off = (uint64_t)((stage * STAGE_BYTES) >> 4);
          umma2_rows(d_tmem, adesc0 + off, bdesc0 + off, idesc, s != 0 ? 1u : 0u,
                     k16_steps(st, s), su32(&sh->empty[stage]));
          any = true;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma2_commit_both(&sh->tfull[acc]);
        if (++acc == 2) { acc = 0; aphase ^= 1u; }
      }
      if (!ok && any) {
        umma2_commit_self(&sh->drain);
        drain_wait(&sh->drain, 0);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------ clearing (both CTAs)
    int stage = 0;
    uint32_t own_phase = 0;  // bit s: parity of own[s]'s next phase
    const uint32_t full_remote0 = map_to_rank(su32(&sh->full[0]), 0);
    WgTile nx{};
    if (pair < total) nx = decode(pair);
    for (int t = pair; t < total; t += npairs) {
      const WgTile st = nx;
      if (t + npairs < total) nx = decode(t + npairs);
      if (st.steps == 0) continue;
      const int last = (stage + st.steps - 1) % STAGES;
      stage = (stage + st.steps) % STAGES;
      if (!has_tail(st)) continue;
      if (!wait_fast(&sh->own[last], (own_phase >> last) & 1u, abort_flag, status)) break;
      own_phase ^= 1u << last;
      // rows r0 .. r1 - 1 of every box, whole 128-byte rows (the swizzle stays
      // inside a row)
      const int r0 = (st.hi - st.lo) - (st.steps - 1) * BR, r1 = (r0 + 15) & ~15;
      const int boxes = 2 + st.kw / 128;
      uint8_t* base = smem + (size_t)last * STAGE_BYTES;
      for (int b = 0; b < boxes; ++b)
        for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
          *reinterpret_cast<uint4*>(base + b * BOX_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(full_remote0 + (uint32_t)(last * sizeof(uint64_t)));
    }
  } else if (warp >= EPI_WARP0) {
    // ------------------------------------------------ epilogue (both CTAs)
    const int quad = warp & 3, grp = (warp - EPI_WARP0) >> 2;
    int acc = 0;
    uint32_t aphase = 0;
    const uint32_t tempty_remote[2] = {map_to_rank(su32(&sh->tempty[0]), 0),
                                       map_to_rank(su32(&sh->tempty[1]), 0)};
    uint8_t* buf = out_stage + (warp - EPI_WARP0) * OUT_BYTES_WARP;
    WgTile nx{};
    if (pair < total) nx = decode(pair);
    for (int t = pair; t < total; t += npairs) {
      const WgTile st = nx;
      if (t + npairs < total) nx = decode(t + npairs);
      const bool zero = st.steps == 0;
      if (!zero) {
        if (!wait_pair_tmem(&sh->tfull[acc], aphase, abort_flag, status)) break;
        tc_fence_after();
      }
      const int n = st.n0 + 128 * (int)rank + 32 * quad;
      const uint32_t tb = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * TK);
#pragma unroll 1
      for (int c = 64 * grp; c < st.kw; c += 128) {
        if (n >= N || st.k0 + c >= K) break;  // warp-uniform
        uint32_t r[2][32];
        if (!zero) {
          tmem_ld32(tb + (uint32_t)c, r[0]);
          tmem_ld32(tb + (uint32_t)c + 32, r[1]);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[0][i] = r[1][i] = 0;
        }
        if (lane == 0) bulk_wait_read<0>();  // the last store from this buffer
        __syncwarp();
        // row `lane` of the box, 16-byte chunk q at q ^ (lane & 7)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t* v = &r[q >> 2][(q & 3) * 8];
          uint4 u;
          u.x = pack2<F16>(__uint_as_float(v[0]), __uint_as_float(v[1]));
          u.y = pack2<F16>(__uint_as_float(v[2]), __uint_as_float(v[3]));
          u.z = pack2<F16>(__uint_as_float(v[4]), __uint_as_float(v[5]));
          u.w = pack2<F16>(__uint_as_float(v[6]), __uint_as_float(v[7]));
          *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) = u;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&tm_out, buf, st.k0 + c, n, st.e);
          bulk_commit();
        }
      }
      if (!zero) {
        tc_fence_before();
        mbar_arrive_cluster_tmem(tempty_remote[acc]);
        if (++acc == 2) { acc = 0; aphase ^= 1u; }
      }
    }
    if (lane == 0) bulk_wait_all();  // every staged box written before the pair exits
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA frees TMEM or exits while its peer still works
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

}  // namespace

cudaError_t launch_gemm_wgrad(const void* d, const void* a, const int32_t* seg_end, int M, int N,
                              int K, int E, bool f16, void* d_w, int* status, cudaStream_t s) {
  if (N % 8 != 0 || K % 8 != 0) return cudaErrorInvalidValue;
  CUtensorMap md, ma, mo;
  auto rows = [&](CUtensorMap* m, const void* p, int cols) {
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)M};
    cuuint64_t str[1] = {(cuuint64_t)cols * 2};
    cuuint32_t box[2] = {64, BR};
    return tmap::encode_bf16(m, p, 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B, f16);
  };
  cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)E};
  cuuint64_t str[2] = {(cuuint64_t)K * 2, (cuuint64_t)N * K * 2};
  cuuint32_t box[3] = {64, 32, 1};
  if (!rows(&md, d, N) || !rows(&ma, a, K) ||
      !tmap::encode_bf16(&mo, d_w, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B, f16))
    return cudaErrorInvalidValue;
  int tn = (N + TN - 1) / TN, tk = (K + TK - 1) / TK;
  int total = E * tn * tk;
  const int pairs = std::max(1, std::min(total, num_sms() / 2));
  const void* kern = f16 ? (const void*)gemm_wgrad_kernel<true> : (const void*)gemm_wgrad_kernel<false>;
  cudaError_t e = set_smem_limit(kern, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_pdl
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {&md, &ma, &mo, &seg_end, &M, &N, &K, &total, &tn, &tk, &status};
  e = cudaLaunchKernelExC(&cfg, kern, args);
  count_launch();
  return e;
}

}  // namespace moe
