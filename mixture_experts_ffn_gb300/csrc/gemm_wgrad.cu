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
//   warp 1        : TMEM allocation (pair); lane 0 of the leader issues the MMAs,
//                   the peer's hands out the tiles
//   warp 2        : clears the rows past an expert's end
//   warp 3        : the bias' gradient, d_bias[e, n] = the sum of d[m, n], beside the
//                   products: 32 columns of an expert at a time, from global memory
//                   (a launch of its own for it cost 8 us of 109 at 999 rows, 2880 x
//                   2880, where d is a hundredth of what is written).  One warp walks
//                   all rows of its columns, 64 a round, also where the products are
//                   cut into parts: free at 31 rows an expert (90 us with and without),
//                   not where they are many (256 on each of 32, 2048 x 1024, 39 us
//                   without and 87 with; 1024 on each of 8, 7168 x 2048, 160 and 249;
//                   16384 of one expert, 512 x 512, 23 and 134)
//   warps 4..11   : epilogue of the CTA's 128 TMEM lanes, 64 columns at a time
// Tiles are as long as their expert has rows, and SMs write at unequal rates, so a
// pair takes the next tile from a counter (in the workspace's status area; the
// launch's last pair resets it): a warp of its own does, a tile ahead of the
// producers, and sends it to every role of both CTAs through a ring of entries.
// Against tiles in turn, 32 rows an expert (2880 x 2880, 32 experts) 89 us instead of
// 102, 256 uneven ones (1536 x 2048, 128 experts) 207 instead of 219, 1024 (7168 x
// 2048, 64 experts) 1148 instead of 1139; by the producer itself, which held up the
// copies, 1200.  An expert without rows has no tiles; the epilogue warps write its
// zeros at the end (found by words of 32 experts; a step an expert cost 2 of the 89 us
// and 9 of the 207).  Every wait is bounded (2 s; the clearing warp's for its next job,
// which the producer always ends, 64 s); on a timeout the block latches the timeout bit,
// drains what it issued and frees TMEM.
//
// Few tiles (SPLIT): where experts have many rows and their tiles leave SM pairs idle,
// the rows are cut into `parts` equal pieces, each a tile of its own whose float32 sums
// go to the workspace, and a second launch adds them up in order (wgrad_parts).
//
// What was measured of it: with many rows an expert a stage takes 590 to 620 cycles for
// MMAs of 512, with or without the copies into shared memory, so these are not what
// holds it up; what does was not established.  (The issuing lane itself waits 98 cycles
// a stage and issues for 342; one elected lane of a converged warp issues in 251, waits
// longer, and the whole gains 1% or nothing.  Stages of 32 rows take it 600 cycles as
// well: 252 us instead of 149 on 8 experts of 1024 rows, 7168 x 2048.)  The ring's depth
// counts, since 32 KB a stage into each SM is most of what L2 delivers (4 stages 1328
// us, 5 stages 1204, 6 stages 1165, 64 uneven experts), more than a second buffer for
// the stores (with 5 stages: 1223).  At 32 rows an expert writing d_w bounds (6 TB/s).
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

// Schedule entries.  Entry j is sent when both producers have taken entry j - AHEAD,
// and no role is further back than STAGES + 2 tiles from a producer: a stage is
// loaded again after the MMAs of STAGES stages before, a tile has at least one, and
// its MMAs wait for the drain of the tile before last.  So an entry is never
// overwritten unread.
constexpr int SCHED = 16, AHEAD = 1;
static_assert(STAGES + 2 + AHEAD < SCHED, "schedule ring");
// A clearing job holds its stage until it is done, so as many entries as stages,
// and one for the job that ends the clearing warp.
constexpr int JOBS = 8;
static_assert(STAGES < JOBS, "clearing jobs");

struct WgShared {
  uint64_t full[STAGES];   // leader: both CTAs' copies of a stage, or both clearing warps
  uint64_t own[STAGES];    // this CTA's copies of a stage whose rows are cleared
  uint64_t empty[STAGES];  // both: the leader's commit frees the stage
  uint64_t tfull[2];       // both: accumulator ready
  uint64_t tempty[2];      // leader: both CTAs drained the accumulator
  uint64_t drain;
  uint64_t sfull[SCHED];   // both: schedule entry written
  uint64_t staken[SCHED];  // peer: both producers have the entry
  uint64_t jfull[JOBS];    // clearing job written
  uint4 sched[SCHED];
  int job[JOBS];           // stage, first row, boxes a byte each; -1 ends
  uint32_t tmem_base;
  int abort;
  uint32_t live[kMaxExperts / 32];      // experts with rows
  int live_before[kMaxExperts / 32 + 1];  // of the words before; all
};
constexpr size_t kSmemBytes =
    (size_t)STAGES * STAGE_BYTES + EPI_WARPS * OUT_BYTES_WARP + sizeof(WgShared) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// A tile: rows [lo, hi) of an expert, e its place in the result (with SPLIT, part * E +
// expert in the partial sums), nt and kt its corner in tiles; none for lo == hi.  In the
// schedule {e, lo, hi, nt << 16 | kt}.
struct WgTile {
  int e, lo, hi, nt, kt;
  __device__ __forceinline__ bool none() const { return lo == hi; }
  __device__ __forceinline__ int steps() const { return (hi - lo + BR - 1) / BR; }
  __device__ __forceinline__ int n0() const { return nt * TN; }
  __device__ __forceinline__ int k0() const { return kt * TK; }
  // columns of a: 128 or 256
  __device__ __forceinline__ int kw(int K) const { return K - kt * TK > TK / 2 ? TK : TK / 2; }
  // rows of the last K16 step past the end
  __device__ __forceinline__ bool has_tail() const { return ((hi - lo) & 15) != 0; }
};
// Rows of each of an expert's `parts` pieces (the last ones may be shorter, or empty).
__device__ __forceinline__ int part_rows(int n, int parts) {
  return ((n + parts - 1) / parts + BR - 1) / BR * BR;
}
// Tile t of the list, by a whole warp: the per = tn * tk tiles of the experts with
// rows, times `parts`, follow one another; `end`: t is past the last.  A piece without
// rows is none.
template <bool SPLIT>
__device__ __forceinline__ WgTile wg_decode(int t, const WgShared* sh,
                                            const int32_t* __restrict__ seg_end, int M, int per,
                                            int tk, int parts, int E, bool& end) {
  const int lane = threadIdx.x & 31;
  WgTile r = {};
  const int q = t / (SPLIT ? per * parts : per);
  int in = t - q * (SPLIT ? per * parts : per);
  // (a counter that was not cleared gives no tile, and no fault)
  end = t < 0 || q >= sh->live_before[kMaxExperts / 32];
  if (end) return r;
  // the word of live experts that holds the q-th, and in it the bit with the rest below
  const int before = sh->live_before[lane];
  const uint32_t word = sh->live[lane];
  const int w = __ffs(__ballot_sync(0xffffffffu, before <= q && q < before + __popc(word))) - 1;
  const uint32_t bits = __shfl_sync(0xffffffffu, word, w);
  const int k = q - __shfl_sync(0xffffffffu, before, w);
  r.e = w * 32 + __ffs(__ballot_sync(0xffffffffu, (bits >> lane & 1u) &&
                                                      __popc(bits & ((1u << lane) - 1u)) == k)) - 1;
  seg_bounds(seg_end, r.e, M, 0, r.lo, r.hi);
  if constexpr (SPLIT) {
    const int part = in / per, rows = part_rows(r.hi - r.lo, parts);
    in -= part * per;
    r.lo = min(r.lo + part * rows, r.hi);
    r.hi = min(r.lo + rows, r.hi);
    r.e += part * E;
  }
  r.nt = in / tk;
  r.kt = in - r.nt * tk;
  return r;
}
// K16 steps of stage s of a tile
__device__ __forceinline__ int k16_steps(const WgTile& t, int s) {
  return min(4, (t.hi - t.lo - s * BR + 15) >> 4);
}

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
// Sums of 32 columns n0 .. of d over the rows [lo, hi), by one warp: four lanes
// read 64 bytes of a row, eight rows at once, eight such loads in flight.
template <bool F16>
__device__ __forceinline__ void bias_columns(const __nv_bfloat16* __restrict__ d, int lo, int hi,
                                             int N, int n0, __nv_bfloat16* __restrict__ out) {
  const int lane = threadIdx.x & 31, n = n0 + 8 * (lane & 3);
  float sum[8] = {};
  if (n < N) {  // N is a multiple of 8
    for (int m = lo + (lane >> 2); m < hi; m += 64) {
      uint4 q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i] = m + 8 * i < hi
                   ? __ldg(reinterpret_cast<const uint4*>(d + (size_t)(m + 8 * i) * N + n))
                   : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[2 * j] += lo16<F16>(u[j]);
          sum[2 * j + 1] += hi16<F16>(u[j]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
  if (lane < 4 && n < N) {
    uint4 u;
    u.x = pack2<F16>(sum[0], sum[1]);
    u.y = pack2<F16>(sum[2], sum[3]);
    u.z = pack2<F16>(sum[4], sum[5]);
    u.w = pack2<F16>(sum[6], sum[7]);
    *reinterpret_cast<uint4*>(out + n) = u;
  }
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
// {64, 32, 1}, or with SPLIT the partial sums [parts * E][N][K] in float32, box {32, 32,
// 1}; all with 128-byte swizzle, zeros read and nothing written outside.
template <bool F16, bool SPLIT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_wgrad_kernel(const __grid_constant__ CUtensorMap tm_d,
                      const __grid_constant__ CUtensorMap tm_a,
                      const __grid_constant__ CUtensorMap tm_out,
                      const int32_t* __restrict__ seg_end, int M, int N, int K, int E, int tn,
                      int tk, int parts, const __nv_bfloat16* __restrict__ d,
                      __nv_bfloat16* __restrict__ d_bias, int* status) {
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
      mbar_init(&sh->tempty[a], 2 * EPI_WARPS);
    }
    mbar_init(&sh->drain, 1);
    for (int i = 0; i < SCHED; ++i) {
      mbar_init(&sh->sfull[i], 1);
      mbar_init(&sh->staken[i], 2);
    }
    for (int i = 0; i < JOBS; ++i) mbar_init(&sh->jfull[i], 1);
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
  for (int w = warp; w < kMaxExperts / 32; w += NUM_THREADS / 32) {
    const int e = w * 32 + lane;
    int lo = 0, hi = 0;
    if (e < E) seg_bounds(seg_end, e, M, 0, lo, hi);
    const uint32_t live = __ballot_sync(0xffffffffu, hi > lo);
    if (lane == 0) sh->live[w] = live;
  }
  __syncthreads();
  if (warp == 0) {
    static_assert(kMaxExperts / 32 == 32, "a word a lane");
    const int n = __popc(sh->live[lane]);
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    sh->live_before[lane] = sum - n;
    if (lane == 31) sh->live_before[32] = sum;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = sh->tmem_base;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int per = tn * tk;
  int* gctr = status + 8;  // tiles taken from the counter, pairs done
  // tile j of the schedule (none at its end, or when the wait failed)
  auto next_tile = [&](int j) -> WgTile {
    WgTile r = {};
    if (!wait_fast<kWaitShared>(&sh->sfull[j % SCHED], (uint32_t)(j / SCHED) & 1u, abort_flag,
                                status))
      return r;
    const uint32_t addr = su32(&sh->sched[j % SCHED]);
    uint32_t corner;
    asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.e), "=r"(r.lo), "=r"(r.hi), "=r"(corner)
                 : "r"(addr)
                 : "memory");
    r.nt = (int)(corner >> 16);
    r.kt = (int)(corner & 0xffffu);
    return r;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------- producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0, own_used = 0, own_phase = 0, last_own = 0, used = 0, used_phase = 0;
      bool ok = true;
      int jobs = 0;
      const uint32_t staken0 = map_to_rank(su32(&sh->staken[0]), 1);
      // (the arrival paces the schedule and orders nothing)
      auto take = [&](int j) -> WgTile {
        const WgTile t = next_tile(j);
        mbar_arrive_cluster_tmem(staken0 + (uint32_t)(j % SCHED * sizeof(uint64_t)));
        return t;
      };
      WgTile st = take(0), nx{};
      for (int j = 0; ok && !st.none(); ++j) {
        const int steps = st.steps(), half = st.kw(K) >> 1, nb = half / 64;
        const uint32_t tx = (uint32_t)(A_BYTES + nb * BOX_BYTES);
        const int nc = st.n0() + 128 * (int)rank, kc = st.k0() + half * (int)rank;
        for (int s = 0; s < steps; ++s) {
          if (!wait_pair(&sh->empty[stage], phase ^ 1u, abort_flag, status)) { ok = false; break; }
          uint8_t* a_dst = smem + (size_t)stage * STAGE_BYTES;
          uint8_t* b_dst = a_dst + A_BYTES;
          uint32_t bar;
          const uint32_t bit = 1u << stage;
          if (s == steps - 1 && st.has_tail()) {
            mbar_expect_tx(&sh->own[stage], tx);
            bar = map_to_rank(su32(&sh->own[stage]), rank);
            own_phase = (own_used & bit) ? own_phase ^ bit : own_phase & ~bit;
            own_used |= bit;
            last_own |= bit;
            *reinterpret_cast<volatile int*>(&sh->job[jobs % JOBS]) =
                stage | (st.hi - st.lo - s * BR) << 8 | (2 + nb) << 16;
            mbar_arrive(&sh->jfull[jobs % JOBS]);
            ++jobs;
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
          if (s == 0) nx = take(j + 1);
        }
        st = nx;
      }
      // no more jobs
      *reinterpret_cast<volatile int*>(&sh->job[jobs % JOBS]) = -1;
      mbar_arrive(&sh->jfull[jobs % JOBS]);
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
      WgTile st = next_tile(0), nx{};
      for (int j = 0; ok && !st.none(); ++j) {
        const int steps = st.steps();
        const uint32_t idesc = idesc_sw(TN, st.kw(K), F16 ? 1 : 0, true, true);
        if (!wait_pair_tmem(&sh->tempty[acc], aphase ^ 1u, abort_flag, status)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * TK);
        for (int s = 0; s < steps; ++s) {
          // copies alone complete a stage at this CTA's scope; after the clearing
          // warps (which order their writes for the async proxy themselves) the
          // peer's shared memory is acquired
          if (!(s == steps - 1 && st.has_tail()
                    ? wait_pair<true>(&sh->full[stage], phase, abort_flag, status)
                    : wait_pair<false>(&sh->full[stage], phase, abort_flag, status))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = (uint64_t)((stage * STAGE_BYTES) >> 4);
          umma2_rows(d_tmem, adesc0 + off, bdesc0 + off, idesc, s != 0 ? 1u : 0u,
                     k16_steps(st, s), su32(&sh->empty[stage]));
          any = true;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          if (s == 0) nx = next_tile(j + 1);  // while the MMAs run
        }
        if (!ok) break;
        umma2_commit_both(&sh->tfull[acc]);
        if (++acc == 2) { acc = 0; aphase ^= 1u; }
        st = nx;
      }
      if (!ok && any) {
        umma2_commit_self(&sh->drain);
        drain_wait(&sh->drain, 0);
      }
    }
    if (!leader) {
      // ---------------------------------------------- schedule (peer, whole warp)
      int t = pair;  // the first tile is the pair's own
      bool ok = true;
      for (int j = 0;; ++j) {
        WgTile st;
        for (bool end = false;;) {
          st = wg_decode<SPLIT>(t, sh, seg_end, M, per, tk, parts, E, end);
          if (end) break;
          int grabbed = 0;
          if (lane == 0) grabbed = npairs + atomicAdd(gctr, 1);
          t = __shfl_sync(0xffffffffu, grabbed, 0);
          if (!st.none()) break;  // (a piece without rows is passed over)
        }
        if (j >= AHEAD) {
          const int i = j - AHEAD;
          ok = wait_fast(&sh->staken[i % SCHED], (uint32_t)(i / SCHED) & 1u, abort_flag, status);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        if (lane < 2)
          publish_remote_v4(map_to_rank(su32(&sh->sched[j % SCHED]), lane),
                            map_to_rank(su32(&sh->sfull[j % SCHED]), lane), (uint32_t)st.e,
                            (uint32_t)st.lo, (uint32_t)st.hi, (uint32_t)(st.nt << 16 | st.kt));
        if (st.none()) break;
      }
      if (lane == 0 && !*abort_flag) {
        __threadfence();  // this pair's last take before its done count
        if (atomicAdd(gctr + 1, 1) == npairs - 1) {
          __threadfence();  // every pair's takes before the reset
          atomicExch(gctr, 0);
          atomicExch(gctr + 1, 0);
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------ clearing (both CTAs)
    uint32_t own_phase = 0;  // bit s: parity of own[s]'s next phase
    const uint32_t full_remote0 = map_to_rank(su32(&sh->full[0]), 0);
    for (int i = 0;; ++i) {
      // there may be no job for as long as the launch takes; the producer, whose own
      // waits are bounded, always sends the last one
      bool ok = false;
      for (int k = 0; k < 32 && !ok; ++k) {
        drain_wait(&sh->jfull[i % JOBS], (uint32_t)(i / JOBS) & 1u);
        ok = mbar_try_wait(su32(&sh->jfull[i % JOBS]), (uint32_t)(i / JOBS) & 1u);
      }
      const int job = *reinterpret_cast<volatile int*>(&sh->job[i % JOBS]);
      // the lanes go on, or give up, together
      if (!__all_sync(0xffffffffu, ok) || job < 0) break;
      const int stage = job & 255, r0 = job >> 8 & 255, r1 = (r0 + 15) & ~15, boxes = job >> 16;
      ok = wait_fast(&sh->own[stage], (own_phase >> stage) & 1u, abort_flag, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      own_phase ^= 1u << stage;
      // rows r0 .. r1 - 1 of every box, whole 128-byte rows (the swizzle stays
      // inside a row)
      uint8_t* base = smem + (size_t)stage * STAGE_BYTES;
      for (int b = 0; b < boxes; ++b)
        for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
          *reinterpret_cast<uint4*>(base + b * BOX_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(full_remote0 + (uint32_t)(stage * sizeof(uint64_t)));
    }
  } else if (warp == 3) {
    // ------------------------------------------------ bias (both CTAs)
    if (d_bias) {
      const int per = (N + 31) / 32;
      for (int u = blockIdx.x; u < E * per; u += gridDim.x) {
        const int e = u / per;
        int lo, hi;
        seg_bounds(seg_end, e, M, 0, lo, hi);
        bias_columns<F16>(d, lo, hi, N, (u - e * per) * 32, d_bias + (size_t)e * N);
      }
    }
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    const int quad = warp & 3, grp = (warp - EPI_WARP0) >> 2;
    int acc = 0;
    uint32_t aphase = 0;
    const uint32_t tempty_remote[2] = {map_to_rank(su32(&sh->tempty[0]), 0),
                                       map_to_rank(su32(&sh->tempty[1]), 0)};
    uint8_t* buf = out_stage + (warp - EPI_WARP0) * OUT_BYTES_WARP;
    // 32 rows of 64 columns from the warp's buffer
    auto store = [&](const WgTile& st, int c, int n) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&tm_out, buf, st.k0() + c, n, st.e);
        bulk_commit();
      }
    };
    for (int j = 0;; ++j) {
      const WgTile st = next_tile(j);
      // the lanes go on, or give up, together
      if (__any_sync(0xffffffffu, st.none())) break;
      if (!__all_sync(0xffffffffu, wait_pair_tmem(&sh->tfull[acc], aphase, abort_flag, status)))
        break;
      tc_fence_after();
      const int n = st.n0() + 128 * (int)rank + 32 * quad;
      const uint32_t tb = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * TK);
#pragma unroll 1
      for (int c = 64 * grp; c < st.kw(K); c += 128) {
        if (n >= N || st.k0() + c >= K) break;  // warp-uniform
        uint32_t r[2][32];
        tmem_ld32(tb + (uint32_t)c, r[0]);
        tmem_ld32(tb + (uint32_t)c + 32, r[1]);
        tmem_wait_ld();
        // boxes of 128-byte rows: 64 results, or twice 32 partial sums
#pragma unroll
        for (int h = 0; h < (SPLIT ? 2 : 1); ++h) {
          if (SPLIT && st.k0() + c + 32 * h >= K) break;  // warp-uniform
          if (lane == 0) bulk_wait_read<0>();  // the last store from this buffer
          __syncwarp();
          // row `lane` of the box, 16-byte chunk q at q ^ (lane & 7)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint4 u;
            if constexpr (SPLIT) {
              u = make_uint4(r[h][4 * q], r[h][4 * q + 1], r[h][4 * q + 2], r[h][4 * q + 3]);
            } else {
              const uint32_t* v = &r[q >> 2][(q & 3) * 8];
              u.x = pack2<F16>(__uint_as_float(v[0]), __uint_as_float(v[1]));
              u.y = pack2<F16>(__uint_as_float(v[2]), __uint_as_float(v[3]));
              u.z = pack2<F16>(__uint_as_float(v[4]), __uint_as_float(v[5]));
              u.w = pack2<F16>(__uint_as_float(v[6]), __uint_as_float(v[7]));
            }
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) = u;
          }
          store(st, c + 32 * h, n);
        }
      }
      // one arrival a warp: those of all 512 threads took their time one by one
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_tmem(tempty_remote[acc]);
      if (++acc == 2) { acc = 0; aphase ^= 1u; }
    }
    // the experts without rows: their tiles follow one another and go to the pairs in
    // turn; `first` is the pair's next one in the expert at hand
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
    for (int i = lane; i < OUT_BYTES_WARP / 16; i += 32)
      reinterpret_cast<uint4*>(buf)[i] = make_uint4(0, 0, 0, 0);
    const int shift = per % npairs;
    int first = pair;
    for (int w = 0; !SPLIT && w * 32 < E; ++w) {  // (adding up the parts writes them too)
      uint32_t empty = ~sh->live[w];
      if (E - w * 32 < 32) empty &= (1u << (E - w * 32)) - 1u;
      for (; empty; empty &= empty - 1u) {
        WgTile st = {w * 32 + __ffs(empty) - 1, 0, 0, 0, 0};
        for (int in = first; in < per; in += npairs) {
          st.nt = in / tk;
          st.kt = in - st.nt * tk;
          const int n = st.n0() + 128 * (int)rank + 32 * quad;
          for (int c = 64 * grp; c < st.kw(K); c += 128)
            if (n < N && st.k0() + c < K) store(st, c, n);
        }
        first -= shift;
        if (first < 0) first += npairs;
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

namespace {

// d_w[e] = the sum of its parts' partial sums in order, rounded once; zeros for an
// expert without rows.  Eight results a thread.
template <bool F16>
__global__ void __launch_bounds__(256)
    wgrad_join_kernel(const float4* __restrict__ partial, const int32_t* __restrict__ seg_end,
                      int M, long long per_expert, int E, int parts, uint4* __restrict__ d_w) {
  pdl_wait();
  const long long count = per_expert * E;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < count; i += gridDim.x * 256LL) {
    int lo, hi;
    seg_bounds(seg_end, (int)(i / per_expert), M, 0, lo, hi);
    const int rows = part_rows(hi - lo, parts), n = hi > lo ? (hi - lo + rows - 1) / rows : 0;
    float v[8] = {};
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const float4 a = __ldcs(partial + (p * count + i) * 2);
      const float4 b = __ldcs(partial + (p * count + i) * 2 + 1);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    d_w[i] = make_uint4(pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]), pack2<F16>(v[4], v[5]),
                        pack2<F16>(v[6], v[7]));
  }
}

// Pieces that an expert's rows are cut into: as many as there are SM pairs for the
// tiles of all experts, of 256 rows at least (on average), and one where that shortens a
// tile by less than 1200 rows, since the partial sums and the second launch cost 3 us or
// more (all without a bias): 2 experts of 6639 rows, 544 x 288, 17.7 us in 6 pieces,
// 38.5 in one; one of 8192, 1024 x 1024, 22 in 4 and 46; but one of 1024, 13.1 in 4 and
// 12.3, and 4 of 1024, 512 x 1024, 14.9 in 2 and 12.4.
// One expert may have nearly all of the rows, whatever their average: a piece is cut to
// 2^26 of them at most, a million stages of 0.3 us, since the drain waits for a piece's
// sum and a wait ends after 2 s (2^30 rows in one piece would take 5).
int wgrad_parts(int M, int N, int K, int E) {
  const int least = (int)std::max(1LL, ((M - 1LL) >> 26) + 1);
  const long long experts = std::max(1, std::min(E, M)), rows = M / experts;
  const long long tiles = ((N + TN - 1LL) / TN) * ((K + TK - 1LL) / TK) * experts;
  const long long parts = std::min<long long>(num_sms() / 2 / tiles, rows / 256);
  return std::max(parts >= 2 && rows - rows / parts >= 1200 ? (int)parts : 1, least);
}

}  // namespace

size_t gemm_wgrad_partial_bytes(int M, int N, int K, int E) {
  const int parts = wgrad_parts(M, N, K, E);
  return parts > 1 ? (size_t)parts * E * N * K * sizeof(float) : 0;
}

// a schedule entry has 16 bits for each coordinate of a tile
bool gemm_wgrad_ok(int N, int K) {
  return N % 8 == 0 && K % 8 == 0 && N <= 0xffff * TN && K <= 0xffff * TK;
}

cudaError_t launch_gemm_wgrad(const void* d, const void* a, const int32_t* seg_end, int M, int N,
                              int K, int E, bool f16, void* d_w, void* d_bias, int* status,
                              float* partial, cudaStream_t s) {
  if (!gemm_wgrad_ok(N, K)) return cudaErrorInvalidValue;
  int parts = wgrad_parts(M, N, K, E);
  const bool split = parts > 1;
  CUtensorMap md, ma, mo;
  auto rows = [&](CUtensorMap* m, const void* p, int cols) {
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)M};
    cuuint64_t str[1] = {(cuuint64_t)cols * 2};
    cuuint32_t box[2] = {64, BR};
    return tmap::encode_bf16(m, p, 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B, f16);
  };
  const cuuint64_t size = split ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)E * parts};
  cuuint64_t str[2] = {(cuuint64_t)K * size, (cuuint64_t)N * K * size};
  cuuint32_t box[3] = {(cuuint32_t)(128 / size), 32, 1};
  if (!rows(&md, d, N) || !rows(&ma, a, K) ||
      !(split ? tmap::encode_f32(&mo, partial, 3, dims, str, box)
              : tmap::encode_bf16(&mo, d_w, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B, f16)))
    return cudaErrorInvalidValue;
  int tn = (N + TN - 1) / TN, tk = (K + TK - 1) / TK;
  const int pairs = std::max(1, std::min(E * tn * tk * parts, num_sms() / 2));
  const void* kern = split ? (f16 ? (const void*)gemm_wgrad_kernel<true, true>
                                  : (const void*)gemm_wgrad_kernel<false, true>)
                           : (f16 ? (const void*)gemm_wgrad_kernel<true, false>
                                  : (const void*)gemm_wgrad_kernel<false, false>);
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
  const __nv_bfloat16* d_p = static_cast<const __nv_bfloat16*>(d);
  __nv_bfloat16* bias_p = static_cast<__nv_bfloat16*>(d_bias);
  void* args[] = {&md, &ma,    &mo,  &seg_end, &M,     &N, &K, &E,
                  &tn, &tk, &parts, &d_p,     &bias_p, &status};
  e = cudaLaunchKernelExC(&cfg, kern, args);
  count_launch();
  if (e != cudaSuccess || !split) return e;
  const long long per_expert = (long long)N * K / 8, count = per_expert * E;
  auto join = [&](auto k) {
    const long long cap = (long long)num_sms() * resident_ctas((const void*)k, 256);
    return launch_pdl(k, dim3((unsigned)std::min((count + 255) / 256, cap)), dim3(256), 0, s,
                      reinterpret_cast<const float4*>(partial), seg_end, M, per_expert, E, parts,
                      static_cast<uint4*>(d_w));
  };
  e = f16 ? join(wgrad_join_kernel<true>) : join(wgrad_join_kernel<false>);
  count_launch();
  return e;
}

}  // namespace moe
