// Grouped GEMM over microscaled operands (mx_dev.cuh): rows of activations in
// MX e4m3 times expert weights in MX e2m1, over the expert-segmented row
// layout, with bias, activation and the output rounding (a 16-bit or float32
// type, or MX e4m3 for the next product) in the epilogue.
//
// Mathematics: p[m, n] = sum over blocks b of 2^(sa[m, b] + sw[n, b]) *
// (codes of a, block b . codes of w, block b).  tcgen05.mma kind::mxf8f6f4
// applies both scales inside the tensor core and accumulates in float32, so
// neither operand is expanded in memory: weights cross HBM at 17/32 byte a
// value.
//
// Layout: the expert's weight rows are the MMA's M operand (128 rows a half),
// the tokens of a chunk of its segment the N operand (a multiple of 16), so a
// segment pads to 16 rows.  Two halves share each token slice: gate and up
// rows of the same 128 outputs (gated kinds), or 256 consecutive output
// columns (plain).  TMEM lane = output column, TMEM column = token; a warp's
// 32 lanes are one MX block of a token's output, so its scale is one
// redux.sync.
//
// Roles (512 threads, one CTA per SM, persistent)
//   warp 0 lane 0 : TMA producer of the weight codes.  The map's type expands
//                   each 16 packed values (8 bytes) into a 16-byte chunk of
//                   shared memory, the form the MMA reads 4-bit values in.
//   warp 1        : TMEM; issues the MMAs
//   warps 2..3    : cp.async loaders of the token rows (gathered through
//                   row_to_route when given)
//   warps 4..7    : both operands' scales, four stages at a time through shared
//                   memory into registers, then tcgen05.st into TMEM, each warp
//                   its own lane quarter (the MMA wants them in all four).  They
//                   have a ring of their own, of two or four stages a slot: tied
//                   to the operands' ring, a stage at a time, these warps set
//                   the pace (585 cycles a stage).
//                   tcgen05.cp would need no warps, but runs in the MMAs' own
//                   pipe and costs it 170 cycles a stage.
//   warps 8..15   : epilogue, two warps a lane quarter
// Stage: 128 columns of K, i.e. four K32 MMA steps; the 4 scale bytes of a
// row and stage are one 32-bit TMEM cell, step j using byte j of it.
// Measured back to back, a stage's eight MMAs take max(313, 4 N) cycles.
// PAIR (cta_group::2): two CTAs share a tile, each with its own weight rows and
// half the tokens; the leader's MMAs read both CTAs' shared memory.  The peer's
// token copies reach the leader's barrier through a forwarding thread, the scale
// warps' and epilogues' arrivals directly.
//
// What bounds it (GB300, median of single launches, L2 flushed): decode (one row
// on each of 128 experts, 2048 x 7168 gate_up) the weights' stream, 312 us for
// 2.0 GB, 0.94 of the measured HBM rate; medium batches (8192 ragged rows on 128
// experts, 2880 x 2880 down: 142 us, 0.66 of HBM) what the ring holds in flight,
// 80 KB of packed weights an SM, half its memory going to the gaps of the expanded
// form, and the weights of experts of several chunks, read again a chunk; many rows
// (65536 ragged ones on 64 experts, 2048 x 7168 gate_up) the MMAs, 1156 us, 0.86 of
// twice the measured bf16 rate (one after another 1324: the power cap), the rest
// shared-memory contention and the one accumulator's epilogue.
// Every wait is bounded (tc_ptx.cuh).
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "gemm_epilogue.cuh"
#include "mx_dev.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace moe {
namespace {

using namespace tc;

constexpr int BK = 128;                    // columns of K per stage
constexpr int W_BYTES = 128 * BK;          // one half's weights, expanded: 16 KB
constexpr int W_TX = W_BYTES / 2;          // bytes its copy counts: the packed ones (the gaps of
                                           // the expanded form are not written)
constexpr int SG = 4;                      // stages whose scales travel together
constexpr int SBUFS = 3;                   // chunks of scales in flight or in use
constexpr int kLoadWarp0 = 2, kScaleWarp0 = 4, kEpiWarp0 = 8, kEpiWarps = 8;
constexpr int kLoaders = 32 * (kScaleWarp0 - kLoadWarp0);
constexpr int NUM_THREADS = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kScaleBar = 1;               // named barrier of the scale warps
constexpr size_t kSmemLimit = 227 * 1024;

// Token columns of a tile and what follows from them: ring depth and TMEM.
// HALVES: 128-row halves of weights a CTA's tile holds.  PAIR: two CTAs of a
// cluster share a tile of twice the weight rows, each holding half its tokens.
template <int NMAX_, int HALVES, bool PAIR>
struct Cfg {
  static constexpr int NMAX = NMAX_;
  static constexpr int kAccs = NMAX <= 112 ? 2 : 1;  // accumulators (512 TMEM columns in all)
  static constexpr int BROWS = PAIR ? NMAX / 2 : NMAX;  // token rows in this CTA's memory
  static constexpr int B_BYTES = BROWS * BK;
  static constexpr int STAGE_BYTES = HALVES * W_BYTES + B_BYTES;
  static constexpr int SF_BYTES = (128 * HALVES + NMAX) * 4 * SG;  // a chunk of every row's scales
  // scales, barriers, tile prefix and segment starts, alignment
  static constexpr int kFixed = SBUFS * SF_BYTES + 10 * 1024;
  static constexpr int STAGES = (int)((kSmemLimit - kFixed) / STAGE_BYTES);
  static constexpr int SFB = (NMAX + 31) / 32;  // TMEM columns of the tokens' scales
  static constexpr int SFB_ST = SFB > 4 ? 8 : SFB > 2 ? 4 : SFB;  // ... as one store writes them
  static constexpr int SFA = 4 * HALVES;        // ... of the weights' scales, in front of them
  static constexpr int SF_COLS = SFA + (SFB_ST + 3) / 4 * 4;  // TMEM columns of a stage's scales
  static constexpr int ACC_COLS = HALVES * NMAX;
  static constexpr int kSf0 = kAccs * ACC_COLS;
  // Scales wait in TMEM in slots of TG stages, a ring of their own: as many
  // slots as the accumulators leave room for.
  static constexpr int TG = 512 - kSf0 >= 2 * 4 * SF_COLS ? 4 : 2;
  static constexpr int kFit = (512 - kSf0) / (TG * SF_COLS);
  static constexpr int SLOTS = kFit > 4 ? 4 : kFit;
  static_assert(SLOTS >= 2, "TMEM columns");
  static_assert(NMAX % 16 == 0 && NMAX <= 256, "N");
};

template <int STAGES, int SLOTS>
struct MxShared {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t sfull[SLOTS];   // a slot's scales are in TMEM
  uint64_t sempty[SLOTS];  // ... and its last MMAs have read them
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int prefix[kMaxExperts + 1];
  int start[kMaxExperts + 1];  // first row of every expert
  int scan_tmp[33];
};

struct MxArgs {
  const uint8_t* a;        // [a_rows, Kp] e4m3 codes
  const uint8_t* a_scale;  // [a_rows, Kp / 32]
  const uint8_t* w_scale;  // [E, N1, Kp / 32]
  const void* bias;        // [E, N1] or null
  const int32_t* seg_end;
  const int32_t* grows;    // row_to_route, or null (row m is row m of a)
  void* out;               // [M, Nout], or e4m3 codes [M, Np]
  uint8_t* out_scale;      // [M, Np / 32]
  int* status;
  int M, Nout, N1, Kp, E, a_rows, gdiv;
  int row_step, half_step;  // weight row of output f, half h: f * row_step + h * half_step
  int bias_t, out_t;        // moe_dtype of the bias and (unless MX) the output
  int even;                 // 16-bit output: Nout is even and out 4-byte aligned
  float limit, alpha, beta;
};

// N consecutive TMEM columns of this warp's lanes from registers
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
  if constexpr (N == 1)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r[0])
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1])
                 : "memory");
  else if constexpr (N == 4)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
  else
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}
// The MMAs of a stage (four K32 steps of each half; half 1's weights
// 16 KB on, its accumulator in d1) and the commit that frees the stage, issued
// by one elected lane of a CONVERGED warp.  All operands are warp-uniform, so
// they stay in uniform registers: the stage then takes max(313, 4 N) cycles,
// against 600 when a diverged lane issues the MMAs one by one and moves every
// operand over first.  Descriptors advance by 32 bytes (2) a step; a step's
// scale byte is selected in the instruction descriptor (bits 4 and 29).
template <int HALVES, bool PAIR>
__device__ __forceinline__ void mma_stage(uint32_t d0, uint32_t d1, uint64_t ad, uint64_t bd,
                                          uint32_t idesc, uint32_t sfa, uint32_t accumulate,
                                          uint32_t bar) {
#define MOE_MX_MMA(G, d, a, b, i, sa, p)                                                      \
  "@e tcgen05.mma.cta_group::" G ".kind::mxf8f6f4.block_scale.scale_vec::1X [" d "], " a ", " \
  b ", " i ", [" sa "], [sb], " p ";\n\t"
#define MOE_MX_STEP2(G, a0, a1, b, i, p) \
  MOE_MX_MMA(G, "%0", a0, b, i, "%5", p) MOE_MX_MMA(G, "%1", a1, b, i, "s1", p)
#define MOE_MX_STEP1(G, a0, a1, b, i, p) MOE_MX_MMA(G, "%0", a0, b, i, "%5", p)
#define MOE_MX_BODY(G, SB, STEP, COMMIT)                                                   \
  "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a0, a1, b0;\n\t.reg .b32 i0, s1, sb;\n\t"       \
  "elect.sync _|e, 0xffffffff;\n\t"                                                        \
  "setp.ne.b32 p, %6, 0;\n\t"                                                              \
  "setp.eq.b32 t, %6, %6;\n\t"                                                             \
  "add.u32 s1, %5, 4;\n\t"                                                                 \
  "add.u32 sb, %5, " SB ";\n\t"                                                            \
  "add.u64 a1, %2, 1024;\n\t"                                                              \
  STEP(G, "%2", "a1", "%3", "%4", "p")                                                     \
  "add.u64 a0, %2, 2;\n\tadd.u64 a1, %2, 1026;\n\tadd.u64 b0, %3, 2;\n\t"                  \
  "add.u32 i0, %4, 0x20000010;\n\t"                                                        \
  STEP(G, "a0", "a1", "b0", "i0", "t")                                                     \
  "add.u64 a0, %2, 4;\n\tadd.u64 a1, %2, 1028;\n\tadd.u64 b0, %3, 4;\n\t"                  \
  "add.u32 i0, %4, 0x40000020;\n\t"                                                        \
  STEP(G, "a0", "a1", "b0", "i0", "t")                                                     \
  "add.u64 a0, %2, 6;\n\tadd.u64 a1, %2, 1030;\n\tadd.u64 b0, %3, 6;\n\t"                  \
  "add.u32 i0, %4, 0x60000030;\n\t"                                                        \
  STEP(G, "a0", "a1", "b0", "i0", "t") "@e " COMMIT
#define MOE_MX_OPS "r"(d0), "r"(d1), "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(accumulate), "r"(bar)
  if constexpr (PAIR) {
    static_assert(HALVES == 2, "pair tiles hold both halves");
    asm volatile(MOE_MX_BODY("2", "8", MOE_MX_STEP2,
                             "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster."
                             "multicast::cluster.b64 [%7], %8;\n\t}")::MOE_MX_OPS,
                 "h"((uint16_t)3)
                 : "memory");
  } else if constexpr (HALVES == 2) {
    asm volatile(MOE_MX_BODY("1", "8", MOE_MX_STEP2,
                             "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster."
                             "b64 [%7];\n\t}")::MOE_MX_OPS
                 : "memory");
  } else {
    asm volatile(MOE_MX_BODY("1", "4", MOE_MX_STEP1,
                             "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster."
                             "b64 [%7];\n\t}")::MOE_MX_OPS
                 : "memory");
  }
#undef MOE_MX_OPS
#undef MOE_MX_BODY
#undef MOE_MX_STEP1
#undef MOE_MX_STEP2
#undef MOE_MX_MMA
}
static_assert((W_BYTES >> 4) == 1024, "half 1's descriptor offset");
// commit by one elected lane of a converged warp, to both CTAs' barriers of a pair
template <bool PAIR>
__device__ __forceinline__ void mx_commit_elect(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bar)
        : "memory");
}
// Wait for a stage's release, which a pair's leader commits to both CTAs: polled as a
// barrier of this CTA alone, then acquired at cluster scope.  Polling at that scope
// takes longer (1024 rows on each of 16 experts, 2048 x 1920 gate_up, 16-bit out: 148
// us, 128 so; 2048 x 7168: 325 and 310).
template <bool PAIR>
__device__ __forceinline__ bool wait_stage(uint64_t* b, uint32_t parity, volatile int* abort_flag,
                                           int* status) {
  return wait_fast(b, parity, abort_flag, status) &&
         (!PAIR || try_wait<kWaitShared>(su32(b), parity));
}
// a load into this CTA's shared memory that completes on a barrier of the
// pair's leader (shared::cluster address)
__device__ __forceinline__ void tma2_4d(void* dst, const CUtensorMap* m, uint32_t bar, int c0,
                                        int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// Instruction descriptor, kind::mxf8f6f4: A e2m1 (format 5 at bit 7), B e4m3
// (format 0 at bit 10), both K-major, N / 8 at bit 17, e8m0 scales (bit 23),
// M / 128 at bit 27 (256 across a pair); the scale byte of K step j at bits 4
// (B) and 29 (A).
template <bool PAIR>
__device__ __forceinline__ uint32_t idesc_mx(int N) {
  return (5u << 7) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((PAIR ? 2u : 1u) << 27);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok, uint64_t pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(ok ? 16 : 0), "l"(pol)
               : "memory");
}

struct MxTile {
  int e, ft, m0, nv, N;  // expert, output tile, first row, rows, MMA columns
};
// row of `a` for tile row r, or -1 (padding, or a map entry out of range)
__device__ __forceinline__ int source_row(const MxArgs& p, const MxTile& t, int r) {
  if (r >= t.nv) return -1;
  int m = t.m0 + r;
  if (p.grows) {
    m = p.grows[m];
    m = m < 0 ? -1 : m / p.gdiv;
  }
  return m < p.a_rows ? m : -1;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// named_sync that returns whether v is true in every thread
__device__ __forceinline__ bool named_and(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
// Rows of expert e: start[e] .. start[e + 1] (start is clamped to [0, M]); a
// segment end below the one before it makes the expert empty.
__device__ __forceinline__ int seg_rows(const int* start, int e) {
  return max(start[e + 1] - start[e], 0);
}
template <int NMAX>
__device__ __forceinline__ MxTile mx_decode(int t, const int* prefix, const int* start, int E) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {  // last e with prefix[e] <= t (skips empty experts)
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int s = start[lo], n = seg_rows(start, lo);
  const int ce = (n + NMAX - 1) / NMAX;  // chunks of equal size, rounded up to 16
  const int local = t - prefix[lo];
  MxTile r;
  r.e = lo;
  r.ft = local / ce;
  const int per = (((n + ce - 1) / ce) + 15) & ~15;
  const int first = min((local % ce) * per, n);
  r.m0 = s + first;
  r.nv = min(per, n - first);  // 0 for a chunk that rounding left empty
  r.N = max(16, (r.nv + 15) & ~15);
  return r;
}

// Exclusive prefix over the experts of their tiles (chunks of up to NMAX rows,
// each crossed with n_ftiles output tiles); prefix has E + 1 entries, scratch
// 33.  The whole block calls it; returns the total.
template <int NMAX>
__device__ int mx_tile_prefix(const int* start, int E, int n_ftiles, int* prefix, int* scratch) {
  const int per = (E + NUM_THREADS - 1) / NUM_THREADS;
  const int lo = threadIdx.x * per, hi = min(E, lo + per);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int mine = 0;
  for (int e = lo; e < hi; ++e) mine += (seg_rows(start, e) + NMAX - 1) / NMAX * n_ftiles;
  int v = mine;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) scratch[wid] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    int acc = 0;
    for (int w = 0; w < NUM_THREADS / 32; ++w) {
      const int x = scratch[w];
      scratch[w] = acc;
      acc += x;
    }
    scratch[32] = acc;
  }
  __syncthreads();
  int run = scratch[wid] + v - mine;
  for (int e = lo; e < hi; ++e) {
    prefix[e] = run;
    run += (seg_rows(start, e) + NMAX - 1) / NMAX * n_ftiles;
  }
  if (threadIdx.x == 0) prefix[E] = scratch[32];
  return scratch[32];  // the caller synchronises before prefix is read
}

// 16 consecutive fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <int ACT>
__device__ __forceinline__ float act_one(float x) {
  if constexpr (ACT == MOE_ACT_RELU) return relu_f(x);
  else if constexpr (ACT == MOE_ACT_GELU) return gelu_f(x);
  else if constexpr (ACT == MOE_ACT_SILU) return x * fast_sigmoid(x);
  else return x;
}

// The calling warp's 32 output columns f0 + lane for 16 tokens m0 .. (nval of
// them): rows of out_t, or MX e4m3 codes with one scale per token.  A lane holds
// one column of every token, memory wants a token's columns together: lanes
// trade columns (pairs for 16-bit values, fours for codes) until each holds a
// 32-bit word of a token, so 16 tokens take 8 or 4 store instructions, not 16.
template <bool MXOUT>
__device__ __forceinline__ void emit16(const float (&v)[16], const MxArgs& p, int m0, int nval,
                                       int f0, int lane) {
  const uint32_t all = 0xffffffffu;
  const int f = f0 + lane;
  if constexpr (MXOUT) {
    const int Np = mx::padded(p.Nout);
    uint32_t r[4] = {0, 0, 0, 0}, mine = 0;  // four tokens' codes a word; scale of token `lane`
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const uint32_t b0 = mx::scale_byte<false>(__reduce_max_sync(all, mx::abs_bits(v[i])));
      const uint32_t b1 = mx::scale_byte<false>(__reduce_max_sync(all, mx::abs_bits(v[i + 1])));
      const float s0 = mx::inv_scale(b0), s1 = mx::inv_scale(b1);
      r[i >> 2] |= mx::e4m3x2(mx::scaled(v[i], s0), mx::scaled(v[i + 1], s1)) << (8 * (i & 3));
      if (lane == i) mine = b0;
      if (lane == i + 1) mine = b1;
    }
    if (lane < nval) p.out_scale[(size_t)(m0 + lane) * (Np / 32) + (f0 >> 5)] = (uint8_t)mine;
    // 4 x 4 bytes between the lanes of each four: lane 4 q + j ends with columns
    // 4 q .. 4 q + 3 of token 4 m + j in word m
    const int j = lane & 3;
    uint8_t* o = static_cast<uint8_t*>(p.out) + (size_t)(m0 + j) * Np + f0 + (lane & ~3);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t w = r[m];
      const uint32_t x = __shfl_xor_sync(all, w, 1);
      // bytes (tokens) of my parity, from the even lane then the odd one
      w = (j & 1) ? __byte_perm(x, w, 0x7351) : __byte_perm(w, x, 0x6240);
      const uint32_t y = __shfl_xor_sync(all, w, 2);
      w = (j & 2) ? __byte_perm(y, w, 0x7632) : __byte_perm(w, y, 0x5410);
      if (4 * m + j < nval) *reinterpret_cast<uint32_t*>(o + (size_t)4 * m * Np) = w;
    }
  } else if (p.out_t == MOE_F32) {
    if (f < p.Nout) {
      float* o = static_cast<float*>(p.out) + (size_t)m0 * p.Nout + f;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < nval) o[(size_t)i * p.Nout] = v[i];
    }
  } else {
    const bool f16 = p.out_t == MOE_F16;
    uint16_t* o = static_cast<uint16_t*>(p.out) + (size_t)m0 * p.Nout;
    if (p.even) {  // words of two columns are aligned
      const int odd = lane & 1;
      o += (size_t)odd * p.Nout + (f - odd);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const uint32_t w = f16 ? pack_f16x2(v[i], v[i + 1]) : pack_bf16x2(v[i], v[i + 1]);
        const uint32_t x = __shfl_xor_sync(all, w, 1);
        const uint32_t u = odd ? __byte_perm(x, w, 0x7632) : __byte_perm(w, x, 0x5410);
        if (i + odd < nval && f - odd < p.Nout)
          *reinterpret_cast<uint32_t*>(o + (size_t)i * p.Nout) = u;
      }
    } else if (f < p.Nout) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < nval)
          o[(size_t)i * p.Nout + f] =
              (uint16_t)(f16 ? pack_f16x2(v[i], 0.0f) : pack_bf16x2(v[i], 0.0f));
    }
  }
}

template <int NMAX, int HALVES, bool PAIR, bool GATED, int ACT, bool MXOUT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_mx_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ MxArgs p) {
  static_assert(HALVES == 2 || !GATED, "gate and up rows");
  using C = Cfg<NMAX, HALVES, PAIR>;
  constexpr int STAGES = C::STAGES;
  const uint32_t rank = PAIR ? cluster_rank() : 0;  // 0: the leader, which issues the MMAs
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, units = PAIR ? gridDim.x >> 1 : gridDim.x;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sf = smem + (size_t)STAGES * C::STAGE_BYTES;
  auto* sh = reinterpret_cast<MxShared<STAGES, C::SLOTS>*>(sf + SBUFS * C::SF_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      // the producer's expect-tx, every loader thread, and the peer's rows; the
      // peer's own barrier counts its loaders
      mbar_init(&sh->full[s], kLoaders + (rank == 0 ? 1 + (PAIR ? 1 : 0) : 0));
      mbar_init(&sh->empty[s], 1);
    }
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&sh->sfull[s], PAIR ? 8 : 4);  // every scale warp
      mbar_init(&sh->sempty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sh->tfull[a], 1);
      mbar_init(&sh->tempty[a], (PAIR ? 2 : 1) * kEpiWarps);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w)) : "memory");
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       su32(&sh->tmem_base)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       su32(&sh->tmem_base)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  pdl_launch();
  constexpr int FT = GATED ? 128 : 128 * HALVES;  // output columns of a tile
  constexpr int FTU = PAIR ? 2 * FT : FT;  // ... and of a pair's
  const int n_ftiles = (p.Nout + FTU - 1) / FTU;
  const int nkb = p.Kp / BK;
  pdl_wait();
  // every expert's rows start where the one before ends
  for (int e = threadIdx.x; e <= p.E; e += NUM_THREADS)
    sh->start[e] = e == 0 ? 0 : min(max(p.seg_end[e - 1], 0), p.M);
  __syncthreads();
  const int total = mx_tile_prefix<NMAX>(sh->start, p.E, n_ftiles, sh->prefix, sh->scan_tmp);
  tc_fence_before();
  if constexpr (PAIR) cluster_sync(); else __syncthreads();  // barriers, TMEM, tile list
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  // tile t as this CTA sees it: its own output tile of the pair's two
  auto decode = [&](int t) {
    MxTile r = mx_decode<NMAX>(t, sh->prefix, sh->start, p.E);
    if constexpr (PAIR) r.ft = 2 * r.ft + (int)rank;
    return r;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------ TMA producer (weights)
      // It also passes on the release of the scale slots: a stage's completion
      // tells it, as it takes the stage again, that the slot whose last stage
      // that was is free.  (A commit of the MMA warp's own for the slots, next
      // to the one for the stage, stalls that warp until the MMAs are done.)
      int stage = 0, slot = 0;
      uint32_t phase = 0;
      uint32_t issued[STAGES];
      int owner[STAGES];  // slot that the stage's last MMAs free, or -1
#pragma unroll
      for (int s = 0; s < STAGES; ++s) {
        issued[s] = 0;
        owner[s] = -1;
      }
      bool ok = true;
      auto take = [&](int freed) {  // waits for the stage; freed: the slot it was to free
        if (!wait_stage<PAIR>(&sh->empty[stage], phase ^ 1u, abort_flag, p.status)) return false;
        if (freed >= 0) {
          tc_fence_after();
          tc_fence_before();
          mbar_arrive(&sh->sempty[freed]);
        }
        return true;
      };
      auto get = [&](int s) {
        int v = -1;
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
          if (i == s) v = owner[i];
        return v;
      };
      for (int tile = unit; tile < total && ok; tile += units) {
        const MxTile t = decode(tile);
        if (t.nv == 0) continue;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!(ok = take(get(stage)))) break;
          uint8_t* dst = smem + (size_t)stage * C::STAGE_BYTES;
          // rows past the operand read as zeros and count in full
          if constexpr (PAIR) {
            if (rank == 0) mbar_expect_tx(&sh->full[stage], 2 * HALVES * W_TX);
            tma2_4d(dst, &tm_w, map_to_rank(su32(&sh->full[stage]), 0), kb * BK, t.ft * FT, 0, t.e);
          } else {
            mbar_expect_tx(&sh->full[stage], HALVES * W_TX);
            tma_4d(dst, &tm_w, &sh->full[stage], kb * BK, t.ft * FT, 0, t.e);
          }
          const bool last = kb % C::TG == C::TG - 1 || kb == nkb - 1;
#pragma unroll
          for (int i = 0; i < STAGES; ++i)
            if (i == stage) {
              ++issued[i];
              owner[i] = last ? slot : -1;
            }
          if (last && ++slot == C::SLOTS) slot = 0;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      for (int i = 0; i < STAGES && ok; ++i) {  // the last stages' releases
        ok = take(get(stage));
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok && rank == 0) {  // let every copy already in flight land before the block exits
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
          if (issued[s]) drain_wait(&sh->full[s], (issued[s] - 1u) & 1u);
      }
    }
  } else if (PAIR && warp == 1 && rank != 0) {
    // ------------------------------------------------ the peer's rows of a stage landed
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = unit; tile < total && ok; tile += units) {
        if (decode(tile).nv == 0) continue;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!wait_fast(&sh->full[stage], phase, abort_flag, p.status)) { ok = false; break; }
          fence_proxy_async_smem();
          mbar_arrive_cluster(map_to_rank(su32(&sh->full[stage]), 0));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (whole warp)
    int stage = 0, acc = 0, slot = 0;
    uint32_t phase = 0, aphase = 0, sphase = 0;
    bool ok = true, any = false;
    const uint64_t ad0 = sw128_desc(su32(smem));
    // a pair's barriers take arrivals of both CTAs
    constexpr int kRows = PAIR ? kWaitShared : kWaitCta, kScales = PAIR ? kWaitTmem : kWaitCta;
    // warp reductions leave their result in a uniform register
    const uint32_t tm0 = __reduce_max_sync(0xffffffffu, tmem);
    for (int tile = unit; tile < total && ok; tile += units) {
      const MxTile t = decode(tile);
      if (t.nv == 0) continue;
      ok = __all_sync(0xffffffffu,
                      wait_pair_tmem<PAIR>(&sh->tempty[acc], aphase ^ 1u, abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tm0 + (uint32_t)(acc * C::ACC_COLS);
      const uint32_t idesc = idesc_mx<PAIR>((int)__reduce_max_sync(0xffffffffu, (uint32_t)t.N));
      for (int kb = 0; kb < nkb; ++kb) {
        // both barriers tried at once, the slow paths only when one is not there yet
        const bool first = kb % C::TG == 0;
        const bool f0 = try_wait<kRows>(su32(&sh->full[stage]), phase);
        const bool f1 = !first || try_wait<kScales>(su32(&sh->sfull[slot]), sphase);
        if (!__all_sync(0xffffffffu, f0 && f1)) {
          ok = wait_bar<kRows>(&sh->full[stage], phase, abort_flag, p.status);
          if (first) ok = wait_bar<kScales>(&sh->sfull[slot], sphase, abort_flag, p.status) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        // the loaders wrote through the generic proxy; tcgen05 reads through
        // the async proxy
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t ad = ad0 + (uint64_t)((stage * C::STAGE_BYTES) >> 4);
        mma_stage<HALVES, PAIR>(d, d + NMAX, ad, ad + (HALVES * W_BYTES >> 4), idesc,
                  tm0 + (uint32_t)(C::kSf0 + (slot * C::TG + kb % C::TG) * C::SF_COLS),
                  kb != 0 ? 1u : 0u, su32(&sh->empty[stage]));
        any = true;
        if (kb % C::TG == C::TG - 1 || kb == nkb - 1)
          if (++slot == C::SLOTS) { slot = 0; sphase ^= 1u; }
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      mx_commit_elect<PAIR>(su32(&sh->tfull[acc]));
      if (++acc == C::kAccs) { acc = 0; aphase ^= 1u; }
    }
    if (!ok && any) {  // every MMA issued so far done before TMEM is freed
      mx_commit_elect<PAIR>(su32(&sh->drain));
      drain_wait(&sh->drain, 0);
    }
  } else if (warp < kScaleWarp0) {
    // ------------------------------------------------ token loaders
    // Thread lt owns 16-byte chunk lt % 8 of rows lt / 8 + 8 i, so eight lanes
    // read one 128-byte row piece; chunk ch of row r lands at chunk
    // ch ^ (r % 8), the 128-byte swizzle.
    const int lt = threadIdx.x - kLoadWarp0 * 32;
    const int ch = lt & 7, r0 = lt >> 3;
    const uint32_t dst0 = (uint32_t)(HALVES * W_BYTES + r0 * 128 + ((ch ^ (r0 & 7)) << 4));
    constexpr int STEP = kLoaders / 8, RI = C::BROWS / STEP;
    static_assert(STEP % 8 == 0 && RI <= 32, "the swizzle and the masks of a thread's rows");
    // the token rows are read again by every output tile of their expert:
    // kept in L2 ahead of the weight stream
    uint64_t keep;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    const uint8_t* a = p.a + ch * 16;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = unit; tile < total && ok; tile += units) {
      const MxTile t = decode(tile);
      if (t.nv == 0) continue;
      // The rows' offsets in 128-byte blocks.  Rows of the MMA's padding are not
      // copied (their columns are never read); a row with a bad map entry is
      // zeroed.
      uint32_t at[RI], mine = 0, good = 0;
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const int b = r0 + STEP * i;  // row of this CTA's buffer
        const int r = PAIR ? b + (int)rank * (t.N / 2) : b, m = source_row(p, t, r);
        if (r < t.nv && (!PAIR || b < t.N / 2)) mine |= 1u << i;
        if (m >= 0) good |= 1u << i;
        at[i] = (uint32_t)max(m, 0) * (uint32_t)nkb;
      }
      for (int kb = 0; kb < nkb; ++kb) {
        if (!wait_stage<PAIR>(&sh->empty[stage], phase ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const uint32_t dst = su32(smem + (size_t)stage * C::STAGE_BYTES) + dst0;
#pragma unroll
        for (int i = 0; i < RI; ++i)
          if (mine & (1u << i))
            cp_async16(dst + i * STEP * 128, a + ((uint64_t)(at[i] + (uint32_t)kb) << 7),
                       (good & (1u << i)) != 0, keep);
        // arrives on the stage's full barrier once this thread's copies land
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         su32(&sh->full[stage]))
                     : "memory");
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // nothing in flight at exit
  } else if (warp < kEpiWarp0) {
    // ------------------------------------------------ scales
    // The first rows of a buffer are the halves' weight rows, the others the
    // tokens; one aligned 16-byte chunk each.  A row's scales start `skew` words
    // into its first chunk (its pitch need not be a multiple of 16 bytes), so a
    // group of SG stages' words lies in chunk g, or in chunks g and g + 1.
    // Reading back, lane l takes rows l, 32 + l, ...: the TMEM cells of its lane.
    const int st = threadIdx.x - kScaleWarp0 * 32, quad = warp & 3;
    constexpr int WR = 128 * HALVES, NA = C::SFA;  // weight rows and their TMEM columns
    constexpr int PER = HALVES + (NMAX + 127) / 128;  // rows a copying thread
    const int sp = p.Kp / 32;                    // scale bytes of a row
    const bool skewed = (sp & 15) != 0;
    const uint32_t sf_dst = su32(sf) + (uint32_t)(st * 16);
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + C::kSf0;
    const int ngr = (nkb + SG - 1) / SG, nch = ngr + (skewed ? 1 : 0);
    // weight row of tile row r (0 .. WR - 1) inside its expert, or -1 past the end
    auto weight_row = [&](int ft, int r) {
      const int f = GATED ? ft * 128 + (r & 127) : ft * FT + r;
      if (f >= p.Nout) return -1;
      return GATED ? f * p.row_step + (r >> 7) * p.half_step : f;
    };
    // Copies run SBUFS chunks ahead of the reads: chunk lc of tile ltile is
    // next, into buffer lbuf; src and left are its rows' next chunk and bytes.
    const uint8_t* src[PER];
    int left[PER];
    int ltile = unit, lc = 0, lbuf = 0, buf = 0;
    auto seek = [&]() {  // rows of the first tile at or after ltile that has any
      for (; ltile < total; ltile += units) {
        const MxTile t = decode(ltile);
        if (t.nv == 0) continue;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int row = i < HALVES ? weight_row(t.ft, st + 128 * i)
                                     : source_row(p, t, st + 128 * (i - HALVES));
          const size_t at = ((i < HALVES ? (size_t)t.e * p.N1 : 0) + max(row, 0)) * sp;
          src[i] = (i < HALVES ? p.w_scale : p.a_scale) + (at & ~size_t(15));
          left[i] = row >= 0 ? sp + (int)(at & 15) : 0;
        }
        return;
      }
    };
    auto copy_chunk = [&]() {
      if (ltile < total) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (i < HALVES || st + 128 * (i - HALVES) < NMAX) {
            // no byte past the row's own scales is read
            const int n = min(16, max(left[i], 0));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             sf_dst + lbuf * C::SF_BYTES + i * 2048),
                         "l"(n ? src[i] : p.w_scale), "r"(n)
                         : "memory");
            src[i] += 16;
            left[i] -= 16;
          }
        }
        if (++lbuf == SBUFS) lbuf = 0;
        if (++lc == nch) {
          lc = 0;
          ltile += units;
          seek();
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    seek();
    for (int i = 0; i < SBUFS; ++i) copy_chunk();
    int slot = 0;
    uint32_t sphase = 0;
    bool ok = true;
    for (int tile = unit; tile < total && ok; tile += units) {
      const MxTile t = decode(tile);
      if (t.nv == 0) continue;
      // where the rows of this lane's cells start in their chunks
      uint32_t skew[NA + C::SFB];
#pragma unroll
      for (int c = 0; c < NA + C::SFB; ++c) {
        const int r = c * 32 + lane;
        const int row = c < NA ? weight_row(t.ft, r) : source_row(p, t, r - WR);
        const size_t at = ((c < NA ? (size_t)t.e * p.N1 : 0) + max(row, 0)) * sp;
        skew[c] = skewed ? (uint32_t)(at & 15) >> 2 : 0u;
      }
      for (int gr = 0; gr < ngr && ok; ++gr) {
        // chunk g, and g + 1 when rows are skewed, landed
        asm volatile("cp.async.wait_group %0;" ::"n"(SBUFS - 2) : "memory");
        named_sync(kScaleBar, 128);
        const int buf1 = buf + 1 == SBUFS ? 0 : buf + 1;
        uint32_t w[SG][NA], b[SG][C::SFB_ST];
#pragma unroll
        for (int c = 0; c < NA + C::SFB_ST; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (c < NA + C::SFB && c * 32 + lane < WR + NMAX) {
            v = *reinterpret_cast<const uint4*>(sf + buf * C::SF_BYTES + (c * 32 + lane) * 16);
            if (skewed) {  // words skew .. skew + 3 of the two chunks
              const uint4 n = *reinterpret_cast<const uint4*>(sf + buf1 * C::SF_BYTES + (c * 32 + lane) * 16);
              const uint32_t k = skew[c < NA + C::SFB ? c : 0];
              const bool one = (k & 1) != 0, two = (k & 2) != 0;
              const uint32_t x0 = one ? v.y : v.x, x1 = one ? v.z : v.y, x2 = one ? v.w : v.z,
                             x3 = one ? n.x : v.w, x4 = one ? n.y : n.x, x5 = one ? n.z : n.y;
              v = make_uint4(two ? x2 : x0, two ? x3 : x1, two ? x4 : x2, two ? x5 : x3);
            }
          }
          if (c < NA) {
            w[0][c] = v.x; w[1][c] = v.y; w[2][c] = v.z; w[3][c] = v.w;
          } else {
            b[0][c - NA] = v.x; b[1][c - NA] = v.y; b[2][c - NA] = v.z; b[3][c - NA] = v.w;
          }
        }
        named_sync(kScaleBar, 128);  // read by all four warps: chunk g is free
        copy_chunk();
        buf = buf1;
        if (skewed && gr == ngr - 1) {  // and so is the tile's last chunk
          copy_chunk();
          if (++buf == SBUFS) buf = 0;
        }
#pragma unroll
        for (int j0 = 0; j0 < SG; j0 += C::TG) {
          if (gr * SG + j0 < nkb && ok) {
            // the slot's TMEM columns are free once its last MMAs completed
            ok = wait_fast(&sh->sempty[slot], sphase ^ 1u, abort_flag, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              tc_fence_after();
              const uint32_t d = taddr + (uint32_t)(slot * C::TG * C::SF_COLS);
#pragma unroll
              for (int j = 0; j < C::TG; ++j) {  // stages past the last: unread
                tmem_st<NA>(d + j * C::SF_COLS, w[j0 + j]);
                tmem_st<C::SFB_ST>(d + j * C::SF_COLS + NA, b[j0 + j]);
              }
              asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if constexpr (PAIR)
                  mbar_arrive_cluster_tmem(map_to_rank(su32(&sh->sfull[slot]), 0));
                else
                  mbar_arrive(&sh->sfull[slot]);
              }
              if (++slot == C::SLOTS) { slot = 0; sphase ^= 1u; }
            }
          }
        }
        // the four warps stop together: they share the barrier
        ok = named_and(kScaleBar, 128, ok);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------ epilogue
    const int quad = warp & 3;  // TMEM lanes 32 * quad ..
    const int c0 = (warp - kEpiWarp0) >> 2;  // 16-token groups c0, c0 + 2, ..
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    int acc = 0;
    uint32_t aphase = 0;
    for (int tile = unit; tile < total; tile += units) {
      const MxTile t = decode(tile);
      if (t.nv == 0) continue;
      // the lane's biases, loaded before the accumulator is ready
      float b[2] = {0.0f, 0.0f};
      const int f0 = t.ft * FT + quad * 32, f = f0 + lane;
      if (p.bias) {
        const size_t be = (size_t)t.e * p.N1;
        auto bias_at = [&](int i) {
          if (p.bias_t == MOE_F32) return static_cast<const float*>(p.bias)[be + i];
          const uint16_t u = static_cast<const uint16_t*>(p.bias)[be + i];
          return p.bias_t == MOE_F16 ? __half2float(__ushort_as_half(u)) : bf16_lo(u);
        };
        if constexpr (GATED) {
          if (f < p.Nout) {
            b[0] = bias_at(f * p.row_step);
            b[1] = bias_at(f * p.row_step + p.half_step);
          }
        } else {
          if (f < p.Nout) b[0] = bias_at(f);
          if (HALVES == 2 && f + 128 < p.Nout) b[1] = bias_at(f + 128);
        }
      }
      if (!wait_pair_tmem<PAIR>(&sh->tfull[acc], aphase, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t base = lanes + (uint32_t)(acc * C::ACC_COLS);
#pragma unroll 1
      for (int c = 16 * c0; c < t.nv; c += 16 * (kEpiWarps / 4)) {
        uint32_t r[HALVES][16];
        tmem_ld16(base + c, r[0]);
        if constexpr (HALVES == 2) tmem_ld16(base + NMAX + c, r[HALVES - 1]);
        tmem_wait_ld();
        const int nval = min(16, t.nv - c);
        float v[16];
        if constexpr (GATED) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = gated<ACT>(__uint_as_float(r[0][i]) + b[0],
                              __uint_as_float(r[HALVES - 1][i]) + b[1],
                              p.limit, p.alpha, p.beta);
          // a pair's second output tile may lie past the padded output
          if (f0 < mx::padded(p.Nout)) emit16<MXOUT>(v, p, t.m0 + c, nval, f0, lane);
        } else {
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = act_one<ACT>(__uint_as_float(r[h][i]) + b[h]);
            // the second half may lie past the padded output
            if (f0 + h * 128 < mx::padded(p.Nout))
              emit16<MXOUT>(v, p, t.m0 + c, nval, f0 + h * 128, lane);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_cluster_tmem(map_to_rank(su32(&sh->tempty[acc]), 0));
        else
          mbar_arrive(&sh->tempty[acc]);
      }
      if (++acc == C::kAccs) { acc = 0; aphase ^= 1u; }
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // neither CTA frees TMEM or exits while its peer works
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                   : "memory");
  }
}

// at most this many chunks of n tokens
long long chunks_bound(const MxArgs& p, int n) { return (long long)p.M / n + std::min(p.M, p.E); }

template <int NMAX, int HALVES, bool PAIR, bool GATED, int ACT, bool MXOUT>
cudaError_t go(const void* w, const MxArgs& p, cudaStream_t s) {
  using C = Cfg<NMAX, HALVES, PAIR>;
  constexpr size_t smem = (size_t)C::STAGES * C::STAGE_BYTES + SBUFS * C::SF_BYTES +
                          sizeof(MxShared<C::STAGES, C::SLOTS>) + 1024;
  static_assert(smem <= kSmemLimit, "shared memory");
  // weights [E][N1][Kp / 2 bytes] as [E][halves][Nout][K]; a box is a stage's rows
  CUtensorMap tm;
  const cuuint64_t row = (cuuint64_t)p.Kp / 2;
  const cuuint64_t dims[4] = {(cuuint64_t)p.Kp, (cuuint64_t)p.Nout, GATED ? 2u : 1u,
                              (cuuint64_t)p.E};
  const cuuint64_t str[3] = {row * p.row_step, GATED ? row * p.half_step : row * p.Nout,
                             row * p.N1};
  const cuuint32_t box[4] = {BK, GATED ? 128u : 128u * HALVES, GATED ? 2u : 1u, 1};
  if (!tmap::encode_u4_expanded(&tm, w, 4, dims, str, box)) return cudaErrorInvalidValue;
  auto kern = gemm_mx_kernel<NMAX, HALVES, PAIR, GATED, ACT, MXOUT>;
  cudaError_t e = set_smem_limit((const void*)kern, (int)smem);
  if (e != cudaSuccess) return e;
  constexpr int CTAS = PAIR ? 2 : 1, FT = CTAS * (GATED ? 128 : 128 * HALVES);
  const long long tiles = chunks_bound(p, NMAX) * ((p.Nout + FT - 1) / FT);
  const int units = (int)std::max<long long>(1, std::min<long long>(tiles, num_sms() / CTAS));
  if constexpr (PAIR) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * units);
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = smem;
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
    e = cudaLaunchKernelEx(&cfg, kern, tm, p);
  } else {
    e = launch_pdl(kern, dim3(units), dim3(NUM_THREADS), smem, s, tm, p);
  }
  count_launch();
  return e;
}

// Tiles: see launch_gemm_mx.
template <bool GATED, int ACT, bool MXOUT>
cudaError_t go_size(const void* w, const MxArgs& p, cudaStream_t s) {
  const int hit = std::min(p.M, p.E);
  const long long avg = ((long long)p.M + hit - 1) / hit;
  if (avg <= 8) {
    if constexpr (!GATED)
      if (chunks_bound(p, 16) * ((p.Nout + 255) / 256) < num_sms())
        return go<16, 1, false, GATED, ACT, MXOUT>(w, p, s);
    return go<16, 2, false, GATED, ACT, MXOUT>(w, p, s);
  }
  if (avg <= 48) return go<64, 2, false, GATED, ACT, MXOUT>(w, p, s);
  if (avg <= 160 || p.Kp / BK <= (MXOUT ? 28 : 14))
    return go<96, 2, true, GATED, ACT, MXOUT>(w, p, s);
  return go<224, 2, true, GATED, ACT, MXOUT>(w, p, s);
}
template <bool GATED, int ACT>
cudaError_t go_out(const void* w, const MxArgs& p, cudaStream_t s) {
  return p.out_scale ? go_size<GATED, ACT, true>(w, p, s) : go_size<GATED, ACT, false>(w, p, s);
}

}  // namespace

cudaError_t launch_gemm_mx(const void* a, const void* a_scale, int a_rows, const int32_t* gather_rows,
                           int gather_div, const void* w, const void* w_scale, const void* bias,
                           const int32_t* seg_end, int M, int Nout, int K, int E,
                           const moe_act_params* act, moe_dtype bias_dt, moe_dtype out_dt, void* out,
                           void* out_scale, int* status, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  const bool gate = act && act_is_gated(act->kind);
  const bool inter = gate && act->kind == MOE_ACT_SWIGLU && act->swiglu_fusion == 1;
  MxArgs p{};
  p.a = static_cast<const uint8_t*>(a);
  p.a_scale = static_cast<const uint8_t*>(a_scale);
  p.w_scale = static_cast<const uint8_t*>(w_scale);
  p.bias = bias;
  p.seg_end = seg_end;
  p.grows = gather_rows;
  p.gdiv = gather_div;
  p.out = out;
  p.out_scale = static_cast<uint8_t*>(out_scale);
  p.status = status;
  p.M = M;
  p.Nout = Nout;
  p.N1 = gate ? 2 * Nout : Nout;
  p.Kp = mx::padded(K);
  p.E = E;
  p.a_rows = a_rows;
  p.row_step = inter ? 2 : 1;
  p.half_step = gate ? (inter ? 1 : Nout) : 0;
  if (act) {
    p.limit = act->limit;
    p.alpha = act->alpha;
    p.beta = act->beta;
  }
  p.bias_t = bias_dt;
  p.out_t = out_dt;
  p.even = Nout % 2 == 0 && (reinterpret_cast<uintptr_t>(out) & 3) == 0;
  // Token columns of a tile, by the rows an expert that has any gets on
  // average (the host does not know the counts; us, single launches, L2 flushed):
  //   up to 8     16 columns, six stages in flight: decode, bound by the weights (one
  //               row on each of 128 experts, 2048 x 7168 gate_up: 312, 314 with 64
  //               columns).  Uneven counts soon need two chunks of 16 (24 rows on each
  //               of 32 experts, 2880 x 2880 gate_up: 91, 68 with 64).  A plain product
  //               whose tiles would not reach every SM takes 128 weight rows a tile
  //               instead of 256.
  //   up to 48    64 columns, five stages (2661 ragged rows on 128 experts, 768 x 2048:
  //               56, 58 with pairs of 96, 64 with 16).  Above, uneven counts start to
  //               need two chunks (8192 ragged rows on 128 experts, 2880 x 2880 down:
  //               152, 142 with pairs of 96), although even ones of up to 64 do not
  //               (64 rows on each of 64 experts: 74, 79 with pairs)
  //   up to 160   96 columns on a pair, two accumulators (the 8192 rows: 142; 146 with
  //               96 on one CTA, 162 with 224 on a pair)
  //   above       224 columns on a pair, one accumulator: the fewest bytes per
  //               product (65536 ragged rows, 2048 x 7168 gate_up: 1156, 1494 with 96,
  //               1293 with 208 on one CTA, whose token copies and shared-memory reads
  //               double), unless the product is so short that the epilogue, which
  //               one accumulator does not hide, costs more than that saves: up to 28
  //               stages of K with MX out (1024 rows on each of 16 experts, 2048 outputs,
  //               gated: 234 and 224 with 96 at 28 stages, 244 and 242 at 29, 357 and 394
  //               at 56; 512 rows, 768 outputs: 105 and 103 at 28, 109 and 111 at 29), up
  //               to 14 with 16-bit out, whose epilogue is half as long.  There the
  //               lengths at which the two cross lie apart: rows that just fill chunks
  //               of 96 stay ahead with 96 (256 an expert, 768 outputs: 70 and 64 at 14
  //               stages, 181 and 177 at 56), others are ahead with 224 from 6 stages on
  //               (1024 an expert, 2048 outputs: 87 and 89 at 6, 124 and 132 at 14).
  switch (act ? act->kind : MOE_ACT_IDENTITY) {
    case MOE_ACT_SILU_AND_MUL: return go_out<true, MOE_ACT_SILU_AND_MUL>(w, p, s);
    case MOE_ACT_SWIGLU: return go_out<true, MOE_ACT_SWIGLU>(w, p, s);
    case MOE_ACT_GELU_AND_MUL: return go_out<true, MOE_ACT_GELU_AND_MUL>(w, p, s);
    case MOE_ACT_RELU: return go_out<false, MOE_ACT_RELU>(w, p, s);
    case MOE_ACT_GELU: return go_out<false, MOE_ACT_GELU>(w, p, s);
    case MOE_ACT_SILU: return go_out<false, MOE_ACT_SILU>(w, p, s);
    default: return go_out<false, MOE_ACT_IDENTITY>(w, p, s);
  }
}

}  // namespace moe
