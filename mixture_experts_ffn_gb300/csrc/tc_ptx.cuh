// Inline-PTX wrappers for the tcgen05 / TMA / mbarrier instructions used by the
// grouped GEMM kernels (sm_100 family, built for sm_103a), plus the bounded
// waits every kernel here uses.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {
namespace tc {

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per wait

__device__ __forceinline__ uint32_t su32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(addr), "r"(parity)
      : "memory");
  return ok != 0;
}

// ---------------------------------------------------------------- pairs of CTAs
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(saddr), "r"(rank));
  return d;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// The CTAs of a pair synchronise at cluster scope, in two ways.
//  TMEM (a drained accumulator, stored scales): tcgen05 fences around relaxed
//    operations on the barrier, before the arrival and after the wait.
//  Shared memory (the peer's token rows, a stage that MMAs have read): release and
//    acquire fences restricted to shared memory around them.  An unrestricted
//    release at this scope also waits for the SM's copies from global memory, a
//    microsecond a stage (gemm_mx.cu, 8192 ragged rows, 2880 x 2880: 138 us, 322
//    with it).
//
// arrivals on a barrier of either CTA of the pair (shared::cluster address): after
// tc_fence_before, and after this thread saw shared memory written
__device__ __forceinline__ void mbar_arrive_cluster_tmem(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar_cluster) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  mbar_arrive_cluster_tmem(bar_cluster);
}
template <bool ACQUIRE = true>
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  if constexpr (ACQUIRE)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "@p fence.acquire.sync_restrict::shared::cluster.cluster;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
  return ok != 0;
}
// How a wait orders what comes after it: after this CTA's accesses; after the TMEM
// (by the caller's tc_fence_after) or the shared memory of both CTAs of a pair.
enum WaitKind { kWaitCta, kWaitTmem, kWaitShared };
template <int W>
__device__ __forceinline__ bool try_wait(uint32_t addr, uint32_t parity) {
  if constexpr (W == kWaitCta) return mbar_try_wait(addr, parity);
  else return mbar_try_wait_cluster<W == kWaitShared>(addr, parity);
}
// Bounded wait for the phase of parity `parity`; false on abort or timeout.
template <int W = kWaitCta>
static __device__ __noinline__ bool wait_bar(uint64_t* b, uint32_t parity, volatile int* abort_flag,
                                      int* status) {
  const uint32_t addr = su32(b);
  if (try_wait<W>(addr, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_wait<W>(addr, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > kTimeoutNs) {
      *abort_flag = 1;
      latch_error(status, kDevTimeout);
      return false;
    }
  }
}
// Fast path inline (no call, no register save/restore when the phase is
// already complete); the bounded spin stays out of line.
template <int W = kWaitCta>
__device__ __forceinline__ bool wait_fast(uint64_t* b, uint32_t parity, volatile int* abort_flag,
                                          int* status) {
  if (try_wait<W>(su32(b), parity)) return true;
  return wait_bar<W>(b, parity, abort_flag, status);
}
// Waits for a barrier that the other CTA of a pair arrives on too, or whose commit
// the other CTA issued, and that hands over shared memory, or TMEM alone.
template <bool PAIR = true>
__device__ __forceinline__ bool wait_pair(uint64_t* b, uint32_t parity, volatile int* abort_flag,
                                          int* status) {
  return wait_fast<PAIR ? kWaitShared : kWaitCta>(b, parity, abort_flag, status);
}
template <bool PAIR = true>
__device__ __forceinline__ bool wait_pair_tmem(uint64_t* b, uint32_t parity,
                                               volatile int* abort_flag, int* status) {
  return wait_fast<PAIR ? kWaitTmem : kWaitCta>(b, parity, abort_flag, status);
}

// Bounded wait used while draining after an abort (ignores the abort flag).
static __device__ __noinline__ void drain_wait(uint64_t* b, uint32_t parity) {
  const uint32_t addr = su32(b);
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(addr, parity)) {
    if (global_ns() - t0 > kTimeoutNs) return;
  }
}

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                       int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(su32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                       int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(su32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                       int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(su32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// TMA loads into this CTA's shared memory that complete on the leader's
// barrier (shared::cluster address); coordinates innermost first.
__device__ __forceinline__ void tma2_2d(void* dst, const CUtensorMap* m, uint32_t bar, int c0,
                                        int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma2_3d(void* dst, const CUtensorMap* m, uint32_t bar, int c0,
                                        int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(su32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void umma2_commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(su32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void umma2_commit_self(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          su32(bar))
      : "memory");
}

// v to the peer's shared memory at addr_cluster, completing on the peer's
// barrier bar_cluster (4 bytes of transaction, and the one arrival the phase
// expects): no fence, the barrier's transaction count orders the data.
__device__ __forceinline__ void publish_remote_u32(uint32_t addr_cluster, uint32_t bar_cluster,
                                                   int v) {
  asm volatile(
      "mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], 4;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%1], %2, [%0];" ::"r"(
          bar_cluster),
      "r"(addr_cluster), "r"(v)
      : "memory");
}

// Four words likewise, 16 bytes of transaction; addr_cluster may be this CTA's own.
__device__ __forceinline__ void publish_remote_v4(uint32_t addr_cluster, uint32_t bar_cluster,
                                                  uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile(
      "mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], 16;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%1], {%2, %3, %4, %5}, [%0];" ::
          "r"(bar_cluster),
      "r"(addr_cluster), "r"(a), "r"(b), "r"(c), "r"(d)
      : "memory");
}

// TMA store of one box from shared memory (bulk async-group completion).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(su32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Wait until at most N committed bulk groups of this thread still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// Wait until every committed bulk group of this thread has completed.
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// Order this thread's generic-proxy shared-memory writes before later
// async-proxy (TMA) reads of them.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory matrix descriptor: K-major operand, 128-byte swizzle, rows of
// 128 bytes, 8-row core groups 1024 bytes apart (stride byte offset).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);  // start address
  d |= (uint64_t)1 << 16;                    // leading byte offset (unused for swizzled K-major)
  d |= (uint64_t)(1024 >> 4) << 32;          // stride byte offset
  d |= (uint64_t)1 << 46;                    // descriptor version
  d |= (uint64_t)2 << 61;                    // 128-byte swizzle
  return d;
}

// Shared-memory matrix descriptor: MN-major operand, 128-byte swizzle.  A box of
// 64 elements (128 bytes) along M or N by `rows` terms of the contraction: groups of
// 8 terms 1024 bytes apart (stride byte offset), the next 64 elements a box further
// (leading byte offset).  A K16 step advances by 16 rows of 128 bytes.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t box_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);  // start address
  d |= (uint64_t)(box_bytes >> 4) << 16;     // leading byte offset
  d |= (uint64_t)(1024 >> 4) << 32;          // stride byte offset
  d |= (uint64_t)1 << 46;                    // descriptor version
  d |= (uint64_t)2 << 61;                    // 128-byte swizzle
  return d;
}
constexpr uint32_t kMnStep = (16 * 128) >> 4;  // descriptor units of a K16 step

#define MOE_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), \
                  "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
// 32 consecutive fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : MOE_R8(0), MOE_R8(8), MOE_R8(16), MOE_R8(24)
      : "r"(taddr));
}
#undef MOE_R8
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// store 32 bf16 (F16: float16) values (64 bytes) of one row; vector path when
// all columns are valid
template <bool F16 = false>
__device__ __forceinline__ void store_row32(__nv_bfloat16* dst, const float (&v)[32], int n_valid) {
  if (n_valid >= 32) {
    uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 u;
      u.x = pack2<F16>(v[8 * q + 0], v[8 * q + 1]);
      u.y = pack2<F16>(v[8 * q + 2], v[8 * q + 3]);
      u.z = pack2<F16>(v[8 * q + 4], v[8 * q + 5]);
      u.w = pack2<F16>(v[8 * q + 6], v[8 * q + 7]);
      d4[q] = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n_valid) {
        if constexpr (F16)
          reinterpret_cast<__half*>(dst)[i] = __float2half_rn(v[i]);
        else
          dst[i] = __float2bfloat16_rn(v[i]);
      }
  }
}

// Instruction descriptor, kind::f16: D f32, A/B bf16, both K-major, M x N.
constexpr uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// The same with A and B float16 (format code 0 in both fields).
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Instruction descriptor, kind::f16 with f32 accumulation, both operands
// K-major: bf16 (or float16 when f16) A and B, M x N; a_mn / b_mn: that operand
// MN-major instead.
__device__ __forceinline__ uint32_t idesc_sw(int M, int N, int f16, bool a_mn = false,
                                             bool b_mn = false) {
  const uint32_t fmt = f16 ? 0u : ((1u << 7) | (1u << 10));
  return (1u << 4) | fmt | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// One 16-bit operand-dtype element (bias) as float.
template <bool F16>
__device__ __forceinline__ float ld16(const __nv_bfloat16* p) {
  if constexpr (F16)
    return __half2float(*reinterpret_cast<const __half*>(p));
  else
    return __bfloat162float(*p);
}

}  // namespace tc
}  // namespace moe
