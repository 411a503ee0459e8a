// What the LM head's training products use of the Blackwell asynchronous
// machinery beyond the sampling kernels' layer (fs_sm100.cuh): operands stored
// along their M or N axis, stores by TMA, narrow TMEM loads, and issue by an
// elected lane of a whole warp.
//
// Descriptor layouts follow the PTX ISA for tcgen05 ("Shared memory
// descriptor", "Instruction descriptor" tables).
#pragma once

#include "fs_sm100.cuh"

namespace fs {
namespace sm100 {

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Bring a box into L2 (no shared memory, no barrier); issued by the lanes that
// reach it.
__device__ __forceinline__ void tma_prefetch_2d(const void* tmap, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y)
               : "memory");
}

// 2-D tiled store of a box from shared memory; out-of-range rows and columns
// of the box are left out.  The writes of ordinary stores to the box are made
// visible to it by fence_async_shared() first; the group that it is committed
// to is waited for before the box is written again (read) or the block ends.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma_store_2d(const void* tmap, const void* smem_src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_u32(smem_src)), "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 TMEM lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
}

// Shared-memory matrix descriptor of a bf16 operand stored along its M or N axis
// (MN-major) with the 128-byte swizzle: boxes of 64 MN elements (128 bytes) by 64 k rows, 8192 bytes each, one after another
// along MN.  Leading byte offset: from one 64-element block to the next;
// stride byte offset: from 8 k rows to the next 8.  Stepping K by 16 rows
// advances the start address by 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);          // start address
  d |= static_cast<uint64_t>(8192u >> 4) << 16;                    // leading byte offset
  d |= static_cast<uint64_t>(1024u >> 4) << 32;                    // stride byte offset
  d |= static_cast<uint64_t>(1u) << 46;                            // descriptor version (sm_100)
  d |= static_cast<uint64_t>(2u) << 61;                            // 128-byte swizzle
  return d;
}

// ---- issue by one elected lane of a warp that runs the loop as a whole: the
// loop's values then stay warp-uniform.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}

// mbar_wait by a whole warp; every lane gets the same answer.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 0;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((it & 63) == 63) {
      if (__any_sync(0xffffffffu, *abort != 0)) return false;
      if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitTimeoutNs)) {
        atomicExch(err, 1);
        *abort = 1;
        return false;
      }
    }
  }
}

__device__ __forceinline__ void mma_bf16_pair_if(uint32_t elected, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void mma_commit_pair_multicast_if(uint32_t elected, uint32_t bar, uint16_t cta_mask) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
          "r"(bar),
      "h"(cta_mask), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx_if(uint32_t elected, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void tma_load_2d_pair_if(uint32_t elected, uint32_t smem_dst, const void* tmap,
                                                    uint32_t bar_cluster_addr, int32_t x, int32_t y, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;\n\t}" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster_addr), "r"(x), "r"(y), "l"(policy), "r"(elected)
      : "memory");
}

// Bits of the instruction descriptor that mark A or B as MN-major.
constexpr uint32_t kIdescMnMajorA = 1u << 15;
constexpr uint32_t kIdescMnMajorB = 1u << 16;

}  // namespace sm100
}  // namespace fs
