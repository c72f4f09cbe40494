// Single-thread instructions (TMA, tcgen05.mma, commits) issued from a whole
// warp in step: the warp runs the loop and its waits together, and each
// instruction elects one lane itself.  Their operands then stay in uniform
// registers; issued under `if (lane == 0)` every one of them is first moved
// there, which took longer than the products it started (a 256 x 256 x 16
// pair MMA 162 clocks instead of 133, a TMA load about 100 ns).
#pragma once
#include "pair.cuh"

namespace lmoe {

// Bounded wait of a warp in step (acquires at cluster scope); false for all
// lanes once the limit passes on any.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait_cluster(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait_cluster(bar, parity))) return true;
    if ((it & 255u) == 0 && __any_sync(0xFFFFFFFFu, globaltimer_ns() - t0 > kWaitLimitNs)) {
      if (lane_id() == 0) atomicExch(err, 1);
      return false;
    }
  }
}

#define LMOE_ELECT "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q "
__device__ __forceinline__ void w_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile(LMOE_ELECT "mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
// Tensor tiles counted on a barrier of this CTA.
__device__ __forceinline__ void w_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1) {
  asm volatile(LMOE_ELECT
               "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
               "%4}], [%2];\n\t}" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void w_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(LMOE_ELECT
               "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
               "%4, %5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
// Counted on a barrier of either CTA of the pair (`bar`: a shared::cluster address).
__device__ __forceinline__ void w_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
  asm volatile(LMOE_ELECT
               "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
               "[%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void w_mma_bf16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The pair's MMA, issued by the even CTA: D rows 0..127 (of 256) in its own
// tensor memory, 128..255 in the odd CTA's; A rows and B rows (N) are split
// the same way over the two shared memories.
__device__ __forceinline__ void w_mma_bf16_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void w_mma_mx_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
          "r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void w_mma_mx(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
          "r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void w_copy_atom(uint32_t taddr, uint64_t sdesc) {
  asm volatile(LMOE_ELECT "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc) : "memory");
}
// Bulk copy (16-byte multiples) counted on a barrier of this CTA.
__device__ __forceinline__ void w_bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(LMOE_ELECT
               "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// A 512-byte scale atom of each CTA's shared memory to its own tensor memory.
__device__ __forceinline__ void w_copy_atom_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile(LMOE_ELECT "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc) : "memory");
}
// Arrive once the MMAs that the electing lane issued so far are done: on a
// barrier of this CTA, or on the same barrier of both CTAs of the pair (`even`:
// the cluster rank of its even CTA).  The lane that elect.sync names is the same for the same member mask.
__device__ __forceinline__ void w_commit(uint64_t* bar) {
  asm volatile(LMOE_ELECT "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                   smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void w_commit_pair(uint64_t* bar, uint32_t even = 0) {
  asm volatile(LMOE_ELECT
               "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
               "%1;\n\t}" ::"r"(smem_u32(bar)),
               "h"(static_cast<uint16_t>(3u << even))
               : "memory");
}
#undef LMOE_ELECT

}  // namespace lmoe
