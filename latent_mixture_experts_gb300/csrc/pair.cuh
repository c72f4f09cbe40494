// Inline-PTX wrappers for clusters: barriers and shared memory of other CTAs,
// and the tensor memory of two CTAs that work on one tile (cta_group::2).
#pragma once
#include "ptx.cuh"

namespace lmoe {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Barrier of all threads of the cluster; orders their memory accesses.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Barrier `id` of the CTA over `threads` threads: arrive and go on, or wait.
__device__ __forceinline__ void named_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Address of CTA `rank`'s copy of a shared variable.
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// 16 bytes to another CTA's shared memory.
__device__ __forceinline__ void st_cluster4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}
// Partial sums that a cluster joins are whole only if no wait of any of its
// CTAs ran out: a thread whose wait did sets `lost`, a flag in the shared memory
// of each CTA, in all `ctas` of them, between the cluster's start and its last
// barrier; behind that barrier every CTA reads its own.
__device__ __forceinline__ void cluster_lost(int* lost, int ctas) {
  for (int r = 0; r < ctas; ++r)
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(map_rank(lost, r)), "r"(1) : "memory");
}
// Without release: for what the arriving thread has waited for itself (loads
// from tensor memory).  A release at cluster scope waits until the thread's
// global stores have arrived: 256 tokens' weight gradients at 7168 x 2048 took
// 50.6 us with it, 42.5 us without.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits of the pair acquire at cluster scope: the arrivals may be the other CTA's.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, int* err, int code) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 255u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicExch(err, code);
      return false;
    }
  }
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Descriptor of an MN-major operand tile written by TMA with 128-byte
// swizzle: blocks of 64 consecutive M (or N) values x K rows of 128 bytes;
// `mn_stride` bytes between 64-value blocks, 8 K rows (1024 bytes) per
// swizzle atom.  A K step of 16 advances the start address by 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr, uint32_t mn_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(mn_stride >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// Instruction descriptor bits for operands stored M (N) contiguous.
constexpr uint32_t kIdescAMajorMn = 1u << 15;
constexpr uint32_t kIdescBMajorMn = 1u << 16;

}  // namespace lmoe
