// cluster.cuh — device helpers for thread-block clusters: addresses and barrier arrivals in
// another CTA's shared memory, waits that acquire at cluster scope (bounded like mbar_wait), and the
// cluster-wide barrier.
#pragma once

#include "common.cuh"

namespace hs {

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_smem(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

// Arrives on a barrier of another CTA (address from remote_smem); releases at cluster scope.
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The same without releasing anything: for barriers that pass on no generic-proxy writes of this thread (what
// they order are tensor-memory accesses, complete by then, and asynchronous copies that count on barriers). A
// releasing arrival waits for the thread's earlier memory operations, about a thousand cycles.
__device__ __forceinline__ void remote_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Orders this thread's generic-proxy accesses of every state space with the async proxy (here: shared
// memory of another CTA that its tensor core reads).
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait that sees what another CTA of the cluster wrote before its arrival.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, int32_t* err) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 63) == 63 && globaltimer() - t0 > kWaitLimitNs) {
      flag_error(err, HS_FLAG_TIMEOUT);
      return false;
    }
  }
}

// Every thread of every CTA of the cluster.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Bulk copy from this CTA's shared memory to another's (addresses from remote_smem; 16-byte aligned, size
// a multiple of 16), its bytes counted on a barrier there.
__device__ __forceinline__ void bulk_s2remote(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// mbarrier.arrive with its default semantics (release at CTA scope) on another CTA's barrier: for handing on what
// a barrier of this CTA has just shown complete (here: operands in its own shared memory, fenced for the async proxy by those who
// wrote them). Released and acquired at cluster scope instead, 64 requests x 4 tokens take 1.98 ms, not 1.14, a chunk of 2,048 tokens
// 7.5, not 6.4.
__device__ __forceinline__ void remote_arrive_cta(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------- two-SM tensor products ---
// cta_group::2: the CTAs with ranks 2k and 2k + 1 work on one product of twice the rows; each holds its rows of A and of the
// accumulator and half of B's columns, the even CTA issues. ts takes A from tensor memory: 16-bit values, two to a 32-bit
// column, row r of a CTA in lane r. commit arrives on the barrier at this offset in every CTA of the mask once this
// thread's products so far are complete.
namespace tc2 {
__device__ __forceinline__ void alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
               "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
               "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void commit(uint64_t* bar, uint16_t mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"(mask)
               : "memory");
}
}  // namespace tc2

}  // namespace hs
