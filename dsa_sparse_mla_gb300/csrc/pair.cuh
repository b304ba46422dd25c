// pair.cuh — device helpers for clusters of two CTAs that work as one (two-SM tensor products): TMA copies and expected bytes
// counted on a barrier of either CTA, 16-byte stores into either CTA's shared memory that count there.
#pragma once

#include <atomic>

#include "cluster.cuh"

namespace hs {
namespace pair {

// Tiled loads into this CTA's shared memory, their bytes counted on a barrier of either CTA of a pair (address from remote_smem), or with
// kSMs = 1 of this CTA. x must be a multiple of 16 bytes.
template <int kSMs = 2>
__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  if constexpr (kSMs == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                     smem_u32(dst)),
                 "l"(map), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}
template <int kSMs = 2>
__device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
  if constexpr (kSMs == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
                     smem_u32(dst)),
                 "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// The same under an L2 cache policy.
__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], [%2], "
      "%5;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5}], "
      "[%2], %6;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// Arrives on a barrier of either CTA and has it expect these bytes. Relaxed: the arrival hands on no writes of this thread.
__device__ __forceinline__ void arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// 16 bytes into either CTA's shared memory, counted on a barrier there; waited for with Mma::wait_writes.
__device__ __forceinline__ void st_async16(uint32_t dst, int4 v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(dst), "r"(bar),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Release and acquire at cluster scope of shared memory alone (remote_arrive and mbar_wait_cluster do so for every memory, and wait for it).
__device__ __forceinline__ void fence_release_smem() { asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory"); }
__device__ __forceinline__ void fence_acquire_smem() { asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory"); }

__device__ __forceinline__ bool try_wait_relaxed(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}

// mbar_wait that sees what another CTA of the cluster wrote to shared memory before its arrival.
__device__ __forceinline__ bool wait_cluster_smem(uint64_t* bar, uint32_t parity, int32_t* err) {
  bool ok = try_wait_relaxed(bar, parity);
  const uint64_t t0 = ok ? 0 : globaltimer();
  for (uint32_t it = 0; !ok; ++it) {
    ok = try_wait_relaxed(bar, parity);
    if (!ok && (it & 63) == 63 && globaltimer() - t0 > kWaitLimitNs) {
      flag_error(err, HS_FLAG_TIMEOUT);
      return false;
    }
  }
  fence_acquire_smem();
  return true;
}

// Whether the phase with this parity is over, without waiting.
__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}

// One SM by itself or a pair's two: tensor products (a commit arrives on the barrier of every CTA that takes part), and barriers of CTA
// `rank` by their address. A CTA by itself is not launched as a cluster and takes the forms of its own shared memory throughout.
template <int kSMs>
struct Mma {
  static __device__ __forceinline__ uint32_t at(const void* p, uint32_t rank) {
    if constexpr (kSMs == 2)
      return remote_smem(p, rank);
    else
      return smem_u32(p);
  }
  static __device__ __forceinline__ void arrive(uint32_t bar) {
    if constexpr (kSMs == 2)
      remote_arrive_cta(bar);
    else
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
  }
  // Hands on this thread's writes of its CTA's shared memory (after __syncwarp its warp's; fenced for the async proxy by those who wrote
  // them) to a thread of CTA 0 that waits with wait_writes: the other forms here order nothing between two CTAs but tensor memory, reads,
  // and copies that count on barriers by themselves.
  static __device__ __forceinline__ void arrive_writes(uint32_t bar) {
    if constexpr (kSMs == 2) {
      fence_release_smem();
      remote_arrive_relaxed(bar);
    } else {
      arrive(bar);
    }
  }
  static __device__ __forceinline__ bool wait_writes(uint64_t* bar, uint32_t parity, int32_t* err) {
    if constexpr (kSMs == 2)
      return wait_cluster_smem(bar, parity, err);
    else
      return mbar_wait(bar, parity, err);
  }
  static __device__ __forceinline__ void arrive_relaxed(uint32_t bar) {
    if constexpr (kSMs == 2)
      remote_arrive_relaxed(bar);
    else
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
  }
  static __device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
    if constexpr (kSMs == 2)
      arrive_expect_tx(bar, bytes);
    else
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
  }
  static __device__ __forceinline__ void alloc(uint32_t* dst, uint32_t ncols) {
    if constexpr (kSMs == 2)
      tc2::alloc(dst, ncols);
    else
      tmem_alloc(dst, ncols);
  }
  static __device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
    if constexpr (kSMs == 2)
      tc2::dealloc(taddr, ncols);
    else
      tmem_dealloc(taddr, ncols);
  }
  static __device__ __forceinline__ void ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (kSMs == 2)
      tc2::ss(d, a, b, idesc, accumulate);
    else
      mma_bf16_ss(d, a, b, idesc, accumulate);
  }
  // A from tensor memory: 16-bit values, two to a column
  static __device__ __forceinline__ void ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (kSMs == 2)
      tc2::ts(d, a, b, idesc, accumulate);
    else
      asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a), "l"(b),
                   "r"(idesc), "r"(accumulate));
  }
  static __device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (kSMs == 2)
      tc2::commit(bar, 0x3);
    else
      mma_commit(bar);
  }
};

// After a wait that ran out: gives copies in flight, which take microseconds, 20 ms to land before the CTA leaves.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 20000000ull) __nanosleep(1000);
}

// Tensor map of a bf16 [rows][heads][cols] tensor (strides in values) with boxes of box_rows x 64 columns of one head, 128-byte swizzle.
inline bool encode_heads(CUtensorMap* map, const void* base, uint64_t cols, uint64_t heads, uint64_t rows, int64_t stride_h, int64_t stride_t,
                         uint32_t box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, heads, rows};
  cuuint64_t strides[2] = {(cuuint64_t)stride_h * 2, (cuuint64_t)stride_t * 2};
  cuuint32_t box[3] = {64, 1, box_rows}, es[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Lets a kernel use this much dynamic shared memory; asked once per kernel and device.
template <typename... P>
inline cudaError_t allow_smem(void (*kernel)(P...), int bytes) {
  struct Seen {
    std::atomic<const void*> kernel[64];
  };
  static Seen seen[8];  // kernels of one signature: a few instances of one template
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const void* k = reinterpret_cast<const void*>(kernel);
  if (dev < 64)
    for (Seen& s : seen)
      if (s.kernel[dev].load(std::memory_order_relaxed) == k) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess || dev >= 64) return e;
  for (Seen& s : seen) {
    const void* none = nullptr;
    if (s.kernel[dev].compare_exchange_strong(none, k) || none == k) break;
  }
  return cudaSuccess;
}

}  // namespace pair
}  // namespace hs
