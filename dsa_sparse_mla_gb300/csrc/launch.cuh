// launch.cuh — launches in a row.
//
// A call's second kernel may be launched while its first still runs (launch_next), so that its blocks stand ready when the first
// ends: the first lets it (let_next), the second waits for the first's end and its writes before it reads or writes
// anything (after_previous). The first kernel of a call, and whatever the caller enqueues next, start as usual; the calls of read.cu,
// heads.cu and expanded.cu let a call of theirs that follows start early, too: every one of their blocks waits for what came before,
// so a kernel's end is still the end of everything before it.
#pragma once

#include <cuda_runtime.h>

namespace hs {

__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace hs
