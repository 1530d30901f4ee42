// Launches whose kernels follow one another in a call: the later kernel's blocks
// are placed while the earlier one still runs, and wait on the device for its
// end (programmatic dependent launch).  The earlier kernel says when with
// let_next_in, the later one calls wait_for_previous before it touches anything.
// What an earlier kernel of the chain writes is read after the wait by ordinary
// loads or __ldcg: __ldg's path is for data that no kernel writes while this one
// is on the device, the call's descriptors.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace gp {

__device__ __forceinline__ void let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace gp
