// dependent.cuh — launches that overlap with the end of the kernel before them
// (programmatic dependent launch): norm and rotation, the paged cache and its
// attention, kernels of a few microseconds each that follow one another in every
// layer of a step.
//
// Every thread of such a kernel passes grid_dependency_wait before it touches
// memory that any earlier kernel may write or read, so each kernel still sees the
// ones before it in the stream as finished.
#pragma once
#include <cuda_runtime.h>

namespace fm {

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" :::); }

// Launch with the programmatic dependency on the kernel before it: the new
// grid's prologue runs while that kernel ends, and its grid_dependency_wait
// returns once it has.
template <typename... Args, typename... Given>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                             Given&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Args(args)...);
}

}  // namespace fm
