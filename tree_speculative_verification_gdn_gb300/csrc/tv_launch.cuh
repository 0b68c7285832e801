// A kernel that is launched while the one in front of it in the stream, a check or a plan, still runs.
#pragma once

#include <cuda_runtime.h>

namespace tv {

// plan_begun() in the first kernel lets the second one begin; wait_for_plan() in that one, before its first read of what
// the first writes and before any write of its own, waits until the first has ended.  Whatever came before the first has
// ended when either runs.  The second one's pointers are not __restrict__: what the first writes is not constant while the
// second lives, and a load of memory declared unaliased or read-only might be moved ahead of the wait.
__device__ __forceinline__ void plan_begun() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_plan() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_behind_plan(void (*kern)(P...), dim3 grid, int block, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid, c.blockDim = dim3(block), c.dynamicSmemBytes = smem, c.stream = s;
  c.attrs = &early, c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, P(args)...);
}

}  // namespace tv
