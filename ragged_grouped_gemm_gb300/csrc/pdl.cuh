// Programmatic dependent launch: a kernel launched with launch_pdl may start
// while the kernel before it on the stream is still running, does what needs
// none of its results (barriers, tensor memory, tensor maps), and then waits
// for it to complete.  Every kernel so launched calls pdl_wait in every thread
// before it touches global memory, so the order of a stream's results is the
// same as without.
#pragma once
#include <cuda_runtime.h>

namespace moe {

// Waits until the kernels before this one have completed and their writes are visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel's blocks start as SMs become free.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// CLUSTER: blocks of a thread block cluster (1: none).
template <int CLUSTER = 1, class... P, class... A>
cudaError_t launch_pdl(void (*kern)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {CLUSTER, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = CLUSTER > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace moe
