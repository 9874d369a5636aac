// Launches that may start while the kernel before them on the stream is ending
// (programmatic dependent launch): block scheduling, barrier set-up and the
// like overlap its tail, and dependent_wait holds back everything that touches
// memory until it is complete and its writes are visible. A kernel launched
// without the attribute waits for its predecessor as always.

#pragma once

#include <cuda_runtime.h>

namespace mxk {

// Every kernel launched by launch_dependent calls this before it reads or
// writes global memory.
__device__ __forceinline__ void dependent_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The next kernel may be scheduled once every CTA has called this or exited.
__device__ __forceinline__ void dependent_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t st, int cluster, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mxk
