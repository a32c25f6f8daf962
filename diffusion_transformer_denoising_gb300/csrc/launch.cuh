// Launches with a cluster shape and programmatic dependence.
#pragma once
#include <cuda_runtime.h>

#include "common.cuh"

namespace dit {

// Programmatic dependence between a kernel and the next of the same call: the
// first lets the second start early, the second waits for the first's results
// before it touches anything that kernel reads or writes.
DIT_DEV void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
DIT_DEV void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch on `s`; cluster > 1: blocks of a cluster along x; after: may start
// before the previous kernel of the stream has ended (it has to wait_previous).
template <class... Params, class... Args>
cudaError_t launch_kernel(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster,
                          bool after, Args... args) {
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute at[2];
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = at;
  if (cluster > 1) {
    at[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[c.numAttrs].val.clusterDim.x = cluster;
    at[c.numAttrs].val.clusterDim.y = at[c.numAttrs].val.clusterDim.z = 1;
    ++c.numAttrs;
  }
  if (after) {
    at[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[c.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++c.numAttrs;
  }
  if (smem > (48 << 10)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&c, kernel, Params(args)...);
}

}  // namespace dit
