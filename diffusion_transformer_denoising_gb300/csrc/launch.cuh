// Launches with a cluster shape and programmatic dependence.
#pragma once
#include <cuda_runtime.h>

#include "common.cuh"

namespace dit {

// Programmatic dependence between a kernel and the next of the same call: the
// first lets the second start early, the second waits for the first's results
// before it touches anything that kernel reads or writes.  One that is marked late reads
// before that wait, and only what the kernels before the previous one wrote: each block of
// the previous one has waited for them (wait_previous) before it let this one start
// (start_next), so they have ended.  It reads past L1 (__ldcg), which may hold what an
// earlier launch found there, and waits before it ends, so that the call's end is that of
// all its kernels.  (Without it the gradient of 64 x 256 x 1024 takes 14.8 us, with it 11.6;
// of 333 x 1000 x 2730 32.3 and 30.5.)
DIT_DEV void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
DIT_DEV void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Clusters of up to 8 blocks (the portable limit): the two halves of the
// cluster barrier, and reads of a peer's shared memory at a cluster_map address.
// Every warp of the cluster reaches both halves, its lanes together.
constexpr int kMaxCluster = 8;
DIT_DEV void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
DIT_DEV void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
DIT_DEV float ld_cluster_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
DIT_DEV float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
DIT_DEV float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Launch on `s` (dynamic shared memory above 48 KB only for kernels without
// static shared memory); cluster > 1: blocks of a cluster along x; after: may start
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
    // one value for every call: another thread's smaller launch of the same
    // kernel must not take the room away in between
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 << 10);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&c, kernel, Params(args)...);
}

}  // namespace dit
