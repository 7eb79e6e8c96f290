// Building blocks of the 4-bit cache, the token weights and the eviction beside
// those of pa_device.cuh: launches that overlap the end of the preceding kernel,
// and 16-byte asynchronous copies.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"

namespace pa {
namespace dev {

// Start of a kernel launched by launch_ordered: plain stream order, and the next
// kernel may be dispatched from here on. The wait comes first, so that what was
// complete before this kernel is also complete before a dependent's own prologue.
__device__ __forceinline__ void griddep_enter() {
  griddep_wait();
  griddep_launch_dependents();
}

// 16 bytes global -> shared, past L1, where `on` (completion: cp_async_commit /
// cp_async_wait). Predicated rather than branched around: the warp stays together.
__device__ __forceinline__ void cp_async16(void* dst_smem, const void* src_gmem, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}\n" ::"r"(smem_addr(dst_smem)),
      "l"(src_gmem), "r"(uint32_t(on))
      : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// until at most N of this thread's newest groups are in flight
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace dev

// Launch of a kernel whose every CTA waits for the preceding kernel
// (griddep_wait, griddep_enter) before it touches memory: its CTAs are
// dispatched while that kernel's last ones still run, which hides the launch
// (about 1.5 us in a chain of small kernels). `cluster`: CTAs of a cluster.
template <typename... Params, typename... Args>
int launch_ordered(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem,
                   cudaStream_t stream, unsigned cluster, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return int(cudaLaunchKernelEx(&cfg, kernel, Params(args)...));
}

}  // namespace pa
