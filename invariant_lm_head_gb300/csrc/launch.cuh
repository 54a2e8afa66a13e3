// Launches that may begin before the kernel ahead of them in the stream has ended.
//
// A kernel launched here starts its CTAs once every CTA of the kernel ahead has said that
// it is nearly done (or has ended), sets itself up, and waits for that kernel's end, with
// all it wrote, before it touches global memory: the launch and the set-up cost nothing
// then. Every thread has to pass ahead_done(), so that a kernel's end means the end of all
// before it. Behind any other kind of work in the stream, and behind a kernel that says
// nothing, such a launch is an ordinary one. A CTA says it late: said at its start, the
// CTAs behind crowd onto the SMs that have room first (256 rows of V=152064 in
// lmhead_top_logprobs, back to back: 33 us for 25.5).
// (4-bit logits back to back: T=64 H=4096 V=32000 17.0 -> 15.3 us, T=200 H=3616 V=32003
// 26.7 -> 23.9, T=1 H=3584 V=152064 48.4 -> 46.7.)
#pragma once

#include <cuda_runtime.h>

namespace lmh {

// This CTA is nearly done: once all are, the kernel behind may start its own.
__device__ __forceinline__ void nearly_done() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// The kernel ahead has ended and its writes are visible.
__device__ __forceinline__ void ahead_done() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// cluster: CTAs of a cluster (1: none asked for here).
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                         cudaStream_t stream, unsigned cluster, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace lmh
