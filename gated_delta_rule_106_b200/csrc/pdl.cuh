// Programmatic dependent launch: a kernel's CTAs may take their places and set up
// shared memory while the kernel before it on the stream ends. Such a kernel
// calls wait_for_previous() before it touches global memory: it returns when the
// kernels before have completed and their writes are visible. let_next_start()
// lets a kernel that is launched this way after it come in once every CTA has called
// it, by any of its threads, or ended; any other kernel after it waits for its end as
// always. Where a kernel calls it only behind its own wait (paged_split_kernel), the
// next one may touch before its wait what that one neither reads nor writes
// (paged_join_kernel's rows without tokens); a kernel that calls it first gives no such
// promise (page_plan_kernel, qk_norm_rope_kernel).
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace gdn {

__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;");
}

template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t stream, A&&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace gdn
