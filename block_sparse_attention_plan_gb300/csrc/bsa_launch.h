// Launches that overlap the end of the kernel ahead of them in the stream.
#pragma once

#include <cuda_runtime.h>

namespace bsa {

// Launch that may become resident before the kernel ahead of it in the stream
// has ended.  Every kernel launched so begins with wait_for_previous(), which
// returns when that one has ended and its writes are visible; it lets its own
// successor queue up right away.  Hides most of the 2 us between dependent
// kernels, which is what calls on a few sequences consist of.
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, int smem, cudaStream_t s,
                         const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// A load of what an earlier kernel of the stream may have written (the library's
// or the caller's: every list, mask and table that a call is given): a kernel
// that launch_after starts may be resident while that one writes, which rules
// out the read-only path (__ldg) for it, whose loads need not stay behind
// wait_for_previous() either.
template <class T>
__device__ __forceinline__ T load_written(const T* p) {
  return *p;
}
__device__ __forceinline__ void next_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

}  // namespace bsa
