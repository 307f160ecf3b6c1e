// Launches that may begin while the kernel before them in the stream ends: its
// last CTAs leave SMs free, and a launch costs microseconds of its own.  Calls issued one
// behind the other, before and after: a decode step's block tables 8.2 and 5.7 us, three
// prompts into the cache and back 81.2 and 77.3, nine requests' attention 16.0 and 14.0.
#pragma once

#include <cuda_runtime.h>

namespace sparge {

// Before a kernel launched by launch_after touches global or tensor memory (its own
// shared memory it may): lets the next kernel's CTAs come to the SMs that have
// room, and waits until all that earlier kernels wrote is there.  Every CTA passes it,
// so a kernel that ends has seen all before it end.
__device__ __forceinline__ void begin_after() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                         cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sparge
