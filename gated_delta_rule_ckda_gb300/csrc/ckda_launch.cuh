// ckda_launch.cuh -- kernels of one call that follow one another.  A kernel launched
// with launch_next may start while the one before it in the stream still runs: its
// launch and its blocks' start hide behind that one's end (linear attention in fp32,
// four kernels: 74 -> 69 us; one long sequence, three: 185 -> 182).  Every kernel that is
// launched so begins with after_previous(), which waits for all of the one before,
// and sees its writes; one that another follows lets it start with let_next_start().
#pragma once
#include <cuda_runtime.h>
#include <utility>

namespace ckda {

__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;");
}

// `next`: a kernel of the same call comes before it.
template <typename... P, typename... A>
cudaError_t launch_next(bool next, void (*kernel)(P...), dim3 grid, unsigned block, size_t smem,
                        cudaStream_t s, A&&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = next ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...);
}

}  // namespace ckda
